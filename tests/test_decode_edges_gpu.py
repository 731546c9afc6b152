"""The decode operators on the GPU at sizes and values beyond those of
test_decode_ops_gpu.py, whose definitions in 64 bits and derived tolerances
they share."""
import pytest
import torch

from epilogue_gemm_amd import binding as gb
from tests.test_decode_ops_gpu import Pool, attend, attend_want, gen, lora_case, lora_check, lora_run, pow2_quantise, rand, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gb.load_library()


@pytest.mark.parametrize("lens,heads,group,head_dim,dtype,cache", [
    # one long sequence, or a few, cut into some one unit a workgroup: as many
    # pieces as units in every column, the last ones too
    ([10300], 4, 7, 128, "bf16", "bf16"), ([12000], 4, 8, 128, "f16", "fp8"), ([20600], 2, 4, 128, "bf16", "bf16"),
    ([20600], 2, 7, 64, "f16", "f16"), ([10500], 4, 16, 64, "bf16", "bf16"), ([21000], 8, 16, 64, "bf16", "fp8"),
    ([4200], 12, 16, 128, "f16", "f16"), ([9000], 1, 160, 128, "bf16", "bf16"), ([11000, 300, 0, 7], 4, 8, 128, "bf16", "bf16"),
    ([6000, 6000], 4, 5, 128, "bf16", "fp8"),
])
@pytest.mark.parametrize("wide", [1, 4])
def test_attend_writes_every_head_of_long_sequences(lens, heads, group, head_dim, dtype, cache, wide):
    pool = Pool(lens, heads, head_dim, 64, dtype, cache, 80, width=wide * -(-max(lens) // 64))
    pool.fill(81)
    q = rand(gen(82), len(lens), heads * group, head_dim, std=1.5, dtype=dtype)
    want, tol = attend_want(pool, q)
    within(attend(pool, q), want, tol, f"{lens} {heads}x{group}")


@pytest.mark.parametrize("page,dtype,cache", [(64, "bf16", "bf16"), (16384, "f16", "fp8")])
def test_attend_over_the_longest_table(page, dtype, cache):
    # 2^31 - 256 tokens at most, all of whose pages are missing but the first
    # and the last
    width = ((1 << 31) - 256) // page
    small = Pool([2 * page], 4, 64, page, dtype, cache, 83)
    small.fill(84)
    table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    table[0, 0], table[0, -1] = int(small.table[0, 0]), int(small.table[0, 1])
    q = rand(gen(85), 1, 8, 64, dtype=dtype)
    want, tol = attend_want(small, q)
    o = torch.full_like(q, float("nan"), device="cuda")
    small.cache.attend(q.cuda(), o, table, torch.tensor([(1 << 31) - 1], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    within(o, want, tol, "the longest table")


@pytest.mark.parametrize("M,N,K,rank,adapters", [(40, 1000, 1024, 16, 3), (100, 264, 4096, 24, 5), (700, 136, 4096, 64, 4),
                                                 (1500, 200, 2048, 32, 6)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_lora_of_a_row_in_any_place(M, N, K, rank, adapters, dtype):
    # one kernel, and two with one range of K and several: the same rows in
    # another order, so in other tiles and beside other adapters, have the same
    # bits
    ids = [(m * 7 + m // 5) % (adapters + 1) - 1 for m in range(M)]
    x, a, b, ids, s, r = lora_case(M, N, K, rank, adapters, dtype, ids, M + N + K)
    want = lora_run(x, a, b, ids, s, r, dtype).cpu()
    lora_check(x, a, b, ids, s, r, want, dtype, "rows in order")
    for seed in (86, 87):
        p = torch.randperm(M, generator=gen(seed))
        assert torch.equal(lora_run(x[p], a, b, ids[p], s, r[p], dtype).cpu(), want[p])


@pytest.mark.parametrize("rank,K", [(8, 64), (16, 64), (24, 64), (40, 64), (64, 64), (72, 64), (8, 8200), (24, 8200)])
def test_lora_infinite_inner_products(rank, K):
    # U[0] of some rows lies beyond fp32: their C is the infinity of B's sign,
    # in one kernel and in two, whatever stands behind the rank
    M, N = 20, 72
    x, a, b, ids, s, r = lora_case(M, N, K, rank, 2, "bf16", [m % 3 - 1 for m in range(M)], 88)
    big = (torch.arange(M) % 2 == 0) & (ids >= 0)
    a[:, 1:, 5] = 0
    a[:, 0, 5] = 64.0
    x[:, 5] = 0
    finite = lora_run(x, a, b, ids, s, r, "bf16").cpu()
    x[big, 5] = 2.0 ** 127
    got = lora_run(x, a, b, ids, s, r, "bf16").cpu()
    assert torch.equal(got[~big], finite[~big]) and bool(finite.isfinite().all())
    sign = b[ids.clamp(min=0).long()][big][:, :, 0].float().sign()
    assert torch.equal(got[big].float(), sign * float("inf"))


@pytest.mark.parametrize("M,K", [(6, 64), (6, 8200)])
def test_lora_finite_inner_products_beside_an_infinite_one(M, K):
    # U = (infinity, 2^17, ...) in F16: the second, beyond the largest F16 but
    # finite, takes nothing from the first
    x, a, b, ids, _, r = lora_case(M, 40, K, 8, 1, "f16", [0] * M, 89)
    a[0, :2], x[:, 7:9] = 0, 0
    a[0, 0, 7], a[0, 1, 8], b[0, :, 0], b[0, :, 1] = float("inf"), 512.0, 1.0, -1.0
    a[0, 1:, 7] = 0
    x[:, 7], x[:, 8] = 1.0, 256.0
    assert bool((lora_run(x, a, b, ids, None, r, "f16") == float("inf")).all())


@pytest.mark.parametrize("M,K", [(20, 64), (20, 8200)])
def test_lora_small_inner_products_beside_a_large_one(M, K):
    # U = (4096, some 2^-8, 0, ...) in F16, of which only the second has a
    # column of B, of ones: C is that product of two F16 values, 22 bits, rounded
    # once
    x, a, b, ids, _, _ = lora_case(M, 40, K, 8, 1, "f16", [0] * M, 96, residual=False)
    a[:], b[:] = 0, 0
    a[0, 0, 3], a[0, 1, 9], b[0, :, 1] = 64.0, 1.3701 * 2.0 ** -8, 1.0
    x[:, 3], x[:, 9] = 64.0, 1 + torch.arange(M) / 37
    got = lora_run(x, a, b, ids, None, None, "f16").cpu()
    assert torch.equal(got, (x[:, 9].double() * a[0, 1, 9].double()).half()[:, None].expand(M, 40))


@pytest.mark.parametrize("head_dim,cache", [(64, "f16"), (128, "f16"), (64, "fp8"), (128, "fp8")])
def test_attend_small_weights_beside_large_ones(head_dim, cache):
    # every 16th key has e^11 to e^13 times the weight of each other, but zeros
    # for a value: the others' weights in F16 would be multiples of 2^-24, a
    # hundredth of them
    n = 3000
    pool = Pool([n], 1, head_dim, 64, "f16", cache, 90)
    k, v = torch.zeros(n, 1, head_dim, dtype=torch.float16), torch.full((n, 1, head_dim), 16.0, dtype=torch.float16)
    k[::16, 0, 0], v[::16] = 12, 0
    pool.held = [(pool.put(pool.k, pool.ks, 0, k), pool.put(pool.v, pool.vs, 0, v))]
    q = torch.zeros(1, 16, head_dim, dtype=torch.float16)
    q[0, :, 0] = (7.5 + torch.arange(16) / 16) * (head_dim / 64) ** 0.5
    want, tol = attend_want(pool, q)
    within(attend(pool, q), want, tol, "small weights")


def test_attend_smallest_f16_values_in_8_bits():
    # rows of 2^-13 and, beside it, 9 2^-24, which E4M3 holds exactly at the
    # rows' scale 2^-21: exact in both products, as a multiple of F16's least
    # step 2^-24
    n, D = 500, 64
    pool = Pool([n], 1, D, 16, "f16", "fp8", 91)
    small, odd = 9 * 2.0 ** -24, torch.arange(n) % 2 == 1
    k, v = torch.zeros(n, 1, D, dtype=torch.float16), torch.full((n, 1, D), small, dtype=torch.float16)
    k[:, 0, 0], v[:, 0, 0] = 2.0 ** -13, 2.0 ** -13
    k[odd, 0, 1:] = small
    v[odd, 0, 1:8] = 2.0 ** -13
    pool.held = [(pool.put(pool.k, pool.ks, 0, k), pool.put(pool.v, pool.vs, 0, v))]
    assert torch.equal(pool.held[0][0], k.double()) and torch.equal(pool.held[0][1], v.double())
    q = torch.zeros(1, 4, D, dtype=torch.float16)
    q[0, 1:, 1:] = torch.tensor([2.0 ** 14, 2.0 ** 15, 65504.0]).half()[:, None]
    want, tol = attend_want(pool, q)
    within(attend(pool, q), want, tol, "smallest values")


def test_attend_scales_beyond_those_of_f16_rows():
    # a cache filled by another's hand: K's scales of any size, V's up to 2^14
    n, D = 300, 64
    pool = Pool([n], 2, D, 32, "f16", "fp8", 92)
    pool.fill(93)
    kv = []
    for values, cache, scale, powers in zip(pool.held[0], (pool.k, pool.v), (pool.ks, pool.vs), ([-90, -20, 0, 16, 20], [-20, 4, 8, 11, 14])):
        q, s = pow2_quantise(values)
        s = torch.exp2(torch.tensor(powers)[torch.randint(0, 5, s.shape, generator=gen(94))].double())
        q = q.clamp(-3, 3)  # (so that O is within F16)
        q = q.float().to(torch.float8_e4m3fn)
        pos = torch.arange(n)
        page, slot = pool.table[0].long()[pos // 32].cuda(), (pos % 32).cuda()
        cache.view(torch.uint8)[page, :, slot] = q.cuda().view(torch.uint8)
        scale[page, :, slot] = s.float().cuda()
        kv.append(q.float().double() * s[..., None])
    pool.held = [tuple(kv)]
    q = torch.randn(1, 4, D, generator=gen(95)) * 2.0 ** -24 * torch.tensor([1.0, 2.0, 4.0, 8.0])[:, None]
    q = q.half()
    want, tol = attend_want(pool, q)
    within(attend(pool, q), want, tol, "large scales")
