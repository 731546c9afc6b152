"""The operators of a decode step on the GPU against their definitions in 64
bits, at the sizes, masks, strides and values where they can go wrong.

Tolerances.  An output in a 16-bit format is off by its rounding, at most
half a step (eps / 2 of the value; half the smallest subnormal near zero),
plus what the fp32 arithmetic before it loses, bounded term by term beside
each operator; E4M3 codes by half a step of theirs (2^-4, or 2^-10 of the
scale below the normal range)."""
import math

import pytest
import torch

from epilogue_gemm_amd import binding as gb

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
SUB = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}  # half the smallest subnormal
U = 2.0 ** -24  # half a step of fp32
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gb.load_library()


def rand(g, *shape, std=1.0, dtype="bf16"):
    return (torch.randn(shape, generator=g) * std).to(DT[dtype])


def gen(seed):
    return torch.Generator().manual_seed(seed)


def strided(t, extra):
    """The rows of a 2-d or 3-d tensor on the GPU, `extra` elements of NaN
    between them."""
    n = t[0].numel()
    pad = 1 << 30 if t.dtype == torch.int32 else NAN  # of a page table: no page
    buf = torch.full((t.shape[0], n + extra), pad, dtype=t.dtype, device="cuda")
    buf[:, :n] = t.reshape(t.shape[0], n).cuda()
    return buf[:, :n].unflatten(1, t.shape[1:]) if t.dim() == 3 else buf[:, :n]


def within(got, want, tol, what):
    """|got - want| <= tol elementwise (fp64), and equally non-finite."""
    got, want = got.detach().cpu().double(), want.double()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), f"{what}: other infinities"
    over = ((got - want).abs() - tol)[fine]
    assert over.numel() == 0 or float(over.max()) <= 0, f"{what}: {int((over > 0).sum())} outside, worst by {float(over.max()):.3g}"


# ---- RMS norm ------------------------------------------------------------------

def rms_want(x, r, w, eps):
    h = x.double() + (r.double() if r is not None else 0.0)
    return h, h / (h.square().mean(1, keepdim=True) + eps).sqrt() * w.double()


def rms_check(x, r, w, eps, dtype, h, y, y_scale, what):
    hw, yw = rms_want(x, r, w, eps)
    e = torch.finfo(DT[dtype]).eps / 2
    # h: the fp32 sum and its rounding.  y: the fp32 sum of squares loses at
    # most cols / 64 + 8 half steps (a lane's chain, then the tree over lanes
    # and waves), halved by the root; h, the root, the quotient, two products
    # and the reciprocal of a scale lose a few more.
    lost = (x.shape[1] / 64 + 24) * U
    if h is not None:
        within(h, hw, hw.abs() * (e + 2 * U) + SUB[dtype], what + " h")
    if y_scale is None:
        within(y, yw, yw.abs() * (e + lost) * (1 + e) + SUB[dtype], what + " y")
        return
    s = y_scale.cpu().double()
    want = (yw.abs().amax(1) / 448).clamp(min=2.0 ** -100)
    assert float(((s - want).abs() / want).max()) <= lost + 2 * U, what + " scale"
    got = y.cpu().float().double() * s[:, None]
    within(got, yw, yw.abs() * (2.0 ** -4 + lost) * (1 + 2.0 ** -4) + 2.0 ** -10 * s[:, None], what + " q")


def rms_run(x, r, w, eps, dtype, out, extra=0, with_h=True):
    xs = strided(x, extra)
    rs = strided(r, 2 * extra) if r is not None else None
    h = strided(torch.full_like(x, NAN), extra) if with_h else None
    y = torch.full((x.shape[0], x.shape[1] + extra), NAN, device="cuda").to(torch.float8_e4m3fn if out == "fp8" else DT[dtype])
    y, ybuf = y[:, :x.shape[1]], y
    s = torch.full((x.shape[0],), NAN, device="cuda") if out == "fp8" else None
    gb.rmsnorm(xs, w.cuda(), y, residual=rs, residual_out=h, y_scale=s, eps=eps)
    torch.cuda.synchronize()
    assert bool(ybuf.float()[:, x.shape[1]:].isnan().all()), "padding of y written"
    return h, y, s


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (70, 8), (2, 64), (5, 130), (9, 256), (33, 512), (17, 1000), (3, 1024),
                                       (2, 2056), (4, 4096), (5, 5120), (3, 8192), (2, 8200), (2, 16384), (1, 20001), (2, 40008)])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "fp8"), ("f16", "fp8")])
@pytest.mark.parametrize("residual", [False, True])
def test_rmsnorm(rows, cols, dtype, out, residual):
    g = gen(rows * 100003 + cols)
    x, w = rand(g, rows, cols, dtype=dtype), (1 + 0.2 * torch.randn(cols, generator=g)).to(DT[dtype])
    r = rand(g, rows, cols, std=3.0, dtype=dtype) if residual else None
    for extra in (0, 8, 3):
        h, y, s = rms_run(x, r, w, 1e-5, dtype, out, extra, with_h=residual)
        rms_check(x, r, w, 1e-5, dtype, h, y, s, f"{rows}x{cols} {dtype}->{out} extra {extra}")


@pytest.mark.parametrize("cols", [77, 1024, 5120])
def test_rmsnorm_in_place_and_misaligned(cols):
    g = gen(cols)
    x, r, w = rand(g, 6, cols), rand(g, 6, cols), rand(g, cols)
    xd, rd = x.cuda(), r.cuda()
    gb.rmsnorm(xd, w.cuda(), xd, residual=rd, residual_out=rd)  # y over x, h over the residual
    torch.cuda.synchronize()
    rms_check(x, r, w, 1e-6, "bf16", rd, xd, None, "in place")
    xd, rd = x.cuda(), r.cuda()
    y = torch.empty_like(xd)
    gb.rmsnorm(xd, w.cuda(), y, residual=rd, residual_out=xd)  # h over x
    torch.cuda.synchronize()
    rms_check(x, r, w, 1e-6, "bf16", xd, y, None, "h over x")
    # every tensor one element off a 16-byte boundary
    off = lambda t: torch.cat([t.reshape(-1)[:1], t.reshape(-1)]).cuda()[1:].view(t.shape)  # noqa: E731
    xd, rd, wd = off(x), off(r), off(w)
    y, h = off(torch.zeros_like(x)), off(torch.zeros_like(x))
    assert xd.data_ptr() % 16 == 2
    gb.rmsnorm(xd, wd, y, residual=rd, residual_out=h)
    torch.cuda.synchronize()
    rms_check(x, r, w, 1e-6, "bf16", h, y, None, "misaligned")


@pytest.mark.parametrize("cols", [64, 1000, 4096, 9000])
@pytest.mark.parametrize("out", ["bf16", "fp8"])
def test_rmsnorm_values(cols, out):
    # rows of zeros (eps > 0), of one huge value, with an infinity, with a
    # NaN, of tiny values, and a plain one between them
    g = gen(cols + 1)
    x = rand(g, 6, cols)
    x[0] = 0
    x[1] = 0
    x[1, cols // 2] = 2.0 ** 60
    x[2, 3] = float("inf")
    x[3, 5] = NAN
    x[4] = x[4].float().mul(2.0 ** -70).bfloat16()
    w = torch.ones(cols, dtype=torch.bfloat16)
    h, y, s = rms_run(x, None, w, 1e-6, "bf16", out, with_h=False)
    y = y.float().cpu()
    # an infinite sum of squares: 0 for the finite values, NaN at the infinity
    assert bool((y[2, :3] == 0).all()) and math.isnan(y[2, 3])
    assert bool(y[3].isnan().all())
    keep = [0, 1, 4, 5]
    rms_check(x[keep], None, w, 1e-6, "bf16", None, y[keep], s[keep] if s is not None else None, "values")
    if s is not None:
        assert float(s[0]) == 2.0 ** -100


def test_rmsnorm_eight_bits_of_zeros_and_a_tiny_eps():
    # 1 / rms of a row of zeros is 1e15, over the least scale more than fp32
    # holds
    x = rand(gen(3), 3, 200)
    x[1] = 0
    w = torch.ones(200, dtype=torch.bfloat16)
    _, y, s = rms_run(x, None, w, 1e-30, "bf16", "fp8", with_h=False)
    assert bool((y[1].float() == 0).all()) and float(s[1]) == 2.0 ** -100
    rms_check(x, None, w, 1e-30, "bf16", None, y, s, "tiny eps")


def test_rmsnorm_many_short_rows():
    # the per-head norm of queries: many rows of 64, more rows than a grid's
    # first workgroups
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(1100003, 64, generator=g, device="cuda").bfloat16()
    w = torch.randn(64, generator=g, device="cuda").bfloat16()
    y = torch.empty_like(x)
    gb.rmsnorm(x, w, y)
    torch.cuda.synchronize()
    pick = torch.cat([torch.arange(100), torch.randint(0, 1100003, (5000,), generator=gen(2)), torch.arange(1100003 - 100, 1100003)])
    rms_check(x[pick.cuda()].cpu(), None, w.cpu(), 1e-6, "bf16", None, y[pick.cuda()], None, "short rows")


def test_rmsnorm_no_rows():
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    gb.rmsnorm(e, torch.ones(64, dtype=torch.bfloat16, device="cuda"), torch.empty_like(e))


# ---- low-rank adapters ------------------------------------------------------------

def lora_case(M, N, K, rank, adapters, dtype, ids, seed, extra=0, residual=True, scale=True):
    g = gen(seed)
    x, a, b = rand(g, M, K, dtype=dtype), rand(g, adapters, rank, K, std=K ** -0.5, dtype=dtype), rand(g, adapters, N, rank, dtype=dtype)
    s = torch.rand(adapters, generator=g) + 0.5 if scale else None
    r = rand(g, M, N, std=2.0, dtype=dtype) if residual else None
    ids = torch.tensor(ids, dtype=torch.int32)
    return x, a, b, ids, s, r


def lora_check(x, a, b, ids, s, r, got, dtype, what):
    want, tol = torch.zeros(got.shape, dtype=torch.float64), torch.zeros(got.shape, dtype=torch.float64)
    if r is not None:
        want += r.double()
    adapters, rank, K = a.shape
    for i in set(ids.tolist()):
        if not 0 <= i < adapters:
            continue
        m = (ids == i).nonzero()[:, 0]
        f = float(s[i].double()) if s is not None else 1.0
        xd, ad, bd = x[m].double(), a[i].double(), b[i].double()
        u = xd @ ad.t()
        # U: an fp32 sum of K products in any order; its two 16-bit parts lose
        # 2^-16 of the value (bf16; f16 less) and 2^-24 of the row's largest;
        # then a sum of at most 2 rank products, the factor and the residual
        du = (K + 16) * U * (xd.abs() @ ad.abs().t()) + 2.0 ** -16 * u.abs() + 2.0 ** -24 * u.abs().amax(1, keepdim=True)
        want[m] += f * (u @ bd.t())
        tol[m] = f * (du @ bd.abs().t() + (2 * rank + 8) * U * (u.abs() @ bd.abs().t()))
    e = torch.finfo(DT[dtype]).eps / 2
    tol = tol * (1 + e) + want.abs() * (e + 4 * U) + SUB[dtype]
    within(got, want, tol, what)


def lora_run(x, a, b, ids, s, r, dtype, extra=0, ws=None):
    N = b.shape[1]
    c = strided(torch.full((x.shape[0], N), NAN, dtype=DT[dtype]), extra)
    gb.lora(strided(x, 8 * (extra > 0)), a.cuda(), b.cuda(), ids.cuda(), c, scale=s.cuda() if s is not None else None,
            residual=strided(r, 2 * extra) if r is not None else None, workspace=ws)
    torch.cuda.synchronize()
    return c


@pytest.mark.parametrize("M,N,K,rank,adapters", [
    (1, 8, 8, 8, 1), (1, 4096, 4096, 16, 3), (16, 64, 64, 16, 1), (17, 65, 72, 24, 5), (5, 1, 128, 8, 2),
    (33, 1000, 1000, 32, 40), (64, 513, 2048, 64, 16), (100, 255, 520, 128, 7), (31, 96, 8200, 40, 3),
    (16, 256, 16, 16, 16), (2, 100000, 64, 8, 2), (300, 320, 256, 72, 9),
    (512, 200, 264, 16, 3), (1000, 65, 2056, 24, 5), (777, 1100, 1032, 128, 2), (520, 8, 8, 8, 20), (8200, 72, 136, 40, 6)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_lora(M, N, K, rank, adapters, dtype):
    # ids in no order, some rows without an adapter (-1, and past the last)
    ids = [(m * 7 + m // 5) % (adapters + 2) - 1 for m in range(M)]
    c = lora_case(M, N, K, rank, adapters, dtype, ids, M + N + K)
    for extra in (0, 8, 3):
        lora_check(*c, lora_run(*c, dtype, extra), dtype, f"{M}x{N}x{K} r{rank} extra {extra}")


@pytest.mark.parametrize("M,N,K,rank,adapters", [
    (20, 300, 8192, 32, 12), (64, 4096, 4096, 64, 6), (3, 40000, 1024, 16, 16), (16, 520, 10000, 8, 20), (48, 1030, 1440, 128, 4),
    (1, 513, 2552, 16, 1), (2, 511, 1024, 64, 3), (128, 512, 1024, 16, 8), (16, 24, 8, 128, 2), (129, 1200, 520, 48, 4)])
def test_lora_few_rows(M, N, K, rank, adapters):
    # sizes on both sides of what one kernel and two are taken for
    ids = [(m * 5 + m // 3) % (adapters + 1) - 1 for m in range(M)]
    c = lora_case(M, N, K, rank, adapters, "bf16", ids, M + N + K)
    for extra in (0, 8, 3):
        lora_check(*c, lora_run(*c, "bf16", extra), "bf16", f"{M}x{N}x{K} r{rank} extra {extra}")


@pytest.mark.parametrize("ids", ["same", "none", "runs", "each"])
@pytest.mark.parametrize("residual,scale", [(True, False), (False, True)])
@pytest.mark.parametrize("M", [80, 600])
def test_lora_ids(ids, residual, scale, M):
    adapters = M
    ids = {"same": [3] * M, "none": [-1] * M, "runs": [m // 23 for m in range(M)], "each": list(range(M))}[ids]
    c = lora_case(M, 192, 512, 16, adapters, "bf16", ids, 5, residual=residual, scale=scale)
    lora_check(*c, lora_run(*c, "bf16"), "bf16", "ids")


def test_lora_out_of_range_ids():
    ids = [0, 1, 2, 3, -1, -2 ** 31, 2 ** 31 - 1, 65536, 1]
    c = lora_case(9, 72, 64, 8, 3, "f16", ids, 6)
    got = lora_run(*c, "f16")
    lora_check(*c, got, "f16", "ids out of range")
    assert torch.equal(got[3:8].cpu(), c[5][3:8])  # without an adapter: the residual's bits


@pytest.mark.parametrize("repeat", [6, 100])
def test_lora_another_adapters_values_stay_out(repeat):
    # adapter 1 is all NaN and infinities: only its own rows see them
    ids = [0, 1, 0, 2, -1, 2] * repeat
    x, a, b, i, s, r = lora_case(6 * repeat, 136, 256, 16, 3, "bf16", ids, 7)
    want = lora_run(x, a, b, i, s, r, "bf16").cpu()
    a[1], b[1] = NAN, float("inf")
    got = lora_run(x, a, b, i, s, r, "bf16").cpu()
    keep = i != 1
    assert torch.equal(got[keep], want[keep])
    assert bool(got[~keep].isnan().all())
    # and a row of NaN in X stays in its row
    x[2] = NAN
    got = lora_run(x, a, b, i, s, r, "bf16").cpu()
    keep[2] = False
    assert torch.equal(got[keep], want[keep]) and bool(got[2].isnan().all())


@pytest.mark.parametrize("M", [20, 640])
@pytest.mark.parametrize("dtype,big", [("f16", 3.0e4), ("bf16", 2.0 ** 90)])
def test_lora_large_inner_products(dtype, big, M):
    # U far beyond the largest f16, C within it: the two parts of U carry a
    # power of two
    x, a, b, i, s, r = lora_case(M, 64, 128, 16, 2, dtype, [0, 1] * (M // 2), 8, residual=False)
    x = (x.float() * big / 8).to(DT[dtype])
    a = (a.float() * 300).to(DT[dtype])
    b = (b.float() * (2.0 ** -14 if dtype == "f16" else 2.0 ** -90)).to(DT[dtype])
    lora_check(x, a, b, i, s, r, lora_run(x, a, b, i, s, r, dtype), dtype, "large U")


def test_lora_many_rows_in_place():
    x, a, b, i, s, r = c = lora_case(700, 264, 320, 24, 4, "bf16", [(m // 9) % 5 - 1 for m in range(700)], 9)
    want = lora_run(*c, "bf16")
    cd = r.cuda()
    gb.lora(x.cuda(), a.cuda(), b.cuda(), i.cuda(), cd, scale=s.cuda(), residual=cd)
    torch.cuda.synchronize()
    assert torch.equal(cd, want)


def test_lora_in_place_and_dirty_workspace():
    c = lora_case(50, 264, 320, 24, 4, "bf16", [(m * 3) % 5 - 1 for m in range(50)], 9)
    x, a, b, i, s, r = c
    n = gb.lora_workspace_size(50, 264, 320, 24, 4)
    ws = torch.full((n // 4,), NAN, device="cuda")
    want = lora_run(*c, "bf16", ws=ws)
    lora_check(*c, want, "bf16", "dirty workspace")
    cd = r.cuda()
    gb.lora(x.cuda(), a.cuda(), b.cuda(), i.cuda(), cd, scale=s.cuda(), residual=cd, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(cd, want)
    with pytest.raises(gb.GemmEpiError):
        gb.lora(x.cuda(), a.cuda(), b.cuda(), i.cuda(), cd, workspace=ws[: n // 4 - 1])


def test_lora_as_the_projections_residual():
    # C = X W^T + bias with the adapters' part through the projection's
    # residual, against the whole in 64 bits
    M, N, K, rank = 24, 512, 512, 16
    ids = [m % 4 - 1 for m in range(M)]
    x, a, b, i, s, _ = lora_case(M, N, K, rank, 3, "bf16", ids, 10, residual=False)
    g = gen(11)
    w, bias = rand(g, N, K, std=K ** -0.5), rand(g, N)
    delta, c = torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    xd = x.cuda()
    gb.lora(xd, a.cuda(), b.cuda(), i.cuda(), delta, scale=s.cuda())
    plan = gb.Plan(M, N, K, "bf16", "bf16", "row", "col", "bias")
    plan.run(xd, w.cuda(), bias.cuda(), c, residual=delta)
    torch.cuda.synchronize()
    plan.close()
    z = x.double() @ w.double().t() + bias.double()
    lora_check(x, a, b, i, s, None, delta, "bf16", "delta")
    want = z + delta.cpu().double()
    tol = want.abs() * (2.0 ** -8 + 4 * U) + (K + 8) * U * (x.double().abs() @ w.double().abs().t() + bias.double().abs())
    within(c, want, tol * (1 + 2.0 ** -8), "projection")


# ---- the paged cache ------------------------------------------------------------------

def pow2_quantise(x):
    """Codes (as fp64 values) and scales of the last axis' rows, from the
    definition: 2^e, e the smallest integer >= -100 with max|x| <= 448 2^e."""
    x = x.double()
    top = x.abs().amax(-1)
    e = torch.ceil(torch.log2(top / 448)).clamp(min=-100)  # log2(0) = -inf
    s = torch.exp2(e)
    q = x / s[..., None]
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
    q = torch.round(q / step) * step
    bad = ~torch.isfinite(top)
    return torch.where(bad[..., None], NAN, q), torch.where(bad, NAN, s)


class Pool:
    """A cache on the GPU whose every slot starts as NaN, a page table in any
    order, and what each token should be, in 64 bits on the CPU."""

    def __init__(self, lens, heads, head_dim, page, dtype, cache, seed, width=None, spare=2):
        g = gen(seed)
        self.dtype, self.heads, self.head_dim, self.page, self.fp8 = dtype, heads, head_dim, page, cache == "fp8"
        held = [max(n, 0) for n in lens]
        self.width = width or max(1, -(-max(held) // page))
        counts = [min(-(-n // page), self.width) for n in held]
        order = torch.randperm(sum(counts) + spare, generator=g).tolist()
        table, at = [], 0
        for n in counts:
            table.append(order[at:at + n] + [-1] * (self.width - n))
            at += n
        self.table = torch.tensor(table, dtype=torch.int32).view(len(lens), self.width)
        self.lens = torch.tensor(lens, dtype=torch.int32)
        shape = (len(order), heads, page, head_dim)
        ct = torch.float8_e4m3fn if self.fp8 else DT[dtype]
        self.k = torch.full(shape, NAN, device="cuda").to(ct)
        self.v = torch.full(shape, NAN, device="cuda").to(ct)
        self.ks = torch.full(shape[:3], NAN, device="cuda") if self.fp8 else None
        self.vs = torch.full(shape[:3], NAN, device="cuda") if self.fp8 else None
        self.cache = gb.PagedCache(self.k, self.v, self.ks, self.vs)

    def put(self, cache, scale, seq, values):
        """Token rows [n, heads, head_dim] of a sequence, positions 0 .. n-1."""
        pos = torch.arange(values.shape[0])
        page, slot = self.table[seq].long()[pos // self.page], pos % self.page
        ok = page >= 0
        page, slot = page[ok].cuda(), slot[ok].cuda()
        if not self.fp8:
            cache[page, :, slot] = values[ok].cuda()
            return values.double()
        q, s = pow2_quantise(values)
        cache.view(torch.uint8)[page, :, slot] = q[ok].float().to(torch.float8_e4m3fn).cuda().view(torch.uint8)
        scale[page, :, slot] = s[ok].float().cuda()
        return q * s[..., None]

    def fill(self, seed, std=1.0):
        g = gen(seed)
        self.held = []
        for i, n in enumerate(self.lens.tolist()):
            n = min(max(n, 0), self.width * self.page)
            kv = [rand(g, n, self.heads, self.head_dim, std=std, dtype=self.dtype) for _ in range(2)]
            self.held.append((self.put(self.k, self.ks, i, kv[0]), self.put(self.v, self.vs, i, kv[1])))


def attend_want(pool, q):
    """O and its tolerance in 64 bits.  An fp32 score is off by at most (D +
    4) half steps of sum |q k| / sqrt(D), and its exponential's argument by a
    few of its own size: a weight by twice that, relative; the weights' two
    16-bit parts lose 2^-16; sums over the keys in fp32 a few half steps more
    in any order of chains of 32 keys and joins."""
    B, hq, D = q.shape
    want, tol = torch.zeros(B, hq, D, dtype=torch.float64), torch.zeros(B, hq, D, dtype=torch.float64)
    e = torch.finfo(q.dtype).eps / 2
    for i in range(B):
        k, v = pool.held[i]
        pos = torch.arange(k.shape[0])
        there = (pool.table[i].long()[pos // pool.page] >= 0) & (pool.table[i].long()[pos // pool.page] < pool.k.shape[0])
        k, v = k[there], v[there]
        if k.shape[0] == 0:
            continue
        for j in range(hq):
            kh, vh, qh = k[:, j * pool.heads // hq], v[:, j * pool.heads // hq], q[i, j].double()
            s = kh @ qh / math.sqrt(D)
            w = torch.softmax(s, 0)
            ds = 2 * (D + 16) * U * float((kh.abs() @ qh.abs()).max()) / math.sqrt(D)
            want[i, j] = w @ vh
            n = k.shape[0]
            tol[i, j] = (2 * ds + 2.0 ** -16 + (n / 32 + 64) * U) * (w @ vh.abs()) * (1 + e) + want[i, j].abs() * (e + 4 * U) + SUB[
                "f16" if q.dtype == torch.float16 else "bf16"]
    return want, tol


def attend(pool, q, extra=0, ws="own"):
    qd = strided(q, extra)
    o = strided(torch.full_like(q, NAN), extra)
    pages = strided(pool.table, 3) if extra else pool.table.cuda()
    workspace = None
    if ws == "dirty":
        n = pool.cache.workspace_size(q.shape[1], pages)
        workspace = torch.full((n // 4,), NAN, device="cuda")
        workspace[:gb.ATTENTION_DECODE_COUNTER_BYTES // 4] = 0
    pool.cache.attend(qd, o, pages, pool.lens.cuda(), workspace=workspace)
    torch.cuda.synchronize()
    if extra:
        tail = o.as_strided((q.shape[0], extra), (o.stride(0), 1), q[0].numel())
        assert bool(tail.isnan().all()), "padding of o written"
    return o


LENS = {
    "one": [1], "short": [1, 2, 15, 16, 17, 31, 32, 33], "empty": [0, 5, 0, 200, 0], "tiles": [127, 128, 129, 255, 256, 257],
    "long": [5003], "mixed": [3000, 1, 0, 777, 64, 2049], "many": [(i * 37) % 301 for i in range(150)],
}


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("heads,group", [(1, 1), (2, 4), (3, 5), (1, 17), (2, 16), (1, 40)])
@pytest.mark.parametrize("head_dim,page,dtype,cache", [(128, 16, "bf16", "bf16"), (64, 48, "f16", "f16"), (128, 64, "f16", "fp8"),
                                                       (64, 16, "bf16", "fp8")])
def test_attend(lens, heads, group, head_dim, page, dtype, cache):
    pool = Pool(LENS[lens], heads, head_dim, page, dtype, cache, 3)
    pool.fill(4)
    q = rand(gen(5), len(LENS[lens]), heads * group, head_dim, std=1.5, dtype=dtype)
    want, tol = attend_want(pool, q)
    within(attend(pool, q), want, tol, f"{lens} {heads}x{group}")


@pytest.mark.parametrize("head_dim,dtype,cache", [(128, "f16", "f16"), (64, "bf16", "bf16"), (128, "bf16", "fp8"), (64, "f16", "fp8")])
def test_attend_strides_and_dirty_workspace(head_dim, dtype, cache):
    pool = Pool(LENS["mixed"], 2, head_dim, 32, dtype, cache, 6, width=100)
    pool.fill(7)
    q = rand(gen(8), 6, 6, head_dim, dtype=dtype)
    want, tol = attend_want(pool, q)
    first = attend(pool, q, extra=24, ws="dirty")
    within(first, want, tol, "strided")
    assert torch.equal(first, attend(pool, q, extra=8, ws="dirty")), "same inputs, other bits"


def test_attend_one_workspace_for_calls_of_any_sizes():
    # large and small calls in turn on one workspace: its counters are zero
    # after each, whatever the call before left behind them
    pools = [Pool(LENS[n], 2, d, 16, "bf16", "bf16", 70) for n, d in (("long", 128), ("mixed", 64), ("one", 128), ("many", 64))]
    need = 0
    for p in pools:
        p.fill(71)
        need = max(need, p.cache.workspace_size(6, p.table))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for p in pools + pools[::-1]:
        q = rand(gen(72), p.table.shape[0], 6, p.head_dim)
        want, tol = attend_want(p, q)
        o = torch.full_like(q, NAN, device="cuda")
        p.cache.attend(q.cuda(), o, p.table.cuda(), p.lens.cuda(), workspace=ws)
        torch.cuda.synchronize()
        within(o, want, tol, "one workspace")
        assert int(ws[:gb.ATTENTION_DECODE_COUNTER_BYTES].count_nonzero()) == 0


def test_attend_more_tiles_than_one_lookup():
    # 34 units a workgroup, so 34 tiles a wave, whose pages are looked up 32
    # tiles at a time; some pages missing
    pool = Pool([70000], 16, 64, 16, "bf16", "bf16", 41)
    pool.table[0, 1500::211] = -1
    g = torch.Generator(device="cuda").manual_seed(42)
    k, v = (torch.randn(70000, 16, 64, generator=g, device="cuda").bfloat16().cpu() for _ in range(2))
    pool.held = [(pool.put(pool.k, None, 0, k), pool.put(pool.v, None, 0, v))]
    q = rand(gen(43), 1, 16, 64, std=2.0)
    want, tol = attend_want(pool, q)
    within(attend(pool, q), want, tol, "two lookups")


def test_attend_missing_pages():
    # pages that do not exist at the front, in the middle, at the end, all of
    # them; entries past the cache and of the lowest value
    pool = Pool([100, 300, 64, 1000, 40], 2, 64, 16, "bf16", "bf16", 9)
    pool.fill(10)
    pool.table[0, 0] = -1
    pool.table[1, 5:9] = torch.tensor([pool.k.shape[0], -2 ** 31, 2 ** 31 - 1, -7], dtype=torch.int32)
    pool.table[2, 3] = -1
    pool.table[3, 2:60] = -1
    pool.table[4] = -1
    q = rand(gen(11), 5, 8, 64)
    want, tol = attend_want(pool, q)
    got = attend(pool, q)
    within(got, want, tol, "missing pages")
    assert bool((got[4] == 0).all())


def test_attend_lengths_outside_the_table():
    pool = Pool([40, 33, 48, 7], 1, 64, 16, "f16", "f16", 12, width=3)
    pool.fill(13)
    q = rand(gen(14), 4, 2, 64, dtype="f16")
    want, tol = attend_want(pool, q)
    pool.lens[1], pool.lens[2] = -5, 2 ** 31 - 1  # nothing, and the whole row of the table
    got = attend(pool, q)
    want[1], tol[1] = 0, 0
    within(got, want, tol, "lengths")


def test_attend_extreme_scores():
    # one key far above the others, scores far below and above zero, equal
    # keys, an infinite key
    pool = Pool([70, 70, 70, 70, 70], 1, 128, 16, "bf16", "bf16", 15)
    pool.fill(16)
    q = rand(gen(17), 5, 4, 128)
    for i, f in ((0, 40.0), (1, -40.0)):
        k = q[i, :1].float().mean(0).repeat(70, 1) * f + pool.held[i][0][:, 0].float()
        pool.held[i] = (pool.put(pool.k, None, i, k.to(torch.bfloat16).view(70, 1, 128)), pool.held[i][1])
    pool.held[2] = (pool.put(pool.k, None, 2, torch.ones(70, 1, 128, dtype=torch.bfloat16)), pool.held[2][1])
    big = pool.held[3][0].to(torch.bfloat16)
    big[33] *= 200
    pool.held[3] = (pool.put(pool.k, None, 3, big), pool.held[3][1])
    want, tol = attend_want(pool, q)
    within(attend(pool, q), want, tol, "extreme scores")
    k = pool.held[4][0].to(torch.bfloat16)
    k[5, 0, 7] = NAN
    pool.put(pool.k, None, 4, k)
    got = attend(pool, q)
    assert bool(got[4].isnan().all())  # a NaN key of the sequence itself
    within(got[:4], want[:4], tol[:4], "beside a NaN")


def test_attend_largest_f16_values_in_8_bits():
    # 65504 is held as 256 times the scale 2^8: 65536, beyond f16
    pool = Pool([200], 1, 64, 16, "f16", "fp8", 18)
    pool.fill(19)
    sign = (torch.arange(200) % 2 * 2 - 1).half()
    k, v = rand(gen(20), 200, 1, 64, dtype="f16"), rand(gen(21), 200, 1, 64, dtype="f16")
    k[:, 0, 0] = 65504 * sign
    v[:, 0, 5] = 65504 * sign
    v[::7, 0, 6] = -65504
    pool.held = [(pool.put(pool.k, pool.ks, 0, k), pool.put(pool.v, pool.vs, 0, v))]
    assert float(pool.held[0][0].max()) == 65536 == -float(pool.held[0][1].min())
    q = rand(gen(22), 1, 2, 64, dtype="f16")
    q[:, :, 0] = 2.0 ** -14
    want, tol = attend_want(pool, q)
    # values of a row whose scale is 2^8 are multiples of 2^-1: exact halved
    within(attend(pool, q), want, tol, "65504")


def test_attend_small_values_in_8_bits():
    # V of an fp8 cache far below f16's normal range times its scale
    pool = Pool([90], 1, 64, 16, "f16", "fp8", 18)
    pool.fill(19, std=2.0 ** -12)
    q = rand(gen(20), 1, 2, 64, dtype="f16")
    want, tol = attend_want(pool, q)
    # a value below f16's normal range is held to 2^-25, half its step there
    within(attend(pool, q), want, tol + 2.0 ** -24, "small values")


@pytest.mark.parametrize("head_dim,dtype,cache", [(128, "bf16", "bf16"), (64, "f16", "f16"), (64, "f16", "fp8"), (128, "bf16", "fp8")])
@pytest.mark.parametrize("new", [None, [3, 0, 40, 1], [0, 0, 0, 0], [100, 17, 64, 9]])
def test_append(head_dim, dtype, cache, new):
    lens = [100, 17, 64, 9]
    pool = Pool(lens, 3, head_dim, 16, dtype, cache, 21)
    before = [t.clone() if t is not None else None for t in (pool.k, pool.v, pool.ks, pool.vs)]
    counts = [1] * 4 if new is None else new
    g = gen(22)
    tokens = sum(counts) + (0 if new is None else 6)  # rows behind the last sequence
    rows = rand(g, tokens, 3 * head_dim * 3 + 8, dtype=dtype).cuda()
    k = rows[:, 8:8 + 3 * head_dim].view(tokens, 3, head_dim)
    v = rows[:, 8 + 6 * head_dim:].view(tokens, 3, head_dim)
    starts = None
    if new is not None:
        starts = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), dtype=torch.int32).cuda()
    pool.cache.append(k, v, pool.table.cuda(), pool.lens.cuda(), starts=starts)
    torch.cuda.synchronize()
    for x, cache_t, scale_t, was, was_s in ((k, pool.k, pool.ks, before[0], before[2]), (v, pool.v, pool.vs, before[1], before[3])):
        want, want_s = was.float().cpu(), was_s.cpu() if was_s is not None else None
        at = 0
        for i, n in enumerate(counts):
            for t in range(n):
                pos = lens[i] - n + t
                page, slot = int(pool.table[i, pos // 16]), pos % 16
                row = x[at + t].cpu()
                if pool.fp8:
                    row, s = pow2_quantise(row)
                    want_s[page, :, slot] = s.float()
                want[page, :, slot] = row.float()
            at += n
        assert torch.equal(cache_t.float().cpu().nan_to_num(nan=12345.0), want.nan_to_num(nan=12345.0))
        if pool.fp8:
            assert torch.equal(scale_t.cpu().nan_to_num(nan=12345.0), want_s.nan_to_num(nan=12345.0))


def test_append_scales_at_their_edges():
    # rows whose largest value is exactly 448 * 2^e, a step above and below,
    # zero, tiny, the largest finite, infinite, NaN
    tops = [448.0, 450.0, 446.0, 1.75, 1.7578125, 0.0, 2.0 ** -126, 2.0 ** -92 * 1.75, 3.3895e38, float("inf"), NAN, 2.0 ** -133]
    n = len(tops)
    pool = Pool([n], 1, 64, 16, "bf16", "fp8", 23)
    x = rand(gen(24), n, 1, 64)
    x = (x.float() / 8).clamp(-0.9, 0.9)
    for i, t in enumerate(tops):
        x[i] *= t if math.isfinite(t) else 1.0
        x[i, 0, 11] = -t
    x = x.to(torch.bfloat16)
    starts = torch.tensor([0, n], dtype=torch.int32).cuda()
    pool.cache.append(x.cuda(), x.cuda(), pool.table.cuda(), pool.lens.cuda(), starts=starts)
    torch.cuda.synchronize()
    q, s = pow2_quantise(x)
    page = int(pool.table[0, 0])
    assert torch.equal(pool.ks[page, 0, :n].cpu().nan_to_num(nan=9.0), s[:, 0].float().nan_to_num(nan=9.0))
    assert torch.equal(pool.k[page, 0, :n].float().cpu().nan_to_num(nan=9.0), q[:, 0].float().nan_to_num(nan=9.0))
    # a single infinity at the scale's edge does not spread to other rows
    assert bool(pool.vs[page, 0, 11].isfinite())


def test_append_to_no_page():
    # rows whose position is outside the sequence or the table, or whose page
    # does not exist, leave the cache as it was
    pool = Pool([40, 33, 20, 48], 2, 64, 16, "bf16", "bf16", 25, width=3)
    was = pool.k.clone().nan_to_num(nan=5.0)
    pool.lens[0] = 2  # three new rows in a sequence of two: the first has no position
    pool.lens[1] = -1
    pool.lens[2] = 2 ** 31 - 1  # past the table
    pool.table[3, 2] = pool.k.shape[0]  # the page of its last rows does not exist
    x = torch.ones(12, 2, 64, dtype=torch.bfloat16, device="cuda")
    starts = torch.tensor([0, 3, 6, 9, 12], dtype=torch.int32).cuda()
    pool.cache.append(x, x, pool.table.cuda(), pool.lens.cuda(), starts=starts)
    torch.cuda.synchronize()
    page = int(pool.table[0, 0])
    was[page, :, :2] = 1
    assert torch.equal(pool.k.nan_to_num(nan=5.0), was)


def test_append_many_sequences():
    # more sequences than a wave's lanes, with empty ones between
    counts = [(i * 5) % 4 for i in range(200)]
    lens = [c + i % 7 for i, c in enumerate(counts)]
    pool = Pool(lens, 1, 64, 16, "f16", "f16", 26)
    x = rand(gen(27), sum(counts), 1, 64, dtype="f16")
    starts = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32)
    pool.cache.append(x.cuda(), -x.cuda(), pool.table.cuda(), pool.lens.cuda(), starts=starts.cuda())
    torch.cuda.synchronize()
    k, v = pool.k.cpu(), pool.v.cpu()
    for i, n in enumerate(counts):
        for t in range(n):
            row, slot = x[int(starts[i]) + t, 0], lens[i] - n + t
            page = int(pool.table[i, 0])
            assert torch.equal(k[page, 0, slot], row) and torch.equal(v[page, 0, slot], -row)
    assert int((~k.isnan().any(-1)).sum()) == sum(counts)


# ---- beyond 32 bits -------------------------------------------------------------------

def test_cache_of_more_than_4_gib():
    # the sequence's pages lie at the end of a cache whose byte offsets pass
    # 2^32 (and element offsets 2^31)
    heads, page, D = 8, 64, 128
    pages = (5 << 30) // (heads * page * D * 2)
    k = torch.zeros(pages, heads, page, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    cache = gb.PagedCache(k, v)
    n = 150
    table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    g = gen(28)
    x, y = rand(g, n, heads, D), rand(g, n, heads, D)
    cache.append(x.cuda(), y.cuda(), table, lens, starts=torch.tensor([0, n], dtype=torch.int32, device="cuda"))
    q = rand(g, 1, heads, D)
    o = torch.empty_like(q, device="cuda")
    cache.attend(q.cuda(), o, table, lens)
    torch.cuda.synchronize()
    assert torch.equal(k[pages - 1].transpose(0, 1).cpu(), x[:64]) and torch.equal(v[pages - 2, :, :22].transpose(0, 1).cpu(), y[128:])
    pool = type("P", (), {})()
    pool.held, pool.table, pool.page, pool.heads, pool.k = [(x.double(), y.double())], table.cpu(), page, heads, k
    want, tol = attend_want(pool, q)
    within(o, want, tol, "far pages")


# ---- together: one decode step, eager and captured -------------------------------------

class Step:
    """Norm, projection with adapters, append, attention, output projection
    onto the residual: the library's calls as a decode step makes them."""

    def __init__(self, cache_fmt):
        self.B, self.hq, self.hkv, self.D, self.K = 6, 8, 2, 64, 512
        g = gen(30)
        self.N = (self.hq + 2 * self.hkv) * self.D
        B, K, N = self.B, self.K, self.N
        self.w_norm = (1 + 0.1 * torch.randn(K, generator=g)).bfloat16().cuda()
        self.w_qkv, self.b_qkv = rand(g, N, K, std=K ** -0.5).cuda(), rand(g, N, std=0.1).cuda()
        self.w_out, self.b_out = rand(g, K, self.hq * self.D, std=(self.hq * self.D) ** -0.5).cuda(), rand(g, K, std=0.1).cuda()
        self.la, self.lb = rand(g, 3, 16, K, std=K ** -0.5).cuda(), rand(g, 3, N, 16, std=0.25).cuda()
        self.ids = torch.tensor([0, -1, 2, 1, 0, 2], dtype=torch.int32).cuda()
        self.pool = Pool([90, 5, 33, 0, 16, 64], self.hkv, self.D, 16, "bf16", cache_fmt, 31, width=12, spare=60)
        free = sorted(set(range(self.pool.k.shape[0])) - set(self.pool.table.flatten().tolist()))
        for i in range(B):  # pages for the tokens to come
            for p in range(12):
                if int(self.pool.table[i, p]) < 0 and free:
                    self.pool.table[i, p] = free.pop()
        self.pool.fill(32)
        self.pages = self.pool.table.cuda()
        self.lens = self.pool.lens.cuda()
        e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.x, self.res = rand(g, B, K).cuda(), rand(g, B, K).cuda()
        self.h, self.y, self.delta, self.qkv, self.o, self.out = e(B, K), e(B, K), e(B, N), e(B, N), e(B, self.hq, self.D), e(B, K)
        self.ws = torch.zeros(self.pool.cache.workspace_size(self.hq, self.pages), dtype=torch.uint8, device="cuda")
        self.lws = torch.empty(gb.lora_workspace_size(B, N, K, 16, 3), dtype=torch.uint8, device="cuda")
        self.p_qkv = gb.Plan(B, N, K, "bf16", "bf16", "row", "col", "bias")
        self.p_out = gb.Plan(B, K, self.hq * self.D, "bf16", "bf16", "row", "col", "bias")

    def run(self, stream=None):
        B, hq, hkv, D = self.B, self.hq, self.hkv, self.D
        gb.rmsnorm(self.x, self.w_norm, self.y, residual=self.res, residual_out=self.h, stream=stream)
        gb.lora(self.y, self.la, self.lb, self.ids, self.delta, workspace=self.lws, stream=stream)
        self.p_qkv.run(self.y, self.w_qkv, self.b_qkv, self.qkv, residual=self.delta, stream=stream)
        rows = self.qkv.view(B, hq + 2 * hkv, D)
        self.pool.cache.append(rows[:, hq:hq + hkv], rows[:, hq + hkv:], self.pages, self.lens, stream=stream)
        self.pool.cache.attend(rows[:, :hq], self.o, self.pages, self.lens, workspace=self.ws, stream=stream)
        self.p_out.run(self.o.view(B, hq * D), self.w_out, self.b_out, self.out, residual=self.h, stream=stream)

    def reset(self):
        self.lens.copy_(self.pool.lens)
        self.x.copy_(self.x0)
        self.res.copy_(self.r0)

    def step(self, call):
        """One step of all sequences: a new token each, its output the next
        step's input."""
        self.lens.add_(1)
        call()
        return self.out.clone()


@pytest.mark.parametrize("cache_fmt", ["bf16", "fp8"])
def test_decode_step_together_and_captured(cache_fmt):
    st = Step(cache_fmt)
    st.x0, st.r0 = st.x.clone(), st.res.clone()
    steps, eager, o_eager = 5, [], []
    for t in range(steps):
        eager.append(st.step(st.run))
        o_eager.append(st.o.clone())
        if t == 0:
            # the step against 64 bits, operator by operator on its own inputs
            h, y = rms_want(st.x.cpu(), st.res.cpu(), st.w_norm.cpu(), 1e-6)
            within(st.h, h, h.abs() * (2.0 ** -8 + 2 * U), "h")
            within(st.y, y, y.abs() * (2.0 ** -8 + 64 * U) * (1 + 2.0 ** -8), "y")
            lora_check(st.y.cpu(), st.la.cpu(), st.lb.cpu(), st.ids.cpu(), None, None, st.delta, "bf16", "delta")
            rows = st.qkv.view(st.B, -1, st.D).cpu()
            for i, n in enumerate(st.pool.lens.tolist()):
                new = []
                for x, held in zip((rows[i, st.hq:st.hq + st.hkv], rows[i, st.hq + st.hkv:]), st.pool.held[i]):
                    val = x.double()
                    if st.pool.fp8:
                        q, s = pow2_quantise(x)
                        val = q * s[..., None]
                    new.append(torch.cat([held, val[None]]))
                st.pool.held[i] = tuple(new)
            want, tol = attend_want(st.pool, rows[:, :st.hq])
            within(st.o, want, tol, "attention")
        st.x.copy_(st.out)
    # the same steps on a side stream
    st.reset()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for t in range(steps):
            assert torch.equal(st.step(st.run), eager[t]), f"side stream, step {t}"
            st.x.copy_(st.out)
    torch.cuda.current_stream().wait_stream(side)
    # captured once and replayed, with eager work of the program between
    st.reset()
    graph = torch.cuda.CUDAGraph()
    st.lens.add_(1)
    st.run()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        st.run()
    st.reset()
    for t in range(steps):
        assert torch.equal(st.step(graph.replay), eager[t]), f"replay {t}"
        assert torch.equal(st.o, o_eager[t])
        st.x.copy_(st.out)
        torch.cuda.synchronize()
        torch.empty(1 << 20, device="cuda").normal_()


def test_two_streams_at_once():
    # independent calls on two streams, each with a workspace of its own
    pools = [Pool([3000, 200, 1], 2, 128, 16, "bf16", "bf16", 40 + i) for i in range(2)]
    qs, os_, wss, tabs, lens = [], [], [], [], []
    for i, p in enumerate(pools):
        p.fill(50 + i)
        qs.append(rand(gen(60 + i), 3, 8, 128))
        tabs.append(p.table.cuda())
        lens.append(p.lens.cuda())
        os_.append(torch.empty(3, 8, 128, dtype=torch.bfloat16, device="cuda"))
        wss.append(torch.zeros(p.cache.workspace_size(8, tabs[i]), dtype=torch.uint8, device="cuda"))
    qd = [q.cuda() for q in qs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            pools[i].cache.attend(qd[i], os_[i], tabs[i], lens[i], workspace=wss[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        want, tol = attend_want(pools[i], qs[i])
        within(os_[i], want, tol, f"stream {i}")


# ---- refusals of the binding ------------------------------------------------------------

def test_binding_refusals():
    d = dict(dtype=torch.bfloat16, device="cuda")
    x, w, y = torch.zeros(4, 64, **d), torch.ones(64, **d), torch.zeros(4, 64, **d)
    for bad in (dict(x=x.float()), dict(x=x.cpu()), dict(x=x.t()), dict(weight=w[:32]), dict(weight=w.half()), dict(y=y[:3]),
                dict(y=y.half()), dict(residual=x[:, :32]), dict(residual_out=x.half()), dict(x=x[0]),
                dict(y_scale=torch.zeros(4, device="cuda")), dict(y=y.to(torch.float8_e4m3fn)), dict(eps=-1.0)):
        with pytest.raises((ValueError, gb.GemmEpiError)):
            gb.rmsnorm(**{**dict(x=x, weight=w, y=y), **bad})
    a, b, i = torch.zeros(2, 8, 64, **d), torch.zeros(2, 64, 8, **d), torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (dict(a=a[0]), dict(a=a.half()), dict(a=a[:, :, :32]), dict(b=b[:1]), dict(ids=i.long()), dict(ids=i[:3]), dict(c=y[:, :32]),
                dict(scale=torch.zeros(3, device="cuda")), dict(residual=x.half()), dict(x=x[:, ::2]), dict(ids=i.cpu()),
                dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), dict(workspace=torch.empty(1 << 20, dtype=torch.uint8))):
        with pytest.raises((ValueError, gb.GemmEpiError)):
            gb.lora(**{**dict(x=x, a=a, b=b, ids=i, c=y), **bad})
    k = torch.zeros(3, 2, 16, 64, **d)
    k8 = k.to(torch.float8_e4m3fn)
    s8 = torch.zeros(3, 2, 16, device="cuda")
    for args in ((k[0], k[0]), (k, k[:2]), (k, k.half()), (k.float(), k.float()), (k, k, s8, s8), (k8, k8), (k8, k8, s8), (k8, k8, s8, s8[:2]),
                 (k.transpose(1, 2), k), (k.cpu(), k.cpu())):
        with pytest.raises(ValueError):
            gb.PagedCache(*args)
    cache = gb.PagedCache(k, k.clone())
    pages, lens = torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.ones(4, dtype=torch.int32, device="cuda")
    kv = torch.zeros(4, 2, 64, **d)
    for bad in (dict(k=kv.half(), v=kv.half()), dict(v=kv[:3]), dict(pages=pages.long()), dict(pages=pages[0]), dict(lens=lens[:3]),
                dict(lens=lens.long()), dict(starts=lens), dict(k=kv[:3], v=kv[:3]), dict(k=kv[:, :1], v=kv[:, :1])):
        with pytest.raises((ValueError, gb.GemmEpiError)):
            cache.append(**{**dict(k=kv, v=kv, pages=pages, lens=lens), **bad})
    q = torch.zeros(4, 4, 64, **d)
    for bad in (dict(q=q.half(), o=q.half()), dict(q=q[:, :3], o=q[:, :3]), dict(o=q[:3]), dict(q=q[0]), dict(o=q.float()),
                dict(workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))):
        with pytest.raises((ValueError, gb.GemmEpiError)):
            cache.attend(**{**dict(q=q, o=q.clone(), pages=pages, lens=lens), **bad})
    torch.cuda.synchronize()
