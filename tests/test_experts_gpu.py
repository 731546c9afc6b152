"""The experts' feed-forward and the 8-bit products on the GPU against their
definitions in 64 bits, at the sizes, masks, strides and values where they can
go wrong.

Tolerances.  An output in a 16-bit format is off by its rounding, at most half
a step (eps / 2 of the value; half the smallest subnormal near zero), plus what
the fp32 arithmetic before it loses, bounded term by term beside each
operator.  Whole numbers are equal."""
import math

import pytest
import torch

from epilogue_gemm_amd import binding as gb

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SUB = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}  # half the smallest subnormal
U = 2.0 ** -24  # half a step of fp32
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gb.load_library()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rand(g, *shape, std=1.0, dtype="f32"):
    return (torch.randn(shape, generator=g) * std).to(DT[dtype])


def codes(g, *shape):
    return torch.randint(-128, 128, shape, generator=g, dtype=torch.int8)


def strided(t, extra):
    """The rows of a 2-d tensor on the GPU, `extra` elements between them (NaN,
    or for integers the lowest value)."""
    pad = NAN if t.is_floating_point() else torch.iinfo(t.dtype).min
    buf = torch.full((t.shape[0], t.shape[1] + extra), pad, dtype=t.dtype, device="cuda")
    buf[:, :t.shape[1]] = t.cuda()
    return buf[:, :t.shape[1]]


def blank(rows, cols, dtype, extra=0):
    """Rows of NaN to be written, and the buffer they stand in."""
    buf = torch.full((rows, cols + extra), NAN, dtype=DT[dtype], device="cuda")
    return buf[:, :cols], buf


def within(got, want, tol, what):
    """|got - want| <= tol elementwise (fp64), and equally non-finite."""
    got, want = got.detach().cpu().double(), want.double()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), f"{what}: other infinities"
    over = ((got - want).abs() - tol)[fine]
    assert over.numel() == 0 or float(over.max()) <= 0, f"{what}: {int((over > 0).sum())} outside, worst by {float(over.max()):.3g}"


# ---- rows in 8-bit integers ----------------------------------------------------

def quantised(x):
    """Codes and scales by the definition: fp32 scales, fp32 quotients (64-bit
    ones rounded to 32 are these), to the nearest integer, ties to even."""
    most = x.float().abs().amax(1)
    s = (most.double() / 127).float().clamp(min=2.0 ** -100)
    bad = ~torch.isfinite(x.float()).all(1)
    q = (x.double() / s.double()[:, None]).float().round()
    s = torch.where(bad, NAN, s)
    return torch.where(bad[:, None], 0.0, q).to(torch.int8), s


def same_scale(got, want):
    return torch.equal(got.cpu().view(torch.int32)[~want.isnan()], want.view(torch.int32)[~want.isnan()]) and \
        torch.equal(got.cpu().isnan(), want.isnan())


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (70, 8), (2, 64), (5, 130), (9, 256), (33, 512), (17, 1000),
                                       (3, 1024), (1200, 520), (4, 4096), (1030, 2055), (5, 5120), (3, 8192),
                                       (2, 8200), (2, 16384), (2, 16391), (1, 32768), (2, 32769), (1, 70001)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_quantise(rows, cols, dtype):
    x = rand(gen(rows * 100003 + cols), rows, cols, std=3.0, dtype=dtype)
    q, s = quantised(x)
    for extra in (0, 8, 3):
        buf = torch.full((rows, cols + extra), 99, dtype=torch.int8, device="cuda")
        scale = torch.full((rows + 1,), -1.0, device="cuda")
        gb.quantise_i8(strided(x, extra), buf[:, :cols], scale[:rows])
        assert torch.equal(buf[:, :cols].cpu(), q) and same_scale(scale[:rows], s)
        assert bool((buf[:, cols:] == 99).all()) and float(scale[rows]) == -1.0, "written past the rows"


def test_quantise_every_value_beside_a_border():
    # all finite values of a format as codes of one scale: multiples of a half
    # of it among them, in a row of each power of two for the largest
    for dtype, bits in (("f16", torch.arange(0, 0x7c00)), ("bf16", torch.arange(0x3000, 0x5000))):
        v = bits.to(torch.int16).view(DT[dtype]).float()
        for top in (127.0, 254.0, 1.0, 3.0, 100.0):
            x = torch.where(v <= top, v, 0.0)
            x = torch.cat([x, torch.tensor([top])])[None].to(DT[dtype])
            q, s = quantised(x)
            y, scale = torch.empty(x.shape, dtype=torch.int8, device="cuda"), torch.empty(1, device="cuda")
            gb.quantise_i8(x.cuda(), y, scale)
            assert torch.equal(y.cpu(), q) and same_scale(scale, s), (dtype, top)


@pytest.mark.parametrize("cols", [5, 128, 1000, 4096, 33000])
def test_quantise_special_rows(cols):
    x = rand(gen(cols), 8, cols, dtype="bf16")
    x[0] = 0
    x[1, cols // 2] = INF
    x[2, cols - 1] = -INF
    x[3, 0] = NAN
    x[4] = 2.0 ** -133  # (a subnormal; below the smallest scale)
    x[5] = 3.3895313892515355e38  # the largest
    x[6] = -x[6].abs()
    q, s = quantised(x)
    y, scale = torch.empty(8, cols, dtype=torch.int8, device="cuda"), torch.empty(8, device="cuda")
    gb.quantise_i8(x.cuda(), y, scale)
    assert torch.equal(y.cpu(), q) and same_scale(scale, s)
    assert scale[1:4].isnan().all() and scale[0] == 2.0 ** -100 and not y[0].any()


# Aligned rows of more than 32 MiB in each of the row kernels (16 lanes a row,
# one to four pieces a thread), and more rows than the 2^20 workgroups of a grid
# take at once.
@pytest.mark.parametrize("rows,cols", [(140000, 128), (35000, 512), (4200, 4096), (1030, 16384), (520, 32768),
                                       ((1 << 20) + 77, 136), ((1 << 20) + 3, 1032), ((1 << 20) + 5, 131), ((1 << 24) + 5, 8)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_quantise_many_rows(rows, cols, dtype):
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    x = torch.empty(rows, cols, dtype=DT[dtype], device="cuda").normal_(generator=g)
    x[torch.tensor([1, rows // 2, rows - 2]), torch.tensor([0, cols // 2, cols - 1])] = torch.tensor([INF, NAN, -INF], dtype=DT[dtype], device="cuda")
    y, s = torch.full((rows, cols), 99, dtype=torch.int8, device="cuda"), torch.full((rows,), -1.0, device="cuda")
    gb.quantise_i8(x, y, s)
    step = max(1, (1 << 27) // cols)
    for i in range(0, rows, step):
        q, sw = quantised(x[i:i + step])
        assert torch.equal(y[i:i + step], q) and same_scale(s[i:i + step], sw.cpu()), i


# ---- products -------------------------------------------------------------------

def act(z, epilogue):
    if epilogue.endswith("relu"):
        return z.clamp(min=0)
    if epilogue.endswith("silu"):
        return z * torch.sigmoid(z)
    if epilogue.endswith("gelu"):
        return z * torch.sigmoid(1.5957691216 * (z + 0.044715 * z ** 3))
    return z


def pre(x, w, xs, ws, bias):
    """z = x w^T (scaled) + bias in 64 bits, and what fp32 may lose of it: a sum
    of K products one half step of sum |x w| each, at most (exact for integers,
    whose conversion and two factors lose three); the bias half a step more."""
    z, a = x.double() @ w.double().T, x.double().abs() @ w.double().abs().T
    if xs is not None:
        f = xs.double()[:, None] * ws.double()[None]
        z, lost = z * f, 3 * U * (z * f).abs()
    else:
        lost = x.shape[1] * U * a
    if bias is not None:
        z = z + bias.double()[None]
    return z, lost + U * z.abs()


def post(z, lost, epilogue, dtype, up=None, residual=None):
    """The epilogue, and what it may be off by: the activations' slopes are at
    most 1.13; their exp, quotient and products lose below 2^-20 of the value,
    and of z where exp's argument does (|z| e^-|z| of it)."""
    y = act(z, epilogue)
    t = 1.13 * lost + 2.0 ** -20 * y.abs() + 2.0 ** -22 * z.abs().clamp(max=30) * (epilogue != "none")
    if up is not None:
        u, ul = up
        y, t = y * u, t * (u.abs() + ul) + ul * y.abs() + U * (y * u).abs()
    if residual is not None:
        y = y + residual.double()
        t = t + U * y.abs()
    e = torch.finfo(DT[dtype]).eps / 2
    return y, t * (1 + e) + e * y.abs() + SUB[dtype]


I8_SIZES = [(1, 1, 16), (1, 64, 64), (3, 33, 112), (16, 16, 128), (17, 130, 144), (31, 100, 4096), (64, 65, 272),
            (33, 256, 1040), (100, 77, 512), (129, 200, 208), (200, 513, 96), (257, 260, 640), (500, 300, 2064),
            (5, 1000, 131056)]


@pytest.mark.parametrize("M,N,K", I8_SIZES)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_i8_gemm(M, N, K, dtype):
    g = gen(M * 1009 + N * 31 + K)
    a, b = codes(g, M, K), codes(g, N, K)
    xs, ws = torch.rand(M, generator=g) * 2.0 ** -8 + 2.0 ** -10, (torch.rand(N, generator=g) + 0.1) / K ** 0.5 * 2.0 ** -5
    bias, r = rand(g, N, dtype=dtype), rand(g, M, N, dtype=dtype)
    for epilogue, extra, res in (("none", 0, False), ("bias", 0, True), ("relu", 3, True), ("bias_gelu", 0, False),
                                 ("silu", 8, False), ("bias_silu", 1, True), ("bias_relu", 0, False)):
        bi = bias if epilogue.startswith("bias") else None
        z, lost = pre(a, b, xs, ws, bi)
        want, tol = post(z, lost, epilogue, dtype, residual=r if res else None)
        c, buf = blank(M, N, dtype, extra)
        gb.i8_gemm(strided(a, 16 * (extra > 0)), xs.cuda(), strided(b, 32 * (extra > 1)), ws.cuda(), c,
                   bias=None if bi is None else bi.cuda(), residual=strided(r, extra) if res else None, epilogue=epilogue)
        within(c, want, tol, f"{M}x{N}x{K} {epilogue}")
        assert bool(buf[:, N:].isnan().all()), "written past the rows"


def test_i8_gemm_in_place_and_extremes():
    g = gen(5)
    M, N, K = 70, 90, 256
    a, b, r = codes(g, M, K), codes(g, N, K), rand(g, M, N, dtype="bf16")
    one = torch.full((90,), 2.0 ** -10)
    z, lost = pre(a, b, one[:M], one, None)
    want, tol = post(z, lost, "none", "bf16", residual=r)
    c = r.cuda()
    gb.i8_gemm(a.cuda(), one[:M].cuda(), b.cuda(), one.cuda(), c, residual=c)
    within(c, want, tol, "in place")
    # the largest sum there can be, exact: (2^17 - 16) 2^14 = 2^31 - 2^18
    K = 131056
    a, b = torch.full((2, K), -128, dtype=torch.int8), torch.full((3, K), -128, dtype=torch.int8)
    b[1] = 127
    ones = torch.tensor([1.0, NAN, INF])
    c, _ = blank(2, 3, "bf16")
    gb.i8_gemm(a.cuda(), ones[:2].cuda(), b.cuda(), ones[[0, 0, 2]].cuda(), c)
    assert c[0].tolist() == [float(torch.tensor(2.0 ** 31 - 2 ** 18, dtype=torch.bfloat16)),
                             float(torch.tensor(-127 * 128.0 * K, dtype=torch.bfloat16)), INF]
    assert bool(c[1].isnan().all())  # a row whose scale is NaN


def grouping(g, counts, away=0):
    """Offsets and a random order of the entries of groups of these sizes."""
    total = sum(counts) + away
    perm = torch.randperm(total, generator=g).int()
    off = [0]
    order = torch.full((total,), -1, dtype=torch.int32)
    for n in counts:
        order[off[-1]:off[-1] + n] = perm[off[-1]:off[-1] + n].sort().values
        off.append(off[-1] + n)
    return torch.tensor(off, dtype=torch.int32), order


def grouped_want(x, w, xs, ws, bias, off, order, per, gather, scatter, gated, epilogue, out, N):
    rows = order.numel()
    want, tol = torch.full((rows, N), NAN, dtype=torch.float64), torch.zeros(rows, N, dtype=torch.float64)
    for e in range(len(off) - 1):
        i = torch.arange(int(off[e]), int(off[e + 1]))
        if not len(i):
            continue
        q = order[i].long()
        xr = q // per if gather else i
        xe, se = x[xr], None if xs is None else xs[xr]
        b = None if bias is None else bias[e]
        z, lost = pre(xe, w[e], se, None if ws is None else ws[e], b)
        up = (z[:, N:], lost[:, N:]) if gated else None
        y, t = post(z[:, :N], lost[:, :N], epilogue, out, up)
        to = q if scatter else i
        want[to], tol[to] = y, t
    return want, tol


def grouped_check(counts, N, K, dtype, away=0, per=1, gather=True, scatter=False, gated=False, epilogue="none",
                  extra=0, out=None, seed=0):
    g = gen(seed + sum(counts) * 7 + N * 13 + K)
    total, E = sum(counts) + away, len(counts)
    assert total % per == 0
    out = out or ("bf16" if dtype == "i8" else dtype)
    off, order = grouping(g, counts, away)
    cols = 2 * N if gated else N
    nx = total // per if gather else total
    xs = ws = None
    if dtype == "i8":
        x, w = codes(g, nx, K), codes(g, E, cols, K)
        xs, ws = torch.rand(nx, generator=g) * 2.0 ** -7, torch.rand(E, cols, generator=g) / K ** 0.5 * 2.0 ** -5
    else:
        x, w = rand(g, nx, K, dtype=dtype), rand(g, E, cols, K, std=K ** -0.5, dtype=dtype)
    bias = rand(g, E, cols, dtype=out) if epilogue.startswith("bias") else None
    want, tol = grouped_want(x, w, xs, ws, bias, off, order, per, gather, scatter, gated, epilogue, out, N)
    c, buf = blank(total, N, out, extra)
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    gb.grouped_gemm(strided(x, 16 * (extra > 0)), dev(w), c, dev(off), dev(order) if gather or scatter else None, per=per,
                    gather=gather, scatter=scatter, gated=gated, bias=dev(bias), epilogue=epilogue, x_scale=dev(xs),
                    w_scale=dev(ws))
    within(c, want, tol, f"{counts[:8]} {N}x{K} {dtype} gather {gather} scatter {scatter} gated {gated} {epilogue}")
    assert bool(buf[:, N:].isnan().all()), "written past the rows"


COUNTS = [[1], [0, 5, 0], [16], [17, 1, 0, 30], [64, 64], [3] * 70, [0] * 100 + [2, 0, 7], [65, 0, 127, 130],
          [1] * 200 + [40], [300, 5]]


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}g{sum(c)}")
@pytest.mark.parametrize("dtype", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("gated", [False, True])
def test_grouped_gemm(counts, dtype, gated):
    epilogue = "silu" if gated else "none"
    grouped_check(counts, 80, 208, dtype, gated=gated, epilogue=epilogue)
    grouped_check(counts, 33, 16 if dtype == "i8" else 8, dtype, gather=False, scatter=True, gated=gated,
                  epilogue="bias_" + epilogue if gated else "bias", extra=3)
    grouped_check(counts, 64, 128, dtype, away=5, gather=False, gated=gated, epilogue="relu")
    grouped_check(counts, 100, 144, dtype, away=(3 - sum(counts)) % 3 + 3, per=3, scatter=True, gated=gated,
                  epilogue=epilogue, extra=8)


# counts around the tiles' heights, columns around their widths, lengths of K
# around their stages
@pytest.mark.parametrize("counts,N,K", [
    ([256, 255, 1], 256, 1024), ([257, 512, 300], 512, 192), ([700, 900], 384, 320), ([128] * 8, 130, 64),
    ([120, 8, 64, 33], 1000, 2048), ([4, 2, 9, 0, 1, 16, 15, 17], 515, 4096), ([40, 32, 31, 20], 260, 1000),
    ([2000], 300, 136), ([1], 2000, 5000), ([600, 650, 0, 700, 640], 513, 72),
])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "i8"])
def test_grouped_gemm_sizes(counts, N, K, dtype):
    K = (K + 15) // 16 * 16
    away = -sum(counts) % 4
    grouped_check(counts, N, K, dtype, away=away, per=4, gated=True, epilogue="silu")
    grouped_check(counts, N, K, dtype, away=away, gather=False, scatter=True, epilogue="bias_gelu")
    grouped_check(counts, N, K, dtype, away=away, gather=False, out="f16" if dtype == "i8" else None)


# One case at least for each kernel and way past the caches that the sizes
# choose, computed in 64 bits on the GPU: rows of K in bytes, off the stages.
KERNELS = [
    ("stream", [1, 0, 3, 17, 2, 0, 0, 1, 4, 0, 1, 0], 130, 4112), ("stream_past", [3, 0, 1, 2] * 16, 520, 4112),
    ("64x64_two", [40, 3, 0, 33, 65], 700, 272), ("64x64_two_past", [10, 0, 25, 4] * 16, 1040, 2064),
    ("64x64_four", [40, 3, 0, 33, 65], 300, 2064), ("64x64_four_past", [20, 17, 0, 64, 30] * 8, 850, 4112),
    ("128x128", [60, 130, 1, 89] * 5, 1700, 1040), ("128x128_past", [60, 130, 1, 89] * 5, 1700, 4016),
    ("128x128_four", [1100, 300], 2300, 4112),
    ("256x256", [1500, 700, 100, 260, 1], 2900, 2064), ("256x256_past", [300, 256, 511, 120, 129, 384, 1, 600], 4100, 4112),
]


@pytest.mark.parametrize("name,counts,cols,row", KERNELS, ids=[k[0] for k in KERNELS])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("gated", [False, True])
def test_grouped_gemm_every_kernel(name, counts, cols, row, dtype, gated):
    g = torch.Generator(device="cuda").manual_seed(len(name) + row)
    per, away = 2, 2 + sum(counts) % 2
    out, K, N, E = "bf16" if dtype == "i8" else dtype, row // (1 if dtype == "i8" else 2), cols // (2 if gated else 1), len(counts)
    total, cols = sum(counts) + away, N * (2 if gated else 1)
    off, order = (t.cuda() for t in grouping(gen(row), counts, away))
    xs = ws = None
    if dtype == "i8":
        x = torch.randint(-128, 128, (total // per, K), generator=g, dtype=torch.int8, device="cuda")
        w = torch.randint(-128, 128, (E, cols, K), generator=g, dtype=torch.int8, device="cuda")
        xs = torch.rand(total // per, generator=g, device="cuda") * 2.0 ** -7
        ws = torch.rand(E, cols, generator=g, device="cuda") / K ** 0.5 * 2.0 ** -5
    else:
        x = torch.randn(total // per, K, generator=g, device="cuda").to(DT[dtype])
        w = (torch.randn(E, cols, K, generator=g, device="cuda") * K ** -0.5).to(DT[dtype])
    bias = torch.randn(E, cols, generator=g, device="cuda").to(DT[out])
    epilogue = "bias_silu" if gated else "bias"
    c, _ = blank(total, N, out)
    gb.grouped_gemm(x, w, c, off, order, per=per, gather=True, scatter=True, gated=gated, bias=bias, epilogue=epilogue,
                    x_scale=xs, w_scale=ws)
    for e, n in enumerate(counts):
        q = order[int(off[e]):int(off[e]) + n].long()
        if not n:
            continue
        z, lost = pre(x[q // per], w[e], None if xs is None else xs[q // per], None if ws is None else ws[e], bias[e])
        y, t = post(z[:, :N], lost[:, :N], epilogue, out, (z[:, N:], lost[:, N:]) if gated else None)
        within(c[q], y.cpu(), t.cpu(), f"{name} group {e}")
        c[q] = NAN
    assert bool(c.isnan().all()), "rows of no entry written"


@pytest.mark.parametrize("M,N,row", [(5, 700, 4112), (40, 700, 4112), (1500, 1800, 4112), (2300, 2100, 1040), (4100, 2900, 2064), (3000, 600, 144)])
def test_i8_gemm_every_kernel(M, N, row):
    g = torch.Generator(device="cuda").manual_seed(M)
    a = torch.randint(-128, 128, (M, row), generator=g, dtype=torch.int8, device="cuda")
    b = torch.randint(-128, 128, (N, row), generator=g, dtype=torch.int8, device="cuda")
    xs, ws = torch.rand(M, generator=g, device="cuda") * 2.0 ** -7, torch.rand(N, generator=g, device="cuda") / row ** 0.5 * 2.0 ** -5
    r, bias = torch.randn(M, N, generator=g, device="cuda").half(), torch.randn(N, generator=g, device="cuda").half()
    z, lost = pre(a, b, xs, ws, bias)
    want, tol = post(z, lost, "bias_gelu", "f16", residual=r)
    gb.i8_gemm(a, xs, b, ws, r, bias=bias, residual=r, epilogue="bias_gelu")  # in place
    within(r, want.cpu(), tol.cpu(), f"{M}x{N}x{row}")


@pytest.mark.parametrize("gated,epilogue", [(g, e) for g in (False, True) for e in gb.EPILOGUES])
def test_grouped_gemm_epilogues(gated, epilogue):
    for dtype in ("bf16", "i8"):
        grouped_check([20, 0, 50], 72, 96, dtype, gated=gated, epilogue=epilogue)


def test_grouped_gemm_of_any_offsets_and_order():
    """Offsets that do not ascend and orders outside the rows: what is named
    is computed, nothing else is read or written."""
    g = gen(3)
    rows, N, K = 40, 64, 64
    x, w = rand(g, rows, K, dtype="bf16"), rand(g, 4, N, K, std=0.125, dtype="bf16")
    off = torch.tensor([-5, 10, 4, 1 << 30, 7], dtype=torch.int32)  # [0, 10), none, [4, 40), none
    order = torch.arange(rows, dtype=torch.int32)
    order[[1, 6, 20]] = torch.tensor([-1, rows, -(1 << 31)], dtype=torch.int32)
    order[30:] = -7
    c, buf = blank(rows + 1, N, "bf16")
    gb.grouped_gemm(x.cuda(), w.cuda(), c[:rows], off.cuda(), order.cuda(), gather=True, scatter=True)
    got = c.cpu().double()
    assert bool(got[rows].isnan().all())
    none = [1, 6, 20] + list(range(30, 40))
    assert bool(got[none].isnan().all())
    for r in range(30):
        if r in none:
            continue
        either = [x[r].double() @ w[e].double().T for e in ([0] if r < 4 else [0, 2] if r < 10 else [2])]
        # (rows of two groups: each column is one of theirs)
        assert float(torch.stack([(got[r] - y).abs() for y in either]).amin(0).max()) < 0.05, r


# Offsets that do not ascend, whose ranges as written would overlap in more tiles
# than the rows and groups of ascending ones have: a case for each of the kernels.
OVERLAPS = [("stream", 64, 16, 300, 4112), ("64x64_two", 1024, 8, 256, 272), ("64x64_four", 400, 16, 128, 2064),
            ("128x128", 3200, 40, 1000, 1040), ("128x128_four", 1280, 20, 1100, 4112), ("256x256", 2560, 10, 4700, 2064),
            ("many_groups", 700, 1000, 40, 144), ("many_groups_stream", 500, 300, 40, 4112)]


@pytest.mark.parametrize("name,rows,groups,cols,row", OVERLAPS, ids=[k[0] for k in OVERLAPS])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("offsets", ["jumps", "steps"])
def test_grouped_gemm_of_offsets_that_descend(name, rows, groups, cols, row, dtype, gated, offsets):
    """Offsets count as no lower than any before them: each place that is then
    named has its group's value, the others stay as they were."""
    g = torch.Generator(device="cuda").manual_seed(rows + groups)
    K, N, out = row // (1 if dtype == "i8" else 2), cols // (2 if gated else 1), "bf16" if dtype == "i8" else dtype
    cols, xs, ws = N * (2 if gated else 1), None, None
    if dtype == "i8":
        x = torch.randint(-128, 128, (rows, K), generator=g, dtype=torch.int8, device="cuda")
        w = torch.randint(-128, 128, (groups, cols, K), generator=g, dtype=torch.int8, device="cuda")
        xs = torch.rand(rows, generator=g, device="cuda") * 2.0 ** -7
        ws = torch.rand(groups, cols, generator=g, device="cuda") / K ** 0.5 * 2.0 ** -5
    else:
        x = torch.randn(rows, K, generator=g, device="cuda").to(DT[dtype])
        w = (torch.randn(groups, cols, K, generator=g, device="cuda") * K ** -0.5).to(DT[dtype])
    if offsets == "jumps":  # to and fro between the first rows and the last
        low = torch.randint(3, rows // 8, (groups // 2 + 1,), generator=gen(rows))
        high = torch.randint(rows // 2, rows - 3, (groups // 2 + 1,), generator=gen(groups))
        off = torch.stack([low, high], 1).reshape(-1)[:groups + 1]
    else:  # up, but for some that fall back, one far below 0
        off = 5 + torch.arange(groups + 1) * (rows - 11) // groups
        back = torch.randint(1, groups, (groups // 4,), generator=gen(groups))
        off[back] -= torch.randint(1, rows // 2, (groups // 4,), generator=gen(rows))
        off[back[0]] = -(1 << 31)
    epilogue = "silu" if gated else "none"
    c, _ = blank(rows, N, out)
    gb.grouped_gemm(x, w, c, off.int().cuda(), gated=gated, epilogue=epilogue, x_scale=xs, w_scale=ws)
    raised = off.clamp(0, rows).cummax(0).values.tolist()
    for e in range(groups):
        i = slice(raised[e], raised[e + 1])
        if i.start == i.stop:
            continue
        z, lost = pre(x[i], w[e], None if xs is None else xs[i], None if ws is None else ws[e], None)
        y, t = post(z[:, :N], lost[:, :N], epilogue, out, (z[:, N:], lost[:, N:]) if gated else None)
        within(c[i], y.cpu(), t.cpu(), f"{name} group {e}")
    assert bool(c[:raised[0]].isnan().all()) and bool(c[raised[-1]:].isnan().all()), "rows that no range names written"


def test_an_order_counts_where_nothing_is_gathered_or_scattered():
    x, w = rand(gen(1), 8, 64, dtype="bf16"), rand(gen(2), 1, 16, 64, dtype="bf16")
    order = torch.tensor([3, -1, 0, 8, 5, 6, 7, 1], dtype=torch.int32)
    c, _ = blank(8, 16, "bf16")
    gb.grouped_gemm(x.cuda(), w.cuda(), c, torch.tensor([0, 7], dtype=torch.int32).cuda(), order.cuda())
    assert c.cpu().isnan().all(1).tolist() == [False, True, False, True, False, False, False, True]


def test_products_keep_no_infinities_from_rows_that_are_none():
    """NaN in rows that no place names reaches no result, and NaN in one row
    that row alone."""
    g = gen(4)
    x, w = rand(g, 50, 64, dtype="f16"), rand(g, 2, 48, 64, dtype="f16")
    off, order = torch.tensor([0, 19, 30], dtype=torch.int32), torch.arange(50, dtype=torch.int32)
    x[30:] = NAN
    x[7, 3] = NAN
    x[9, 5] = INF
    c, _ = blank(50, 48, "f16")
    gb.grouped_gemm(x.cuda(), w.cuda(), c, off.cuda(), order.cuda(), gather=True)
    got = c.cpu()
    assert bool(got[30:].isnan().all()) and bool(got[7].isnan().all()) and not bool(got[9].isfinite().any())
    assert bool(got[[i for i in range(30) if i not in (7, 9)]].isfinite().all())


def test_rows_far_apart():
    """Rows of C and of X more than 2^31 elements from the first."""
    g = gen(6)
    ld, N, K, rows = (1 << 30) + 8, 24, 32, 3
    x, w = rand(g, rows, K, dtype="bf16"), rand(g, 1, N, K, dtype="bf16")
    buf = torch.empty(ld * (rows - 1) + N, dtype=torch.bfloat16, device="cuda")
    c = buf.as_strided((rows, N), (ld, 1))
    off = torch.tensor([0, rows], dtype=torch.int32)
    gb.grouped_gemm(x.cuda(), w.cuda(), c, off.cuda())
    z, lost = pre(x, w[0], None, None, None)
    within(c, *post(z, lost, "none", "bf16"), "far rows of c")
    wt = torch.tensor([[1.0, 0.5, 2.0]])
    y2 = torch.empty(1, N, dtype=torch.bfloat16, device="cuda")
    gb.combine(c, wt.cuda(), None, y2, experts=1)
    want = (c.cpu().double() * wt.double().T).sum(0, keepdim=True)
    within(y2, want, want.abs() * (2.0 ** -8 + 8 * U) + 4 * U * (c.cpu().double() * wt.double().T).abs().sum(0, keepdim=True), "far rows of z")
    q, s = torch.empty(rows, N, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    gb.quantise_i8(c, q, s)
    qw, sw = quantised(c.cpu())
    assert torch.equal(q.cpu(), qw) and same_scale(s, sw)


def test_products_of_rows_16_mib_apart():
    """The largest distance between rows, in both operands: the last rows of a
    tile lie a GiB behind its first."""
    g, ld, M, N, K = gen(16), 1 << 24, 70, 66, 4112
    a, b, r = codes(g, M, K), codes(g, N, K), rand(g, M, N, dtype="bf16")
    xs, ws = torch.rand(M, generator=g) * 2.0 ** -8, torch.rand(N, generator=g) * 2.0 ** -10
    far = [torch.empty((n - 1) * ld + K, dtype=torch.int8, device="cuda").as_strided((n, K), (ld, 1)) for n in (M, N)]
    far[0].copy_(a)
    far[1].copy_(b)
    for m in (16, M):  # (streamed, and in tiles)
        z, lost = pre(a[:m], b, xs[:m], ws, None)
        c, _ = blank(m, N, "bf16")
        gb.i8_gemm(far[0][:m], xs[:m].cuda(), far[1], ws.cuda(), c, residual=r[:m].cuda())
        within(c, *post(z, lost, "none", "bf16", residual=r[:m]), f"{m} rows")


@pytest.mark.parametrize("name,rows,ld,K,groups", [("tiles", 65534, 32760, 32760, 1), ("stream", 4095, 1 << 19, 2056, 1024)])
def test_gathered_rows_up_to_4_gib(name, rows, ld, K, groups):
    """A gathered X just below the largest one: its first and last rows."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.zeros(rows * ld, dtype=torch.bfloat16, device="cuda").as_strided((rows, K), (ld, 1))
    q = torch.tensor([rows - 1, 0, rows // 2, rows - 2], device="cuda")
    x[q] = torch.randn(4, K, generator=g, device="cuda").to(torch.bfloat16)
    w = (torch.randn(groups, 24, K, generator=g, device="cuda") * K ** -0.5).to(torch.bfloat16)
    off = torch.full((groups + 1,), 4, dtype=torch.int32, device="cuda")
    off[0] = 0  # all of group 0
    order = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    order[:4] = q.int()
    c, _ = blank(rows, 24, "bf16")
    gb.grouped_gemm(x, w, c, off, order, gather=True)
    z, lost = pre(x[q], w[0], None, None, None)
    y, t = post(z, lost, "none", "bf16")
    within(c[:4], y.cpu(), t.cpu(), name)
    assert bool(c[4:].isnan().all())


@pytest.mark.parametrize("rows", [3, 20, 200])
def test_gates_of_2_gib(rows):
    """The most that a group's gates may have: its values lie 2 GiB behind."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    N, K = 1 << 14, 1 << 16
    x = torch.randn(rows, K, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.empty(1, 2 * N, K, dtype=torch.bfloat16, device="cuda").normal_(0.0, K ** -0.5, generator=g)
    c, _ = blank(rows, N, "bf16")
    gb.grouped_gemm(x, w, c, torch.tensor([0, rows], dtype=torch.int32, device="cuda"), gated=True, epilogue="silu")
    assert bool(c.isfinite().all())
    for at in (0, N // 2 - 32, N - 64):
        n = torch.arange(at, at + 64, device="cuda")
        z, lost = pre(x, w[0][n], None, None, None)
        y, t = post(z, lost, "silu", "bf16", pre(x, w[0][n + N], None, None, None))
        within(c[:, at:at + 64], y.cpu(), t.cpu(), f"columns from {at}")


# ---- the router --------------------------------------------------------------------

def route_want(logits, per, score, renormalise, scale):
    l = logits.double()
    l = torch.where(l.isnan(), -INF, l)
    rank = torch.argsort(-l, dim=1, stable=True)[:, :per]
    top = l.gather(1, rank)
    there = top > -INF
    m = l.amax(1, keepdim=True)
    if score == "sigmoid":
        p = torch.sigmoid(top)
        if renormalise:
            # relative to the largest: e^-|l| may be too small for any number
            d = torch.where(there, top - m, -INF)
            low = torch.exp(d) * (1 + torch.exp(m.clamp(max=0))) / (1 + torch.exp(top.clamp(max=0)))
            p = torch.where(m < 0, low, p)
    else:
        shifted = torch.where(l == m, 0.0, l - m)  # (infinities share)
        e = torch.where(l > -INF, torch.exp(shifted), 0.0)
        p = e.gather(1, rank)
        if not renormalise:
            p = p / e.sum(1, keepdim=True)
    p = torch.where(there, p, 0.0)
    if renormalise:
        p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
    return torch.where(there, rank, -1).int(), torch.where(there, p * scale, 0.0)


def group_want(ids, groups):
    flat = ids.reshape(-1)
    order, off = [], [0]
    for e in range(groups):
        order += (flat == e).nonzero()[:, 0].tolist()
        off.append(len(order))
    order += [-1] * (flat.numel() - len(order))
    return torch.tensor(off, dtype=torch.int32), torch.tensor(order, dtype=torch.int32)


def route_check(logits, per, score, renormalise, scale=1.0, extra=0):
    t, e = logits.shape
    ids = torch.full((t, per), 77, dtype=torch.int32, device="cuda")
    w = torch.full((t, per), NAN, device="cuda")
    off, order = torch.full((e + 2,), 5, dtype=torch.int32, device="cuda"), torch.full((t * per,), 5, dtype=torch.int32, device="cuda")
    gb.route(strided(logits, extra), ids, w, score=score, renormalise=renormalise, scale=scale, offsets=off[:-1], order=order)
    iw, ww = route_want(logits, per, score, renormalise, scale)
    assert torch.equal(ids.cpu(), iw), "ids"
    # exp of a 32-bit difference (half a step of up to 40, where it counts: 40
    # U), its own two or three, sums of up to 1024 terms in 64 lanes (16 + 6
    # additions) and four further operations
    within(w, ww, ww.abs() * 80 * U + 2.0 ** -126, "weights")
    ow, rw = group_want(iw, e)
    assert torch.equal(off[:-1].cpu(), ow) and torch.equal(order.cpu(), rw) and int(off[-1]) == 5
    return ids, w


@pytest.mark.parametrize("tokens,experts,per", [(1, 1, 1), (1, 8, 2), (5, 4, 4), (3, 64, 6), (33, 60, 4), (2, 65, 8), (32, 128, 8),
                                                (70, 129, 7), (9, 256, 8), (300, 160, 6), (4, 384, 8), (7, 1024, 64), (130, 512, 8), (9, 300, 6), (3, 600, 20),
                                                (2000, 16, 2), (5, 100, 64), (1030, 256, 8), (3000, 8, 2)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("score,renormalise", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_route(tokens, experts, per, dtype, score, renormalise):
    logits = rand(gen(tokens * 31 + experts), tokens, experts, std=2.0, dtype=dtype)
    route_check(logits, per, score, renormalise, 2.5, extra=tokens % 3)


def test_route_ties_go_to_the_lower_expert():
    for experts in (7, 64, 128, 256, 300, 1024):
        logits = torch.zeros(20, experts)
        logits[1] = -0.0
        logits[2, ::2] = -0.0
        logits[3:] = torch.randint(-2, 3, (17, experts), generator=gen(experts)).float()
        for score in ("softmax", "sigmoid"):
            ids, _ = route_check(logits, 5, score, True)
            assert ids[0].tolist() == [0, 1, 2, 3, 4] == ids[1].tolist() == ids[2].tolist()


@pytest.mark.parametrize("score,renormalise", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_route_special_logits(score, renormalise):
    x = rand(gen(2), 16, 70)
    x[0] = -INF
    x[1] = NAN
    x[2, 3:] = -INF
    x[3, :68] = NAN
    x[4] -= 500
    x[5] = 3e38
    x[6] = -3e38
    x[7] *= 40
    x[8, 5] = 1000
    if score == "softmax":
        x[9, [4, 60]] = INF
        x[10] = INF
    ids, w = route_check(x, 4, score, renormalise)
    assert ids[0].tolist() == [-1] * 4 == ids[1].tolist() and not w[:2].any()
    assert ids[2].tolist()[3] == -1 and sorted(ids[2].tolist()[:3]) == [0, 1, 2]
    assert sorted(ids[3].tolist()) == [-1, -1, 68, 69]


@pytest.mark.parametrize("rows,groups", [(0, 3), (1, 1), (1, 1024), (63, 5), (64, 64), (65, 2), (1000, 7), (1025, 64), (5000, 1024),
                                         (100001, 60), (262144, 256)])
def test_group_rows(rows, groups):
    g = gen(rows + groups)
    ids = torch.randint(-2, groups + 2, (rows,), generator=g, dtype=torch.int32)
    if rows > 70:
        ids[-3:] = torch.tensor([-(1 << 31), (1 << 31) - 1, groups], dtype=torch.int32)
        ids[10:70] = 0
    off = torch.full((groups + 1,), 9, dtype=torch.int32, device="cuda")
    order = torch.full((rows,), 9, dtype=torch.int32, device="cuda")
    gb.group_rows(ids.cuda(), off, order)
    key = torch.where((ids >= 0) & (ids < groups), ids, groups)
    key, want = key.sort(stable=True)
    assert torch.equal(order.cpu(), torch.where(key < groups, want, -1).int())
    assert torch.equal(off.cpu(), torch.searchsorted(key, torch.arange(groups + 1, dtype=torch.int32)).int())


# Ids beside the most of which a lane keeps its own (131072), partial and odd
# rounds of 32768 among them.
@pytest.mark.parametrize("rows,groups", [(98305, 33), (131071, 5), (131072, 256), (131073, 60), (163878, 1024), (196608, 3), (229377, 64), (400000, 16)])
def test_group_rows_of_many_ids(rows, groups):
    test_group_rows(rows, groups)
    # nearly all in one group, then all in it
    for others in (0.01, 0.0):
        for most in (0, groups - 1):
            g = gen(rows + most)
            ids = torch.where(torch.rand(rows, generator=g) < others, torch.randint(-1, groups, (rows,), generator=g), most).int()
            off = torch.full((groups + 2,), 9, dtype=torch.int32, device="cuda")
            order = torch.full((rows + 1,), 9, dtype=torch.int32, device="cuda")
            gb.group_rows(ids.cuda(), off[:-1], order[:-1])
            key, want = torch.where(ids >= 0, ids, groups).sort(stable=True)
            assert torch.equal(order[:-1].cpu(), torch.where(key < groups, want, -1).int()), (others, most)
            assert torch.equal(off[:-1].cpu(), torch.searchsorted(key, torch.arange(groups + 1, dtype=torch.int32)).int())
            assert int(off[-1]) == 9 == int(order[-1]), "written past the end"


def test_route_without_tokens():
    off = torch.full((9,), 7, dtype=torch.int32, device="cuda")
    empty = torch.empty(0, 2, device="cuda")
    gb.route(torch.empty(0, 8, device="cuda"), empty.int(), empty, offsets=off, order=torch.empty(0, dtype=torch.int32, device="cuda"))
    assert not off.any()


# ---- a token's rows brought together --------------------------------------------------

@pytest.mark.parametrize("tokens,per,cols", [(1, 1, 1), (3, 2, 7), (5, 8, 64), (32, 4, 2048), (7, 3, 2055), (2, 64, 130), (40, 6, 5000),
                                             (1, 5, 16384), (3000, 2, 8)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_combine(tokens, per, cols, dtype):
    g = gen(tokens * 17 + per * 3 + cols)
    z, r, w = rand(g, tokens * per, cols, dtype=dtype), rand(g, tokens, cols, dtype=dtype), torch.rand(tokens, per, generator=g)
    ids = torch.randint(-1, 4, (tokens, per), generator=g, dtype=torch.int32)
    z[(ids.reshape(-1) < 0) | (ids.reshape(-1) >= 3)] = NAN  # read into nothing
    w[ids < 0] = NAN
    for extra, res, masked in ((0, True, True), (3, False, True), (8, True, False), (0, False, False)):
        there = ((ids >= 0) & (ids < 3)) if masked else torch.ones_like(ids, dtype=torch.bool)
        zz = z if masked else torch.nan_to_num(z)
        ww = w if masked else torch.nan_to_num(w)
        terms = torch.where(there[..., None], ww.double()[..., None] * zz.double().view(tokens, per, cols), 0.0)
        want = terms.sum(1) + (r.double() if res else 0.0)
        # a product and an addition a term, and the residual's
        lost = (per + 1) * U * (terms.abs().sum(1) + want.abs())
        e = torch.finfo(DT[dtype]).eps / 2
        y, buf = blank(tokens, cols, dtype, extra)
        gb.combine(strided(zz, extra), ww.cuda(), ids.cuda() if masked else None, y, experts=3, residual=strided(r, 2 * extra) if res else None)
        within(y, want, lost * (1 + e) + e * want.abs() + SUB[dtype], f"{tokens}x{per}x{cols} extra {extra}")
        assert bool(buf[:, cols:].isnan().all()), "written past the rows"


# Aligned rows of more than 32 MiB, and more tokens than the 2^20 workgroups of a
# grid take at once.
@pytest.mark.parametrize("tokens,per,cols", [(1100, 4, 4096), (2050, 3, 2880), ((1 << 20) + 9, 2, 16), ((1 << 20) + 9, 2, 15)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_combine_many_rows(tokens, per, cols, dtype):
    g = torch.Generator(device="cuda").manual_seed(tokens + cols)
    z, r = (torch.empty(n, cols, dtype=DT[dtype], device="cuda").normal_(generator=g) for n in (tokens * per, tokens))
    w = torch.rand(tokens, per, generator=g, device="cuda")
    ids = torch.randint(-1, 4, (tokens, per), generator=g, dtype=torch.int32, device="cuda")
    there = (ids >= 0) & (ids < 3)
    z[~there.reshape(-1)] = NAN
    terms = torch.where(there[..., None], w.double()[..., None] * z.double().view(tokens, per, cols), 0.0)
    e = torch.finfo(DT[dtype]).eps / 2
    for res in (False, True):  # (in place the second time)
        want = terms.sum(1) + (r.double() if res else 0.0)
        lost = (per + 1) * U * (terms.abs().sum(1) + want.abs())
        y = r if res else torch.full_like(r, NAN)
        gb.combine(z, w, ids, y, experts=3, residual=r if res else None)
        within(y, want.cpu(), (lost * (1 + e) + e * want.abs() + SUB[dtype]).cpu(), f"{tokens}x{per}x{cols} residual {res}")


def test_combine_in_place():
    g = gen(8)
    z, r, w = rand(g, 12, 100, dtype="bf16"), rand(g, 4, 100, dtype="bf16"), torch.rand(4, 3, generator=g)
    y, apart = r.cuda(), torch.empty(4, 100, dtype=torch.bfloat16, device="cuda")
    gb.combine(z.cuda(), w.cuda(), None, apart, experts=1, residual=y)
    gb.combine(z.cuda(), w.cuda(), None, y, experts=1, residual=y)
    assert torch.equal(y, apart)


# ---- a layer of experts ------------------------------------------------------------------

class Layer:
    """A layer of experts after a norm, in 16 bits or 8."""

    def __init__(self, tokens, experts, per, D, H, dtype, seed):
        g = gen(seed)
        self.tokens, self.experts, self.per, self.dtype = tokens, experts, per, dtype
        out = self.out = "bf16" if dtype == "i8" else dtype
        self.norm = (1 + 0.1 * rand(g, D)).to(DT[out]).cuda()
        self.router = rand(g, experts, D, std=D ** -0.5, dtype=out).cuda()
        up, down = rand(g, experts, 2 * H, D, std=D ** -0.5), rand(g, experts, D, H, std=H ** -0.5)
        self.up_scale = self.down_scale = None
        if dtype == "i8":
            (qu, su), (qd, sd) = quantised(up.reshape(-1, D)), quantised(down.reshape(-1, H))
            self.up, self.down = qu.view(up.shape).cuda(), qd.view(down.shape).cuda()
            self.up_scale, self.down_scale = su.view(experts, -1).cuda(), sd.view(experts, -1).cuda()
        else:
            self.up, self.down = up.to(DT[out]).cuda(), down.to(DT[out]).cuda()
        new = lambda *s, t=DT[out]: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
        n = tokens * per
        self.x, self.y, self.h, self.z, self.o = new(tokens, D), new(tokens, D), new(n, H), new(n, D), new(tokens, D)
        self.logits, self.ids, self.w = new(tokens, experts), new(tokens, per, t=torch.int32), new(tokens, per, t=torch.float32)
        self.off, self.order = new(experts + 1, t=torch.int32), new(n, t=torch.int32)
        self.qy, self.sy, self.qh, self.sh = new(tokens, D, t=torch.int8), new(tokens, t=torch.float32), new(n, H, t=torch.int8), new(n, t=torch.float32)
        self.plan = gb.Plan(tokens, experts, D, out, out, "row", "col", "none")

    def run(self, stream=None):
        gb.rmsnorm(self.x, self.norm, self.y, stream=stream)
        self.plan.run(self.y, self.router, None, self.logits, stream=stream)
        gb.route(self.logits, self.ids, self.w, offsets=self.off, order=self.order, stream=stream)
        y, h, sy, sh = self.y, self.h, None, None
        if self.dtype == "i8":
            gb.quantise_i8(self.y, self.qy, self.sy, stream=stream)
            y, sy = self.qy, self.sy
        gb.grouped_gemm(y, self.up, self.h, self.off, self.order, per=self.per, gather=True, gated=True, epilogue="silu",
                        x_scale=sy, w_scale=self.up_scale, stream=stream)
        if self.dtype == "i8":
            gb.quantise_i8(self.h, self.qh, self.sh, stream=stream)
            h, sh = self.qh, self.sh
        gb.grouped_gemm(h, self.down, self.z, self.off, self.order, per=self.per, scatter=True, x_scale=sh,
                        w_scale=self.down_scale, stream=stream)
        gb.combine(self.z, self.w, self.ids, self.o, experts=self.experts, residual=self.x, stream=stream)

    def want(self):
        """The layer in 64 bits from what its own steps rounded: the chosen
        experts and their weights, and the rows in 8 bits."""
        y = self.y.cpu().double() if self.dtype != "i8" else self.qy.cpu().double() * self.sy.cpu().double()[:, None]
        up, down = self.up.cpu().double(), self.down.cpu().double()
        if self.dtype == "i8":
            up, down = up * self.up_scale.cpu().double()[..., None], down * self.down_scale.cpu().double()[..., None]
        ids, w = self.ids.cpu(), self.w.cpu().double()
        o = self.x.cpu().double()
        H = up.shape[1] // 2
        for t in range(self.tokens):
            for j in range(self.per):
                e = int(ids[t, j])
                z = up[e] @ y[t]
                o[t] += w[t, j] * (down[e] @ (act(z[:H], "silu") * z[H:]))
        return o


@pytest.mark.parametrize("dtype", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("tokens", [1, 5, 150])
def test_layer_of_experts(tokens, dtype):
    layer = Layer(tokens, 12, 3, 128, 96, dtype, tokens)
    layer.x.copy_(rand(gen(tokens + 1), tokens, 128, dtype=layer.out))
    layer.run()
    want = layer.want()
    e = torch.finfo(DT[layer.out]).eps / 2
    # h and z are rounded once each, and o: of values whose sums are below 2 in
    # the mean; in 8 bits h's codes are half a step of 1/127 of its largest
    # value off, in sums of 96 of either sign
    off = (layer.o.cpu().double() - want).abs()
    scale = float(want.square().mean().sqrt())
    lost = 8 * e + (8 * 0.5 / 127 if dtype == "i8" else 0.0)
    assert float(off.max()) <= lost * scale * 4, (float(off.max()), scale)


def test_layer_captured_in_graphs():
    """Two layers in graphs of their own, replayed in turn between eager work
    on other inputs: every replay gives the eager bits."""
    layers = [Layer(9, 12, 3, 128, 96, "bf16", 1), Layer(40, 8, 2, 128, 64, "i8", 2)]
    graphs = []
    s = torch.cuda.Stream()
    for layer in layers:
        layer.x.copy_(rand(gen(1), layer.tokens, 128, dtype="bf16"))
        layer.run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            layer.run()
        graphs.append(graph)
    for i in range(6):
        layer, graph = layers[i % 2], graphs[i % 2]
        x = rand(gen(10 + i), layer.tokens, 128, std=1.0 + i, dtype="bf16").cuda()
        layer.x.copy_(x)
        layer.run()
        eager = layer.o.clone()
        layer.o.fill_(NAN)
        for t in (layer.ids, layer.off, layer.order):
            t.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(layer.o, eager), i


def test_other_stream_and_order_of_work():
    layer = Layer(30, 12, 3, 128, 96, "bf16", 3)
    x = rand(gen(5), 30, 128, dtype="bf16").cuda()
    layer.x.copy_(x)
    layer.run()
    want = layer.o.clone()
    layer.o.fill_(NAN)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    layer.run(stream=s)
    s.synchronize()
    assert torch.equal(layer.o, want)
    with torch.cuda.stream(s):
        layer.o.fill_(NAN)
        layer.run()
    s.synchronize()
    assert torch.equal(layer.o, want)


def test_two_streams_at_once():
    """The same calls on two streams without an order between them, on inputs
    of their own: each gives the bits that it gives alone."""
    layers = [Layer(700, 12, 3, 512, 384, "i8", 7), Layer(800, 16, 4, 512, 256, "bf16", 8)]
    for i, layer in enumerate(layers):
        layer.x.copy_(rand(gen(i), layer.tokens, 512, dtype="bf16"))
        layer.run()
    want = [(layer.o.clone(), layer.order.clone(), layer.w.clone()) for layer in layers]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for layer, stream in zip(layers, streams):
            layer.run(stream=stream)
    torch.cuda.synchronize()
    for layer, (o, order, w) in zip(layers, want):
        assert torch.equal(layer.o, o) and torch.equal(layer.order, order) and torch.equal(layer.w, w)


# ---- refusals of the tensor calls ------------------------------------------------------

def test_tensor_calls_refuse():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    q, s = torch.zeros(4, 64, dtype=torch.int8, device="cuda"), torch.zeros(4, device="cuda")
    w, ws = torch.zeros(2, 32, 64, dtype=torch.int8, device="cuda"), torch.zeros(2, 32, device="cuda")
    c = torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda")
    i = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    off, order = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    f = torch.zeros(4, 2, device="cuda")
    bad = [
        lambda: gb.quantise_i8(x.float(), q, s), lambda: gb.quantise_i8(x, q[:3], s), lambda: gb.quantise_i8(x, q.short(), s),
        lambda: gb.quantise_i8(x, q, s[:3]), lambda: gb.quantise_i8(x.t(), q.t(), s), lambda: gb.quantise_i8(x.cpu(), q, s),
        lambda: gb.i8_gemm(q, s, w[0], ws[1], c.float()), lambda: gb.i8_gemm(x, s, w[0], ws[0], c),
        lambda: gb.i8_gemm(q, s[:2], w[0], ws[0], c), lambda: gb.i8_gemm(q, s, w[0], ws[0], c, epilogue="bias"),
        lambda: gb.i8_gemm(q, s, w[0], ws[0], c, bias=c[0]), lambda: gb.i8_gemm(q, s, w[0], ws[0], c, residual=c.half()),
        lambda: gb.i8_gemm(q, s, w[0], ws[0], c[:, :31]),
        lambda: gb.route(f, i.long(), f), lambda: gb.route(f, i, f[:, :1]), lambda: gb.route(f, i, f, offsets=off),
        lambda: gb.route(f.double(), i, f), lambda: gb.route(f, i, f, offsets=off[:2], order=order),
        lambda: gb.route(f, i, f, offsets=off, order=order),
        lambda: gb.group_rows(i, off, order), lambda: gb.group_rows(i.t(), off, order.repeat(2)), lambda: gb.group_rows(order, off[:1], order),
        lambda: gb.grouped_gemm(q, w, c, off), lambda: gb.grouped_gemm(q, w, c, off, x_scale=s),
        lambda: gb.grouped_gemm(x, w, c, off), lambda: gb.grouped_gemm(q, w, c, off, x_scale=s, w_scale=ws, gated=True),
        lambda: gb.grouped_gemm(q, w, c, off[:2], x_scale=s, w_scale=ws), lambda: gb.grouped_gemm(q, w, c, off, order[:3], x_scale=s, w_scale=ws),
        lambda: gb.grouped_gemm(q, w, c, off, order, per=3, gather=True, x_scale=s, w_scale=ws),
        lambda: gb.grouped_gemm(q, w, c, off, order, per=0, x_scale=s, w_scale=ws),
        lambda: gb.grouped_gemm(q, w, c, off, bias=c, x_scale=s, w_scale=ws),
        lambda: gb.combine(c, f[:1], i[:1], c, experts=2), lambda: gb.combine(c, f[:2].int(), i[:2], c[:2], experts=2),
        lambda: gb.combine(c, f[:2], i[:2].long(), c[:2], experts=2), lambda: gb.combine(c.half(), f[:2], i[:2], c[:2], experts=2),
    ]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {k} was taken")
    for call in (lambda: gb.combine(c, f[:2], i[:2], c[:2], experts=0), lambda: gb.i8_gemm(q[:, :40], s, w[0][:, :40], ws[0], c),
                 lambda: gb.grouped_gemm(q, w, c, off, gather=True, x_scale=s, w_scale=ws)):
        with pytest.raises(gb.GemmEpiError):
            call()


def test_calls_without_rows_do_nothing():
    dev = dict(device="cuda")
    e = torch.empty(0, 64, dtype=torch.bfloat16, **dev)
    q, s = torch.empty(0, 64, dtype=torch.int8, **dev), torch.empty(0, **dev)
    gb.quantise_i8(e, q, s)
    gb.i8_gemm(q, s, torch.zeros(8, 64, dtype=torch.int8, **dev), torch.zeros(8, **dev), torch.empty(0, 8, dtype=torch.bfloat16, **dev))
    gb.grouped_gemm(e, torch.zeros(2, 8, 64, dtype=torch.bfloat16, **dev), torch.empty(0, 8, dtype=torch.bfloat16, **dev),
                    torch.zeros(3, dtype=torch.int32, **dev), torch.empty(0, dtype=torch.int32, **dev), gather=True)
    gb.combine(e, torch.empty(0, 3, **dev), None, e, experts=4)
    torch.cuda.synchronize()
