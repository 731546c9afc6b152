"""The experts' feed-forward and the 8-bit products without a GPU: every
refusal of the C ABI (all are decided on the host, before any HIP call)."""
import pytest

from epilogue_gemm_amd import binding as gb

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = 0x10000  # stands for a device pointer: nothing here is launched
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gb.load_library()


# Each valid call below has no rows, which does nothing, so that no refused
# argument can hide behind a launch.

def _quantise(**kw):
    a = dict(X=P, ldx=64, Y=P, ldy=64, scale=P, rows=0, cols=64, dtype="bf16", stream=None)
    a.update(kw)
    return gb.gemm_epi_quantise_i8(*a.values())


@pytest.mark.parametrize("kw,want", [
    ({}, OK), ({"dtype": "f16"}, OK), ({"Y": P + 1, "ldx": 65, "ldy": 67}, OK), ({"cols": 1 << 30, "ldx": 1 << 30, "ldy": 1 << 30}, OK),
    ({"X": None}, INVALID), ({"Y": None}, INVALID), ({"scale": None}, INVALID), ({"rows": -1}, INVALID),
    ({"cols": 0}, INVALID), ({"ldx": 63}, INVALID), ({"ldy": 63}, INVALID), ({"dtype": "f32"}, INVALID),
    ({"dtype": "i8"}, INVALID), ({"X": P + 1}, INVALID), ({"scale": P + 2}, INVALID),
    ({"rows": 1 << 31}, UNSUPPORTED), ({"cols": (1 << 30) + 1, "ldx": 1 << 31, "ldy": 1 << 31}, UNSUPPORTED),
])
def test_quantise_refusals(kw, want):
    assert _quantise(**kw) == want


def _i8(**kw):
    a = dict(A=P, lda=64, a_scale=P, B=P, ldb=64, b_scale=P, bias=P, R=P, ldr=40, C=P, ldc=40, M=0, N=40, K=64,
             epilogue="bias_gelu", out_dtype="bf16", stream=None)
    a.update(kw)
    return gb.gemm_epi_i8_gemm(*a.values())


@pytest.mark.parametrize("kw,want", [
    ({}, OK), ({"R": None, "ldr": 0}, OK), ({"bias": None, "epilogue": "silu"}, OK), ({"out_dtype": "f16"}, OK),
    ({"K": 131056, "lda": 131056, "ldb": 131056}, OK), ({"N": 41, "ldc": 41, "ldr": 41}, OK),
    ({"M": -1}, INVALID), ({"N": 0}, INVALID), ({"K": 0}, INVALID), ({"lda": 48}, INVALID), ({"ldb": 48}, INVALID),
    ({"ldc": 39}, INVALID), ({"ldr": 39}, INVALID), ({"out_dtype": "f32"}, INVALID), ({"out_dtype": "i8"}, INVALID),
    ({"C": P + 1}, INVALID), ({"R": P + 1}, INVALID), ({"bias": P + 1}, INVALID), ({"a_scale": P + 2}, INVALID),
    ({"b_scale": P + 2}, INVALID),
    ({"K": 24, "lda": 32, "ldb": 32}, UNSUPPORTED), ({"K": 1 << 17, "lda": 1 << 17, "ldb": 1 << 17}, UNSUPPORTED),
    ({"lda": 72}, UNSUPPORTED), ({"ldb": 72}, UNSUPPORTED), ({"lda": 1 << 24}, OK), ({"ldb": 1 << 24}, OK),
    ({"lda": (1 << 24) + 16}, UNSUPPORTED), ({"ldb": (1 << 24) + 16}, UNSUPPORTED), ({"M": 1 << 31}, UNSUPPORTED),
    ({"M": 1 << 24, "N": 8192, "ldc": 8192, "ldr": 8192}, UNSUPPORTED), ({"ldc": 1 << 31}, UNSUPPORTED),
    ({"M": 5, "A": None}, INVALID), ({"M": 5, "B": None}, INVALID), ({"M": 5, "C": None}, INVALID),
    ({"M": 5, "a_scale": None}, INVALID), ({"M": 5, "b_scale": None}, INVALID), ({"M": 5, "bias": None}, INVALID),
    ({"M": 5, "A": P + 8}, UNSUPPORTED), ({"M": 5, "B": P + 8}, UNSUPPORTED),
])
def test_i8_gemm_refusals(kw, want):
    assert _i8(**kw) == want


def test_unknown_enum_values_are_refused():
    lib = gb.load_library()
    args = [P, 64, P, P, 64, P, P, None, 0, P, 40, 0, 40, 64]
    for epilogue in (-1, 7, 100):
        assert lib.gemm_epi_i8_gemm(*args, epilogue, gb.DTYPES["bf16"], None) == INVALID
    assert lib.gemm_epi_i8_gemm(*args, 0, 9, None) == INVALID
    assert lib.gemm_epi_route(P, 16, 9, 0, 16, 2, 0, 0, 1.0, P, P, None, None, None) == INVALID
    assert lib.gemm_epi_route(P, 16, 2, 0, 16, 2, 2, 0, 1.0, P, P, None, None, None) == INVALID
    assert lib.gemm_epi_plan_set_ld is not None and gb.gemm_epi_plan_status(64, 64, 64, "i8", "bf16", "row", "col", "none") == INVALID


def _route(**kw):
    a = dict(logits=P, ldl=16, dtype="f32", tokens=0, experts=16, per=4, score="softmax", renormalise=True, scale=1.0,
             ids=P, weights=P, offsets=None, order=None, stream=None)
    a.update(kw)
    return gb.gemm_epi_route(*a.values())


@pytest.mark.parametrize("kw,want", [
    ({}, OK), ({"dtype": "bf16"}, OK), ({"dtype": "f16", "logits": P + 2}, OK), ({"per": 16}, OK), ({"scale": -2.0}, OK),
    ({"logits": None, "ids": None, "weights": None}, OK),  # (no tokens)
    ({"tokens": -1}, INVALID), ({"experts": 0}, INVALID), ({"per": 0}, INVALID), ({"per": 17}, INVALID),
    ({"ldl": 15}, INVALID), ({"scale": NAN}, INVALID), ({"scale": INF}, INVALID), ({"scale": -INF}, INVALID),
    ({"dtype": "fp8"}, INVALID), ({"dtype": "i8"}, INVALID), ({"order": P}, INVALID),
    ({"logits": P + 2}, INVALID), ({"dtype": "bf16", "logits": P + 1}, INVALID), ({"ids": P + 2}, INVALID),
    ({"weights": P + 2}, INVALID), ({"offsets": P + 2, "order": P}, INVALID), ({"offsets": P, "order": P + 2}, INVALID),
    ({"tokens": 5, "logits": None}, INVALID), ({"tokens": 5, "ids": None}, INVALID),
    ({"tokens": 5, "weights": None}, INVALID), ({"tokens": 5, "offsets": P}, INVALID),
    ({"experts": 1025, "ldl": 1025}, UNSUPPORTED), ({"experts": 100, "ldl": 100, "per": 65}, UNSUPPORTED),
    ({"tokens": (1 << 25) + 1}, UNSUPPORTED), ({"ldl": 1 << 31}, UNSUPPORTED),
    ({"tokens": 1 << 25, "experts": 64, "ldl": 64, "per": 64}, UNSUPPORTED),
])
def test_route_refusals(kw, want):
    assert _route(**kw) == want


@pytest.mark.parametrize("kw,want", [
    ({"rows": -1}, INVALID), ({"groups": 0}, INVALID), ({"offsets": None}, INVALID), ({"ids": None}, INVALID),
    ({"order": None}, INVALID), ({"ids": P + 2}, INVALID), ({"offsets": P + 2}, INVALID), ({"order": P + 2}, INVALID),
    ({"groups": 1025}, UNSUPPORTED), ({"rows": 1 << 31}, UNSUPPORTED),
])
def test_group_rows_refusals(kw, want):
    a = dict(ids=P, rows=5, groups=4, offsets=P, order=P, stream=None)
    a.update(kw)
    assert gb.gemm_epi_group_rows(*a.values()) == want


_GROUPS = dict(offsets=P, order=P, groups=3, rows=0, per=2)


def _grouped(places={}, **kw):
    a = dict(groups=gb.groups_struct(*{**_GROUPS, **places}.values()), X=P, ldx=64, x_scale=None, W=P, w_scale=None,
             bias=None, C=P, ldc=40, N=40, K=64, flags=gb.GATHER | gb.GATED, epilogue="silu", dtype="bf16", out_dtype="bf16",
             stream=None)
    a.update(kw)
    return gb.gemm_epi_grouped_gemm(*a.values())


_I8 = dict(dtype="i8", x_scale=P, w_scale=P)
_SIX = {"rows": 6}


@pytest.mark.parametrize("places,kw,want", [
    ({}, {}, OK), ({}, {"flags": 0}, OK), ({}, {"flags": 7}, OK), ({}, _I8, OK), ({}, {**_I8, "out_dtype": "f16"}, OK),
    ({}, {"dtype": "f16", "out_dtype": "f16"}, OK), ({}, {"epilogue": "bias_silu", "bias": P}, OK),
    ({}, {"groups": None}, INVALID), ({}, {"flags": 8}, INVALID), ({}, {"flags": -1}, INVALID),
    ({"rows": -2}, {}, INVALID), ({"groups": 0}, {}, INVALID), ({"per": 0}, {}, INVALID), ({"rows": 5}, {}, INVALID),
    ({}, {"N": 0}, INVALID), ({}, {"K": 0}, INVALID), ({}, {"ldx": 56}, INVALID), ({}, {"ldc": 39}, INVALID),
    ({}, {"dtype": "f32", "out_dtype": "f32"}, INVALID), ({}, {"out_dtype": "f16"}, INVALID),
    ({}, {**_I8, "out_dtype": "i8"}, INVALID), ({}, {"dtype": "fp8", "out_dtype": "fp8"}, INVALID),
    ({"offsets": P + 2}, {}, INVALID), ({"order": P + 2}, {}, INVALID), ({}, {"C": P + 1}, INVALID),
    ({}, {**_I8, "x_scale": P + 2}, INVALID), ({}, {**_I8, "w_scale": P + 2}, INVALID),
    ({}, {"epilogue": "bias_silu", "bias": P + 1}, INVALID),
    ({}, {"K": 60}, UNSUPPORTED), ({}, {**_I8, "K": 56}, UNSUPPORTED), ({}, {"ldx": 68}, UNSUPPORTED),
    ({}, {**_I8, "ldx": 72}, UNSUPPORTED), ({}, {"K": 1 << 17, "ldx": 1 << 17}, UNSUPPORTED),
    ({"groups": 1025}, {}, UNSUPPORTED), ({"rows": 1 << 31}, {}, UNSUPPORTED), ({}, {"ldc": 1 << 31}, UNSUPPORTED),
    ({}, {"ldx": 1 << 23}, OK), ({}, {"ldx": (1 << 23) + 8}, UNSUPPORTED),
    ({"rows": 1 << 16}, {"ldx": 1 << 16}, UNSUPPORTED),  # X of 4 GiB, gathered
    ({"rows": 1 << 20, "groups": 1024}, {"N": 1 << 14, "ldc": 1 << 14}, UNSUPPORTED),
    ({**_SIX, "offsets": None}, {}, INVALID), ({**_SIX, "order": None}, {}, INVALID),
    ({**_SIX, "order": None}, {"flags": gb.SCATTER}, INVALID), (_SIX, {"X": None}, INVALID), (_SIX, {"W": None}, INVALID),
    (_SIX, {"C": None}, INVALID), (_SIX, {"x_scale": P}, INVALID), (_SIX, {"w_scale": P}, INVALID),
    (_SIX, {"dtype": "i8"}, INVALID), (_SIX, {"epilogue": "bias"}, INVALID),
    (_SIX, {"X": P + 8}, UNSUPPORTED), (_SIX, {"W": P + 8}, UNSUPPORTED),
])
def test_grouped_gemm_refusals(places, kw, want):
    assert _grouped(places, **kw) == want


@pytest.mark.parametrize("kw", [
    {"ldx": 1 << 62}, {"ldx": (1 << 62) + 8}, {"ldx": (1 << 63) - 8}, {"ldx": 1 << 31}, {"ldx": 1 << 61, "dtype": "f16", "out_dtype": "f16"},
    {**_I8, "ldx": 1 << 62}, {**_I8, "ldx": (1 << 63) - 16}, {"K": 1 << 62, "ldx": 1 << 62}, {"K": (1 << 63) - 8, "ldx": (1 << 63) - 1},
    {**_I8, "K": 1 << 62, "ldx": 1 << 62}, {"N": (1 << 62) + 8, "ldc": 1 << 62 | 16},
])
@pytest.mark.parametrize("flags", [0, gb.GATHER, gb.GATED, gb.GATHER | gb.GATED])
def test_grouped_gemm_refuses_sizes_whose_bytes_pass_64_bits(kw, flags):
    """Sizes and distances near 2^63: their bytes are no number of 64 bits."""
    assert _grouped(**{"flags": flags, **kw}) == UNSUPPORTED


def _combine(**kw):
    a = dict(Z=P, ldz=64, weights=P, ids=P, experts=4, R=P, ldr=64, Y=P, ldy=64, tokens=0, per=4, cols=64, dtype="bf16",
             stream=None)
    a.update(kw)
    return gb.gemm_epi_combine(*a.values())


@pytest.mark.parametrize("kw,want", [
    ({}, OK), ({"ids": None}, OK), ({"R": None, "ldr": 0}, OK), ({"Z": P + 2, "cols": 63}, OK),
    ({"Z": None}, INVALID), ({"Y": None}, INVALID), ({"weights": None}, INVALID), ({"tokens": -1}, INVALID),
    ({"per": 0}, INVALID), ({"cols": 0}, INVALID), ({"experts": 0}, INVALID), ({"ldz": 63}, INVALID),
    ({"ldr": 63}, INVALID), ({"ldy": 63}, INVALID), ({"dtype": "f32"}, INVALID), ({"Z": P + 1}, INVALID),
    ({"R": P + 1}, INVALID), ({"Y": P + 1}, INVALID), ({"weights": P + 2}, INVALID), ({"ids": P + 2}, INVALID),
    ({"per": 65}, UNSUPPORTED), ({"tokens": 1 << 31}, UNSUPPORTED), ({"tokens": 1 << 26, "per": 32}, UNSUPPORTED),
    ({"cols": (1 << 30) + 1, "ldz": 1 << 31, "ldr": 1 << 31, "ldy": 1 << 31}, UNSUPPORTED),
])
def test_combine_refusals(kw, want):
    assert _combine(**kw) == want
