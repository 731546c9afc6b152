"""The operators of a decode step without a GPU: every refusal of the C ABI
(all are decided on the host, before any HIP call), the workspace sizes, and
the index arithmetic of the paged cache, compiled for the host and checked
against brute force -- pages that do not exist, lengths outside the table,
the split of a batch's keys into pieces."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from epilogue_gemm_amd import binding as gb

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED = 0, 1, 2
P = 0x10000  # stands for a device pointer: nothing here is launched


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gb.load_library()


# ---- refusals ---------------------------------------------------------------
# Each valid call below has rows, batch or M = 0, which does nothing, so that
# no refused argument can hide behind a launch.

def _rms(**kw):
    a = dict(X=P, ldx=64, R=P, ldr=64, W=P, H=P, ldh=64, Y=P, ldy=64, y_scale=None, rows=0, cols=64, eps=1e-6,
             dtype="bf16", out_dtype="bf16", stream=None)
    a.update(kw)
    return gb.gemm_epi_rmsnorm(*a.values())


@pytest.mark.parametrize("kw,want", [
    ({}, OK), ({"R": None, "ldr": 0}, OK), ({"H": None, "ldh": 0}, OK),
    ({"out_dtype": "fp8", "y_scale": P}, OK), ({"out_dtype": "fp8", "y_scale": P, "Y": P + 1}, OK),
    ({"X": None}, INVALID), ({"W": None}, INVALID), ({"Y": None}, INVALID),
    ({"rows": -1}, INVALID), ({"cols": 0}, INVALID), ({"cols": 65}, INVALID),
    ({"ldx": 63}, INVALID), ({"ldr": 63}, INVALID), ({"ldh": 63}, INVALID), ({"ldy": 63}, INVALID),
    ({"eps": -1e-6}, INVALID), ({"eps": float("nan")}, INVALID), ({"eps": float("inf")}, INVALID), ({"eps": 0.0}, OK),
    ({"dtype": "f32"}, INVALID), ({"dtype": "fp8"}, INVALID), ({"out_dtype": "f16"}, INVALID),
    ({"out_dtype": "f32"}, INVALID), ({"out_dtype": "fp8"}, INVALID), ({"y_scale": P}, INVALID),
    ({"X": P + 1}, INVALID), ({"R": P + 1}, INVALID), ({"W": P + 1}, INVALID), ({"H": P + 1}, INVALID),
    ({"Y": P + 1}, INVALID), ({"out_dtype": "fp8", "y_scale": P + 2}, INVALID),
    ({"rows": 1 << 31}, UNSUPPORTED), ({"cols": 1 << 31, "ldx": 1 << 31, "ldr": 1 << 31, "ldh": 1 << 31,
                                        "ldy": 1 << 31}, UNSUPPORTED),
])
def test_rmsnorm_refusals(kw, want):
    assert _rms(**kw) == want


def _lora(**kw):
    a = dict(X=P, ldx=64, A=P, B=P, scale=P, ids=P, R=P, ldr=40, C=P, ldc=40, M=0, N=40, K=64, rank=8, adapters=3,
             dtype="f16", ws=P, ws_bytes=1 << 30, stream=None)
    a.update(kw)
    return gb.gemm_epi_lora(*a.values())


@pytest.mark.parametrize("kw,want", [
    ({}, OK), ({"R": None, "ldr": 0}, OK), ({"scale": None}, OK), ({"ws": None, "ws_bytes": 0}, OK),
    ({"M": -1}, INVALID), ({"N": 0}, INVALID), ({"K": 0}, INVALID), ({"rank": 0}, INVALID), ({"adapters": 0}, INVALID),
    ({"ldx": 63}, INVALID), ({"ldr": 39}, INVALID), ({"ldc": 39}, INVALID), ({"dtype": "fp8"}, INVALID),
    ({"rank": 12}, UNSUPPORTED), ({"rank": 136}, UNSUPPORTED), ({"K": 60}, UNSUPPORTED),
    ({"adapters": 65536}, UNSUPPORTED), ({"M": 1 << 28}, UNSUPPORTED),
    ({"N": 65535 * 256 + 1, "ldc": 1 << 30, "ldr": 1 << 30}, UNSUPPORTED),
    ({"K": 1 << 31, "ldx": 1 << 31}, UNSUPPORTED),
    # with rows, refused before anything is launched
    ({"M": 5, "X": None}, INVALID), ({"M": 5, "A": None}, INVALID), ({"M": 5, "B": None}, INVALID),
    ({"M": 5, "ids": None}, INVALID), ({"M": 5, "C": None}, INVALID), ({"M": 5, "ws": None}, INVALID),
    ({"M": 5, "ws_bytes": 16}, INVALID), ({"M": 5, "C": P + 1}, INVALID), ({"M": 5, "R": P + 1}, INVALID),
    ({"M": 5, "ids": P + 2}, INVALID), ({"M": 5, "scale": P + 2}, INVALID),
    ({"M": 5, "X": P + 8}, UNSUPPORTED), ({"M": 5, "A": P + 8}, UNSUPPORTED), ({"M": 5, "B": P + 8}, UNSUPPORTED),
    ({"M": 5, "ws": P + 8}, UNSUPPORTED), ({"M": 5, "ldx": 68}, UNSUPPORTED),
])
def test_lora_refusals(kw, want):
    assert _lora(**kw) == want


def test_lora_workspace_size():
    # a multiple of one fp32 row of the padded rank for each row and range of
    # K; nothing for sizes that are refused
    size = gb.gemm_epi_lora_workspace_size
    for M, K, rank, pad in ((1, 8, 8, 16), (16, 4096, 16, 16), (100, 4096, 40, 64), (33, 1000, 128, 128), (20000, 4096, 8, 16)):
        n = size(M, 100, K, rank, 4)
        assert n > 0 and n % (M * pad * 4) == 0
    assert size(0, 100, 64, 8, 4) == 0 == size(4, 100, 64, 12, 4) == size(4, 100, 64, 8, 0)
    assert max(size(M, 100, K, 128, 4) for M in range(1, 2000) for K in (8, 4096, 1 << 20)) < 256 << 20


_CACHE = dict(k=P, v=P, k_scale=None, v_scale=None, num_pages=9, page_size=16, heads=2, head_dim=64, dtype="bf16")
_TABLE = dict(pages=P, ld=4, width=4, lens=P, batch=0)
_CACHE_CASES = [
    ({"k": None}, INVALID), ({"v": None}, INVALID), ({"k_scale": P}, INVALID), ({"v_scale": P}, INVALID),
    ({"dtype": "fp8"}, INVALID), ({"dtype": "fp8", "k_scale": P}, INVALID), ({"dtype": "fp8", "v_scale": P}, INVALID),
    ({"dtype": "fp8", "k_scale": P, "v_scale": P}, OK), ({"dtype": "f32"}, INVALID), ({"dtype": "f16"}, INVALID),
    ({"num_pages": 0}, INVALID), ({"page_size": 0}, INVALID), ({"heads": 0}, INVALID), ({"head_dim": 0}, INVALID),
    ({"head_dim": 80}, UNSUPPORTED), ({"head_dim": 256}, UNSUPPORTED), ({"page_size": 8}, UNSUPPORTED),
    ({"page_size": 24}, UNSUPPORTED), ({"page_size": 65552}, UNSUPPORTED), ({"page_size": 48}, OK),
    ({"heads": 1026}, UNSUPPORTED), ({"num_pages": 1 << 28}, UNSUPPORTED), ({"num_pages": 1 << 31}, UNSUPPORTED),
    ({"k": P + 8}, UNSUPPORTED), ({"v": P + 8}, UNSUPPORTED),
    ({"dtype": "fp8", "k_scale": P + 8, "v_scale": P}, UNSUPPORTED),
]
_TABLE_CASES = [
    ({"ld": 3}, INVALID), ({"width": 0}, INVALID), ({"batch": -1}, INVALID), ({"batch": 65536}, UNSUPPORTED),
    ({"width": 1 << 31, "ld": 1 << 31}, UNSUPPORTED), ({"width": 1 << 27, "ld": 1 << 27}, UNSUPPORTED),
    ({"width": (1 << 27) - 16, "ld": 1 << 27}, OK), ({"ld": 1 << 31}, UNSUPPORTED),
    ({"batch": 1024, "width": 1 << 24, "ld": 1 << 24}, UNSUPPORTED),
    ({"batch": 1, "pages": None}, INVALID), ({"batch": 1, "lens": None}, INVALID), ({"batch": 1, "pages": P + 2}, INVALID),
    ({"batch": 1, "lens": P + 2}, INVALID),
]


def _structs(cache, table):
    return gb.paged_cache_struct(*{**_CACHE, **cache}.values()), gb.page_table_struct(*{**_TABLE, **table}.values())


def _append(cache={}, table={}, **kw):
    c, t = _structs(cache, table)
    a = dict(K=P, ldk=2048, V=P, ldv=2048, starts=None, tokens=t.batch, dtype="bf16", stream=None)
    a.update(kw)
    return gb.gemm_epi_cache_append(c, t, *a.values())


def _decode(cache={}, table={}, **kw):
    c, t = _structs(cache, table)
    a = dict(Q=P, ldq=4096, O=P, ldo=4096, q_heads=c.heads * 2 if 0 < c.heads < 16 else max(c.heads, 1), dtype="bf16",
             ws=P, ws_bytes=1 << 40, stream=None)
    a.update(kw)
    return gb.gemm_epi_attention_decode(c, t, *a.values())


@pytest.mark.parametrize("kw,want", _CACHE_CASES)
def test_cache_refusals(kw, want):
    assert _append(kw) == want
    assert _decode(kw) == want


@pytest.mark.parametrize("kw,want", _TABLE_CASES)
def test_table_refusals(kw, want):
    assert _append({}, kw) == want
    assert _decode({}, kw) == want


@pytest.mark.parametrize("kw,want", [
    ({}, OK), ({"K": None, "V": None}, OK), ({"ldk": 127}, INVALID), ({"ldv": 127}, INVALID), ({"tokens": 1}, INVALID),
    ({"tokens": -1, "starts": P}, INVALID), ({"tokens": 7, "starts": P}, OK), ({"starts": P + 2}, INVALID),
    ({"dtype": "f16"}, INVALID), ({"dtype": "fp8"}, INVALID), ({"ldk": 132}, UNSUPPORTED), ({"ldv": 132}, UNSUPPORTED),
    ({"tokens": 1 << 26, "starts": P}, UNSUPPORTED),
    ({"table": {"batch": 1}, "tokens": 0}, INVALID), ({"table": {"batch": 1}, "tokens": 0, "starts": P}, OK),
    ({"table": {"batch": 1}, "K": None}, INVALID), ({"table": {"batch": 1}, "V": None}, INVALID),
    ({"table": {"batch": 1}, "K": P + 8}, UNSUPPORTED), ({"table": {"batch": 1}, "V": P + 8}, UNSUPPORTED),
])
def test_append_refusals(kw, want):
    assert _append(**kw) == want


@pytest.mark.parametrize("kw,want", [
    ({}, OK), ({"q_heads": 0}, INVALID), ({"q_heads": 3}, INVALID), ({"q_heads": 16386, "ldq": 1 << 21, "ldo": 1 << 21},
                                                                     UNSUPPORTED),
    ({"ldq": 255}, INVALID), ({"ldo": 255}, INVALID), ({"ldq": 260}, UNSUPPORTED), ({"ldo": 260}, UNSUPPORTED),
    ({"dtype": "f16"}, INVALID), ({"dtype": "fp8"}, INVALID), ({"dtype": "f32"}, INVALID),
    ({"table": {"batch": 1}, "Q": None}, INVALID), ({"table": {"batch": 1}, "O": None}, INVALID),
    ({"table": {"batch": 1}, "ws": None}, INVALID), ({"table": {"batch": 1}, "ws_bytes": 64}, INVALID),
    ({"table": {"batch": 1}, "Q": P + 8}, UNSUPPORTED), ({"table": {"batch": 1}, "O": P + 8}, UNSUPPORTED),
    ({"table": {"batch": 1}, "ws": P + 8}, UNSUPPORTED),
])
def test_decode_refusals(kw, want):
    assert _decode(**kw) == want


def test_null_structs():
    c, t = _structs({}, {})
    assert gb.gemm_epi_cache_append(None, t, P, 128, P, 128, None, 0, "bf16", None) == INVALID
    assert gb.gemm_epi_cache_append(c, None, P, 128, P, 128, None, 0, "bf16", None) == INVALID
    assert gb.gemm_epi_attention_decode(None, t, P, 256, P, 256, 4, "bf16", P, 1 << 20, None) == INVALID
    assert gb.gemm_epi_attention_decode(c, None, P, 256, P, 256, 4, "bf16", P, 1 << 20, None) == INVALID
    assert gb.gemm_epi_attention_decode_workspace_size(None, 1, 1, 4) == 0


def test_decode_workspace_size():
    c, _ = _structs({}, {})
    size = gb.gemm_epi_attention_decode_workspace_size
    assert size(c, 0, 4, 4) == 0 and size(c, 1, 0, 4) == 0 and size(c, 1, 4, 3) == 0 and size(c, 65536, 4, 4) == 0
    # grows with the batch and the width, and stays small for wide tables
    assert 0 < size(c, 1, 4, 4) <= size(c, 2, 4, 4) <= size(c, 2, 64, 4)
    assert size(c, 64, 1 << 16, 4) < 64 << 20


# ---- index arithmetic of the paged cache, on the host ------------------------

_WRAP = r'''
#include "paged.hpp"
using namespace ge::paged;
extern "C" {
int c_seq_len(int s, int cap) { return seq_len(s, cap); }
int c_page_or_none(int e, int n) { return page_or_none(e, n); }
int c_divide(int n, int d) { return divide(n, make_divider(d)); }
int64_t c_row_of(int p, int hs, int h, int ps, int s) { return row_of(p, hs, h, ps, s); }
int c_new_position(int len, int end, int row, int cap) { return new_position(len, end, row, cap); }
int c_units_of(int len) { return units_of(len); }
int c_shares(int F, int n) { return make_shares(F, n).n; }
int c_share_begin(int F, int n, int w) { return share_begin(make_shares(F, n), w); }
int c_share_of(int F, int n, int f) { return share_of(make_shares(F, n), f); }
int c_workgroups_of(int F, int most) { return workgroups_of(F, most); }
int c_joined_here(int pieces, int rows, int d) { return joined_here(pieces, rows, d); }
int64_t c_pieces_bound(int64_t cap, int columns, int n) { return pieces_bound(cap, columns, n); }
}
'''


@pytest.fixture(scope="module")
def paged(tmp_path_factory):
    d = tmp_path_factory.mktemp("paged")
    src, so = d / "wrap.cpp", d / "wrap.so"
    src.write_text(_WRAP)
    r = subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                        "-static-libubsan", "-shared", "-fPIC", "-I", os.path.join(ROOT, "epilogue_gemm_amd", "csrc"),
                        str(src), "-o", str(so)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lib = ctypes.CDLL(str(so))
    lib.c_row_of.restype = ctypes.c_int64
    lib.c_pieces_bound.restype = ctypes.c_int64
    lib.c_pieces_bound.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int]
    return lib


INT_MIN, INT_MAX = -(1 << 31), (1 << 31) - 1


def test_lengths_and_pages_outside_the_table(paged):
    for stored in (INT_MIN, -1, 0, 1, 63, 64, 65, INT_MAX):
        assert paged.c_seq_len(stored, 64) == min(max(stored, 0), 64)
    for entry in (INT_MIN, -2, -1, 0, 1, 8, 9, 10, INT_MAX):
        assert paged.c_page_or_none(entry, 9) == (entry if 0 <= entry < 9 else -1)


def test_page_of_a_position(paged):
    rng = np.random.default_rng(0)
    for d in [*range(1, 200), 255, 256, 257, 1000, 4093, 4095, 4096]:
        top = (1 << 27) - 1
        ns = {0, 1, d - 1, d, d + 1, top, top - 1, top // d * d, top // d * d - 1, *rng.integers(0, 1 << 27, 50).tolist()}
        for n in ns:
            assert paged.c_divide(n, d) == n // d, (n, d)


def test_every_row_of_every_page_is_inside_and_its_own(paged):
    pages, heads, ps = 5, 3, 16
    seen = {paged.c_row_of(p, heads, h, ps, s) for p in range(pages) for h in range(heads) for s in range(ps)}
    assert seen == set(range(pages * heads * ps))
    # the largest cache: 2^31 - 1 slots, 1024 heads
    assert paged.c_row_of((1 << 27) - 2, 1024, 1023, 16, 15) == (((1 << 27) - 2) * 1024 + 1023) * 16 + 15


def test_new_positions(paged):
    cap = 64
    for length in (INT_MIN, -3, 0, 1, 5, 64, 65, 200, INT_MAX):
        for end, row in ((1, 0), (5, 0), (5, 4), (70, 0), (0, 3), (INT_MAX, 0), (INT_MIN, INT_MAX), (INT_MIN, 0)):
            p = length - (end - row)
            assert paged.c_new_position(length, end, row, cap) == (p if 0 <= p < cap else -1)


def test_units(paged):
    for n in (0, 1, 127, 128, 129, 4096, INT_MAX - 256, INT_MAX):
        assert paged.c_units_of(n) == -(-n // 128)


@pytest.mark.parametrize("seed", range(40))
def test_shares_cover_every_unit_once(paged, seed):
    rng = np.random.default_rng(seed)
    F = int(rng.choice([1, 2, 7, 511, 512, 513, 100003, 1 << 30, INT_MAX]))
    given = int(rng.choice([1, 2, 8, 63, 512]))
    W = paged.c_shares(F, given)
    assert W == min(F, given) and paged.c_shares(0, given) == 0
    begins = [paged.c_share_begin(F, given, w) for w in range(W + 1)]
    assert begins[0] == 0 and begins[-1] == F
    sizes = np.diff(np.array(begins, dtype=np.int64))
    assert sizes.min() >= 1 and sizes.max() - sizes.min() <= 1  # even
    for f in {0, F - 1, *[int(x) for x in rng.integers(0, F, 50)], *[b for b in begins if b < F], *[b - 1 for b in begins if b > 0]}:
        w = paged.c_share_of(F, given, f)
        assert begins[w] <= f < begins[w + 1], (F, W, f)


@pytest.mark.parametrize("seed", range(20))
def test_pieces_stay_within_their_bound(paged, seed):
    # a batch's sequences, column by column, cut where shares end
    rng = np.random.default_rng(100 + seed)
    cap = int(rng.choice([16, 128, 1000, 8192, 100000]))
    units = [paged.c_units_of(int(n)) for n in rng.integers(0, cap + 1, size=int(rng.integers(1, 40)))]
    columns, given = int(rng.choice([1, 2, 8, 30, 600])), 512
    F = sum(units) * columns
    bound = paged.c_pieces_bound(cap, columns, given)
    at = 0
    for _ in range(min(columns, 3)):
        for u in units:
            if u:
                pieces = paged.c_share_of(F, given, at + u - 1) - paged.c_share_of(F, given, at) + 1
                assert pieces <= bound, (pieces, bound)
            at += u


def test_who_joins(paged):
    # more pieces or rows never move a join into the main kernel
    for d in (64, 128):
        for rows in range(1, 17):
            here = [paged.c_joined_here(p, rows, d) for p in range(1, 600)]
            assert here[0] and here == sorted(here, reverse=True)
            if rows > 1:
                assert all(a <= b for a, b in zip(here, [paged.c_joined_here(p, rows - 1, d) for p in range(1, 600)]))


def test_workgroups_of_few_units(paged):
    for most in (1, 100, 256, 300, 512):
        n = [paged.c_workgroups_of(F, most) for F in (0, 1, 2047, 2048, 2056, 3000, 4096, 1 << 20, INT_MAX)]
        assert all(1 <= x <= most for x in n) and n == sorted(n) and n[0] == min(most, 256) and n[-3:] == [most] * 3


@pytest.mark.parametrize("seed", range(10))
def test_pieces_of_few_units_stay_within_the_bound_for_all_workgroups(paged, seed):
    # the host bounds the pieces by the most workgroups, the kernels may take fewer
    rng = np.random.default_rng(200 + seed)
    cap, columns = int(rng.choice([1000, 8192, 100000])), int(rng.choice([1, 2, 8, 30]))
    units = [paged.c_units_of(int(n)) for n in rng.integers(0, cap + 1, size=int(rng.integers(1, 9)))]
    F = sum(units) * columns
    n, bound = paged.c_workgroups_of(F, 512), paged.c_pieces_bound(cap, columns, 512)
    at = 0
    for u in units:
        if u:
            assert paged.c_share_of(F, n, at + u - 1) - paged.c_share_of(F, n, at) + 1 <= bound
        at += u


def test_tensor_calls_refuse_what_is_not_a_cuda_tensor():
    # the host-only module's own checks; the device's index and stream are not used before them
    torch = pytest.importorskip("torch")
    gb.load_library()
    from epilogue_gemm_amd import _calls
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    t = torch.zeros(2, 8, 8, dtype=torch.bfloat16)
    for f, args in ((_calls.rmsnorm, (x, x[0], x, None, None, None, 1e-6)), (_calls.rmsnorm, (1, x[0], x, None, None, None, 1e-6)),
                    (_calls.rmsnorm, (x[0], x[0], x, None, None, None, 1e-6)), (_calls.rmsnorm, (x.float(), x[0], x, None, None, None, 1e-6)),
                    (_calls.lora, (x, t, t, x, x, None, None, None)), (_calls.lora, (x, x, t, x, x, None, None, None))):
        with pytest.raises(ValueError):
            f(0, 0, *args)
    with pytest.raises(TypeError):
        _calls.attend(0, 0)
