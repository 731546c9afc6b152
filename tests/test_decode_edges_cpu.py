"""The decode operators' index arithmetic (csrc/paged.hpp) over whole ranges of
sizes, compiled for the host with the checks for undefined behaviour on."""
import ctypes
import os
import subprocess

import pytest

from epilogue_gemm_amd import binding as gb

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def compiled(tmp_path, text):
    src, so = tmp_path / "wrap.cpp", tmp_path / "wrap.so"
    src.write_text('#include "paged.hpp"\nusing namespace ge::paged;\nextern "C" {\n' + text + "\n}\n")
    r = subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                        "-static-libubsan", "-shared", "-fPIC", "-I", os.path.join(ROOT, "epilogue_gemm_amd", "csrc"),
                        str(src), "-o", str(so)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return ctypes.CDLL(str(so))


@pytest.mark.parametrize("most", [256, 512])
def test_every_cut_sequence_is_joined(tmp_path, most):
    # One sequence of U units in each of `columns` columns (the batch whose
    # sequences are cut into the most pieces), all columns, and tables of its
    # length and wider: the pieces stay within the host's bound, so a join
    # that the main kernel leaves is one that the host launches.
    lib = compiled(tmp_path, r'''
    int sweep(int most, int columns, int units, int* at) {
      for (int U = 1; U <= units; ++U)
        for (int wide = 0; wide < 2; ++wide) {
          const int64_t cap = wide ? 1 << 22 : (int64_t)U * kUnit, full = cap / kUnit * columns;
          const int wgs = full < most ? (int)full : most, F = U * columns;
          const Shares s = make_shares(F, workgroups_of(F, wgs));
          const int bound = (int)pieces_bound(cap, columns, wgs);
          for (int c = 0; c < columns; ++c) {
            const int pieces = share_of(s, c * U + U - 1) - share_of(s, c * U) + 1;
            bool left = pieces > bound;
            for (int rows = 1; rows <= 16; ++rows)
              for (int d = 64; d <= 128; d += 64)
                left = left || (joined_here(bound, rows, d) && !joined_here(pieces, rows, d));
            if (left) {
              at[0] = U; at[1] = c; at[2] = pieces; at[3] = bound;
              return 1;
            }
          }
        }
      return 0;
    }''')
    at = (ctypes.c_int * 4)()
    for columns in range(1, 65):
        assert lib.sweep(most, columns, 600, at) == 0, (columns, "units, column, pieces, bound", list(at))


def test_shares_are_even_and_every_number_is_in_its_own(tmp_path):
    # floor(w F / n) exactly, and the share of every number, for all small F
    # and at the largest
    lib = compiled(tmp_path, r'''
    int sweep(int from, int to, int given) {
      for (int F = from;; ++F) {
        const Shares s = make_shares(F, given);
        if (s.n != (F < given ? F : given)) return F;
        for (int w = 0; w < s.n; ++w) {
          const int a = share_begin(s, w), b = share_begin(s, w + 1);
          if (a != (int)((int64_t)w * F / s.n) || b <= a || b - a - s.base > 1) return F;
          if (share_of(s, a) != w || share_of(s, b - 1) != w || share_of(s, a + (b - a) / 2) != w) return F;
        }
        if (share_begin(s, s.n) != F) return F;
        if (F == to) return 0;
      }
    }''')
    for given in (1, 2, 3, 100, 255, 256, 257, 509, 511, 512):
        for start, to in ((1, 3000), ((1 << 24) - 100, (1 << 24) + 100), ((1 << 30) - 100, (1 << 30) + 100), ((1 << 31) - 300, (1 << 31) - 1)):
            assert lib.sweep(start, to, given) == 0, (start, given)


def test_every_share_is_one_workgroups(tmp_path):
    # and the larger shares are spread over the workgroups that share an XCD
    lib = compiled(tmp_path, r"""
    int c_shares(int F, int given) { return make_shares(F, given).n; }
    int c_share_at(int F, int given, int workgroup) { return share_at(make_shares(F, given), workgroup); }
    int c_size(int F, int given, int w) { const Shares s = make_shares(F, given); return share_begin(s, w + 1) - share_begin(s, w); }
    """)
    for given in (1, 7, 8, 100, 256, 512):
        for F in (1, 5, 8, 250, 256, 257, 300, 528, 1000, 4100, 100003):
            n = lib.c_shares(F, given)
            at = [lib.c_share_at(F, given, b) for b in range(n)]
            assert sorted(at) == list(range(n))
            if n % 8 == 0:
                units = [sum(lib.c_size(F, given, w) for w in at[x::8]) for x in range(8)]
                assert max(units) - min(units) <= 1, (F, given, units)


def test_looked_up_keys_stay_inside_up_to_the_longest_table(tmp_path):
    # the lookups that every wave makes in the shares of one sequence, at the
    # largest table (2^31 - 256 tokens) and at small sizes: the key in 64 bits,
    # or none past the last tile
    lib = compiled(tmp_path, r'''
    int64_t sweep(int len, int columns, int most) {
      const int U = units_of(len), F = U * columns;
      const Shares s = make_shares(F, workgroups_of(F, most));
      int64_t keys = 0;
      for (int w = 0; w < s.n; ++w)
        for (int f = share_begin(s, w), end = share_begin(s, w + 1); f < end;) {
          const int u = f % U, take = end - f < U - u ? end - f : U - u;
          const int kbeg = u * kUnit, kend = len < kbeg + take * kUnit ? len : kbeg + take * kUnit;
          for (int wave = 0; wave < 4; ++wave) {
            const int k1 = kbeg + 32 * wave, last = k1 < kend ? (kend - 1 - k1) / 128 : -1;
            for (int n = 0; n <= last; n += 32) {
              if (n == 64 && last > 256) n = (last - 64) / 32 * 32;  // the middle ones are alike
              for (int lane = 0; lane < 64; ++lane) {
                const int64_t k = (int64_t)k1 + 128 * (int64_t)(n + (lane >> 1)), kg = k + 16 * (lane & 1);
                if (looked_up_key(k1, kend, last, n + (lane >> 1), lane & 1) != (k >= kend ? -1 : kg < kend ? kg : k)) return -1;
                keys += k < kend;
              }
            }
          }
          f += take;
        }
      return keys;
    }''')
    lib.sweep.restype = ctypes.c_int64
    for length in (1, 16, 17, 33, 127, 128, 129, 5003, 100000):
        for columns in (1, 3):
            # two lookups a tile
            assert lib.sweep(length, columns, 256) == 2 * columns * -(-length // 32)
    for most in (256, 512):
        for columns in (1, 2, 4, 100):
            for length in ((1 << 31) - 256, (1 << 31) - 256 - 15, (1 << 31) - 65536):
                assert lib.sweep(length, columns, most) > 0


def test_the_library_builds_without_torch(monkeypatch, tmp_path, capsys):
    # build() up to its end on a machine without torch: the C library linked,
    # the tensor calls left out
    from epilogue_gemm_amd import build as b
    monkeypatch.setattr(b, "BUILD", str(tmp_path))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(b, "CALLS", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(b, "sources", lambda: [os.path.join(b.CSRC, "tuning.cpp")])
    found = b.importlib.util.find_spec
    monkeypatch.setattr(b.importlib.util, "find_spec", lambda name, *a: None if name == "torch" else found(name, *a))
    b.build(verbose=True)
    assert os.path.exists(b.LIB) and not os.path.exists(b.CALLS)
    assert "torch is not installed" in capsys.readouterr().out


def test_sizes_that_no_grid_holds_are_refused():
    # 2^24 workgroups of 256 would be 2^32 threads
    OK, INVALID, UNSUPPORTED, P = 0, 1, 2, 0x10000
    cache = gb.paged_cache_struct(P, P, None, None, 9, 16, 2, 64, "bf16")
    table = gb.page_table_struct(P, 4, 4, P, 0)  # (no sequences: nothing is launched)
    for tokens, want in (((1 << 26) - 4, OK), ((1 << 26) - 3, UNSUPPORTED), ((1 << 26) - 1, UNSUPPORTED)):
        assert gb.gemm_epi_cache_append(cache, table, P, 128, P, 128, P, tokens, "bf16", None) == want
    for M, want in (((1 << 28) - 16, INVALID), ((1 << 28) - 15, UNSUPPORTED), ((1 << 28) - 1, UNSUPPORTED)):
        # (no ids: refused before anything is launched)
        assert gb.gemm_epi_lora(P, 64, P, P, None, None, None, 0, P, 64, M, 64, 64, 8, 2, "f16", P, 1 << 60, None) == want
        assert (gb.gemm_epi_lora_workspace_size(M, 64, 64, 8, 2) > 0) == (want == INVALID)


def test_rmsnorm_takes_any_finite_eps():
    for eps, want in ((0.0, 0), (3.4e38, 0), (3.5e38, 1), (float("inf"), 1), (float("nan"), 1), (-1e-45, 1)):
        # (no rows: nothing is launched; 3.5e38 is an infinity in fp32)
        assert gb.gemm_epi_rmsnorm(0x10000, 64, None, 0, 0x10000, None, 0, 0x10000, 64, None, 0, 64, eps, "bf16", "bf16", None) == want
