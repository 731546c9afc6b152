"""Python binding of libgemm_epi.so (include/gemm_epi.h) -- argument
marshalling only.

The functions below carry the C names and call straight into the library;
every step of the computation runs in its HIP kernels.  ``Plan`` is a thin
convenience over them that takes torch CUDA tensors (used only as device
memory) and torch's current stream.  There is no fallback: if the library
is missing, loading fails with an error that says how to build it.
"""
from __future__ import annotations

import ctypes
import os
import re

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgemm_epi.so")
CALLS_PATH = os.path.join(_HERE, "_calls.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "gemm_epi.h")

# Enum values of include/gemm_epi.h
DTYPES = {"f16": 0, "bf16": 1, "f32": 2, "fp8": 3, "i8": 4}
LAYOUTS = {"row": 0, "col": 1}
EPILOGUES = {"none": 0, "relu": 1, "bias_relu": 2, "bias_gelu": 3, "bias": 4, "silu": 5, "bias_silu": 6}
KERNELS = {"auto": 0, "generic": 1, "tile": 2, "skinny": 3}
SCORES = {"softmax": 0, "sigmoid": 1}  # include/gemm_epi_experts.h
GATHER, SCATTER, GATED = 1, 2, 4
KERNEL_NAMES = {v: k for k, v in KERNELS.items()}
STATUS = {0: "OK", 1: "ERR_INVALID_ARG", 2: "ERR_UNSUPPORTED", 3: "ERR_HIP", 4: "ERR_NO_MEMORY"}
OK = 0


class Extras(ctypes.Structure):
    """struct gemm_epi_extras: optional column scale, residual and output
    scale pointers."""
    _fields_ = [("col_scale", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("out_scale", ctypes.c_void_p)]


class _PagedCache(ctypes.Structure):
    """struct gemm_epi_paged_cache (include/gemm_epi_decode.h)."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int64),
                ("heads", ctypes.c_int64), ("head_dim", ctypes.c_int64), ("dtype", ctypes.c_int)]


class _PageTable(ctypes.Structure):
    """struct gemm_epi_page_table (include/gemm_epi_decode.h)."""
    _fields_ = [("pages", ctypes.c_void_p), ("ld", ctypes.c_int64), ("width", ctypes.c_int64),
                ("lens", ctypes.c_void_p), ("batch", ctypes.c_int64)]


class _Groups(ctypes.Structure):
    """struct gemm_epi_groups (include/gemm_epi_experts.h)."""
    _fields_ = [("offsets", ctypes.c_void_p), ("order", ctypes.c_void_p), ("groups", ctypes.c_int64),
                ("rows", ctypes.c_int64), ("per", ctypes.c_int64)]


class GemmEpiError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        msg = f"{fn} returned {gemm_epi_status_string(status)}"
        if status == 3:
            msg += f" (hipError_t {gemm_epi_last_hip_error()})"
        super().__init__(msg)


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libgemm_epi.so once.  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: the HIP library has not been built. "
            "Run `python -c 'import __graft_entry__ as g; g.build()'` or "
            "`python epilogue_gemm_amd/build.py` first.")
    lib = ctypes.CDLL(path)
    i64, i32, vp, cp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_char_p
    lib.gemm_epi_plan.argtypes = [ctypes.POINTER(vp), i64, i64, i64, i32, i32, i32, i32, i32]
    lib.gemm_epi_plan.restype = i32
    lib.gemm_epi_plan_set_ld.argtypes = [vp, i64, i64, i64]
    lib.gemm_epi_plan_set_ld.restype = i32
    lib.gemm_epi_run.argtypes = [vp, vp, vp, vp, vp, vp]
    lib.gemm_epi_run.restype = i32
    lib.gemm_epi_workspace_size.argtypes = [vp]
    lib.gemm_epi_workspace_size.restype = ctypes.c_size_t
    lib.gemm_epi_run_ws.argtypes = [vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    lib.gemm_epi_run_ws.restype = i32
    lib.gemm_epi_run_noalloc.argtypes = [vp, vp, vp, vp, vp, vp]
    lib.gemm_epi_run_noalloc.restype = i32
    lib.gemm_epi_run_ex.argtypes = [vp, vp, vp, vp, ctypes.POINTER(Extras), vp, vp, ctypes.c_size_t, vp]
    lib.gemm_epi_run_ex.restype = i32
    lib.gemm_epi_tune.argtypes = [vp, vp, vp, vp, vp, i32, i32, vp, ctypes.POINTER(ctypes.c_float)]
    lib.gemm_epi_tune.restype = i32
    lib.gemm_epi_tuning_save.argtypes = [cp]
    lib.gemm_epi_tuning_save.restype = i32
    lib.gemm_epi_tuning_load.argtypes = [cp]
    lib.gemm_epi_tuning_load.restype = i32
    lib.gemm_epi_tuning_clear.argtypes = []
    lib.gemm_epi_tuning_clear.restype = None
    lib.gemm_epi_tuning_size.argtypes = []
    lib.gemm_epi_tuning_size.restype = i32
    lib.gemm_epi_attention_fwd.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, i32, i32, vp]
    lib.gemm_epi_attention_fwd.restype = i32
    lib.gemm_epi_destroy.argtypes = [vp]
    lib.gemm_epi_destroy.restype = i32
    lib.gemm_epi_status_string.argtypes = [i32]
    lib.gemm_epi_status_string.restype = cp
    lib.gemm_epi_last_hip_error.argtypes = []
    lib.gemm_epi_last_hip_error.restype = i32
    lib.gemm_epi_plan_select.argtypes = [vp, i32, i32]
    lib.gemm_epi_plan_select.restype = i32
    lib.gemm_epi_num_configs.argtypes = [i32]
    lib.gemm_epi_num_configs.restype = i32
    lib.gemm_epi_plan_describe.argtypes = [vp, ctypes.POINTER(i32), ctypes.POINTER(i32)]
    lib.gemm_epi_plan_describe.restype = cp
    # the operators of a decode step (include/gemm_epi_decode.h)
    sz, f32 = ctypes.c_size_t, ctypes.c_float
    pc, pt = ctypes.POINTER(_PagedCache), ctypes.POINTER(_PageTable)
    lib.gemm_epi_rmsnorm.argtypes = [vp, i64, vp, i64, vp, vp, i64, vp, i64, vp, i64, i64, f32, i32, i32, vp]
    lib.gemm_epi_rmsnorm.restype = i32
    lib.gemm_epi_lora.argtypes = [vp, i64, vp, vp, vp, vp, vp, i64, vp, i64, i64, i64, i64, i64, i64, i32, vp, sz, vp]
    lib.gemm_epi_lora.restype = i32
    lib.gemm_epi_lora_workspace_size.argtypes = [i64, i64, i64, i64, i64]
    lib.gemm_epi_lora_workspace_size.restype = sz
    lib.gemm_epi_cache_append.argtypes = [pc, pt, vp, i64, vp, i64, vp, i64, i32, vp]
    lib.gemm_epi_cache_append.restype = i32
    lib.gemm_epi_attention_decode.argtypes = [pc, pt, vp, i64, vp, i64, i64, i32, vp, sz, vp]
    lib.gemm_epi_attention_decode.restype = i32
    lib.gemm_epi_attention_decode_workspace_size.argtypes = [pc, i64, i64, i64]
    lib.gemm_epi_attention_decode_workspace_size.restype = sz
    # the experts' feed-forward and 8-bit products (include/gemm_epi_experts.h)
    lib.gemm_epi_quantise_i8.argtypes = [vp, i64, vp, i64, vp, i64, i64, i32, vp]
    lib.gemm_epi_quantise_i8.restype = i32
    lib.gemm_epi_i8_gemm.argtypes = [vp, i64, vp, vp, i64, vp, vp, vp, i64, vp, i64, i64, i64, i64, i32, i32, vp]
    lib.gemm_epi_i8_gemm.restype = i32
    lib.gemm_epi_route.argtypes = [vp, i64, i32, i64, i64, i64, i32, i32, f32, vp, vp, vp, vp, vp]
    lib.gemm_epi_route.restype = i32
    lib.gemm_epi_group_rows.argtypes = [vp, i64, i64, vp, vp, vp]
    lib.gemm_epi_group_rows.restype = i32
    lib.gemm_epi_grouped_gemm.argtypes = [ctypes.POINTER(_Groups), vp, i64, vp, vp, vp, vp, vp, i64, i64, i64, i32,
                                          i32, i32, i32, vp]
    lib.gemm_epi_grouped_gemm.restype = i32
    lib.gemm_epi_combine.argtypes = [vp, i64, vp, vp, i64, vp, i64, vp, i64, i64, i64, i64, i32, vp]
    lib.gemm_epi_combine.restype = i32
    # measurement helpers (include/gemm_epi_probes.h)
    lib.gemm_epi_probe_hbm_read.argtypes = [vp, ctypes.c_size_t, vp, vp]
    lib.gemm_epi_probe_hbm_read.restype = i32
    lib.gemm_epi_probe_mfma.argtypes = [i32, i32, vp, vp]
    lib.gemm_epi_probe_mfma.restype = i32
    lib.gemm_epi_probe_mfma_flops.argtypes = [i32, i32]
    lib.gemm_epi_probe_mfma_flops.restype = ctypes.c_double
    _lib = lib
    return lib


def headers():
    """Every header of the C ABI (include/*.h)."""
    d = os.path.dirname(HEADER)
    return sorted(os.path.join(d, f) for f in os.listdir(d) if f.endswith(".h"))


def header_functions(header: str | None = None):
    """Names of the functions the C ABI headers declare (all of include/*.h,
    or the one given)."""
    names = set()
    for h in [header] if header else headers():
        text = open(h).read()
        text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
        names.update(re.findall(r"\b(gemm_epi_\w+)\s*\(", text))
    return sorted(names)


# ---- the C entry points, same names ----------------------------------------

def gemm_epi_plan(M, N, K, in_dtype, out_dtype, layout_a, layout_b, epilogue) -> int:
    """Returns the plan handle (an int); raises GemmEpiError on failure."""
    h = ctypes.c_void_p()
    st = load_library().gemm_epi_plan(ctypes.byref(h), int(M), int(N), int(K), DTYPES[in_dtype], DTYPES[out_dtype],
                                      LAYOUTS[layout_a], LAYOUTS[layout_b], EPILOGUES[epilogue])
    if st != OK:
        raise GemmEpiError("gemm_epi_plan", st)
    return h.value


def gemm_epi_plan_status(M, N, K, in_dtype, out_dtype, layout_a, layout_b, epilogue, raw=False) -> int:
    """Status code of gemm_epi_plan for raw (possibly invalid) enum values;
    destroys the plan if one was made.  For tests of argument validation."""
    h = ctypes.c_void_p()
    lib = load_library()
    if raw:
        args = (in_dtype, out_dtype, layout_a, layout_b, epilogue)
    else:
        args = (DTYPES[in_dtype], DTYPES[out_dtype], LAYOUTS[layout_a], LAYOUTS[layout_b], EPILOGUES[epilogue])
    st = lib.gemm_epi_plan(ctypes.byref(h), int(M), int(N), int(K), *args)
    if st == OK:
        lib.gemm_epi_destroy(h)
    return st


def gemm_epi_plan_set_ld(plan, lda=0, ldb=0, ldc=0) -> int:
    return load_library().gemm_epi_plan_set_ld(plan, int(lda), int(ldb), int(ldc))


def gemm_epi_run(plan, A_ptr, B_ptr, bias_ptr, C_ptr, stream) -> int:
    return load_library().gemm_epi_run(plan, A_ptr, B_ptr, bias_ptr, C_ptr, stream)


def gemm_epi_run_noalloc(plan, A_ptr, B_ptr, bias_ptr, C_ptr, stream) -> int:
    return load_library().gemm_epi_run_noalloc(plan, A_ptr, B_ptr, bias_ptr, C_ptr, stream)


def gemm_epi_workspace_size(plan) -> int:
    return int(load_library().gemm_epi_workspace_size(plan))


def gemm_epi_run_ws(plan, A_ptr, B_ptr, bias_ptr, C_ptr, ws_ptr, ws_bytes, stream) -> int:
    return load_library().gemm_epi_run_ws(plan, A_ptr, B_ptr, bias_ptr, C_ptr, ws_ptr, int(ws_bytes), stream)


def gemm_epi_run_ex(plan, A_ptr, B_ptr, bias_ptr, scale_ptr, residual_ptr, C_ptr, ws_ptr, ws_bytes, stream,
                    extras_null=False, out_scale_ptr=None) -> int:
    """extras_null passes a NULL gemm_epi_extras pointer (the three extras
    pointers are then ignored)."""
    ex = None if extras_null else ctypes.byref(Extras(scale_ptr, residual_ptr, out_scale_ptr))
    return load_library().gemm_epi_run_ex(plan, A_ptr, B_ptr, bias_ptr, ex, C_ptr, ws_ptr, int(ws_bytes), stream)


TUNE_COLD = 1


def gemm_epi_tune(plan, A_ptr, B_ptr, bias_ptr, C_ptr, iters, stream, flags=0):
    """Returns (status, best microseconds per launch)."""
    us = ctypes.c_float(0.0)
    st = load_library().gemm_epi_tune(plan, A_ptr, B_ptr, bias_ptr, C_ptr, int(iters), int(flags), stream,
                                      ctypes.byref(us))
    return st, float(us.value)


def gemm_epi_tuning_save(path: str) -> int:
    return load_library().gemm_epi_tuning_save(None if path is None else str(path).encode())


def gemm_epi_tuning_load(path: str) -> int:
    return load_library().gemm_epi_tuning_load(None if path is None else str(path).encode())


def gemm_epi_tuning_clear() -> None:
    load_library().gemm_epi_tuning_clear()


def gemm_epi_tuning_size() -> int:
    return int(load_library().gemm_epi_tuning_size())


def gemm_epi_attention_fwd(Q_ptr, K_ptr, V_ptr, O_ptr, B, S, H, D, dtype, causal, stream) -> int:
    return load_library().gemm_epi_attention_fwd(Q_ptr, K_ptr, V_ptr, O_ptr, int(B), int(S), int(H), int(D),
                                                 DTYPES[dtype], int(bool(causal)), stream)


def attention_fwd(q, k, v, o, causal=False, stream=None):
    """Scaled dot-product attention on torch CUDA tensors [B, S, H, D]
    (contiguous, fp16 or bf16): fills `o`; enqueued on torch's current
    stream (or `stream`), not synchronised."""
    import torch

    for name, t in (("q", q), ("k", k), ("v", v), ("o", o)):
        if not t.is_cuda or not t.is_contiguous() or t.dim() != 4:
            raise ValueError(f"{name}: expected a contiguous 4-d CUDA tensor [B, S, H, D]")
        if t.shape != q.shape or t.dtype != q.dtype:
            raise ValueError(f"{name}: shape/dtype differ from q")
    B, S, H, D = q.shape
    if _dtype_name(q) not in ("f16", "bf16"):
        raise ValueError(f"q: dtype {q.dtype}; expected float16 or bfloat16")
    s = stream.cuda_stream if stream is not None else _current_stream_handle(torch)
    st = gemm_epi_attention_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), B, S, H, D,
                                _dtype_name(q), causal, s)
    if st != OK:
        raise GemmEpiError("gemm_epi_attention_fwd", st)


# ---- the operators of a decode step (include/gemm_epi_decode.h) --------------

def gemm_epi_rmsnorm(X, ldx, R, ldr, W, H, ldh, Y, ldy, y_scale, rows, cols, eps, dtype, out_dtype, stream) -> int:
    return load_library().gemm_epi_rmsnorm(X, ldx, R, ldr, W, H, ldh, Y, ldy, y_scale, rows, cols, eps,
                                           DTYPES[dtype], DTYPES[out_dtype], stream)


def gemm_epi_lora(X, ldx, A, B, scale, ids, R, ldr, C, ldc, M, N, K, rank, adapters, dtype, ws, ws_bytes,
                  stream) -> int:
    return load_library().gemm_epi_lora(X, ldx, A, B, scale, ids, R, ldr, C, ldc, M, N, K, rank, adapters,
                                        DTYPES[dtype], ws, ws_bytes, stream)


def gemm_epi_lora_workspace_size(M, N, K, rank, adapters) -> int:
    return int(load_library().gemm_epi_lora_workspace_size(M, N, K, rank, adapters))


def paged_cache_struct(k, v, k_scale, v_scale, num_pages, page_size, heads, head_dim, dtype):
    """A gemm_epi_paged_cache of pointers and sizes (for the two calls below)."""
    return _PagedCache(k, v, k_scale, v_scale, num_pages, page_size, heads, head_dim, DTYPES[dtype])


def page_table_struct(pages, ld, width, lens, batch):
    """A gemm_epi_page_table of pointers and sizes."""
    return _PageTable(pages, ld, width, lens, batch)


def gemm_epi_cache_append(cache, table, K, ldk, V, ldv, starts, tokens, dtype, stream) -> int:
    return load_library().gemm_epi_cache_append(cache, table, K, ldk, V, ldv, starts, tokens, DTYPES[dtype], stream)


def gemm_epi_attention_decode(cache, table, Q, ldq, O, ldo, q_heads, dtype, ws, ws_bytes, stream) -> int:
    return load_library().gemm_epi_attention_decode(cache, table, Q, ldq, O, ldo, q_heads, DTYPES[dtype], ws,
                                                    ws_bytes, stream)


def gemm_epi_attention_decode_workspace_size(cache, batch, width, q_heads) -> int:
    return int(load_library().gemm_epi_attention_decode_workspace_size(cache, batch, width, q_heads))


ATTENTION_DECODE_COUNTER_BYTES = 2048  # GEMM_EPI_ATTENTION_DECODE_COUNTER_BYTES


# The tensor calls below check their arguments and call the library in
# _calls.so (torch_calls.cpp): 4.0 us a call, most of it the launch, where
# checks written here and ctypes took 6.7.

class _Calls:
    """That module, and torch's current device and stream as plain numbers,
    looked up at the first call."""
    m = None


def _load_calls():
    import torch

    load_library()
    if not os.path.exists(CALLS_PATH):
        raise RuntimeError(f"{CALLS_PATH} is missing: it is built beside the HIP library. "
                           "Run `python -c 'import __graft_entry__ as g; g.build()'` or "
                           "`python epilogue_gemm_amd/build.py` first.")
    from . import _calls

    C = _Calls
    C.device, C.raw = getattr(torch._C, "_cuda_getDevice", None), getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if C.device is None or C.raw is None:
        C.device, C.raw = torch.cuda.current_device, lambda index: torch.cuda.current_stream(index).cuda_stream
    torch.cuda.current_device()  # (initialises the device)
    C.m = _calls


def _stream_of(stream, index):
    """hipStream_t of a given stream, which has to be the current device's."""
    if stream.device.index != index:
        raise ValueError(f"stream: on device {stream.device.index}, the current device is {index}")
    return stream.cuda_stream


def _workspace(nbytes, stream, zeros=0):
    """A workspace from torch's allocator on the stream of the call, its first
    `zeros` bytes zero."""
    import torch

    with torch.cuda.stream(stream):  # (None: the current one)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        if zeros:
            workspace[:zeros].zero_()
    return workspace


def rmsnorm(x, weight, y, residual=None, residual_out=None, y_scale=None, eps=1e-6, stream=None):
    """h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight over the last
    axis of [rows, cols] tensors of one 16-bit format (the rows may be
    strided); ``residual_out`` receives h, and may be ``residual`` or ``x``
    itself.  ``y`` is of the same format, or float8_e4m3fn with
    ``y_scale`` ([rows] float32) receiving each row's scale.  Enqueued on
    torch's current stream (or `stream`), not synchronised."""
    C = _Calls
    if C.m is None:
        _load_calls()
    index = C.device()
    st = C.m.rmsnorm(index, C.raw(index) if stream is None else _stream_of(stream, index), x, weight, y, residual,
                     residual_out, y_scale, eps)
    if st != OK:
        raise GemmEpiError("gemm_epi_rmsnorm", st)


def lora_workspace_size(M, N, K, rank, adapters) -> int:
    """Bytes of workspace ``lora`` uses for these sizes."""
    return gemm_epi_lora_workspace_size(M, N, K, rank, adapters)


def lora(x, a, b, ids, c, scale=None, residual=None, workspace=None, stream=None):
    """c[m] = residual[m] + scale[i] (x[m] a[i]^T) b[i]^T with i = ids[m]; a
    row whose id is outside [0, adapters) has no adapter.  x [M, K], c and
    residual [M, N] (rows may be strided; ``residual`` may be ``c`` itself, or
    None for 0), a [adapters, rank, K] and b [adapters, N, rank], all of one
    16-bit format; ids [M] int32, scale [adapters] float32 or None for 1.
    ``workspace``: an optional CUDA tensor of ``lora_workspace_size`` bytes,
    else one is allocated.  With residual None, c is what ``Plan.run`` of the
    projection takes as its residual."""
    C = _Calls
    if C.m is None:
        _load_calls()
    index = C.device()
    s = C.raw(index) if stream is None else _stream_of(stream, index)
    st = C.m.lora(index, s, x, a, b, ids, c, scale, residual, workspace)
    if st < 0:
        st = C.m.lora(index, s, x, a, b, ids, c, scale, residual, _workspace(-st, stream))
    if st != OK:
        raise GemmEpiError("gemm_epi_lora", st)


class PagedCache:
    """The paged key-value cache of one layer over the caller's tensors: k and
    v [num_pages, heads, page_size, head_dim] in float16, bfloat16 or
    float8_e4m3fn, the latter with k_scale and v_scale [num_pages, heads,
    page_size] float32.  ``append`` and ``attend`` enqueue on torch's current
    stream (or the given one) and return without synchronising.

    Both take ``pages`` [batch, width] int32 (rows may be strided; an entry
    outside [0, num_pages) is no page) and ``lens`` [batch] int32, the tokens
    each sequence holds, those of the current step included."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        import torch

        shape = k.shape
        if len(shape) != 4:
            raise ValueError("k: expected a 4-d tensor [num_pages, heads, page_size, head_dim]")
        if not k.is_cuda:
            raise ValueError("k: expected a CUDA tensor")
        fmt = _dtype_name(k)
        if fmt not in ("f16", "bf16", "fp8"):
            raise ValueError(f"k: dtype {k.dtype}; expected float16, bfloat16 or float8_e4m3fn")
        self.device_index = k.get_device()

        def at(name, t, dtype, shape):
            if not t.is_cuda or t.get_device() != self.device_index or t.dtype != dtype or t.shape != shape or \
                    not t.is_contiguous():
                raise ValueError(f"{name}: expected a contiguous {dtype} tensor {tuple(shape)} on k's device")
            return t.data_ptr()

        pk, pv = at("k", k, k.dtype, shape), at("v", v, k.dtype, shape)
        if (fmt == "fp8") != (k_scale is not None) or (fmt == "fp8") != (v_scale is not None):
            raise ValueError("k_scale, v_scale: for a float8_e4m3fn cache, and only then")
        pks = pvs = None
        if fmt == "fp8":
            pks = at("k_scale", k_scale, torch.float32, shape[:3])
            pvs = at("v_scale", v_scale, torch.float32, shape[:3])
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_pages, self.heads, self.page_size, self.head_dim = shape
        self._struct = paged_cache_struct(pk, pv, pks, pvs, shape[0], shape[2], shape[1], shape[3], fmt)
        self._address = ctypes.addressof(self._struct)

    def append(self, k, v, pages, lens, starts=None, stream=None):
        """Writes the rows k and v [tokens, heads, head_dim] (rows may be
        strided) to their sequences' last positions.  ``starts`` [batch + 1]
        int32: the rows of sequence i are starts[i] .. starts[i + 1] - 1, rows
        from starts[batch] on are ignored; None: one row a sequence."""
        C = _Calls
        if C.m is None:
            _load_calls()
        index = C.device()
        st = C.m.append(index, C.raw(index) if stream is None else _stream_of(stream, index), self._address,
                        self.device_index, k, v, pages, lens, starts)
        if st != OK:
            raise GemmEpiError("gemm_epi_cache_append", st)

    def workspace_size(self, q_heads, pages) -> int:
        """Bytes of workspace ``attend`` uses for this page table."""
        return gemm_epi_attention_decode_workspace_size(self._struct, pages.shape[0], pages.shape[1], q_heads)

    def attend(self, q, o, pages, lens, workspace=None, stream=None):
        """o[i, h] = attention of query q[i, h] over the tokens of sequence i
        (0 where there are none).  q and o [batch, q_heads, head_dim] (rows
        may be strided), float16 or bfloat16, the cache's format unless that
        is float8_e4m3fn.  ``workspace``: an optional CUDA tensor of
        ``workspace_size`` bytes, its first ATTENTION_DECODE_COUNTER_BYTES
        zero before its first use (every completed run leaves them zero), else
        one is allocated."""
        C = _Calls
        if C.m is None:
            _load_calls()
        index = C.device()
        s = C.raw(index) if stream is None else _stream_of(stream, index)
        args = (self._address, self.device_index, q, o, pages, lens)
        st = C.m.attend(index, s, *args, workspace)
        if st < 0:
            st = C.m.attend(index, s, *args, _workspace(-st, stream, ATTENTION_DECODE_COUNTER_BYTES))
        if st != OK:
            raise GemmEpiError("gemm_epi_attention_decode", st)


# ---- the experts' feed-forward and 8-bit products (include/gemm_epi_experts.h) ----

def gemm_epi_quantise_i8(X, ldx, Y, ldy, scale, rows, cols, dtype, stream) -> int:
    return load_library().gemm_epi_quantise_i8(X, ldx, Y, ldy, scale, rows, cols, DTYPES[dtype], stream)


def gemm_epi_i8_gemm(A, lda, a_scale, B, ldb, b_scale, bias, R, ldr, C, ldc, M, N, K, epilogue, out_dtype,
                     stream) -> int:
    return load_library().gemm_epi_i8_gemm(A, lda, a_scale, B, ldb, b_scale, bias, R, ldr, C, ldc, M, N, K,
                                           EPILOGUES[epilogue], DTYPES[out_dtype], stream)


def gemm_epi_route(logits, ldl, dtype, tokens, experts, per, score, renormalise, scale, ids, weights, offsets, order,
                   stream) -> int:
    return load_library().gemm_epi_route(logits, ldl, DTYPES[dtype], tokens, experts, per, SCORES[score],
                                         int(bool(renormalise)), scale, ids, weights, offsets, order, stream)


def gemm_epi_group_rows(ids, rows, groups, offsets, order, stream) -> int:
    return load_library().gemm_epi_group_rows(ids, rows, groups, offsets, order, stream)


def groups_struct(offsets, order, groups, rows, per):
    """A gemm_epi_groups of pointers and sizes (for the call below)."""
    return _Groups(offsets, order, groups, rows, per)


def gemm_epi_grouped_gemm(groups, X, ldx, x_scale, W, w_scale, bias, C, ldc, N, K, flags, epilogue, dtype, out_dtype,
                          stream) -> int:
    return load_library().gemm_epi_grouped_gemm(groups, X, ldx, x_scale, W, w_scale, bias, C, ldc, N, K, flags,
                                                EPILOGUES[epilogue], DTYPES[dtype], DTYPES[out_dtype], stream)


def gemm_epi_combine(Z, ldz, weights, ids, experts, R, ldr, Y, ldy, tokens, per, cols, dtype, stream) -> int:
    return load_library().gemm_epi_combine(Z, ldz, weights, ids, experts, R, ldr, Y, ldy, tokens, per, cols,
                                           DTYPES[dtype], stream)


def _called(fn, name, stream, *args):
    """A call of _calls.so on the current device and the given or torch's
    current stream."""
    C = _Calls
    if C.m is None:
        _load_calls()
    index = C.device()
    st = getattr(C.m, fn)(index, C.raw(index) if stream is None else _stream_of(stream, index), *args)
    if st != OK:
        raise GemmEpiError(name, st)


def quantise_i8(x, y, scale, stream=None):
    """scale = max(max|x| / 127, 2^-100), y = x / scale rounded to the nearest
    integer, over the last axis of x [rows, cols] float16 or bfloat16 and y
    [rows, cols] int8 (rows may be strided); scale [rows] float32.  A row that
    holds an infinity or a NaN gets scale NaN.  Enqueued on torch's current
    stream (or `stream`), not synchronised, as all calls below."""
    _called("quantise_i8", "gemm_epi_quantise_i8", stream, x, y, scale)


def i8_gemm(a, a_scale, b, b_scale, c, bias=None, residual=None, epilogue="none", stream=None):
    """c = act((a b^T) a_scale[:, None] b_scale[None] + bias) + residual for
    int8 rows a [M, K] and weights b [N, K], a_scale [M] and b_scale [N]
    float32; c and residual [M, N] float16 or bfloat16 (``residual`` may be
    ``c`` itself), bias [N] of that format for an epilogue with one.  Rows may
    be strided.  ``epilogue``: a name of EPILOGUES."""
    _called("i8_gemm", "gemm_epi_i8_gemm", stream, a, a_scale, b, b_scale, c, bias, residual, EPILOGUES[epilogue])


def route(logits, ids, weights, score="softmax", renormalise=True, scale=1.0, offsets=None, order=None, stream=None):
    """The experts of each token: ids [tokens, per] int32 of the largest
    logits [tokens, experts] (float32, float16 or bfloat16, rows may be
    strided), of equal ones the lower first, and their weights [tokens, per]
    float32: the softmax over all experts or each logit's sigmoid
    (``score``), divided by its sum over the chosen ones (``renormalise``), times
    ``scale``.  An expert at minus infinity or NaN is not chosen: id -1, weight
    0.  With ``offsets`` [experts + 1] and ``order`` [tokens * per] int32, those
    of ``group_rows`` too."""
    _called("route", "gemm_epi_route", stream, logits, ids, weights, SCORES[score], bool(renormalise), scale, offsets,
            order)


def group_rows(ids, offsets, order, stream=None):
    """The entries of ids (int32, contiguous) by group: order [entries] int32
    holds their numbers, group by group and ascending in each, those of group
    g from offsets[g] to offsets[g + 1] - 1 (offsets [groups + 1] int32); an id
    outside [0, groups) is in no group, and as many -1 stand behind the last."""
    _called("group_rows", "gemm_epi_group_rows", stream, ids, offsets, order)


def grouped_gemm(x, w, c, offsets, order=None, per=1, gather=False, scatter=False, gated=False, bias=None,
                 epilogue="none", x_scale=None, w_scale=None, stream=None):
    """For place i of group g, offsets[g] <= i < offsets[g + 1] (offsets that
    descend count as no lower than any before them), and entry q = order[i]
    (without ``order``: i): row q of c (``scatter``, else row i) = act(row
    q // per of x (``gather``, else row i) w[g]^T + bias[g]).  w [groups, N, K],
    and with ``gated`` [groups, 2 N, K], N rows of gates, then N of values: act(x
    gate^T + bias) * (x value^T + bias).  c [rows, N], x [rows, K], or with ``gather``
    [rows / per, K] (rows may be strided), bias [groups, N or 2 N].  x, w, c and
    bias of one 16-bit format, or x and w int8 with x_scale [rows of x] and
    w_scale [groups, N or 2 N] float32.  Rows of c that no place writes are left
    as they were."""
    _called("grouped_gemm", "gemm_epi_grouped_gemm", stream, x, w, c, offsets, order, per,
            (GATHER if gather else 0) | (SCATTER if scatter else 0) | (GATED if gated else 0), bias,
            EPILOGUES[epilogue], x_scale, w_scale)


def combine(z, weights, ids, y, experts, residual=None, stream=None):
    """y[t] = residual[t] + the sum over j of weights[t, j] z[t * per + j], over
    the j with 0 <= ids[t, j] < experts (``ids`` None: all).  z [tokens * per,
    cols], y and residual [tokens, cols] of one 16-bit format (rows may be
    strided; ``residual`` may be ``y`` itself), weights [tokens, per] float32, ids
    [tokens, per] int32."""
    _called("combine", "gemm_epi_combine", stream, z, weights, ids, y, experts, residual)


# ---- measurement helpers (include/gemm_epi_probes.h) -------------------------

def gemm_epi_probe_hbm_read(buf_ptr, nbytes, sink_ptr, stream) -> int:
    return load_library().gemm_epi_probe_hbm_read(buf_ptr, int(nbytes), sink_ptr, stream)


def gemm_epi_probe_mfma(iters, workgroups, out_ptr, stream) -> int:
    return load_library().gemm_epi_probe_mfma(int(iters), int(workgroups), out_ptr, stream)


def gemm_epi_probe_mfma_flops(iters, workgroups) -> float:
    return float(load_library().gemm_epi_probe_mfma_flops(int(iters), int(workgroups)))


def gemm_epi_destroy(plan) -> int:
    return load_library().gemm_epi_destroy(plan)


def gemm_epi_status_string(status: int) -> str:
    return load_library().gemm_epi_status_string(int(status)).decode()


def gemm_epi_last_hip_error() -> int:
    return int(load_library().gemm_epi_last_hip_error())


def gemm_epi_plan_select(plan, kernel: str, config: int = -1) -> int:
    return load_library().gemm_epi_plan_select(plan, KERNELS[kernel], int(config))


def gemm_epi_num_configs(kernel: str) -> int:
    return int(load_library().gemm_epi_num_configs(KERNELS[kernel]))


def gemm_epi_plan_describe(plan):
    """(kernel family name, config index, config name)."""
    k, c = ctypes.c_int(), ctypes.c_int()
    name = load_library().gemm_epi_plan_describe(plan, ctypes.byref(k), ctypes.byref(c))
    if name is None:
        raise ValueError("NULL plan")
    return KERNEL_NAMES[k.value], c.value, name.decode()


# ---- convenience over torch tensors (device memory + stream only) ----------

_TORCH_DTYPE_NAMES = {"float16": "f16", "bfloat16": "bf16", "float32": "f32", "float8_e4m3fn": "fp8"}
_NAME_OF_DTYPE = {}  # torch.dtype -> format name (None: not a format of the library), filled on use


def _dtype_name(t):
    d = t.dtype
    try:
        return _NAME_OF_DTYPE[d]
    except KeyError:
        n = _NAME_OF_DTYPE[d] = _TORCH_DTYPE_NAMES.get(str(d).replace("torch.", ""))
        return n


def _current_stream_handle(torch) -> int:
    """hipStream_t of torch's current stream on the current device (the raw
    handle without building a Stream object, where torch offers it)."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None:
        return raw(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


class Plan:
    """A planned problem.  ``run(A, B, bias, C)`` enqueues on torch's current
    CUDA stream (or the given one) and returns without synchronising."""

    def __init__(self, M, N, K, in_dtype, out_dtype, layout_a="row", layout_b="row", epilogue="none",
                 kernel: str = "auto", config: int = -1, lda: int = 0, ldb: int = 0, ldc: int = 0):
        self.M, self.N, self.K = int(M), int(N), int(K)
        self.in_dtype, self.out_dtype = in_dtype, out_dtype
        self.layout_a, self.layout_b, self.epilogue = layout_a, layout_b, epilogue
        self.handle = gemm_epi_plan(M, N, K, in_dtype, out_dtype, layout_a, layout_b, epilogue)
        # stored extents (elements) of A, B and C: (rows - 1) * ld + row length
        a_rows, a_cols = (self.M, self.K) if layout_a == "row" else (self.K, self.M)
        b_rows, b_cols = (self.K, self.N) if layout_b == "row" else (self.N, self.K)
        self.lda, self.ldb, self.ldc = int(lda) or a_cols, int(ldb) or b_cols, int(ldc) or self.N
        self._extent = {"A": (a_rows - 1) * self.lda + a_cols, "B": (b_rows - 1) * self.ldb + b_cols,
                        "C": (self.M - 1) * self.ldc + self.N}
        if lda or ldb or ldc:
            st = gemm_epi_plan_set_ld(self.handle, lda, ldb, ldc)
            if st != OK:
                gemm_epi_destroy(self.handle)
                self.handle = None
                raise GemmEpiError("gemm_epi_plan_set_ld", st)
        if kernel != "auto":
            st = gemm_epi_plan_select(self.handle, kernel, config)
            if st != OK:
                gemm_epi_destroy(self.handle)
                self.handle = None
                raise GemmEpiError("gemm_epi_plan_select", st)
        self.kernel, self.config, self.name = gemm_epi_plan_describe(self.handle)
        self._run = load_library().gemm_epi_run

    def _check(self, t, name, dtype, numel):
        if t is None:
            return None
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous CUDA tensor")
        if _dtype_name(t) != dtype:
            raise ValueError(f"{name}: dtype {t.dtype} does not match {dtype}")
        n = t.numel()
        if n < numel or (n != numel and name not in ("A", "B", "C", "residual")):
            raise ValueError(f"{name}: {n} elements, expected {numel}")
        return t.data_ptr()

    @property
    def workspace_size(self) -> int:
        """Bytes of workspace that let ``run`` split K (0: never splits)."""
        return gemm_epi_workspace_size(self.handle)

    def run(self, A, B, bias, C, stream=None, workspace=None, scale=None, residual=None, out_scale=None):
        """``workspace``: an optional zero-filled uint8 CUDA tensor of at least
        ``workspace_size`` bytes (left zero-filled by every completed run).
        ``scale``: optional fp32 per-column factors (N); ``residual``:
        optional M x N tensor of the output format, added after the
        activation (must not overlap C); ``out_scale``: optional one-element
        fp32 CUDA tensor multiplying the final value (the quantisation
        scale of an fp8 output)."""
        import torch

        a = self._check(A, "A", self.in_dtype, self._extent["A"])
        b = self._check(B, "B", self.in_dtype, self._extent["B"])
        bi = self._check(bias, "bias", self.in_dtype, self.N)
        c = self._check(C, "C", self.out_dtype, self._extent["C"])
        s = stream.cuda_stream if stream is not None else _current_stream_handle(torch)
        if scale is not None or residual is not None or out_scale is not None:
            sc = self._check(scale, "scale", "f32", self.N)
            r = self._check(residual, "residual", self.out_dtype, self._extent["C"])
            q = self._check(out_scale, "out_scale", "f32", 1)
            ws, nbytes = None, 0
            if workspace is not None:
                if not workspace.is_cuda or not workspace.is_contiguous():
                    raise ValueError("workspace: expected a contiguous CUDA tensor")
                ws, nbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
            st = gemm_epi_run_ex(self.handle, a, b, bi, sc, r, c, ws, nbytes, s, out_scale_ptr=q)
            if st != OK:
                raise GemmEpiError("gemm_epi_run_ex", st)
            return
        if workspace is None:
            st = self._run(self.handle, a, b, bi, c, s)
            fn = "gemm_epi_run"
        else:
            if not workspace.is_cuda or not workspace.is_contiguous():
                raise ValueError("workspace: expected a contiguous CUDA tensor")
            nbytes = workspace.numel() * workspace.element_size()
            st = gemm_epi_run_ws(self.handle, a, b, bi, c, workspace.data_ptr(), nbytes, s)
            fn = "gemm_epi_run_ws"
        if st != OK:
            raise GemmEpiError(fn, st)

    def tune(self, A, B, bias, C, iters=10, stream=None, cold=False) -> float:
        """Measure every configuration that can run this problem on these
        buffers and keep the fastest (also recorded in the tuning table).
        ``cold``: evict the caches before every timed launch.  Returns the
        winner's mean microseconds per launch; synchronises the stream."""
        import torch

        a = self._check(A, "A", self.in_dtype, self._extent["A"])
        b = self._check(B, "B", self.in_dtype, self._extent["B"])
        bi = self._check(bias, "bias", self.in_dtype, self.N)
        c = self._check(C, "C", self.out_dtype, self._extent["C"])
        s = stream.cuda_stream if stream is not None else _current_stream_handle(torch)
        st, us = gemm_epi_tune(self.handle, a, b, bi, c, iters, s, TUNE_COLD if cold else 0)
        if st != OK:
            raise GemmEpiError("gemm_epi_tune", st)
        self.kernel, self.config, self.name = gemm_epi_plan_describe(self.handle)
        return us

    def close(self):
        if self.handle is not None:
            gemm_epi_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
