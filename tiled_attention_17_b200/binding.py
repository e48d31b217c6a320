"""ctypes binding of libtiledattn.so (argument marshalling only).

Every function here passes device pointers, sizes and the CUDA stream through
to the C ABI declared in include/tiledattn.h; all computation happens in the
library's kernels.  There is no fallback: if the shared object cannot be
loaded, every call raises.

Functions with the C names take raw integers (device pointers) or torch
tensors (their data_ptr() is passed).  `attention()` and `paged_decode()` are
conveniences that allocate outputs with torch and call the C entry points.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libtiledattn.so")

TA_OK = 0
STATUS_NAMES = {0: "TA_OK", 1: "TA_ERR_INVALID_ARG", 2: "TA_ERR_UNSUPPORTED", 3: "TA_ERR_CUDA",
                4: "TA_ERR_BAD_BLOCK_TABLE", 5: "TA_ERR_DEVICE_TIMEOUT"}
TA_DEV_TIMEOUT = 1
TA_DEV_BAD_BLOCK_TABLE = 2
TA_DEV_BAD_SEQ_LEN = 4

EXPORTS = ["ta_status_string", "ta_version", "ta_last_error", "attn_fwd", "attn_fwd_fp8", "attn_bwd_workspace_size",
           "attn_bwd",
           "attn_rope", "attn_paged_append",
           "attn_paged_prefill", "attn_lse_merge", "attn_lse_merge_finish",
           "attn_paged_decode_workspace_size",
           "attn_paged_decode_shared_workspace_size", "attn_paged_decode_shared",
           "attn_paged_decode", "attn_paged_decode_noalloc", "attn_paged_decode_check", "attn_paged_gather_debug",
           "ta_device_status", "ta_selftest_bounded_wait", "ta_exp2_poly_debug"]


class TiledAttnError(RuntimeError):
    def __init__(self, fn, code, detail=""):
        self.code = code
        msg = f"{fn} returned {STATUS_NAMES.get(code, code)}"
        super().__init__(msg + (f": {detail}" if detail else ""))


_lib = None


def load(path: str | None = None):
    """Load (once) and return the ctypes handle of libtiledattn.so."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libtiledattn.so not found at {p}; build it with "
                           f"`python -m tiled_attention_17_b200.build`")
    L = ctypes.CDLL(p)
    vp, i32, f32, sz, u32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_uint
    L.ta_status_string.argtypes = [i32]
    L.ta_status_string.restype = ctypes.c_char_p
    L.ta_version.restype = i32
    L.ta_last_error.restype = ctypes.c_char_p
    L.attn_fwd.argtypes = [vp, vp, vp, vp, vp] + [i32] * 6 + [f32, i32, vp]
    L.attn_fwd.restype = i32
    L.attn_fwd_fp8.argtypes = [vp, vp, vp, f32, f32, f32, vp, vp] + [i32] * 6 + [f32, i32, vp]
    L.attn_fwd_fp8.restype = i32
    L.attn_paged_prefill.argtypes = [vp] * 6 + [i32] * 9 + [f32, i32, vp, vp, vp]
    L.attn_paged_prefill.restype = i32
    i64 = ctypes.c_int64
    L.attn_lse_merge.argtypes = [vp, vp, vp, vp, i64, i32, i32, vp]
    L.attn_lse_merge.restype = i32
    L.attn_lse_merge_finish.argtypes = [vp, vp, i64, i32, vp]
    L.attn_lse_merge_finish.restype = i32
    L.attn_rope.argtypes = [vp] * 4 + [i32] * 7 + [f32] + [i64] * 7 + [vp]
    L.attn_rope.restype = i32
    L.attn_paged_append.argtypes = [vp] * 11 + [i32] * 10 + [f32] + [i64] * 6 + [vp]
    L.attn_paged_append.restype = i32
    L.attn_bwd_workspace_size.argtypes = [i32] * 3
    L.attn_bwd_workspace_size.restype = sz
    L.attn_bwd.argtypes = [vp] * 10 + [sz] + [i32] * 6 + [f32, i32, vp]
    L.attn_bwd.restype = i32
    L.attn_paged_decode_workspace_size.argtypes = [i32] * 6
    L.attn_paged_decode_workspace_size.restype = sz
    L.attn_paged_decode.argtypes = [vp, vp, vp, vp, vp] + [i32] * 7 + [f32, vp, vp, vp, sz, vp]
    L.attn_paged_decode.restype = i32
    L.attn_paged_decode_shared_workspace_size.argtypes = [i32] * 5
    L.attn_paged_decode_shared_workspace_size.restype = sz
    L.attn_paged_decode_shared.argtypes = [vp] * 7 + [i32] * 9 + [f32, vp, vp, vp, sz, vp]
    L.attn_paged_decode_shared.restype = i32
    L.attn_paged_decode_noalloc.argtypes = [vp, vp, vp, vp, vp] + [i32] * 7 + [f32, vp, vp, vp]
    L.attn_paged_decode_noalloc.restype = i32
    L.attn_paged_decode_check.argtypes = [vp, ctypes.POINTER(u32), vp]
    L.attn_paged_decode_check.restype = i32
    L.attn_paged_gather_debug.argtypes = [vp, vp, vp, vp] + [i32] * 7 + [vp, vp, vp]
    L.attn_paged_gather_debug.restype = i32
    L.ta_device_status.argtypes = [ctypes.POINTER(u32), i32]
    L.ta_device_status.restype = i32
    L.ta_selftest_bounded_wait.argtypes = [u32, vp]
    L.ta_selftest_bounded_wait.restype = i32
    L.ta_exp2_poly_debug.argtypes = [vp, vp, i64, vp]
    L.ta_exp2_poly_debug.restype = i32
    if path is None:
        _lib = L
    return L


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # 0.1 us; a Stream object costs 3 us
        return raw(torch.cuda.current_device()) if raw else torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn, code):
    if code != TA_OK:
        raise TiledAttnError(fn, code, ta_last_error())


# ---------------------------------------------------------------------------
# C-named entry points
# ---------------------------------------------------------------------------

def ta_status_string(code: int) -> str:
    return load().ta_status_string(code).decode()


def ta_version() -> int:
    return load().ta_version()


def ta_last_error() -> str:
    return load().ta_last_error().decode()


def attn_fwd(q, k, v, o, lse, B, Hq, Hkv, Nq, Nkv, d, scale, causal, stream=None, check=True) -> int:
    code = load().attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Nq, Nkv, d,
                           float(scale), int(causal), _stream(stream))
    if check:
        _check("attn_fwd", code)
    return code


def attn_fwd_fp8(q, k, v, q_descale, k_descale, v_descale, o, lse, B, Hq, Hkv, Nq, Nkv, d, scale, causal,
                 stream=None, check=True) -> int:
    code = load().attn_fwd_fp8(_ptr(q), _ptr(k), _ptr(v), float(q_descale), float(k_descale), float(v_descale),
                               _ptr(o), _ptr(lse), B, Hq, Hkv, Nq, Nkv, d, float(scale), int(causal), _stream(stream))
    if check:
        _check("attn_fwd_fp8", code)
    return code


def attn_paged_prefill(q, k_cache, v_cache, block_table, cu_seqlens, seq_lens, page_size, num_seqs, total_q,
                       max_q_len, Hq, Hkv, d, max_pages, num_pages_total, scale, causal, o, lse, stream=None,
                       check=True) -> int:
    code = load().attn_paged_prefill(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(cu_seqlens),
                                     _ptr(seq_lens), page_size, num_seqs, total_q, max_q_len, Hq, Hkv, d, max_pages,
                                     num_pages_total, float(scale), int(causal), _ptr(o), _ptr(lse),
                                     _stream(stream))
    if check:
        _check("attn_paged_prefill", code)
    return code


def attn_lse_merge(acc_o, acc_lse, part_o, part_lse, rows, d, first, stream=None, check=True) -> int:
    code = load().attn_lse_merge(_ptr(acc_o), _ptr(acc_lse), _ptr(part_o), _ptr(part_lse), int(rows), d, int(first),
                                 _stream(stream))
    if check:
        _check("attn_lse_merge", code)
    return code


def attn_lse_merge_finish(acc_o, out, rows, d, stream=None, check=True) -> int:
    code = load().attn_lse_merge_finish(_ptr(acc_o), _ptr(out), int(rows), d, _stream(stream))
    if check:
        _check("attn_lse_merge_finish", code)
    return code


def attn_rope(x, y, positions, inv_freq, B, H, N, d, rotary_dim, interleaved, inverse, amplitude, x_stride_b,
              x_stride_h, x_stride_n, y_stride_b, y_stride_h, y_stride_n, pos_stride_b, stream=None,
              check=True) -> int:
    code = load().attn_rope(_ptr(x), _ptr(y), _ptr(positions), _ptr(inv_freq), B, H, N, d, rotary_dim,
                            int(interleaved), int(inverse), float(amplitude), x_stride_b, x_stride_h, x_stride_n,
                            y_stride_b, y_stride_h, y_stride_n, pos_stride_b, _stream(stream))
    if check:
        _check("attn_rope", code)
    return code


def attn_paged_append(q, k, v, q_out, k_cache, v_cache, block_table, cu_seqlens, seq_lens, positions, inv_freq,
                      page_size, num_seqs, total, Hq, Hkv, d, max_pages, num_pages_total, rotary_dim, interleaved,
                      amplitude, q_stride_t, q_stride_h, k_stride_t, k_stride_h, v_stride_t, v_stride_h, stream=None,
                      check=True) -> int:
    code = load().attn_paged_append(_ptr(q), _ptr(k), _ptr(v), _ptr(q_out), _ptr(k_cache), _ptr(v_cache),
                                    _ptr(block_table), _ptr(cu_seqlens), _ptr(seq_lens), _ptr(positions),
                                    _ptr(inv_freq), page_size, num_seqs, total, Hq, Hkv, d, max_pages,
                                    num_pages_total, rotary_dim, int(interleaved), float(amplitude), q_stride_t,
                                    q_stride_h, k_stride_t, k_stride_h, v_stride_t, v_stride_h, _stream(stream))
    if check:
        _check("attn_paged_append", code)
    return code


def attn_bwd_workspace_size(B, Hq, Nq) -> int:
    return load().attn_bwd_workspace_size(B, Hq, Nq)


def attn_bwd(q, k, v, o, dout, lse, dq, dk, dv, workspace, workspace_bytes, B, Hq, Hkv, Nq, Nkv, d, scale,
             causal, stream=None, check=True) -> int:
    code = load().attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv),
                           _ptr(workspace), int(workspace_bytes), B, Hq, Hkv, Nq, Nkv, d, float(scale), int(causal),
                           _stream(stream))
    if check:
        _check("attn_bwd", code)
    return code


def attn_paged_decode_workspace_size(num_seqs, Hq, Hkv, d, max_pages, page_size) -> int:
    return load().attn_paged_decode_workspace_size(num_seqs, Hq, Hkv, d, max_pages, page_size)


def attn_paged_decode(q, k_cache, v_cache, block_table, seq_lens, page_size, num_seqs, Hq, Hkv, d,
                      max_pages, num_pages_total, scale, o, lse, workspace, workspace_bytes,
                      stream=None, check=True) -> int:
    code = load().attn_paged_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(seq_lens),
                                    page_size, num_seqs, Hq, Hkv, d, max_pages, num_pages_total, float(scale),
                                    _ptr(o), _ptr(lse), _ptr(workspace), int(workspace_bytes), _stream(stream))
    if check:
        _check("attn_paged_decode", code)
    return code


def attn_paged_decode_noalloc(q, k_cache, v_cache, block_table, seq_lens, page_size, num_seqs, Hq, Hkv, d,
                              max_pages, num_pages_total, scale, o, lse, stream=None, check=True) -> int:
    """attn_paged_decode without a workspace argument, for callers that cannot
    allocate device memory: the library uses its own fixed 64 MiB scratch array
    (shared by all calls on a device; overlapping calls race)."""
    code = load().attn_paged_decode_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                                            _ptr(seq_lens), page_size, num_seqs, Hq, Hkv, d, max_pages,
                                            num_pages_total, float(scale), _ptr(o), _ptr(lse), _stream(stream))
    if check:
        _check("attn_paged_decode_noalloc", code)
    return code


def attn_paged_decode_shared_workspace_size(num_seqs, num_groups, Hq, Hkv, d) -> int:
    return load().attn_paged_decode_shared_workspace_size(num_seqs, num_groups, Hq, Hkv, d)


def attn_paged_decode_shared(q, k_cache, v_cache, block_table, seq_lens, group_offsets, prefix_lens, page_size,
                             num_seqs, num_groups, max_own_len, Hq, Hkv, d, max_pages, num_pages_total, scale, o, lse,
                             workspace, workspace_bytes, stream=None, check=True) -> int:
    code = load().attn_paged_decode_shared(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(seq_lens),
                                           _ptr(group_offsets), _ptr(prefix_lens), page_size, num_seqs, num_groups,
                                           max_own_len, Hq, Hkv, d, max_pages, num_pages_total, float(scale), _ptr(o),
                                           _ptr(lse), _ptr(workspace), int(workspace_bytes), _stream(stream))
    if check:
        _check("attn_paged_decode_shared", code)
    return code


def attn_paged_decode_check(workspace, stream=None):
    flags = ctypes.c_uint(0)
    code = load().attn_paged_decode_check(_ptr(workspace), ctypes.byref(flags), _stream(stream))
    return code, flags.value


def attn_paged_gather_debug(k_cache, v_cache, block_table, seq_lens, seq, hkv, page_size, Hkv, d, max_pages,
                            num_pages_total, k_out, v_out, stream=None, check=True) -> int:
    code = load().attn_paged_gather_debug(_ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(seq_lens),
                                          seq, hkv, page_size, Hkv, d, max_pages, num_pages_total,
                                          _ptr(k_out), _ptr(v_out), _stream(stream))
    if check:
        _check("attn_paged_gather_debug", code)
    return code


def ta_device_status(reset: bool = True):
    flags = ctypes.c_uint(0)
    code = load().ta_device_status(ctypes.byref(flags), int(reset))
    return code, flags.value


def ta_selftest_bounded_wait(limit_us: int, stream=None) -> int:
    return load().ta_selftest_bounded_wait(int(limit_us), _stream(stream))


def ta_exp2_poly_debug(x, y, n: int, stream=None, check: bool = True) -> int:
    code = load().ta_exp2_poly_debug(_ptr(x), _ptr(y), int(n), _stream(stream))
    if check:
        _check("ta_exp2_poly_debug", code)
    return code


# ---------------------------------------------------------------------------
# torch conveniences (allocate outputs, then call the C entry points)
# ---------------------------------------------------------------------------

def attention(q, k, v, causal: bool, scale: float | None = None, out=None, lse=None, stream=None):
    """q [B,Hq,Nq,d], k/v [B,Hkv,Nkv,d] bf16 CUDA tensors -> (o, lse)."""
    import torch
    B, Hq, Nq, d = q.shape
    _, Hkv, Nkv, _ = k.shape
    for t in (q, k, v):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous bf16 CUDA tensors")
    if scale is None:
        scale = d ** -0.5
    o = out if out is not None else torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device)
    attn_fwd(q, k, v, o, lse, B, Hq, Hkv, Nq, Nkv, d, scale, causal, stream)
    return o, lse


def attention_fp8(q, k, v, descale, causal: bool, scale: float | None = None, out=None, lse=None, stream=None):
    """q [B,Hq,Nq,128], k/v [B,Hkv,Nkv,128] contiguous CUDA tensors of E4M3
    codes (torch.float8_e4m3fn or uint8); descale = (q_descale, k_descale,
    v_descale) -> (o bf16, lse fp32)."""
    import torch
    B, Hq, Nq, d = q.shape
    _, Hkv, Nkv, _ = k.shape
    for t in (q, k, v):
        if t.dtype not in (torch.float8_e4m3fn, torch.uint8) or not t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous float8_e4m3fn (or uint8) CUDA tensors")
    if scale is None:
        scale = d ** -0.5
    o = out if out is not None else torch.empty((B, Hq, Nq, d), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device)
    dq, dk, dv = descale
    attn_fwd_fp8(q, k, v, dq, dk, dv, o, lse, B, Hq, Hkv, Nq, Nkv, d, scale, causal, stream)
    return o, lse


def attention_backward(q, k, v, o, lse, dout, causal: bool, scale: float | None = None, workspace=None,
                       stream=None):
    """Gradients (dq, dk, dv) of `attention` for the loss gradient dout (all bf16
    CUDA tensors; o and lse from the forward call with the same arguments)."""
    import torch
    B, Hq, Nq, d = q.shape
    _, Hkv, Nkv, _ = k.shape
    for t in (q, k, v, o, dout):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k, v, o, dout must be contiguous bf16 CUDA tensors")
    if scale is None:
        scale = d ** -0.5
    ws_bytes = attn_bwd_workspace_size(B, Hq, Nq)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    attn_bwd(q, k, v, o, dout, lse, dq, dk, dv, workspace, workspace.numel(), B, Hq, Hkv, Nq, Nkv, d, scale,
             causal, stream)
    return dq, dk, dv


def paged_prefill(q, k_cache, v_cache, block_table, cu_seqlens, seq_lens, max_q_len: int, causal: bool,
                  scale: float | None = None, out=None, lse=None, stream=None):
    """q [total_q, Hq, d] packed by cu_seqlens [S+1] (int32, device); caches
    [P, Hkv, page, d]; block_table [S, max_pages]; seq_lens [S] -> (o, lse)."""
    import torch
    T, Hq, d = q.shape
    P, Hkv, ps, _ = k_cache.shape
    S = seq_lens.shape[0]
    if scale is None:
        scale = d ** -0.5
    o = out if out is not None else torch.empty_like(q)
    if lse is None:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device)
    attn_paged_prefill(q, k_cache, v_cache, block_table, cu_seqlens, seq_lens, ps, S, T, max_q_len, Hq, Hkv, d,
                       block_table.shape[1], P, scale, causal, o, lse, stream)
    return o, lse


def paged_decode(q, k_cache, v_cache, block_table, seq_lens, scale: float | None = None, workspace=None,
                 out=None, lse=None, stream=None):
    """q [S,Hq,d]; caches [P,Hkv,page,d] bf16; block_table [S,max_pages] int32; seq_lens [S] int32."""
    import torch
    S, Hq, d = q.shape
    P, Hkv, ps, _ = k_cache.shape
    max_pages = block_table.shape[1]
    if scale is None:
        scale = d ** -0.5
    ws_bytes = attn_paged_decode_workspace_size(S, Hq, Hkv, d, max_pages, ps)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=q.device)
    o = out if out is not None else torch.empty_like(q)
    if lse is None:
        lse = torch.empty((S, Hq), dtype=torch.float32, device=q.device)
    attn_paged_decode(q, k_cache, v_cache, block_table, seq_lens, ps, S, Hq, Hkv, d, max_pages, P, scale,
                      o, lse, workspace, workspace.numel(), stream)
    return o, lse, workspace


_raw_stream = _raw_device = None


def _here(device):
    """The handle of the current stream if `device` is the current device, else None.  (The calls below are a few
    microseconds of kernel in their small sizes, so a Stream object, 3 us, or a device guard is too much.)"""
    global _raw_stream, _raw_device
    if _raw_stream is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda index: torch.cuda.current_stream(index).cuda_stream)
        _raw_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    index = device.index
    return _raw_stream(index) if _raw_device() == index else None


def _scope(device, stream):
    """The device and stream a convenience call allocates and launches on: the
    tensors' device, and `stream` (a torch stream or its handle) or that
    device's current one.  What the call allocates belongs to that stream."""
    import contextlib
    import torch
    if stream is not None:
        if isinstance(stream, int):   # 0 is the default stream's handle (an ExternalStream of 0 is one of torch's pool)
            stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
        if stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
    stack = contextlib.ExitStack()
    stack.enter_context(torch.cuda.device(device))
    if stream is not None:
        stack.enter_context(torch.cuda.stream(stream))
    return stack


def _rows(name, t, shape=None):
    """A bf16 CUDA tensor whose last dimension is contiguous."""
    import torch
    if t.dtype is not torch.bfloat16 or not t.is_cuda or t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must be a bf16 CUDA tensor with contiguous rows")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _ints(name, t, shape, device):
    import torch
    if t.dtype is not torch.int32 or t.shape != shape or t.get_device() != device.index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor {tuple(shape)} on {device}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t


def _frequencies(inv_freq, device):
    """rotary_dim of an inv_freq tensor (0 for None)."""
    import torch
    if inv_freq is None:
        return 0
    if inv_freq.dtype is not torch.float64 or inv_freq.device != device or inv_freq.dim() != 1 \
            or not inv_freq.is_contiguous():
        raise ValueError(f"inv_freq must be a contiguous float64 tensor [rotary_dim / 2] on {device}")
    return 2 * inv_freq.shape[0]


def _rope(x, inv_freq, positions, interleaved, amplitude, out, stream, inverse):
    import torch
    if x.dim() != 4:
        raise ValueError(f"x must be [B, H, N, d], got {tuple(x.shape)}")
    B, H, N, d = x.shape
    if x.dtype is not torch.bfloat16 or not x.is_cuda or x.stride(3) != 1:
        _rows("x", x)
    device = x.device
    rotary_dim = _frequencies(inv_freq, device)
    pos_stride = 0
    if positions is not None:
        if positions.dim() == 1:
            _ints("positions", positions, (N,), device)
        else:
            _ints("positions", positions, (B, N), device)
            pos_stride = N
    if out is not None and _rows("out", out, x.shape).device != device:
        raise ValueError("out must be on x's device")
    handle = _here(device) if stream is None else None
    if handle is None:
        with _scope(device, stream):
            return _rope(x, inv_freq, positions, interleaved, amplitude, out, None, inverse)
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    xb, xh, xn, _ = x.stride()
    yb, yh, yn, _ = out.stride()
    code = (_lib or load()).attn_rope(
        x.data_ptr(), out.data_ptr(), None if positions is None else positions.data_ptr(),
        None if inv_freq is None else inv_freq.data_ptr(), B, H, N, d, rotary_dim, int(interleaved), inverse,
        float(amplitude), xb, xh, xn, yb, yh, yn, pos_stride, handle)
    if code:
        _check("attn_rope", code)
    return out


def rope(x, inv_freq, positions=None, interleaved: bool = False, amplitude: float = 1.0, out=None, stream=None):
    """Rotary positions of x, a bf16 CUDA tensor or view [B, H, N, d] (e.g. the
    heads of a fused projection's [B, N, heads, d] rows, transposed): the
    rotated tensor, contiguous [B, H, N, d] as `attention` takes it, or written
    to `out` (any view of that shape; x itself rotates in place).  inv_freq and
    amplitude from `rope.frequencies` (None: copy only); positions int32 [N] or
    [B, N], by default 0..N-1."""
    return _rope(x, inv_freq, positions, interleaved, amplitude, out, stream, 0)


def rope_backward(dout, inv_freq, positions=None, interleaved: bool = False, amplitude: float = 1.0, out=None,
                  stream=None):
    """The gradient of `rope`'s input for the output gradient dout (same
    arguments); `out` may be a view of a fused projection's gradient rows."""
    return _rope(dout, inv_freq, positions, interleaved, amplitude, out, stream, 1)


def paged_append(k, v, k_cache, v_cache, block_table, seq_lens, cu_seqlens=None, q=None, q_out=None, inv_freq=None,
                 positions=None, interleaved: bool = False, amplitude: float = 1.0, stream=None):
    """Write new tokens' keys (rotated) and values into the paged cache and
    return their rotated queries (None without q).

    k, v [total, Hkv, d] and q [total, Hq, d]: bf16 CUDA tensors or views with
    contiguous rows; caches [P, Hkv, page, d]; block_table [S, max_pages];
    seq_lens [S] the lengths after the append; cu_seqlens [S+1] packs the new
    tokens as in `paged_prefill` (None: one token per sequence, total = S).
    All index tensors int32.  inv_freq None appends without rotation."""
    import torch
    T, Hkv, d = k.shape
    P, _, ps, _ = k_cache.shape
    S, max_pages = block_table.shape
    dev = k.device
    rows, pool = k.shape, k_cache.shape
    rotary_dim = _frequencies(inv_freq, dev)
    bf16, i32, index = torch.bfloat16, torch.int32, k.get_device()
    if (k.dtype is not bf16 or v.dtype is not bf16 or k_cache.dtype is not bf16 or v_cache.dtype is not bf16
            or v.shape != rows or pool != (P, Hkv, ps, d) or v_cache.shape != pool or index < 0
            or v.get_device() != index or k_cache.get_device() != index or v_cache.get_device() != index
            or k.stride(2) != 1 or v.stride(2) != 1 or not k_cache.is_contiguous() or not v_cache.is_contiguous()):
        _rows("k", k)
        _rows("v", v, rows)
        for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
            if not _rows(name, t, (P, Hkv, ps, d)).is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        if not index == v.get_device() == k_cache.get_device() == v_cache.get_device():
            raise ValueError("all tensors must be on one device")
    _ints("block_table", block_table, (S, max_pages), dev)
    _ints("seq_lens", seq_lens, (S,), dev)
    if cu_seqlens is not None:
        _ints("cu_seqlens", cu_seqlens, (S + 1,), dev)
    if positions is not None:
        _ints("positions", positions, (T,), dev)
    Hq, qt, qh = 0, 0, 0
    if q is None:
        q_out = None
    else:
        Hq = q.shape[1]
        _rows("q", q, (T, Hq, d))
        qt, qh, _ = q.stride()
        if q_out is not None and not _rows("q_out", q_out, (T, Hq, d)).is_contiguous():
            raise ValueError("q_out must be contiguous")
        if q.get_device() != index or q_out is not None and q_out.get_device() != index:
            raise ValueError("all tensors must be on one device")
    handle = _here(dev) if stream is None else None
    if handle is None:
        with _scope(dev, stream):
            return paged_append(k, v, k_cache, v_cache, block_table, seq_lens, cu_seqlens, q, q_out, inv_freq, positions,
                                interleaved, amplitude)
    if q is not None and q_out is None:
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
    kt, kh, _ = k.stride()
    vt, vh, _ = v.stride()
    code = (_lib or load()).attn_paged_append(
        None if q is None else q.data_ptr(), k.data_ptr(), v.data_ptr(), None if q is None else q_out.data_ptr(),
        k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(),
        None if cu_seqlens is None else cu_seqlens.data_ptr(), seq_lens.data_ptr(),
        None if positions is None else positions.data_ptr(), None if inv_freq is None else inv_freq.data_ptr(),
        ps, S, T, Hq, Hkv, d, max_pages, P, rotary_dim, int(interleaved), float(amplitude), qt, qh, kt, kh, vt, vh,
        handle)
    if code:
        _check("attn_paged_append", code)
    return q_out


def paged_decode_shared(q, k_cache, v_cache, block_table, seq_lens, group_offsets, prefix_lens,
                        max_own_len: int | None = None, scale: float | None = None, workspace=None, out=None,
                        lse=None, stream=None):
    """`paged_decode` where groups of sequences share a prefix, which is read
    once per group: group g is sequences [group_offsets[g],
    group_offsets[g+1]), whose first prefix_lens[g] tokens are the same (read
    through the first sequence's block-table row).  max_own_len: most tokens a
    sequence has after its prefix (by default what the table can hold).
    group_offsets [G+1] and prefix_lens [G] are int32 device tensors, the rest
    as `paged_decode`; returns (o, lse, workspace)."""
    import torch
    S, Hq, d = q.shape
    P, Hkv, ps, _ = k_cache.shape
    max_pages = block_table.shape[1]
    groups = prefix_lens.shape[0]
    dev = q.device
    bf16, index, pool = torch.bfloat16, q.get_device(), k_cache.shape
    if (q.dtype is not bf16 or k_cache.dtype is not bf16 or v_cache.dtype is not bf16 or pool[3] != d
            or v_cache.shape != pool or index < 0 or k_cache.get_device() != index or v_cache.get_device() != index
            or not q.is_contiguous() or not k_cache.is_contiguous() or not v_cache.is_contiguous()):
        for name, t, shape in (("q", q, (S, Hq, d)), ("k_cache", k_cache, (P, Hkv, ps, d)),
                               ("v_cache", v_cache, (P, Hkv, ps, d))):
            if not _rows(name, t, shape).is_contiguous() or t.device != dev:
                raise ValueError(f"{name} must be contiguous and on {dev}")
    _ints("block_table", block_table, (S, max_pages), dev)
    _ints("seq_lens", seq_lens, (S,), dev)
    _ints("group_offsets", group_offsets, (groups + 1,), dev)
    _ints("prefix_lens", prefix_lens, (groups,), dev)
    if out is not None and (not _rows("out", out, (S, Hq, d)).is_contiguous() or out.device != dev):
        raise ValueError(f"out must be contiguous and on {dev}")
    if lse is not None and (lse.dtype is not torch.float32 or lse.shape != (S, Hq) or lse.device != dev
                            or not lse.is_contiguous()):
        raise ValueError(f"lse must be a contiguous float32 tensor {(S, Hq)} on {dev}")
    if workspace is not None and (workspace.device != dev or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be contiguous and on {dev}")
    if max_own_len is None:
        max_own_len = max_pages * ps
    if scale is None:
        scale = d ** -0.5
    handle = _here(dev) if stream is None else None
    if handle is None:
        with _scope(dev, stream):
            return paged_decode_shared(q, k_cache, v_cache, block_table, seq_lens, group_offsets, prefix_lens,
                                       max_own_len, scale, workspace, out, lse)
    if workspace is None:
        need = attn_paged_decode_shared_workspace_size(S, groups, Hq, Hkv, d)
        workspace = q.new_empty(max(need, 256), dtype=torch.uint8)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = q.new_empty((S, Hq), dtype=torch.float32)
    code = (_lib or load()).attn_paged_decode_shared(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
        group_offsets.data_ptr(), prefix_lens.data_ptr(), ps, S, groups, max_own_len, Hq, Hkv, d, max_pages, P,
        float(scale), out.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), handle)
    if code:
        _check("attn_paged_decode_shared", code)
    return out, lse, workspace
