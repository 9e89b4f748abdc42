"""Python binding of libi4rt: INT4 weight-only batch-1 decode on B200 (sm_100a).

Argument marshalling only. Every computation runs in the CUDA kernels of
``libi4rt.so`` (built by ``python -m int4_weight_only_02_b200.build``); there
is no CPU or PyTorch fallback, and a missing library raises at first use.
PyTorch provides device memory and streams: tensors are passed by
``data_ptr()``, and calls run on ``torch.cuda.current_stream()`` unless a
stream is given.

Layouts (see include/i4rt.h): INT4 weights [N][K/8] uint32 (8 consecutive k
per word, field i at bits 4i..4i+3, two's complement), fp16 group-128 scales
[N][K/128], KV pools [pages][kv heads][page_size][128] fp16.
"""
from __future__ import annotations

import array
import ctypes
import operator
import os
import struct

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libi4rt.so")
_lib = None

I4_OK, I4_EINVAL, I4_EALIGN, I4_EUNSUPPORTED, I4_ECUDA, I4_ENOMEM = 0, -1, -2, -3, -4, -5

_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t


class I4Error(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"i4rt status {status}: {msg}")
        self.status = status


class ModelDesc(ctypes.Structure):
    _fields_ = [("n_layers", _i), ("hidden", _i), ("intermediate", _i), ("n_q_heads", _i), ("n_kv_heads", _i),
                ("head_dim", _i), ("vocab", _i), ("group", _i), ("page_size", _i), ("max_ctx", _i),
                ("rope_theta", _f), ("rms_eps", _f)]


class LayerWeights(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("w_qkv", "s_qkv", "b_qkv", "w_o", "s_o", "w_gate_up", "s_gate_up", "w_down",
                                   "s_down", "ln_in", "ln_post")]


class ModelWeights(ctypes.Structure):
    _fields_ = [("embed", _vp), ("layers", ctypes.POINTER(LayerWeights)), ("ln_final", _vp), ("w_lm", _vp),
                ("s_lm", _vp)]


class SeqState(ctypes.Structure):
    _fields_ = [("token", _vp), ("pos", _vp), ("ctx_len", _vp), ("page_table", _vp),
                ("k_pools", ctypes.POINTER(_vp)), ("v_pools", ctypes.POINTER(_vp)), ("num_pages", _i),
                ("logits", _vp), ("prompt", _vp), ("n_prompt", _i), ("history", _vp), ("status", _vp)]


class RmsnormRopeArgs(ctypes.Structure):
    _fields_ = [("x_in", _vp), ("resid", _vp), ("gamma", _vp), ("out", _vp), ("M", _i), ("H", _i), ("eps", _f),
                ("qkv", _vp), ("pos", _vp), ("B", _i), ("Hq", _i), ("Hkv", _i), ("D", _i), ("theta", _f),
                ("k_pool", _vp), ("v_pool", _vp), ("page_table", _vp), ("page_size", _i),
                ("max_pages_per_seq", _i)]


class RopeChunkArgs(ctypes.Structure):
    _fields_ = [("qkv", _vp), ("qkv_stride", ctypes.c_longlong), ("q_start", _vp), ("ctx_len", _vp), ("cs", _vp),
                ("q_out", _vp), ("k_pool", _vp), ("v_pool", _vp), ("page_table", _vp), ("max_pos", _i), ("rotary_dim", _i),
                ("interleaved", _i), ("T", _i), ("B", _i), ("Hq", _i), ("Hkv", _i), ("D", _i), ("page_size", _i),
                ("max_pages_per_seq", _i), ("num_pages", _i)]


class ChunkAttnArgs(ctypes.Structure):
    _fields_ = [("q", _vp), ("q_stride", ctypes.c_longlong), ("k_pool", _vp), ("v_pool", _vp), ("page_table", _vp),
                ("q_start", _vp), ("ctx_len", _vp), ("out", _vp), ("ws", _vp), ("ws_bytes", _sz), ("T", _i), ("B", _i),
                ("Hq", _i), ("Hkv", _i), ("D", _i), ("page_size", _i), ("max_pages_per_seq", _i), ("num_pages", _i),
                ("window", _i), ("max_q", _i), ("scale", _f)]


class KvCacheDesc(ctypes.Structure):
    _fields_ = [("page_table", _vp), ("ctx_len", _vp), ("refs", _vp), ("n_seqs", _i), ("max_pages_per_seq", _i),
                ("page_size", _i), ("num_pages", _i)]


_ll, _d = ctypes.c_longlong, ctypes.c_double

_SIGS = {
    "i4_last_error": (ctypes.c_char_p, []),
    "i4_version": (ctypes.c_char_p, []),
    "int4_gemv": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp]),
    "int4_gemm": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _sz, _vp]),
    "int4_gemm_ws_bytes": (_sz, [_i, _i, _i]),
    "i4_int4_gemv_variant": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp]),
    "i4_int4_unpack": (_i, [_vp, _vp, _i, _i, _vp]),
    "paged_gqa_decode_ws_bytes": (_sz, [_i, _i, _i, _i, _i, _i]),
    "paged_gqa_decode": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp, _sz, _vp]),
    "paged_gqa_decode_static": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp]),
    "i4_paged_gqa_decode_strided": (_i, [_vp, ctypes.c_longlong, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i,
                                         _f, _vp, _sz, _vp]),
    "i4_embed_gather": (_i, [_vp, _vp, _vp, _i, _i, _i, _vp]),
    "i4_argmax_rows": (_i, [_vp, _vp, _vp, _vp, _i, _i, _vp]),
    "i4_paged_gather": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp]),
    "rmsnorm_rope": (_i, [ctypes.POINTER(RmsnormRopeArgs), _vp]),
    "i4_rmsnorm": (_i, [_vp, _vp, _vp, _vp, _i, _i, _f, _vp]),
    "i4_rope_kv_append": (_i, [_vp, _vp, _i, _i, _i, _i, _f, _vp, _vp, _vp, _i, _i, _vp]),
    "silu_mul": (_i, [_vp, _vp, _i, _i, _vp]),
    "i4_rope_table": (_i, [_vp, _i, _i, _d, _i, _d, _i, _vp]),
    "i4_rope_append_chunk": (_i, [_vp, _vp]),
    "i4_paged_gqa_chunk_ws_bytes": (_sz, []),
    "i4_paged_gqa_chunk": (_i, [_vp, _vp]),
    "i4_kv_pages_ws_bytes": (_sz, [_i, _i]),
    "i4_kv_pages_copy": (_i, [_vp, _i, _i, _i, _i, _i, _vp, _vp, _i, _vp]),
    "i4_kv_pages_reserve": (_i, [_vp, _vp, _vp, _i, _vp, _vp, _sz, _vp]),
    "i4_kv_pages_fork": (_i, [_vp, _vp, _i, _i, _i, _vp, _vp, _i, _vp, _vp, _sz, _vp]),
    "i4_kv_pages_free": (_i, [_vp, _vp, _i, _vp]),
    "i4_kv_pages_compact": (_i, [_vp, _vp, _i, _i, _i, _vp, _vp, _sz, _vp]),
    "decode_step_graph_create": (_i, [ctypes.POINTER(ModelDesc), ctypes.POINTER(ModelWeights),
                                      ctypes.POINTER(SeqState), ctypes.POINTER(_vp)]),
    "decode_step_graph_replay": (_i, [_vp, _vp]),
    "decode_step_eager": (_i, [_vp, _vp]),
    "decode_step_kernel_count": (_i, [_vp]),
    "decode_step_phase_count": (_i, [_vp]),
    "decode_step_is_persistent": (_i, [_vp]),
    "decode_step_trace": (_i, [_vp, ctypes.POINTER(ctypes.c_ulonglong), _sz]),
    "decode_step_graph_destroy": (_i, [_vp]),
    "decode_step_launch_kernel": (_i, [_vp, _i, _vp]),
    "decode_step_buffer_copy": (_i, [_vp, _i, _vp, _sz, _i, _vp]),
    "i4_set_option": (_i, [ctypes.c_char_p, _i]),
    "i4_device_error": (_i, [_i]),
}


def lib() -> ctypes.CDLL:
    """Load libi4rt.so; raises if it has not been built (there is no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libi4rt.so not found at {LIB_PATH}; build it with "
                               "`python -m int4_weight_only_02_b200.build` (nvcc, sm_100a)")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def exported_symbols():
    return sorted(_SIGS)


def _check(status: int, name: str):
    if status != I4_OK:
        raise I4Error(status, f"{name}: {lib().i4_last_error().decode()}")


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def device_error(reset: bool = True) -> int:
    """0, or 1 when a bounded in-kernel wait gave up (synchronises the device)."""
    v = int(lib().i4_device_error(int(reset)))
    if v < 0:
        _check(v, "i4_device_error")
    return v


def set_option(name: str, value: int):
    _check(lib().i4_set_option(name.encode(), int(value)), "i4_set_option")


# ------------------------------------------------------------------ kernels

def int4_gemv(w, scales, x, bias=None, y=None, out_fp32: bool = False, group: int = 128, stream=None,
              unpack: int | None = None, max_ctas: int = 0):
    """y[M][N] = x[M][K] . dequant(w, scales)^T (+ bias), fp32 accumulation."""
    import torch
    x2 = x if x.dim() == 2 else x.view(1, -1)
    M, K = x2.shape
    N = w.shape[0]
    if y is None:
        y = torch.empty((M, N), device=x.device, dtype=torch.float32 if out_fp32 else torch.float16)
    if unpack is None and max_ctas == 0:
        st = lib().int4_gemv(_p(w), _p(scales), _p(x2), _p(bias), _p(y), int(out_fp32), M, N, K, group,
                             _stream(stream))
    else:
        st = lib().i4_int4_gemv_variant(_p(w), _p(scales), _p(x2), _p(bias), _p(y), int(out_fp32), M, N, K,
                                        0 if unpack is None else unpack, max_ctas, _stream(stream))
    _check(st, "int4_gemv")
    return y if x.dim() == 2 else y.view(-1)


def int4_gemm_ws_bytes(M: int, N: int, K: int) -> int:
    return int(lib().int4_gemm_ws_bytes(M, N, K))


def int4_gemm(w, scales, x, bias=None, y=None, out_fp32: bool = False, group: int = 128, ws=None, stream=None):
    """y[M][N] = x[M][K] . dequant(w, scales)^T (+ bias) on the tcgen05 tensor cores (any M). With `ws` (a
    zeroed uint8 device tensor of at least int4_gemm_ws_bytes(M, N, K) bytes) K may be split over CTAs."""
    import torch
    M, K = x.shape
    N = w.shape[0]
    if y is None:
        y = torch.empty((M, N), device=x.device, dtype=torch.float32 if out_fp32 else torch.float16)
    nb = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().int4_gemm(_p(w), _p(scales), _p(x), _p(bias), _p(y), int(out_fp32), M, N, K, group, _p(ws), nb,
                           _stream(stream)), "int4_gemm")
    return y


def int4_unpack(w, K: int, stream=None):
    import torch
    q = torch.empty((w.shape[0], K), device=w.device, dtype=torch.int8)
    _check(lib().i4_int4_unpack(_p(w), _p(q), w.shape[0], K, _stream(stream)), "i4_int4_unpack")
    return q


def paged_gqa_decode_ws_bytes(B, Hq, Hkv, D, page_size, max_pages_per_seq) -> int:
    return int(lib().paged_gqa_decode_ws_bytes(B, Hq, Hkv, D, page_size, max_pages_per_seq))


def paged_gqa_decode(q, k_pool, v_pool, page_table, ctx_len, out=None, scale=None, ws=None, stream=None):
    """out [B][Hq][D] fp16; the workspace is allocated zeroed when not given."""
    import torch
    B, Hq, D = q.shape
    _, Hkv, P, _ = k_pool.shape
    max_pages = page_table.shape[1]
    if out is None:
        out = torch.empty_like(q)
    nbytes = paged_gqa_decode_ws_bytes(B, Hq, Hkv, D, P, max_pages)
    if ws is None:
        ws = torch.zeros(nbytes, device=q.device, dtype=torch.uint8)
    scale = 1.0 / D ** 0.5 if scale is None else scale
    _check(lib().paged_gqa_decode(_p(q), _p(k_pool), _p(v_pool), _p(page_table), _p(ctx_len), _p(out), B, Hq, Hkv, D,
                                  P, max_pages, float(scale), _p(ws), ws.numel() * ws.element_size(),
                                  _stream(stream)), "paged_gqa_decode")
    return out


def paged_gqa_decode_static(q, k_pool, v_pool, page_table, ctx_len, out=None, scale=None, stream=None):
    """paged_gqa_decode with the library's fixed device scratch instead of a workspace (allocates nothing
    besides `out` when it is not given)."""
    import torch
    B, Hq, D = q.shape
    _, Hkv, P, _ = k_pool.shape
    if out is None:
        out = torch.empty_like(q)
    scale = 1.0 / D ** 0.5 if scale is None else scale
    _check(lib().paged_gqa_decode_static(_p(q), _p(k_pool), _p(v_pool), _p(page_table), _p(ctx_len), _p(out), B, Hq,
                                         Hkv, D, P, page_table.shape[1], float(scale), _stream(stream)),
           "paged_gqa_decode_static")
    return out


def paged_gqa_decode_strided(q, q_stride: int, Hq: int, k_pool, v_pool, page_table, ctx_len, out, ws, scale=None,
                             stream=None):
    """paged_gqa_decode reading the q rows of sequence b at q[b * q_stride ...] (e.g. inside qkv rows)."""
    B = page_table.shape[0]
    _, Hkv, P, D = k_pool.shape
    scale = 1.0 / D ** 0.5 if scale is None else scale
    _check(lib().i4_paged_gqa_decode_strided(_p(q), int(q_stride), _p(k_pool), _p(v_pool), _p(page_table),
                                             _p(ctx_len), _p(out), B, Hq, Hkv, D, P, page_table.shape[1],
                                             float(scale), _p(ws), ws.numel() * ws.element_size(),
                                             _stream(stream)), "i4_paged_gqa_decode_strided")
    return out


def embed_gather(table, tokens, out, stream=None):
    """out[b] = table[tokens[b]] (token ids clamped to the table)."""
    V, H = table.shape
    _check(lib().i4_embed_gather(_p(table), _p(tokens), _p(out), tokens.numel(), H, V, _stream(stream)),
           "i4_embed_gather")
    return out


def argmax_rows(logits, tokens, pos=None, ctx_len=None, stream=None):
    """tokens[b] = argmax(logits[b]) (lowest index on ties); pos and ctx_len advance by one when given."""
    B, N = logits.shape
    _check(lib().i4_argmax_rows(_p(logits), _p(tokens), _p(pos), _p(ctx_len), B, N, _stream(stream)),
           "i4_argmax_rows")
    return tokens


def paged_gather(pool, page_table, ctx_len, max_ctx: int, out=None, stream=None):
    import torch
    _, Hkv, P, D = pool.shape
    B, max_pages = page_table.shape
    if out is None:
        out = torch.zeros((B, Hkv, max_ctx, D), device=pool.device, dtype=pool.dtype)
    _check(lib().i4_paged_gather(_p(pool), _p(page_table), _p(ctx_len), _p(out), B, Hkv, D, P, max_pages, max_ctx,
                                 _stream(stream)), "i4_paged_gather")
    return out


def rmsnorm(x, gamma, out=None, resid=None, eps: float = 1e-6, stream=None):
    import torch
    x2 = x if x.dim() == 2 else x.view(1, -1)
    if out is None:
        out = torch.empty_like(x2)
    _check(lib().i4_rmsnorm(_p(x2), _p(resid), _p(gamma), _p(out), x2.shape[0], x2.shape[1], float(eps),
                            _stream(stream)), "i4_rmsnorm")
    return out if x.dim() == 2 else out.view(-1)


def rope_kv_append(qkv, pos, Hq: int, Hkv: int, theta: float = 1e6, k_pool=None, v_pool=None, page_table=None,
                   stream=None):
    """Rotates the q and k heads of qkv [B][(Hq+2Hkv)*128] in place; appends k, v to the pools when given."""
    B = qkv.shape[0] if qkv.dim() == 2 else 1
    P = k_pool.shape[2] if k_pool is not None else 0
    max_pages = page_table.shape[-1] if page_table is not None else 0
    _check(lib().i4_rope_kv_append(_p(qkv), _p(pos), B, Hq, Hkv, 128, float(theta), _p(k_pool), _p(v_pool),
                                   _p(page_table), P, max_pages, _stream(stream)), "i4_rope_kv_append")
    return qkv


def rmsnorm_rope(args: RmsnormRopeArgs, stream=None):
    _check(lib().rmsnorm_rope(ctypes.byref(args), _stream(stream)), "rmsnorm_rope")


def silu_mul(gate_up, out=None, stream=None):
    import torch
    g2 = gate_up if gate_up.dim() == 2 else gate_up.view(1, -1)
    M, I2 = g2.shape
    if out is None:
        out = torch.empty((M, I2 // 2), device=gate_up.device, dtype=torch.float16)
    _check(lib().silu_mul(_p(g2), _p(out), M, I2 // 2, _stream(stream)), "silu_mul")
    return out if gate_up.dim() == 2 else out.view(-1)


# ------------------------------------------------------------------ several new tokens of several sequences

# The argument structures of the header (RopeChunkArgs, ChunkAttnArgs, KvCacheDesc) as the calls below build them: packing
# takes a quarter of a ctypes structure's time, and one pointer less of ctypes' conversion than twenty arguments.
_ROPE_CHUNK = struct.Struct("@Qq7Q11i0q")
_CHUNK_ATTN = struct.Struct("@Qq8Q10if0q")
_CACHE = struct.Struct("@3Q4i0q")


def _refuse(name: str, what: str):
    raise I4Error(I4_EINVAL, f"{name}: {what}")


def _tensors(name: str, dims_of, f16=(), i32=(), other=()) -> int:
    """Refuses tensors that the call could not follow: all are contiguous and lie on the current CUDA device (whose
    current stream the call uses), those of ``f16`` and ``i32`` have that type and ``other`` is (tensor, dtype) pairs;
    ``dims_of`` gives the numbers of dimensions in the same order. Returns the device's index. The calls take
    microseconds on the GPU, so each tensor is asked four cheap questions."""
    import torch
    dev = (f16 or i32)[0].get_device()
    half, whole = torch.float16, torch.int32
    ok = dev >= 0 and dev == torch.cuda.current_device()
    i = 0
    for t in f16:
        ok = ok and t.dtype is half and t.dim() == dims_of[i] and t.is_contiguous() and t.get_device() == dev
        i += 1
    for t in i32:
        ok = ok and t.dtype is whole and t.dim() == dims_of[i] and t.is_contiguous() and t.get_device() == dev
        i += 1
    for t, dtype in other:
        ok = ok and t.dtype is dtype and t.dim() == dims_of[i] and t.is_contiguous() and t.get_device() == dev
        i += 1
    if ok:
        return dev
    every = [(t, half) for t in f16] + [(t, whole) for t in i32] + list(other)
    for (t, dtype), dims in zip(every, dims_of):
        if t.dtype is not dtype or t.dim() != dims or not t.is_contiguous():
            _refuse(name, f"a contiguous {dtype} tensor of {dims} dimensions is needed, got {t.dtype} {tuple(t.shape)}")
    _refuse(name, f"tensors on the current CUDA device are needed, got {sorted({str(t.device) for t, _ in every})}")


def _alloc(stream, make, *args, **kw):
    """make(*args, **kw) on the call's stream: what a call allocates for itself is filled, used and given back there."""
    if stream is None:
        return make(*args, **kw)
    import torch
    with torch.cuda.stream(stream):
        return make(*args, **kw)


def _raw_stream(stream, dev: int) -> int:
    """cudaStream_t of `stream`, or of device dev's current stream (without the stream object that
    torch.cuda.current_stream() makes)."""
    if stream is not None:
        return stream.cuda_stream
    import torch
    return torch._C._cuda_getCurrentRawStream(dev)


ROPE_SCALINGS = {"none": 0, "linear": 1, "yarn": 2}


def rope_table(max_pos: int, rotary_dim: int = 128, theta: float = 1e6, scaling: str = "none", factor: float = 1.0,
               original_ctx: int = 0, device="cuda", stream=None):
    """Angles of positions 0..max_pos-1 for ``rope_append_chunk``: [max_pos][rotary_dim/2][2] fp32 (cos, sin).
    ``scaling``: "none", "linear" (positions / factor) or "yarn" (frequencies blended over original_ctx)."""
    import torch
    if scaling not in ROPE_SCALINGS:
        _refuse("rope_table", f"scaling {scaling!r} is none of {sorted(ROPE_SCALINGS)}")
    cs = _alloc(stream, torch.empty, (max(int(max_pos), 0), max(int(rotary_dim), 0) // 2, 2), dtype=torch.float32, device=device)
    if cs.device.type != "cuda" or cs.device.index != torch.cuda.current_device():
        _refuse("rope_table", f"the current CUDA device is needed, got {cs.device}")
    _check(lib().i4_rope_table(_p(cs), int(max_pos), int(rotary_dim), float(theta), ROPE_SCALINGS[scaling],
                               float(factor), int(original_ctx), _stream(stream)), "rope_table")
    return cs


def rope_append_chunk(qkv, q_start, ctx_len, cs, Hq: int, Hkv: int, k_pool, v_pool, page_table, q_out=None,
                      interleaved: bool = False, stream=None):
    """Rotates the q and k heads of new tokens (qkv [T][(Hq+2Hkv)*128], rows may be strided) by the angles ``cs`` of
    their positions; q goes to q_out [T][Hq][128] (returned; rows behind the last sequence are left alone), k and v to
    the pages. The rotated part of a head is cs.shape[1] * 2 values."""
    import torch
    name = "rope_append_chunk"
    f16 = torch.float16
    if qkv.dim() != 2 or qkv.dtype is not f16 or (qkv.stride(1) != 1 and qkv.shape[1] > 1):
        _refuse(name, "qkv [T][(Hq+2Hkv)*128] fp16 with adjacent columns is needed")
    T, width = qkv.shape
    B, max_pages = page_table.shape
    if q_out is None:
        q_out = _alloc(stream, torch.zeros, (T, Hq, 128), device=qkv.device, dtype=f16)
    dev = _tensors(name, (4, 4, 3, 1, 1, 2, 3), (k_pool, v_pool, q_out), (q_start, ctx_len, page_table),
                   ((cs, torch.float32),))
    num_pages, hkv, P, D = shape = k_pool.shape
    max_pos, half, two = cs.shape
    if (qkv.get_device() != dev or width != (Hq + 2 * Hkv) * D or hkv != Hkv or v_pool.shape != shape
            or q_out.shape != (T, Hq, D) or q_start.numel() != B + 1 or ctx_len.numel() != B or two != 2):
        _refuse(name, f"shapes do not match: qkv {tuple(qkv.shape)}, pools {tuple(k_pool.shape)} {tuple(v_pool.shape)}, "
                      f"q_out {tuple(q_out.shape)}, {B} page-table rows, q_start {q_start.numel()}")
    if T == 0 or B == 0:
        return q_out
    _check(lib().i4_rope_append_chunk(
        _ROPE_CHUNK.pack(qkv.data_ptr(), qkv.stride(0) if T > 1 else width, q_start.data_ptr(), ctx_len.data_ptr(),
                         cs.data_ptr(), q_out.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), page_table.data_ptr(),
                         max_pos, half * 2, 1 if interleaved else 0, T, B, Hq, Hkv, D, P, max_pages, num_pages),
        _raw_stream(stream, dev)), name)
    return q_out


def paged_gqa_chunk_ws_bytes() -> int:
    return int(lib().i4_paged_gqa_chunk_ws_bytes())


def paged_gqa_chunk(q, k_pool, v_pool, page_table, q_start, ctx_len, out=None, window: int = 0, max_q: int = 0,
                    scale=None, ws=None, stream=None):
    """Attention of new tokens (q [T][Hq][128], token rows may be strided) over the pages that hold their own K/V
    already: row i of sequence b sees the positions up to ctx_len[b] - n + i, the last ``window`` of them if not 0.
    ``max_q``: the longest chunk if known on the host (a hint). ``ws``: paged_gqa_chunk_ws_bytes() bytes, any contents;
    allocated when not given. Rows behind the last sequence are left alone (zeros in an ``out`` made here)."""
    import torch
    name = "paged_gqa_chunk"
    f16 = torch.float16
    if q.dim() != 3 or q.dtype is not f16 or q.stride(2) != 1 or (q.stride(1) != q.shape[2] and q.shape[1] > 1):
        _refuse(name, "q [T][Hq][128] fp16 with adjacent heads is needed")
    T, Hq, D = shape = q.shape
    B, max_pages = page_table.shape
    if out is None:
        out = _alloc(stream, torch.zeros, (T, Hq, D), device=q.device, dtype=f16)
    if ws is None:
        ws = _alloc(stream, torch.empty, paged_gqa_chunk_ws_bytes(), device=q.device, dtype=torch.uint8)
    dev = _tensors(name, (4, 4, 3, 2, 1, 1, 1), (k_pool, v_pool, out), (page_table, q_start, ctx_len), ((ws, torch.uint8),))
    num_pages, Hkv, P, dk = pool = k_pool.shape
    if (q.get_device() != dev or dk != D or v_pool.shape != pool or out.shape != shape or q_start.numel() != B + 1
            or ctx_len.numel() != B):
        _refuse(name, f"shapes do not match: q {tuple(q.shape)}, pools {tuple(k_pool.shape)} {tuple(v_pool.shape)}, out "
                      f"{tuple(out.shape)}, {B} page-table rows, q_start {q_start.numel()}")
    if T == 0 or B == 0:
        return out
    _check(lib().i4_paged_gqa_chunk(
        _CHUNK_ATTN.pack(q.data_ptr(), q.stride(0) if T > 1 else Hq * D, k_pool.data_ptr(), v_pool.data_ptr(),
                         page_table.data_ptr(), q_start.data_ptr(), ctx_len.data_ptr(), out.data_ptr(), ws.data_ptr(),
                         ws.numel(), T, B, Hq, Hkv, D, P, max_pages, num_pages, window, max_q,
                         D ** -0.5 if scale is None else scale),
        _raw_stream(stream, dev)), name)
    return out


_SHAPE = operator.attrgetter("shape")


def _pool_array(name: str, pools):
    """(host array of the pools' addresses, their shape) of a sequence of pools of 16-bit values and one layout: pages of another
    would be moved by the first one's."""
    import torch
    T = torch.Tensor
    shape = pools[0].shape if len(pools) else ()
    if len(shape) != 4:
        _refuse(name, "pools [num_pages][Hkv][page_size][D] are needed")
    dev = pools[0].get_device()
    if dev < 0 or dev != torch.cuda.current_device():
        _refuse(name, f"pools on the current CUDA device are needed, got {pools[0].device}")
    if (list(map(_SHAPE, pools)) != [shape] * len(pools) or set(map(T.element_size, pools)) != {2}
            or not all(map(T.is_contiguous, pools)) or set(map(T.get_device, pools)) != {dev}):
        _refuse(name, "pools of one shape, two bytes a value, contiguous and on one device are needed")
    return array.array("Q", map(T.data_ptr, pools)), shape


def _cache_desc(name: str, page_table, ctx_len, refs, page_size: int, ws, *lists):
    """(the cache's descriptor, its device)."""
    import torch
    n = lists[0].numel()
    dev = _tensors(name, _CACHE_DIMS, (), (page_table, ctx_len, refs, *lists), () if ws is None else ((ws, torch.uint8),))
    S, width = page_table.shape
    if ctx_len.numel() != S or any([t.numel() != n for t in lists]):
        _refuse(name, f"shapes do not match: page_table {tuple(page_table.shape)}, ctx_len {tuple(ctx_len.shape)}, lists of "
                      f"{[t.numel() for t in lists]}")
    return _CACHE.pack(page_table.data_ptr(), ctx_len.data_ptr(), refs.data_ptr(), S, width, page_size, refs.numel()), dev


_CACHE_DIMS = (2, 1, 1, 1, 1, 1, 1)  # page_table, then lists and the workspace


def kv_pages_ws_bytes(num_pages: int, n_seqs: int) -> int:
    return int(lib().i4_kv_pages_ws_bytes(num_pages, n_seqs))


def _kv_ws(ws, page_table, refs, stream):
    import torch
    if ws is None:
        ws = _alloc(stream, torch.empty, max(kv_pages_ws_bytes(refs.numel(), page_table.shape[0]), 256), dtype=torch.uint8,
                         device=refs.device)
    return ws


def kv_pages_copy(pools, src, dst, stream=None):
    """Page src[i] -> dst[i] in every pool (device int32 lists; no page may be both source and target)."""
    arr, (num_pages, Hkv, P, D) = _pool_array("kv_pages_copy", pools)
    dev = _tensors("kv_pages_copy", (1, 1), (), (src, dst))
    if src.numel() != dst.numel():
        _refuse("kv_pages_copy", f"{src.numel()} sources and {dst.numel()} targets")
    _check(lib().i4_kv_pages_copy(arr.buffer_info()[0], len(pools), num_pages, Hkv, P, D, src.data_ptr(), dst.data_ptr(), src.numel(),
                                  _raw_stream(stream, dev)), "kv_pages_copy")


def kv_pages_reserve(page_table, ctx_len, refs, page_size: int, seqs, add, status=None, ws=None, stream=None):
    """Room for add[i] more tokens of sequence seqs[i]: free pages into its row, ctx_len += add[i]. Returns status [n]
    (0 done, 1 not enough free pages, 2 refused)."""
    import torch
    if status is None:
        status = _alloc(stream, torch.empty_like, seqs)
    ws = _kv_ws(ws, page_table, refs, stream)
    desc, dev = _cache_desc("kv_pages_reserve", page_table, ctx_len, refs, page_size, ws, seqs, add, status)
    _check(lib().i4_kv_pages_reserve(desc, seqs.data_ptr(), add.data_ptr(), seqs.numel(), status.data_ptr(),
                                     ws.data_ptr(), ws.numel(), _raw_stream(stream, dev)), "kv_pages_reserve")
    return status


def kv_pages_fork(pools, page_table, ctx_len, refs, src, dst, status=None, ws=None, stream=None):
    """Sequence dst[i] becomes a continuation of src[i]: full pages shared, a last page that is not full copied in every
    pool. Returns status [n] (0 done, 1 no free page and dst left empty, 2 refused)."""
    import torch
    arr, (num_pages, Hkv, P, D) = _pool_array("kv_pages_fork", pools)
    if status is None:
        status = _alloc(stream, torch.empty_like, src)
    ws = _kv_ws(ws, page_table, refs, stream)
    desc, dev = _cache_desc("kv_pages_fork", page_table, ctx_len, refs, P, ws, src, dst, status)
    if refs.numel() != num_pages:
        _refuse("kv_pages_fork", f"{refs.numel()} reference counts for {num_pages} pages")
    _check(lib().i4_kv_pages_fork(desc, arr.buffer_info()[0], len(pools), Hkv, D, src.data_ptr(), dst.data_ptr(), src.numel(),
                                  status.data_ptr(), ws.data_ptr(), ws.numel(), _raw_stream(stream, dev)), "kv_pages_fork")
    return status


def kv_pages_free(page_table, ctx_len, refs, page_size: int, seqs, stream=None):
    """The pages of the sequences are given back; their rows become -1 and their ctx_len 0."""
    desc, dev = _cache_desc("kv_pages_free", page_table, ctx_len, refs, page_size, None, seqs)
    _check(lib().i4_kv_pages_free(desc, seqs.data_ptr(), seqs.numel(), _raw_stream(stream, dev)),
           "kv_pages_free")


def kv_pages_compact(pools, page_table, ctx_len, refs, n_live=None, ws=None, stream=None):
    """Moves the pages in use to the lowest ids in every pool; page_table and refs follow. Returns n_live [1], the number
    of pages in use."""
    import torch
    arr, (num_pages, Hkv, P, D) = _pool_array("kv_pages_compact", pools)
    if n_live is None:
        n_live = _alloc(stream, torch.empty, 1, dtype=torch.int32, device=refs.device)
    ws = _kv_ws(ws, page_table, refs, stream)
    desc, dev = _cache_desc("kv_pages_compact", page_table, ctx_len, refs, P, ws, n_live)
    if refs.numel() != num_pages or n_live.numel() != 1:
        _refuse("kv_pages_compact", f"{refs.numel()} reference counts for {num_pages} pages, n_live of {n_live.numel()}")
    _check(lib().i4_kv_pages_compact(desc, arr.buffer_info()[0], len(pools), Hkv, D, n_live.data_ptr(), ws.data_ptr(),
                                     ws.numel(), _raw_stream(stream, dev)), "kv_pages_compact")
    return n_live


from .runtime import (BatchedDecode, ChunkedDecoder, DecodeGraph, DeviceModel, PagedCache, Prefill,  # noqa: E402,F401
                      Sequence)  # noqa: E402,F401
