"""Python binding of libggufdq (the GB300 GGUF block-dequant GEMV / MoE library).

Argument marshalling only: every function here passes device pointers, sizes and the CUDA
stream of PyTorch tensors to the C ABI declared in ``include/ggufdq.h`` and raises
``QGError`` on a non-zero status.  All arithmetic runs in the library's CUDA kernels; there
is no other code path.  If the shared library has not been built, importing works but the
first call raises, naming the build step (``gguf_block_dequant_gb300.build.build()``).
"""
from __future__ import annotations

import ctypes
import os
import threading

from . import build as _build

Q4_0, Q8_0, Q4_K, Q6_K = 2, 8, 12, 14
BLOCK = {Q8_0: (32, 34), Q4_0: (32, 18), Q4_K: (256, 144), Q6_K: (256, 210)}

QG_OK, QG_EINVAL_SHAPE, QG_EINVAL_PTR, QG_EALIGN, QG_EUNSUPPORTED, QG_ECUDA, QG_EDEVICE_ID, QG_ETIMEOUT, \
    QG_EWORKSPACE = range(9)

_lock = threading.Lock()
_lib = None


class QGError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {strerror(status)} (status {status})")


def lib_path() -> str:
    return _build.LIB


def load():
    """Load libggufdq.so (no fallback: raises if it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_build.LIB):
            raise RuntimeError(f"{_build.LIB} is not built; run gguf_block_dequant_gb300.build.build()")
        L = ctypes.CDLL(_build.LIB)
        P, I, I64, SZ, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p
        sig = {
            "qg_version": ([], I),
            "qg_strerror": ([I], ctypes.c_char_p),
            "qg_block_shape": ([I, P, P], I),
            "qg_device_status": ([P, I], I),
            "qg_set_static_weights": ([S, I], I),
            "qgemv_q8_0": ([P, P, P, I64, I64, S], I),
            "qgemv_q4_0": ([P, P, P, I64, I64, S], I),
            "qgemv_q4_k": ([P, P, P, I64, I64, S], I),
            "qgemv_q6_k": ([P, P, P, I64, I64, S], I),
            "qgemv_t": ([I, P, P, P, I64, I64, I, S], I),
            "qgemv_multi": ([I, I, P, P, P, I64, P, I, S], I),
            "qgemm_workspace_size": ([I, I64, I64, I64], SZ),
            "qgemm": ([I, P, P, P, I64, I64, I64, P, SZ, S], I),
            "moe_workspace_size": ([I, I, I, I, I], SZ),
            "moe_route_topk": ([P, P, I, I, I, I, P, P, P, P, SZ, S], I),
            "moe_route_topk_noalloc": ([P, P, I, I, I, I, P, P, P, S], I),
            "moe_expert_swiglu": ([I, P, P, I64, P, I, I, P, P, I, I, I, I, P, P, SZ, S], I),
            "moe_combine": ([I, P, I64, P, I, I, P, P, P, I, I, I, I, P, I, P, SZ, S], I),
            "moe_layer": ([I, P, P, P, P, P, I64, P, I, I, I, I, I, I, P, P, P, P, P, SZ, S], I),
            "qg_embed_rows": ([I, P, I64, I64, P, I, ctypes.c_float, P, S], I),
            "qg_rmsnorm": ([P, P, I, I64, ctypes.c_float, ctypes.c_float, P, S], I),
            "moe_expert_act": ([I, P, P, I64, P, I, I, P, P, I, I, I, I, P, P, P, SZ, S], I),
            "moe_combine_ex": ([I, P, I64, P, I, I, P, P, P, I, I, I, I, P, P, I, P, SZ, S], I),
            "moe_layer_ex": ([I, P, P, P, P, P, I64, P, I, I, I, I, I, I, P, P, P, P, P, P, SZ, S], I),
            "qg_argmax_rows": ([P, I, I64, P, S], I),
            "qg_head_argmax": ([I, P, I64, I64, P, I, P, P, S], I),
            "qg_rope_freqs": ([I, ctypes.c_double, P, P], I),
            "qg_kv_append": ([P, P, I, P, I64, P, I64, P, I64, P, P, ctypes.c_float, P, I, I, P, S], I),
            "qg_attn_workspace_size": ([P, P, I], SZ),
            "qg_attn_paged": ([P, P, I, P, I64, ctypes.c_float, P, I, P, SZ, S], I),
            "qg_beam_workspace_size": ([I, I, I, I64], SZ),
            "qg_beam_select": ([P, P, P, I, I, I, I, I64, P, P, P, P, P, SZ, S], I),
            "qg_beam_reorder": ([P, I, P, I, P, S], I),
        }
        for name, (args, res) in sig.items():
            if hasattr(L, name):
                f = getattr(L, name)
                f.argtypes = args
                f.restype = res
        _lib = L
        return L


def strerror(status: int) -> str:
    try:
        return load().qg_strerror(int(status)).decode()
    except Exception:  # noqa: BLE001 - message only
        return f"status {status}"


def _ptr(t):
    return None if t is None else t.data_ptr()


_raw_stream = None  # the current stream's handle, without a Stream object where torch offers it


def _current_stream():
    global _raw_stream
    if _raw_stream is None:
        import torch

        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        device = torch.cuda.current_device
        current = torch.cuda.current_stream
        _raw_stream = (lambda: raw(device())) if raw else (lambda: current().cuda_stream)
    return _raw_stream()


def _stream(stream):
    if stream is None:
        return _current_stream()
    return stream if isinstance(stream, int) else stream.cuda_stream


def _call(name, *args):
    rc = getattr(_lib or load(), name)(*args)
    if rc != QG_OK:
        raise QGError(rc, name)


def version() -> int:
    return load().qg_version()


def device_status(clear: bool = True) -> int:
    v = ctypes.c_uint32(0)
    _call("qg_device_status", ctypes.byref(v), int(clear))
    return v.value


def set_static_weights(enable: bool, stream=None) -> bool:
    """Declare the weight buffers read on `stream` (default: the current stream) immutable:
    GEMVs enqueued there may start streaming them before the preceding kernel finishes.
    Returns the stream's previous setting."""
    prev = load().qg_set_static_weights(_stream(stream), int(bool(enable)))
    if prev < 0:
        raise QGError(QG_ECUDA, "qg_set_static_weights")
    return bool(prev)


def row_bytes(qtype: int, n: int) -> int:
    qk, bb = BLOCK[qtype]
    return (n // qk) * bb


# ---- GEMV / GEMM ---------------------------------------------------------------------------

_GEMV1 = {Q8_0: "qgemv_q8_0", Q4_0: "qgemv_q4_0", Q4_K: "qgemv_q4_k", Q6_K: "qgemv_q6_k"}


def qgemv(qtype, w, x, M, N, y, stream=None):
    """y[m] = W[m] . x for one token (qgemv_q8_0 / _q4_0 / _q4_k / _q6_k)."""
    _call(_GEMV1[qtype], _ptr(w), _ptr(x), _ptr(y), M, N, _stream(stream))
    return y


def qgemv_q8_0(w, x, y, M, N, stream=None):
    return qgemv(Q8_0, w, x, M, N, y, stream)


def qgemv_q4_0(w, x, y, M, N, stream=None):
    return qgemv(Q4_0, w, x, M, N, y, stream)


def qgemv_q4_k(w, x, y, M, N, stream=None):
    return qgemv(Q4_K, w, x, M, N, y, stream)


def qgemv_q6_k(w, x, y, M, N, stream=None):
    return qgemv(Q6_K, w, x, M, N, y, stream)


def qgemv_t(qtype, w, x, y, M, N, T, stream=None):
    """Y[t][m] = W[m] . X[t] for T <= 16 token rows, one weight pass."""
    _call("qgemv_t", qtype, _ptr(w), _ptr(x), _ptr(y), M, N, T, _stream(stream))
    return y


def qgemv_multi(qtype, ws, ys, x, N, T, stream=None):
    """Y_j = W_j . X for up to 4 matrices sharing the activations X [T][N], one launch.
    ws: weight tensors (raw blocks), ys: f32 [T][M_j] outputs; M_j from ys."""
    n = len(ws)
    if n != len(ys):
        raise ValueError("one output per weight tensor")
    W = (ctypes.c_void_p * n)(*[w.data_ptr() for w in ws])
    Y = (ctypes.c_void_p * n)(*[y.data_ptr() for y in ys])
    M = (ctypes.c_int64 * n)(*[int(y.shape[-1]) for y in ys])
    _call("qgemv_multi", qtype, n, W, Y, M, N, _ptr(x), T, _stream(stream))
    return ys


def embed_rows(qtype, table, V, N, ids, out, scale=1.0, stream=None):
    """out[i] = scale * dequantized row ids[i] of the [V][N] table (raw blocks)."""
    _call("qg_embed_rows", qtype, _ptr(table), V, N, _ptr(ids), int(ids.numel()), float(scale), _ptr(out),
          _stream(stream))
    return out


def rmsnorm(x, w, eps, y, k=1.0, stream=None):
    """y[t] = ((x[t] / sqrt(mean(x[t]^2) + eps)) * k) * w for x [T][N] (k = 1: plain RMSNorm)."""
    T, N = (1, x.shape[-1]) if x.dim() == 1 else (x.shape[0], x.shape[1])
    _call("qg_rmsnorm", _ptr(x), _ptr(w), T, N, float(eps), float(k), _ptr(y), _stream(stream))
    return y


def argmax_rows(logits, ids, stream=None):
    """ids[t] = lowest index of the largest value of logits[t] (NaN never picked)."""
    T, n = (1, logits.shape[-1]) if logits.dim() == 1 else (logits.shape[0], logits.shape[1])
    _call("qg_argmax_rows", _ptr(logits), T, n, _ptr(ids), _stream(stream))
    return ids


def head_argmax(qtype, w, x, M, N, T, logits, ids, stream=None):
    """Tied-head GEMV over T <= 16 tokens into logits [T][M], then ids[t] = argmax logits[t]."""
    _call("qg_head_argmax", qtype, _ptr(w), M, N, _ptr(x), T, _ptr(logits), _ptr(ids), _stream(stream))
    return ids


def qgemm_workspace_size(qtype, M, N, T) -> int:
    return int(load().qgemm_workspace_size(qtype, M, N, T))


def qgemm(qtype, w, x, y, M, N, T, workspace=None, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _call("qgemm", qtype, _ptr(w), _ptr(x), _ptr(y), M, N, T, _ptr(workspace), ws_bytes, _stream(stream))
    return y


# ---- MoE -------------------------------------------------------------------------------------

def moe_workspace_size(T, k, E, H, F) -> int:
    return int(load().moe_workspace_size(T, k, E, H, F))


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def moe_route_topk(xn, wr, T, H, E, k, ids, weights, logits=None, workspace=None, stream=None):
    _call("moe_route_topk", _ptr(xn), _ptr(wr), T, H, E, k, _ptr(ids), _ptr(weights), _ptr(logits),
          _ptr(workspace), _nbytes(workspace), _stream(stream))
    return ids, weights


def moe_route_topk_noalloc(xn, wr, T, H, E, k, ids, weights, logits=None, stream=None):
    """moe_route_topk without a workspace argument (library-held scratch, T * E <= 16384)."""
    _call("moe_route_topk_noalloc", _ptr(xn), _ptr(wr), T, H, E, k, _ptr(ids), _ptr(weights), _ptr(logits),
          _stream(stream))
    return ids, weights


def moe_expert_swiglu(qtype, w_gate, w_up, expert_stride, slots, n_slots, E, ids, xn, T, k, H, F, act,
                      workspace=None, stream=None):
    _call("moe_expert_swiglu", qtype, _ptr(w_gate), _ptr(w_up), expert_stride, _ptr(slots), n_slots, E, _ptr(ids),
          _ptr(xn), T, k, H, F, _ptr(act), _ptr(workspace), _nbytes(workspace), _stream(stream))
    return act


def moe_combine(qtype, w_down, expert_stride, slots, n_slots, E, ids, weights, act, T, k, H, F, x_inout,
                add_residual=1, workspace=None, stream=None):
    _call("moe_combine", qtype, _ptr(w_down), expert_stride, _ptr(slots), n_slots, E, _ptr(ids), _ptr(weights),
          _ptr(act), T, k, H, F, _ptr(x_inout), int(add_residual), _ptr(workspace), _nbytes(workspace),
          _stream(stream))
    return x_inout


ACT_SILU, ACT_GELU_TANH = 0, 1


class MoeVariant(ctypes.Structure):
    """qg_moe_variant: expert activation, per-expert down scale, sigmoid-gated shared expert."""
    _fields_ = [("act", ctypes.c_int), ("down_scale", ctypes.c_void_p), ("shared_out", ctypes.c_void_p),
                ("shared_gate", ctypes.c_void_p)]


def moe_variant(act=ACT_SILU, down_scale=None, shared_out=None, shared_gate=None):
    """A qg_moe_variant from tensors (None for the fields not used).  The struct keeps the
    tensors alive: it holds their addresses, and the kernels read them when they run."""
    dp = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    v = MoeVariant(int(act), dp(down_scale), dp(shared_out), dp(shared_gate))
    v.tensors = (down_scale, shared_out, shared_gate)
    return v


def _var(v):
    return None if v is None else ctypes.byref(v)


def moe_expert_act(qtype, w_gate, w_up, expert_stride, slots, n_slots, E, ids, xn, T, k, H, F, variant, act,
                   workspace=None, stream=None):
    _call("moe_expert_act", qtype, _ptr(w_gate), _ptr(w_up), expert_stride, _ptr(slots), n_slots, E, _ptr(ids),
          _ptr(xn), T, k, H, F, _var(variant), _ptr(act), _ptr(workspace), _nbytes(workspace), _stream(stream))
    return act


def moe_combine_ex(qtype, w_down, expert_stride, slots, n_slots, E, ids, weights, act, T, k, H, F, variant, x_inout,
                   add_residual=1, workspace=None, stream=None):
    _call("moe_combine_ex", qtype, _ptr(w_down), expert_stride, _ptr(slots), n_slots, E, _ptr(ids), _ptr(weights),
          _ptr(act), T, k, H, F, _var(variant), _ptr(x_inout), int(add_residual), _ptr(workspace),
          _nbytes(workspace), _stream(stream))
    return x_inout


def moe_layer_ex(qtype, xn, wr, w_gate, w_up, w_down, expert_stride, slots, n_slots, T, H, F, E, k, variant, ids,
                 weights, act, x_inout, workspace=None, stream=None):
    _call("moe_layer_ex", qtype, _ptr(xn), _ptr(wr), _ptr(w_gate), _ptr(w_up), _ptr(w_down), expert_stride,
          _ptr(slots), n_slots, T, H, F, E, k, _var(variant), _ptr(ids), _ptr(weights), _ptr(act), _ptr(x_inout),
          _ptr(workspace), _nbytes(workspace), _stream(stream))
    return x_inout


def moe_layer(qtype, xn, wr, w_gate, w_up, w_down, expert_stride, slots, n_slots, T, H, F, E, k, ids, weights, act,
              x_inout, workspace=None, stream=None):
    _call("moe_layer", qtype, _ptr(xn), _ptr(wr), _ptr(w_gate), _ptr(w_up), _ptr(w_down), expert_stride,
          _ptr(slots), n_slots, T, H, F, E, k, _ptr(ids), _ptr(weights), _ptr(act), _ptr(x_inout),
          _ptr(workspace), _nbytes(workspace), _stream(stream))
    return x_inout


# ---- paged cache, attention, beam search ------------------------------------------------------

DT_F32, DT_F16, DT_BF16 = 0, 1, 2


_dtypes = {}


def _dtype(t):
    if not _dtypes:
        import torch

        _dtypes.update({torch.float32: DT_F32, torch.float16: DT_F16, torch.bfloat16: DT_BF16})
    try:
        return _dtypes[t.dtype]
    except KeyError:
        raise ValueError(f"unsupported dtype {t.dtype}") from None


class KVCache(ctypes.Structure):
    """qg_kv_cache: one layer's page pools."""
    device = None  # the pools' GPU (kv_cache sets it: what goes with the cache has to be there too)
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int), ("n_pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("n_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class KVBatch(ctypes.Structure):
    """qg_kv_batch: the sequences, their lengths and page lists, and the prefixes they share."""
    device = None
    _fields_ = [("n_seqs", ctypes.c_int), ("n_tokens", ctypes.c_int), ("n_groups", ctypes.c_int),
                ("max_pages", ctypes.c_int), ("max_prefix_pages", ctypes.c_int), ("q_start", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("pages", ctypes.c_void_p), ("group_start", ctypes.c_void_p),
                ("prefix_len", ctypes.c_void_p), ("prefix_pages", ctypes.c_void_p)]


_f32_i64 = None


def _types():
    global _f32_i64
    if _f32_i64 is None:
        import torch

        _f32_i64 = (torch.float32, torch.int64)
    return _f32_i64


def _check(t, dtype, what):
    """A contiguous tensor of the named torch dtype (None passes)."""
    import torch

    if t is not None and (t.dtype is not getattr(torch, dtype) or not t.is_contiguous()):
        raise ValueError(f"{what} must be contiguous and {dtype}")


def _on(device, names, *tensors):
    """Refuses tensors that are not on the GPU `device` (None: unknown, from a struct filled by hand): the
    kernels take addresses, and one of host memory or of another GPU would fault."""
    if device is None:
        return
    if device < 0:
        raise ValueError("the cached-decode calls take GPU tensors")
    for i, t in enumerate(tensors):
        if t is not None and t.get_device() != device:
            raise ValueError(f"{names.split()[i]} must be on GPU {device} with the rest")


def _cache_device(cache, batch):
    d, b = cache.device, batch.device
    if d is not None and b is not None and d != b:
        raise ValueError("the batch must be on the cache's GPU")
    return b if d is None else d


def kv_cache(k, v):
    """A qg_kv_cache of two pools [pages][tokens][heads][D] of one f16 or bf16 type (any strides
    with the last one 1: a head-major pool is passed as its permuted view).  Keeps them alive."""
    if k.shape != v.shape or k.dtype != v.dtype or k.dim() != 4:
        raise ValueError("k and v must be 4-D pools of one shape and type")
    if k.stride() != v.stride() or k.stride(3) != 1:
        raise ValueError("k and v must have equal strides with heads' elements side by side")
    if k.device != v.device:
        raise ValueError("k and v must be on one device")
    c = KVCache(k.data_ptr(), v.data_ptr(), _dtype(k), *k.shape, *k.stride()[:3])
    c.tensors = (k, v)
    c.device = k.get_device()
    return c


def kv_caches(ks, vs):
    """The layers' caches as one array (beam_reorder), each of them a cache for the other calls."""
    cs = [kv_cache(k, v) for k, v in zip(ks, vs, strict=True)]
    if any(c.device != cs[0].device for c in cs):
        raise ValueError("the layers' pools must be on one device")

    class Caches(KVCache * len(cs)):
        def __getitem__(self, i):
            c = super().__getitem__(i)
            if isinstance(c, KVCache):
                c.device = self.device
            return c

    arr = Caches(*cs)
    arr.tensors = [c.tensors for c in cs]
    arr.device = cs[0].device if cs else None
    return arr


def _i32(t, what, dim, device):
    import torch

    if t is None:
        return
    if t.dtype != torch.int32 or t.dim() != dim or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{what} must be a contiguous {dim}-D int32 tensor on {device}")


def kv_batch(kv_len, pages, q_start=None, n_tokens=None, group_start=None, prefix_len=None, prefix_pages=None):
    """A qg_kv_batch from int32 device tensors: kv_len [B], pages [B][max_pages], q_start [B + 1] with the
    number of token rows (None: one token per sequence), group_start [G + 1], prefix_len [G],
    prefix_pages [G][max_prefix_pages].  Keeps them alive."""
    dev = kv_len.device
    _i32(kv_len, "kv_len", 1, dev)
    _i32(pages, "pages", 2, dev)
    _i32(q_start, "q_start", 1, dev)
    _i32(group_start, "group_start", 1, dev)
    _i32(prefix_len, "prefix_len", 1, dev)
    _i32(prefix_pages, "prefix_pages", 2, dev)
    B = kv_len.shape[0]
    G = 0 if prefix_len is None else prefix_len.shape[0]
    if pages.shape[0] != B:
        raise ValueError("pages must have a row per sequence")
    if q_start is None:
        if n_tokens not in (None, B):
            raise ValueError("without q_start there is one token per sequence")
        n_tokens = B
    elif q_start.shape[0] != B + 1 or n_tokens is None:
        raise ValueError("q_start must have n_seqs + 1 entries, and n_tokens be given")
    if G and (group_start is None or group_start.shape[0] != G + 1 or
              (prefix_pages is not None and prefix_pages.shape[0] != G)):
        raise ValueError("group_start must have n_groups + 1 entries and prefix_pages a row per group")
    b = KVBatch(B, n_tokens, G, pages.shape[1], 0 if prefix_pages is None else prefix_pages.shape[1],
                *[None if t is None else t.data_ptr()
                  for t in (q_start, kv_len, pages, group_start, prefix_len, prefix_pages)])
    b.tensors = (kv_len, pages, q_start, group_start, prefix_len, prefix_pages)
    b.device = kv_len.get_device()
    return b


def rope_freqs(rot, theta, factors=None):
    """The rotation table of kv_append (qg_rope_freqs), int64 [rot / 2] on the host; factors from anywhere."""
    import torch

    out = torch.empty((max(rot // 2, 1),), dtype=torch.int64)
    f = None if factors is None else torch.as_tensor(factors, dtype=torch.float32, device="cpu").contiguous()
    if f is not None and f.numel() != rot // 2:
        raise ValueError("one factor per pair")
    _call("qg_rope_freqs", rot, float(theta), _ptr(f), _ptr(out))
    return out


def _rows(t, T, n, what):
    """Row stride of a tensor whose T rows of n elements may be slices of wider ones."""
    if t is None:
        return 0
    shape, st = t.shape, t.stride()
    if len(shape) == 3 and (st[2] != 1 or (shape[1] > 1 and st[1] != shape[2])):
        raise ValueError(f"{what}: a token's heads must lie side by side")
    if len(shape) not in (2, 3) or st[-1] != 1 or shape[0] != T or t.numel() != T * n:
        raise ValueError(f"{what} must have {T} rows of {n} elements")
    return st[0] if T > 1 else n


def kv_append(cache, batch, q, k, v, q_out, freqs, pairs=False, q_norm=None, k_norm=None, eps=1e-6, stream=None):
    """Norm, rotate and append a step's tokens (qg_kv_append).  q [T][Hq*D], k, v [T][heads*D]: f32, rows
    may be slices of one projection's; q_out [T][Hq][D] of the cache's type; freqs a device copy of
    rope_freqs (None: no rotation)."""
    T, D, Hkv = batch.n_tokens, cache.head_dim, cache.n_heads
    f32, i64 = _types()
    if (k.dtype is not f32 or v.dtype is not f32 or (q is not None and q.dtype is not f32) or
            (freqs is not None and (freqs.dtype is not i64 or not freqs.is_contiguous()))):
        raise ValueError("q, k and v must be f32 and freqs contiguous int64")
    Hq = 0
    if q is not None:
        Hq = q_out.numel() // (T * D) if T else Hkv
        if _dtype(q_out) != cache.dtype or not q_out.is_contiguous() or q_out.numel() != T * Hq * D:
            raise ValueError("q_out must be contiguous, of the cache's type and have whole heads for every token")
    for t in (q_norm, k_norm):
        if t is not None and (t.dtype is not f32 or t.numel() != D or not t.is_contiguous()):
            raise ValueError("q_norm and k_norm must be contiguous f32 of head_dim elements")
    qs, ks, vs = _rows(q, T, Hq * D, "q"), _rows(k, T, Hkv * D, "k"), _rows(v, T, Hkv * D, "v")
    _on(_cache_device(cache, batch), "k v q q_out freqs q_norm k_norm", k, v, q, q_out, freqs, q_norm, k_norm)
    _call("qg_kv_append", ctypes.byref(cache), ctypes.byref(batch), Hq, _ptr(q), qs, _ptr(k),
          ks, _ptr(v), vs, _ptr(q_norm), _ptr(k_norm), float(eps),
          _ptr(freqs), 0 if freqs is None else 2 * freqs.numel(), int(bool(pairs)), _ptr(q_out), _stream(stream))
    return q_out


def attn_workspace_size(cache, batch, Hq) -> int:
    return int(load().qg_attn_workspace_size(ctypes.byref(cache), ctypes.byref(batch), Hq))


def attn_paged(cache, batch, q, out, scale, workspace, stream=None):
    """Causal attention of the batch's new tokens over the cache (qg_attn_paged).  q [T][Hq][D] of the
    cache's type (rows may be slices), out [T][Hq][D] of that type or f32."""
    T, D = batch.n_tokens, cache.head_dim
    Hq = out.numel() // (T * D) if T else cache.n_heads
    if _dtype(q) != cache.dtype or not out.is_contiguous():
        raise ValueError("q must be of the cache's type and out contiguous")
    if out.numel() != T * Hq * D:
        raise ValueError(f"out must have {T} rows of whole heads")
    qs = _rows(q, T, Hq * D, "q")
    _on(_cache_device(cache, batch), "q out workspace", q, out, workspace)
    _call("qg_attn_paged", ctypes.byref(cache), ctypes.byref(batch), Hq, _ptr(q), qs, float(scale),
          _ptr(out), _dtype(out), _ptr(workspace), _nbytes(workspace), _stream(stream))
    return out


def beam_workspace_size(N, W, K, V) -> int:
    return int(load().qg_beam_workspace_size(N, W, K, V))


def beam_select(logits, scores, N, W, out_scores, parents, tokens, workspace, done=None, eos=-1, done_out=None,
                stream=None):
    """The K best continuations of N requests' W beams (qg_beam_select); K from the outputs' [N][K]."""
    V, K = logits.shape[-1], out_scores.shape[-1]
    if logits.numel() != N * W * V or scores.numel() != N * W:
        raise ValueError("logits must be [N*W][V] and scores [N*W]")
    for t, dtype, what in ((logits, "float32", "logits"), (scores, "float32", "scores"),
                           (out_scores, "float32", "out_scores"), (parents, "int32", "parents"),
                           (tokens, "int32", "tokens"), (done, "uint8", "done"), (done_out, "uint8", "done_out")):
        _check(t, dtype, what)
    if any(t is not None and t.numel() != N * K for t in (out_scores, parents, tokens, done_out)):
        raise ValueError("outputs must be [N][K]")
    if done is not None and done.numel() != N * W:
        raise ValueError("done must be [N*W]")
    _on(logits.get_device(), "scores out_scores parents tokens done done_out workspace", scores, out_scores, parents, tokens,
        done, done_out, workspace)
    _call("qg_beam_select", _ptr(logits), _ptr(scores), _ptr(done), int(eos), N, W, K, V, _ptr(out_scores),
          _ptr(parents), _ptr(tokens), _ptr(done_out), _ptr(workspace), _nbytes(workspace), _stream(stream))
    return out_scores, parents, tokens


def beam_reorder(caches, batch, parents, W, stream=None):
    """Beam i of each request takes the cached tokens of beam parents[n][i], in place (qg_beam_reorder).
    caches: kv_caches of all layers; batch: kv_batch(kv_len, pages)."""
    if parents.numel() != batch.n_seqs:
        raise ValueError("parents must be [N][W]")
    _check(parents, "int32", "parents")
    _on(_cache_device(caches, batch), "parents", parents)
    _call("qg_beam_reorder", caches, len(caches), ctypes.byref(batch), W, _ptr(parents), _stream(stream))
