"""ctypes binding of libpi.so (the C ABI in include/pi.h).

Argument marshalling only: every function takes torch tensors (device memory)
or plain integers, converts them to pointers / sizes, calls the entry point of
the same name and raises PiError on a nonzero status.  All computation runs in
the library's HIP kernels.  There is no fallback: if libpi.so is missing or
cannot be loaded, `lib()` raises.
"""
from __future__ import annotations

import ctypes as C
import os
from typing import Optional, Sequence

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libpi.so")

PI_OK, PI_ERR_ARG, PI_ERR_SHAPE, PI_ERR_ALIGN, PI_ERR_DTYPE, PI_ERR_WORKSPACE, PI_ERR_BUDGET, \
    PI_ERR_HIP = range(8)
PI_F32, PI_F16, PI_Q4_0 = 0, 1, 2
PI_RELU, PI_REGLU, PI_SQRELU = 0, 1, 2
PI_MAX_BATCH = 64
(PI_K_PRED_L1, PI_K_PRED_L2, PI_K_COMPACT, PI_K_UP, PI_K_DOWN, PI_K_MERGE, PI_K_PROFILE,
 PI_K_INDEX, PI_K_COPY, PI_K_REDUCE, PI_K_FFN, PI_K_ACCUMULATE, PI_K_STREAM, PI_K_UP_FINISH,
 PI_K_ROPE_APPEND, PI_K_ATTN, PI_K_ATTN_JOIN, PI_K_PAGES, PI_K_PAGE_COPY, PI_K_COUNT) = range(20)
PI_STREAM_SINK_WORDS = 2048
PI_SCRATCH_BYTES = 32 << 20
PI_MAX_HEAD_DIM, PI_MAX_PAGE_SIZE = 256, 1024
PI_ROPE_HALVES, PI_ROPE_PAIRS = 0, 1
PI_SCALE_NONE, PI_SCALE_LINEAR, PI_SCALE_BASE, PI_SCALE_BANDS = range(4)

# every symbol include/pi.h declares
EXPORTS = ("pi_workspace_bytes", "pi_workspace_init", "pi_predict", "pi_compact_active",
           "pi_sparse_ffn", "pi_sparse_ffn_split", "pi_sparse_ffn_split_noalloc",
           "pi_sparse_ffn_crossover", "pi_merge",
           "pi_dense_ffn",
           "pi_profile_counts", "pi_build_neuron_index", "pi_plan_hot_split",
           "pi_calibrate_workspace_bytes", "pi_calibrate_threshold", "pi_true_mask",
           "pi_host_sparse_ffn", "pi_hybrid_host_bytes", "pi_sparse_ffn_hybrid",
           "pi_accumulate_mask", "pi_permute_rows",
           "pi_copy", "pi_stream_read",
           "pi_rope_turns", "pi_rope_append", "pi_attention_workspace_bytes",
           "pi_paged_attention", "pi_pages_workspace_bytes", "pi_pages_extend", "pi_pages_fork",
           "pi_pages_free", "pi_pages_compact", "pi_pages_copy",
           "pi_kernel_timer_start", "pi_kernel_timer_stop", "pi_kernel_name", "pi_status_string",
           "pi_last_error")


class PiError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{msg} (status {status})")
        self.status = status


class HybridInfo(C.Structure):
    _fields_ = [("cold_count", C.c_int32), ("threads", C.c_int32), ("wait_us", C.c_double),
                ("host_us", C.c_double)]


class Predictor(C.Structure):
    _fields_ = [("d", C.c_int32), ("n", C.c_int32), ("r", C.c_int32), ("wdtype", C.c_int32),
                ("P1t", C.c_void_p), ("P2t", C.c_void_p), ("b2", C.c_void_p),
                ("threshold", C.c_float)]


class FfnPart(C.Structure):
    _fields_ = [("d", C.c_int32), ("rows", C.c_int32), ("wdtype", C.c_int32), ("act", C.c_int32),
                ("W_up", C.c_void_p), ("W_gate", C.c_void_p), ("b_up", C.c_void_p),
                ("b_gate", C.c_void_p), ("W_downT", C.c_void_p)]


class ActiveLists(C.Structure):
    _fields_ = [("n_hot", C.c_int32), ("hot_idx", C.c_void_p), ("cold_idx", C.c_void_p),
                ("counts", C.c_void_p)]


class KvCache(C.Structure):
    _fields_ = [("dtype", C.c_int32), ("layers", C.c_int32), ("pages", C.c_int32),
                ("kv_heads", C.c_int32), ("page_size", C.c_int32), ("head_dim", C.c_int32),
                ("k", C.c_void_p), ("v", C.c_void_p)]


class SeqBatch(C.Structure):
    _fields_ = [("n_seqs", C.c_int32), ("n_tokens", C.c_int32), ("max_new", C.c_int32),
                ("max_len", C.c_int32), ("q_start", C.c_void_p), ("kv_len", C.c_void_p),
                ("table", C.c_void_p), ("table_stride", C.c_int32)]


class Rows(C.Structure):
    _fields_ = [("data", C.c_void_p), ("token_stride", C.c_int64), ("head_stride", C.c_int64)]


class Rope(C.Structure):
    _fields_ = [("rotary_dim", C.c_int32), ("layout", C.c_int32), ("turns", C.c_void_p),
                ("magnitude", C.c_float)]


class ScoreRule(C.Structure):
    _fields_ = [("scale", C.c_float), ("cap", C.c_float), ("window", C.c_int32),
                ("slopes", C.c_void_p), ("prefix", C.c_void_p), ("first", C.c_void_p)]


class PageState(C.Structure):
    _fields_ = [("pages", C.c_int32), ("max_seqs", C.c_int32), ("table_stride", C.c_int32),
                ("page_size", C.c_int32), ("refs", C.c_void_p), ("table", C.c_void_p),
                ("lens", C.c_void_p)]


_lib = None


def lib() -> C.CDLL:
    """Load libpi.so (built by sparse_activation_ffn_amd.build); raise if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m sparse_activation_ffn_amd.build`")
    L = C.CDLL(LIB_PATH)
    P, I32, I64, SZ = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t
    sig = {
        "pi_workspace_bytes": ([I32, I32, I32, I32], SZ),
        "pi_workspace_init": ([P, SZ, P], I32),
        "pi_predict": ([P, P, I32, I32, P, P, P, P, SZ, P], I32),
        "pi_compact_active": ([P, I32, P, P], I32),
        "pi_sparse_ffn": ([P, P, I32, I32, P, P, P, P, SZ, P], I32),
        "pi_sparse_ffn_split": ([P, P, P, I32, I32, P, P, P, P, P, P, SZ, P], I32),
        "pi_sparse_ffn_split_noalloc": ([P, P, P, I32, I32, P, P, P, P, P, P], I32),
        "pi_sparse_ffn_crossover": ([P, P, P, I32, I32, P, P, I32, P, P, P, P, SZ, P], I32),
        "pi_merge": ([P, P, I32, I32, P, P], I32),
        "pi_dense_ffn": ([P, P, I32, I32, P, P, SZ, P], I32),
        "pi_profile_counts": ([P, P, I32, I32, P, P], I32),
        "pi_build_neuron_index": ([P, I32, I64, I64, P, P, P], I32),
        "pi_plan_hot_split": ([P, I32, I64, I64, C.c_double, C.c_double, P], I32),
        "pi_calibrate_workspace_bytes": ([I32, I32, I32, I32], SZ),
        "pi_calibrate_threshold": ([P, P, P, I32, I32, C.c_double, P, P, P, SZ, P], I32),
        "pi_true_mask": ([P, P, I32, I32, P, P], I32),
        "pi_host_sparse_ffn": ([P, P, I32, I32, P, I32, P, I32], I32),
        "pi_hybrid_host_bytes": ([I32, I32, I32], SZ),
        "pi_sparse_ffn_hybrid": ([P, P, P, I32, I32, P, P, P, P, P, SZ, P, SZ, I32, P, P], I32),
        "pi_accumulate_mask": ([P, I32, P, P], I32),
        "pi_permute_rows": ([P, P, P, I32, I64, P], I32),
        "pi_copy": ([P, P, I64, P], I32),
        "pi_stream_read": ([P, I64, P, P], I32),
        "pi_rope_turns": ([I32, C.c_double, I32, C.c_double, C.c_double, C.c_double, C.c_double, P],
                          I32),
        "pi_rope_append": ([P, I32, P, P, P, I32, P, P, P, P, P], I32),
        "pi_attention_workspace_bytes": ([P, P, I32], SZ),
        "pi_paged_attention": ([P, I32, P, P, I32, P, P, P, P, SZ, P], I32),
        "pi_pages_workspace_bytes": ([P, I32], SZ),
        "pi_pages_extend": ([P, P, P, P, I32, P, P, P, SZ, P], I32),
        "pi_pages_fork": ([P, P, P, I32, P, SZ, P], I32),
        "pi_pages_free": ([P, P, I32, P], I32),
        "pi_pages_compact": ([P, P, P, P, SZ, P], I32),
        "pi_pages_copy": ([P, P, P, I32, P], I32),
        "pi_kernel_timer_start": ([I32, I32], I32),
        "pi_kernel_timer_stop": ([I32, P, P], I32),
        "pi_kernel_name": ([I32], C.c_char_p),
        "pi_status_string": ([I32], C.c_char_p),
        "pi_last_error": ([], C.c_char_p),
    }
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    _lib = L
    return L


def _check(status: int):
    if status != PI_OK:
        L = lib()
        raise PiError(status, f"{L.pi_status_string(status).decode()}: "
                              f"{L.pi_last_error().decode()}")


def ptr(t) -> Optional[int]:
    """Device pointer of a tensor (or an int passed through, None stays None)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def stream_handle(stream=None) -> Optional[int]:
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


_dtypes: dict = {}


def dtype_code(t) -> int:
    code = _dtypes.get(t.dtype)
    if code is None:
        import torch
        _dtypes.update({torch.float32: PI_F32, torch.float16: PI_F16})
        code = _dtypes.get(t.dtype)
        if code is None:
            raise TypeError(f"no pi dtype for {t.dtype}")
    return code


# ---- the C entry points, same names -----------------------------------------

def pi_workspace_bytes(d: int, n: int, r: int, B: int) -> int:
    return int(lib().pi_workspace_bytes(d, n, r, B))


def pi_workspace_init(ws, stream=None):
    _check(lib().pi_workspace_init(ptr(ws), ws.numel() * ws.element_size(), stream_handle(stream)))


def pi_predict(pred: Predictor, x, mask, logits=None, lists: Optional[ActiveLists] = None,
               ws=None, stream=None):
    _check(lib().pi_predict(C.byref(pred), ptr(x), x.shape[0], dtype_code(x), ptr(mask),
                            ptr(logits), None if lists is None else C.byref(lists), ptr(ws),
                            0 if ws is None else ws.numel() * ws.element_size(),
                            stream_handle(stream)))


def pi_compact_active(mask, n: int, lists: ActiveLists, stream=None):
    _check(lib().pi_compact_active(ptr(mask), n, C.byref(lists), stream_handle(stream)))


def pi_sparse_ffn(part: FfnPart, x, idx, count, y, ws, stream=None):
    _check(lib().pi_sparse_ffn(C.byref(part), ptr(x), x.shape[0], dtype_code(x), ptr(idx),
                               ptr(count), ptr(y), ptr(ws), ws.numel() * ws.element_size(),
                               stream_handle(stream)))


def pi_sparse_ffn_split(hot: FfnPart, cold: Optional[FfnPart], x, lists: ActiveLists,
                        y_hot=None, y_cold=None, y=None, ws=None, stream=None, mask=None):
    """mask given: compaction fused, `lists` are outputs; mask None: `lists` are inputs."""
    _check(lib().pi_sparse_ffn_split(C.byref(hot), None if cold is None else C.byref(cold),
                                     ptr(x), x.shape[0], dtype_code(x), ptr(mask), C.byref(lists),
                                     ptr(y_hot), ptr(y_cold), ptr(y), ptr(ws),
                                     0 if ws is None else ws.numel() * ws.element_size(),
                                     stream_handle(stream)))


def pi_sparse_ffn_split_noalloc(hot: FfnPart, cold: Optional[FfnPart], x, lists: ActiveLists,
                                y_hot=None, y_cold=None, y=None, stream=None, mask=None):
    """pi_sparse_ffn_split with the library's static scratch instead of a workspace."""
    _check(lib().pi_sparse_ffn_split_noalloc(C.byref(hot), None if cold is None else C.byref(cold),
                                             ptr(x), x.shape[0], dtype_code(x), ptr(mask),
                                             C.byref(lists), ptr(y_hot), ptr(y_cold), ptr(y),
                                             stream_handle(stream)))


def pi_sparse_ffn_crossover(hot: FfnPart, cold: Optional[FfnPart], x, lists: ActiveLists,
                            dense_from: int, y_hot=None, y_cold=None, y=None, ws=None, stream=None,
                            mask=None):
    """pi_sparse_ffn_split, but every row is computed when the device active count
    reaches dense_from (the prompt-phase crossover)."""
    _check(lib().pi_sparse_ffn_crossover(C.byref(hot), None if cold is None else C.byref(cold),
                                         ptr(x), x.shape[0], dtype_code(x), ptr(mask),
                                         C.byref(lists), int(dense_from), ptr(y_hot), ptr(y_cold),
                                         ptr(y), ptr(ws),
                                         0 if ws is None else ws.numel() * ws.element_size(),
                                         stream_handle(stream)))


def pi_merge(y_hot, y_cold, y, stream=None):
    B, d = y_hot.shape
    _check(lib().pi_merge(ptr(y_hot), ptr(y_cold), B, d, ptr(y), stream_handle(stream)))


def pi_dense_ffn(part: FfnPart, x, y, ws, stream=None):
    _check(lib().pi_dense_ffn(C.byref(part), ptr(x), x.shape[0], dtype_code(x), ptr(y), ptr(ws),
                              ws.numel() * ws.element_size(), stream_handle(stream)))


def pi_profile_counts(part: FfnPart, X, counts, stream=None):
    _check(lib().pi_profile_counts(C.byref(part), ptr(X), X.shape[0], dtype_code(X), ptr(counts),
                                   stream_handle(stream)))


def pi_build_neuron_index(counts, budget_bytes: int, bytes_per_neuron: int, perm,
                          stream=None) -> int:
    n_hot = C.c_int32(0)
    _check(lib().pi_build_neuron_index(ptr(counts), counts.numel(), int(budget_bytes),
                                       int(bytes_per_neuron), ptr(perm), C.byref(n_hot),
                                       stream_handle(stream)))
    return int(n_hot.value)


def pi_plan_hot_split(counts_slot, budget_bytes: int, bytes_per_neuron: int, hbm_gbps: float,
                      link_gbps: float) -> int:
    """counts_slot: host array (numpy uint32) of activation counts in slot order."""
    import numpy as np
    c = np.ascontiguousarray(counts_slot, dtype=np.uint32)
    n_hot = C.c_int32(0)
    _check(lib().pi_plan_hot_split(c.ctypes.data if c.size else None, c.size, int(budget_bytes),
                                   int(bytes_per_neuron), float(hbm_gbps), float(link_gbps),
                                   C.byref(n_hot)))
    return int(n_hot.value)


def pi_calibrate_workspace_bytes(d: int, n: int, r: int, S: int) -> int:
    return int(lib().pi_calibrate_workspace_bytes(d, n, r, S))


def pi_calibrate_threshold(pred: Predictor, part: FfnPart, X, target_recall: float, tau, stats,
                           ws, stream=None):
    _check(lib().pi_calibrate_threshold(C.byref(pred), C.byref(part), ptr(X), X.shape[0],
                                        dtype_code(X), float(target_recall), ptr(tau), ptr(stats),
                                        ptr(ws), ws.numel() * ws.element_size(),
                                        stream_handle(stream)))


def pi_true_mask(part: FfnPart, x, mask, stream=None):
    _check(lib().pi_true_mask(C.byref(part), ptr(x), x.shape[0], dtype_code(x), ptr(mask),
                              stream_handle(stream)))


def pi_host_sparse_ffn(part: FfnPart, x, idx, count: int, y, threads: int = 0):
    """Every tensor here is a CPU tensor (host memory); runs on the host cores."""
    _check(lib().pi_host_sparse_ffn(C.byref(part), ptr(x), x.shape[0], dtype_code(x), ptr(idx),
                                    int(count), ptr(y), int(threads)))


def pi_hybrid_host_bytes(d: int, n: int, B: int) -> int:
    return lib().pi_hybrid_host_bytes(d, n, B)


def pi_sparse_ffn_hybrid(hot: FfnPart, cold: FfnPart, x, mask, lists: ActiveLists, y_cold, y, ws,
                         host_ws, threads: int = 0, stream=None) -> HybridInfo:
    """hot on the device, cold (host-memory weights) on the host cores; host_ws is a pinned
    CPU tensor of at least pi_hybrid_host_bytes bytes.  Returns the call's HybridInfo."""
    info = HybridInfo()
    _check(lib().pi_sparse_ffn_hybrid(C.byref(hot), C.byref(cold), ptr(x), x.shape[0],
                                      dtype_code(x), ptr(mask), C.byref(lists), ptr(y_cold),
                                      ptr(y), ptr(ws), ws.numel() * ws.element_size(),
                                      ptr(host_ws), host_ws.numel() * host_ws.element_size(),
                                      int(threads), C.byref(info), stream_handle(stream)))
    return info


def pi_accumulate_mask(mask, n: int, counts, stream=None):
    _check(lib().pi_accumulate_mask(ptr(mask), n, ptr(counts), stream_handle(stream)))


def pi_permute_rows(src, dst, perm, rows: int, row_bytes: int, stream=None):
    _check(lib().pi_permute_rows(ptr(src), ptr(dst), ptr(perm), rows, row_bytes,
                                 stream_handle(stream)))


def pi_copy(src, dst, nbytes: int, stream=None):
    _check(lib().pi_copy(ptr(src), ptr(dst), nbytes, stream_handle(stream)))


def pi_stream_read(src, nbytes: int, sink, stream=None):
    _check(lib().pi_stream_read(ptr(src), nbytes, ptr(sink), stream_handle(stream)))


# ---- paged key/value cache and the attention over it ----------------------------

def pi_rope_turns(rotary_dim: int, base: float = 10000.0, scaling: int = PI_SCALE_NONE,
                  factor: float = 1.0, low: float = 1.0, high: float = 4.0, context: float = 0.0):
    """Turns per position of each pair (float64 CPU tensor; copy it to the device for make_rope)."""
    import torch
    turns = torch.empty(max(rotary_dim // 2, 0), dtype=torch.float64)
    _check(lib().pi_rope_turns(rotary_dim, base, scaling, factor, low, high, context,
                               turns.data_ptr() or None))
    return turns


def pi_rope_append(cache: KvCache, layer: int, batch: SeqBatch, rope: Rope, q, q_out, k, v,
                   positions=None, stream=None):
    """q, q_out [tokens][q_heads][head_dim] (both None: keys and values only), k and v
    [tokens][kv_heads][head_dim]; the elements of a head contiguous, other strides free."""
    hq = 0 if q is None else q.shape[1]
    hk, dt, d, n = cache.kv_heads, cache.dtype, cache.head_dim, batch.n_tokens
    _vector("positions", positions, "int32", n)
    _check(lib().pi_rope_append(
        C.byref(cache), layer, C.byref(batch), C.byref(rope), ptr(positions), hq,
        None if q is None else _rows(q, dt, d, n, hq),
        None if q_out is None else _rows(q_out, dt, d, n, hq),
        _rows(k, dt, d, n, hk), _rows(v, dt, d, n, hk), stream_handle(stream)))


def pi_attention_workspace_bytes(cache: KvCache, batch: SeqBatch, q_heads: int) -> int:
    return int(lib().pi_attention_workspace_bytes(C.byref(cache), C.byref(batch), q_heads))


def pi_paged_attention(cache: KvCache, layer: int, batch: SeqBatch, rule: ScoreRule, q, out,
                       lse=None, ws=None, stream=None):
    """q and out [tokens][q_heads][head_dim], lse [tokens][q_heads] float32 or None."""
    hq, dt, d, n = q.shape[1], cache.dtype, cache.head_dim, batch.n_tokens
    _vector("lse", lse, "float32", n * hq)
    for (name, have), need in zip(getattr(rule, "_sizes", ()), (hq, batch.n_seqs, n)):
        if have is not None and have < need:
            raise ValueError(f"{name} must have at least {need} elements, has {have}")
    _check(lib().pi_paged_attention(
        C.byref(cache), layer, C.byref(batch), C.byref(rule), hq, _rows(q, dt, d, n, hq),
        _rows(out, dt, d, n, hq), ptr(lse), ptr(ws),
        0 if ws is None else ws.numel() * ws.element_size(), stream_handle(stream)))


def pi_pages_workspace_bytes(state: PageState, n: int) -> int:
    return int(lib().pi_pages_workspace_bytes(C.byref(state), n))


def pi_pages_extend(state: PageState, cache: Optional[KvCache], seqs, add, granted, copies, ws,
                    stream=None):
    """seqs, add, granted: int32 [n]; copies: int32 [2][n]."""
    n = seqs.numel()
    for name, t, size in (("seqs", seqs, n), ("add", add, n), ("granted", granted, n), ("copies", copies, 2 * n)):
        _vector(name, t, "int32", size)
    _check(lib().pi_pages_extend(C.byref(state), None if cache is None else C.byref(cache),
                                 ptr(seqs), ptr(add), n, ptr(granted), ptr(copies),
                                 ptr(ws), ws.numel() * ws.element_size(), stream_handle(stream)))


def pi_pages_fork(state: PageState, src, dst, ws, stream=None):
    _vector("src", src, "int32", 0)
    _vector("dst", dst, "int32", src.numel())
    _check(lib().pi_pages_fork(C.byref(state), ptr(src), ptr(dst), src.numel(), ptr(ws),
                               ws.numel() * ws.element_size(), stream_handle(stream)))


def pi_pages_free(state: PageState, seqs, stream=None):
    _vector("seqs", seqs, "int32", 0)
    _check(lib().pi_pages_free(C.byref(state), ptr(seqs), seqs.numel(), stream_handle(stream)))


def pi_pages_compact(state: PageState, cache: Optional[KvCache], moved, ws, stream=None):
    _vector("moved", moved, "int32", state.pages)
    _check(lib().pi_pages_compact(C.byref(state), None if cache is None else C.byref(cache),
                                  ptr(moved), ptr(ws), ws.numel() * ws.element_size(),
                                  stream_handle(stream)))


def pi_pages_copy(cache: KvCache, src, dst, stream=None):
    _vector("src", src, "int32", 0)
    _vector("dst", dst, "int32", src.numel())
    _check(lib().pi_pages_copy(C.byref(cache), ptr(src), ptr(dst), src.numel(),
                               stream_handle(stream)))


def pi_kernel_timer_start(kid: int, max_launches: int):
    _check(lib().pi_kernel_timer_start(kid, max_launches))


def pi_kernel_timer_stop(kid: int):
    ms, k = C.c_float(0.0), C.c_int32(0)
    _check(lib().pi_kernel_timer_stop(kid, C.byref(ms), C.byref(k)))
    return float(ms.value), int(k.value)


def pi_kernel_name(kid: int) -> str:
    return lib().pi_kernel_name(kid).decode()


# ---- descriptors from device tensors ------------------------------------------

def make_predictor(P1t, P2t, b2, threshold: float = 0.0) -> Predictor:
    r, d = P1t.shape
    n = P2t.shape[0]
    p = Predictor(d, n, r, dtype_code(P1t), ptr(P1t), ptr(P2t), ptr(b2), float(threshold))
    p._keep = (P1t, P2t, b2)
    return p


def make_part(d: int, W_up, W_downT, act: int = PI_RELU, W_gate=None, b_up=None, b_gate=None,
              q4: bool = False) -> FfnPart:
    rows = W_up.shape[0]
    wdtype = PI_Q4_0 if q4 else dtype_code(W_up)
    p = FfnPart(d, rows, wdtype, act, ptr(W_up), ptr(W_gate), ptr(b_up), ptr(b_gate),
                ptr(W_downT))
    p._keep = (W_up, W_gate, b_up, b_gate, W_downT)
    return p


def make_lists(n_hot: int, hot_idx, cold_idx, counts) -> ActiveLists:
    L = ActiveLists(n_hot, ptr(hot_idx), ptr(cold_idx), ptr(counts))
    L._keep = (hot_idx, cold_idx, counts)
    return L


def make_kv_cache(k, v) -> KvCache:
    """k and v: [layers][pages][kv_heads][page_size][head_dim] device tensors."""
    if k.shape != v.shape or k.dtype != v.dtype or not (k.is_contiguous() and v.is_contiguous()):
        raise ValueError("k and v must be contiguous and alike in shape and dtype")
    layers, pages, heads, page_size, head_dim = k.shape
    c = KvCache(dtype_code(k), layers, pages, heads, page_size, head_dim, ptr(k), ptr(v))
    c._keep = (k, v)
    return c


def make_seq_batch(q_start, kv_len, table, n_tokens: int, max_new: int, max_len: int) -> SeqBatch:
    """q_start int32 [n_seqs + 1], kv_len int32 [n_seqs], table int32 [n_seqs][table_stride]."""
    n = kv_len.numel()
    _int32("q_start", q_start, (n + 1,))
    _int32("kv_len", kv_len, (n,))
    _int32("table", table, (n, table.shape[-1]))
    b = SeqBatch(n, n_tokens, max_new, max_len, ptr(q_start), ptr(kv_len), ptr(table),
                 table.shape[-1])
    b._keep = (q_start, kv_len, table)
    return b


def make_score_rule(scale: float, cap: float = 0.0, slopes=None, window: int = 0, prefix=None,
                    first=None) -> ScoreRule:
    """slopes float32 [q_heads], prefix int32 [n_seqs], first int32 [n_tokens] (device) or None."""
    _vector("slopes", slopes, "float32", 0)
    _vector("prefix", prefix, "int32", 0)
    _vector("first", first, "int32", 0)
    r = ScoreRule(float(scale), float(cap), int(window), ptr(slopes), ptr(prefix), ptr(first))
    r._keep = (slopes, prefix, first)
    # how many there are is compared where the batch is known
    r._sizes = [(name, t.numel() if hasattr(t, "numel") else None)
                for name, t in (("slopes", slopes), ("prefix", prefix), ("first", first))]
    return r


def make_rope(turns, pairs: bool = False, magnitude: float = 1.0) -> Rope:
    """turns: float64 device tensor [rotary_dim / 2] (pi_rope_turns)."""
    _vector("turns", turns, "float64", 0)
    r = Rope(2 * turns.numel(), PI_ROPE_PAIRS if pairs else PI_ROPE_HALVES, ptr(turns) or None,
             float(magnitude))
    r._keep = turns
    return r


def make_page_state(refs, table, lens, page_size: int) -> PageState:
    """refs int32 [pages], table int32 [max_seqs][table_stride], lens int32 [max_seqs]."""
    n = lens.numel()
    _int32("refs", refs, (refs.numel(),))
    _int32("table", table, (n, table.shape[-1]))
    _int32("lens", lens, (n,))
    s = PageState(refs.numel(), n, table.shape[-1], page_size, ptr(refs), ptr(table), ptr(lens))
    s._keep = (refs, table, lens)
    return s


def _int32(name: str, t, shape):
    if str(t.dtype) != "torch.int32" or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {tuple(shape)}")


_torch_dtypes: dict = {}


def _vector(name: str, t, dtype: str, n: int):
    """Refuses a tensor (None and addresses pass) that does not hold n elements of dtype one after the other."""
    if t is None or isinstance(t, int):
        return
    if t.dtype is _torch_dtypes.get(dtype) and t.numel() >= n and t.is_contiguous():
        return
    if not _torch_dtypes:
        import torch
        _torch_dtypes.update(int32=torch.int32, float32=torch.float32, float64=torch.float64)
        return _vector(name, t, dtype, n)
    raise ValueError(f"{name} must be a contiguous {dtype} tensor of at least {n} elements, "
                     f"got {tuple(t.shape)} of {t.dtype}")


def _rows(t, dtype: int, head_dim: int, n_tokens: int, heads: int):
    """Reference to [tokens][heads][head_dim] as the library sees it; checked here, where the
    shape is known."""
    shape, strides = t.shape, t.stride()
    if len(shape) != 3 or shape[0] < n_tokens or shape[1] != heads or shape[2] != head_dim or \
            strides[2] != 1:
        raise ValueError(f"need [{n_tokens}][{heads}][{head_dim}] with contiguous heads, "
                         f"got {tuple(shape)} with strides {strides}")
    if dtype_code(t) != dtype:
        raise TypeError("q, k, v and the output have the cache's dtype")
    return C.byref(Rows(t.data_ptr(), strides[0], strides[1]))


def row_slice(t, lo: int, hi: int):
    """Rows [lo, hi) of a per-neuron device tensor (a view, no copy)."""
    return None if t is None else t[lo:hi]
