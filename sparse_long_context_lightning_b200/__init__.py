"""Token-level sparse attention for one long-context layer on B200 (sm_100a).

Python binding of ``liblsa.so`` (C ABI declared in ``include/lsa.h``).  The functions below only
marshal arguments (device pointers, sizes, the current CUDA stream) into the C calls: every step of
the path runs in the library's CUDA kernels.  Importing this package does not load the library;
the first call does, and raises ``LsaError`` if the built library is missing.
"""

from __future__ import annotations

import ctypes
import os
import struct

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "liblsa.so")

LSA_OK = 0
LSA_BF16 = 0
LSA_FP8_E4M3 = 1
LSA_OP_TOPK, LSA_OP_BUCKET, LSA_OP_ATTN, LSA_OP_REFINE, LSA_OP_BUCKET_MIN, LSA_OP_HYBRID_ATTN = 1, 2, 3, 4, 5, 6

_bf16, _f32, _f64, _i64, _i32 = torch.bfloat16, torch.float32, torch.float64, torch.int64, torch.int32
_NORMS = {"none": 0, "rms": 1, "layer": 2}
_LAYOUTS = {"interleaved": 0, "half": 1}
_SCALINGS = {"none": 0, "linear": 1, "yarn": 2}

_STATUS = {0: "LSA_OK", -1: "LSA_ERR_INVALID_ARG", -2: "LSA_ERR_UNSUPPORTED", -3: "LSA_ERR_WORKSPACE",
           -4: "LSA_ERR_CUDA", -5: "LSA_ERR_DEVICE_CHECK", -6: "LSA_ERR_TIMEOUT"}

# exported symbol -> (restype, argtypes)
_P, _I64, _I32, _F32, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
SIGNATURES = {
    "lsa_index_score": (_I32, [_P, _P, _P, _P, _P, _I32, _I64, _I32, _I32, _I64, _P, _P, _I64, _P]),
    "lsa_topk_select": (_I32, [_P, _I64, _I64, _I64, _I32, _I32, _I32, _P, _P, _I64, _P, _P]),
    "lsa_topk_refine": (_I32, [_P, _P, _P, _I64, _I32, _I32, _I64, _P, _I64, _P, _I32, _I32, _I32, _P, _P, _I64, _P,
                               _P, _SZ, _P]),
    "lsa_pool_keys": (_I32, [_P, _I32, _P, _I64, _I32, _P, _I32, _I64, _P, _P]),
    "lsa_bucket_select": (_I32, [_P, _P, _P, _I32, _I64, _I32, _I32, _P, _I64, _P, _I32, _I32, _I32, _I32, _I64,
                                 _P, _P, _I64, _P, _P, _SZ, _P]),
    "lsa_bucket_select_noalloc": (_I32, [_P, _P, _P, _I32, _I64, _I32, _I32, _P, _I64, _P, _I32, _I32, _I32, _I32,
                                         _I64, _P, _P, _I64, _P, _P]),
    "lsa_split_representatives": (_I32, [_P, _I64, _I32, _P, _P]),
    "lsa_bucket_select_split": (_I32, [_P, _P, _I64, _I32, _I32, _P, _I64, _P, _I32, _I32, _I32, _I32, _I64, _P, _P,
                                       _I64, _P, _P, _SZ, _P]),
    "lsa_hi_select": (_I32, [_P, _P, _P, _I64, _I32, _I32, _I64, _P, _I32, _I32, _I32, _I32, _I32, _I32, _P, _P, _I64,
                             _P, _P, _SZ, _P]),
    "lsa_hi_workspace_size": (_SZ, [_I64, _I64, _I32, _I32, _I32, _I32, _I32, _I32]),
    "lsa_hybrid_attn": (_I32, [_P, _P, _I64, _P, _I64, _P, _I64, _I32, _I32, _I32, _I32, _I32, _P, _F32, _P, _P, _P,
                               _SZ, _P]),
    "lsa_tree_parents": (_I32, [_P, _I64, _I32, _I32, _P, _P]),
    "lsa_tree_workspace_size": (_SZ, [_I64, _I64, _I32, _I32, _I32]),
    "lsa_tree_select": (_I32, [_P, _P, _I64, _I32, _I32, _P, _I64, _P, _I64, _I32, _P, _I32, _I32, _I32, _I32, _I32,
                               _I64, _P, _P, _I64, _P, _P, _SZ, _P]),
    "lsa_tree_select_split": (_I32, [_P, _P, _I64, _I32, _I32, _P, _I64, _P, _I64, _I32, _P, _I32, _I32, _I32, _I32,
                                     _I32, _I64, _P, _P, _I64, _P, _P, _SZ, _P]),
    "lsa_msa_select": (_I32, [_P, _P, _P, _I64, _I32, _I32, _I64, _I32, _I32, _P, _P, _P, _I64, _P, _P, _SZ, _P]),
    "lsa_msa_workspace_size": (_SZ, [_I64, _I64, _I32, _I32]),
    "lsa_msa_attn_workspace_size": (_SZ, [_I64, _I64, _I32]),
    "lsa_msa_attn": (_I32, [_P, _P, _I64, _P, _P, _I64, _P, _I64, _I32, _I32, _I32, _I32, _F32, _P, _P, _P, _SZ, _P]),
    "lsa_sparse_attn": (_I32, [_P, _P, _I64, _P, _I64, _P, _I64, _I32, _I32, _I32, _F32, _P, _P, _P, _SZ, _P]),
    "lsa_rope_freqs": (_I32, [_I32, ctypes.c_double, _I32, ctypes.c_double, _I64, ctypes.c_double, ctypes.c_double, _P,
                              _P]),
    "lsa_norm_rope": (_I32, [_P, _I64, _I64, _I64, _I32, _I32, _I32, _P, _P, _F32, _P, _I32, _I32, _I32, _F32, _P, _P,
                             _I64, _I64, _I32, _P, _P]),
    "lsa_cache_append": (_I32, [_P, _I64, _I64, _I32, _I32, _P, _F32, _P, _I32, _F32, _P, _P, _P, _I64, _P, _I64, _I32,
                                _I32, _P, _P, _F32, _I32, _I32, _P, _I32, _P, _P]),
    "lsa_prefix_attn": (_I32, [_P, _I64, _I32, _I32, _I32, _P, _I64, _P, _I64, _I32, _P, _I64, _P, _F32, _P, _P, _P,
                               _SZ, _P]),
    "lsa_prefix_attn_workspace_size": (_SZ, [_I64, _I32]),
    "lsa_norm_rope_packed": (_I32, [ctypes.c_char_p]),
    "lsa_cache_append_packed": (_I32, [ctypes.c_char_p]),
    "lsa_prefix_attn_packed": (_I32, [ctypes.c_char_p]),
    "lsa_workspace_size": (_SZ, [_I32, _I64, _I64, _I32, _I32, _I32, _I32]),
    "lsa_device_status": (_I32, [_P]),
    "lsa_selftest_wait": (_I32, [ctypes.c_uint64, _P]),
    "lsa_strerror": (ctypes.c_char_p, [_I32]),
    "lsa_last_error": (ctypes.c_char_p, []),
    "lsa_version": (ctypes.c_char_p, []),
}


class LsaError(RuntimeError):
    def __init__(self, fn: str, status: int, detail: str = ""):
        super().__init__(f"{fn} failed: {_STATUS.get(status, status)} {detail}".strip())
        self.status = status


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load liblsa.so (once).  Raises LsaError when it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise LsaError("load_library", -4, f"{path} is missing: run `python -m sparse_long_context_lightning_b200.build`")
        lib = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(lib, name)
            f.restype = res
            f.argtypes = args
        _lib = lib
    return _lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(fn: str, st: int):
    if st != LSA_OK:
        lib = load_library()
        raise LsaError(fn, st, lib.lsa_last_error().decode() if st in (-4, -5, -6) else "")


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return LSA_BF16
    if t.dtype in (torch.uint8, torch.float8_e4m3fn):
        return LSA_FP8_E4M3
    raise LsaError("dtype", -2, f"index tensors must be bf16 or e4m3 codes, got {t.dtype}")


def lsa_workspace_size(op: int, B: int, L: int, K: int, H: int = 0, sink: int = 0, window: int = 0) -> int:
    return int(load_library().lsa_workspace_size(op, B, L, K, H, sink, window))


def lsa_index_score(q_idx, w, k_idx, q_pos, scores, q_scale=None, k_scale=None, stream=None):
    """scores[b, s] = sum_j w[b,j] ReLU(q_idx[b,j] . k_idx[s]) (s <= q_pos[b]), else -inf."""
    B, H_I, d_I = q_idx.shape
    L = k_idx.shape[0]
    st = load_library().lsa_index_score(_ptr(q_idx), _ptr(q_scale), _ptr(w), _ptr(k_idx), _ptr(k_scale),
                                        _dtype_code(q_idx), B, H_I, d_I, L, _ptr(q_pos), _ptr(scores),
                                        scores.stride(0), _stream(stream))
    _check("lsa_index_score", st)


def lsa_topk_select(scores, L, K, sink, window, q_pos, idx, count, stream=None):
    """Top-K of each score row over [0, q_pos] minus sink/window, unioned with sink and window."""
    st = load_library().lsa_topk_select(_ptr(scores), scores.stride(0), scores.shape[0], L, K, sink, window,
                                        _ptr(q_pos), _ptr(idx), idx.stride(0), _ptr(count), _stream(stream))
    _check("lsa_topk_select", st)


def lsa_topk_refine(q_idx, w, k_idx, cand, cand_count, K, sink, window, q_pos, idx, count, ws, stream=None):
    """Re-rank the dynamic candidates of `cand` (a K' top-K row) with bf16 scores; keep the top K."""
    B, H_I, d_I = q_idx.shape
    st = load_library().lsa_topk_refine(_ptr(q_idx), _ptr(w), _ptr(k_idx), B, H_I, d_I, k_idx.shape[0], _ptr(cand),
                                        cand.stride(0), _ptr(cand_count), K, sink, window, _ptr(q_pos), _ptr(idx),
                                        idx.stride(0), _ptr(count), _ptr(ws),
                                        0 if ws is None else ws.numel() * ws.element_size(), _stream(stream))
    _check("lsa_topk_refine", st)


def lsa_pool_keys(k_idx, centroids, bsz, members=None, k_scale=None, stream=None):
    """centroids[c] = mean of the bsz member index keys (explicit members, or contiguous blocks)."""
    L, d_I = k_idx.shape
    st = load_library().lsa_pool_keys(_ptr(k_idx), _dtype_code(k_idx), _ptr(k_scale), L, d_I, _ptr(members), bsz,
                                      centroids.shape[0], _ptr(centroids), _stream(stream))
    _check("lsa_pool_keys", st)


def lsa_bucket_select(q_idx, w, centroids, members, bsz, M, sink, window, L, q_pos, idx, count, ws, stream=None):
    """Flat buckets (members given) or micro-blocks (members None): top-M representatives, expanded."""
    B, H_I, d_I = q_idx.shape
    st = load_library().lsa_bucket_select(_ptr(q_idx), None, _ptr(w), _dtype_code(q_idx), B, H_I, d_I,
                                          _ptr(centroids), centroids.shape[0], _ptr(members), bsz, M, sink, window,
                                          L, _ptr(q_pos), _ptr(idx), idx.stride(0), _ptr(count), _ptr(ws),
                                          0 if ws is None else ws.numel() * ws.element_size(), _stream(stream))
    _check("lsa_bucket_select", st)


def lsa_split_representatives(centroids, split, stream=None):
    """split[p] (bf16 [3, NB, d_I]): centroids == split[0] + split[1] + split[2] exactly."""
    NB, d_I = centroids.shape
    st = load_library().lsa_split_representatives(_ptr(centroids), NB, d_I, _ptr(split), _stream(stream))
    _check("lsa_split_representatives", st)


def lsa_bucket_select_split(q_idx, w, split, members, bsz, M, sink, window, L, q_pos, idx, count, ws, stream=None):
    """lsa_bucket_select from the representatives' cached bf16 split (lsa_split_representatives)."""
    B, H_I, d_I = q_idx.shape
    st = load_library().lsa_bucket_select_split(_ptr(q_idx), _ptr(w), B, H_I, d_I, _ptr(split), split.shape[1],
                                                _ptr(members), bsz, M, sink, window, L, _ptr(q_pos), _ptr(idx),
                                                idx.stride(0), _ptr(count), _ptr(ws),
                                                0 if ws is None else ws.numel() * ws.element_size(), _stream(stream))
    _check("lsa_bucket_select_split", st)


def lsa_device_status(stream=None):
    """Synchronise the stream and raise if a kernel gave up a bounded wait (LSA_ERR_TIMEOUT) or failed a
    device-side index check (LSA_ERR_DEVICE_CHECK) since the last check."""
    _check("lsa_device_status", load_library().lsa_device_status(_stream(stream)))


def lsa_selftest_wait(limit_ns, stream=None):
    """Launch a kernel whose bounded wait on an mbarrier nothing completes runs out after limit_ns."""
    _check("lsa_selftest_wait", load_library().lsa_selftest_wait(int(limit_ns), _stream(stream)))


def lsa_tree_parents(centroids, F, parents, stream=None):
    """Level-2 centres of the tree search: parent p = mean of the centres of buckets [pF, min((p+1)F, NB))."""
    NB, d_I = centroids.shape
    st = load_library().lsa_tree_parents(_ptr(centroids), NB, d_I, F, _ptr(parents), _stream(stream))
    _check("lsa_tree_parents", st)


def lsa_tree_workspace_size(B, NP, F, M2, M):
    return load_library().lsa_tree_workspace_size(B, NP, F, M2, M)


def lsa_tree_select(q_idx, w, centroids, parents, F, members, M2, M, sink, window, L, q_pos, idx, count, ws,
                    stream=None):
    """Two-level tree search: top-M2 parents, then the top-M of their children, expanded as Flat buckets."""
    B, H_I, d_I = q_idx.shape
    NB, bsz = members.shape
    st = load_library().lsa_tree_select(_ptr(q_idx), _ptr(w), B, H_I, d_I, _ptr(centroids), NB, _ptr(parents),
                                        parents.shape[0], F, _ptr(members), bsz, M2, M, sink, window, L,
                                        _ptr(q_pos), _ptr(idx), idx.stride(0), _ptr(count), _ptr(ws),
                                        0 if ws is None else ws.numel() * ws.element_size(), _stream(stream))
    _check("lsa_tree_select", st)


def lsa_tree_select_split(q_idx, w, split, parents, F, members, M2, M, sink, window, L, q_pos, idx, count, ws,
                          stream=None):
    """lsa_tree_select with the children scored on the tensor cores from the centres' cached bf16 split."""
    B, H_I, d_I = q_idx.shape
    NB, bsz = members.shape
    st = load_library().lsa_tree_select_split(_ptr(q_idx), _ptr(w), B, H_I, d_I, _ptr(split), NB, _ptr(parents),
                                              parents.shape[0], F, _ptr(members), bsz, M2, M, sink, window, L,
                                              _ptr(q_pos), _ptr(idx), idx.stride(0), _ptr(count), _ptr(ws),
                                              0 if ws is None else ws.numel() * ws.element_size(), _stream(stream))
    _check("lsa_tree_select_split", st)


def lsa_hi_workspace_size(B, L, P, Bsub, M, K, sink, window):
    return load_library().lsa_hi_workspace_size(B, L, P, Bsub, M, K, sink, window)


def lsa_hi_select(q_idx, w, k_idx, sub_split, P, Bsub, M, K, sink, window, q_pos, idx, count, ws, stream=None):
    """Two-stage selection: top-M pages from the sub-block means' split, then token top-K on their tokens."""
    B, H_I, d_I = q_idx.shape
    L = k_idx.shape[0]
    st = load_library().lsa_hi_select(_ptr(q_idx), _ptr(w), _ptr(k_idx), B, H_I, d_I, L, _ptr(sub_split), P, Bsub, M,
                                      K, sink, window, _ptr(q_pos), _ptr(idx), idx.stride(0), _ptr(count), _ptr(ws),
                                      0 if ws is None else ws.numel() * ws.element_size(), _stream(stream))
    _check("lsa_hi_select", st)


def lsa_bucket_select_noalloc(q_idx, w, centroids, members, bsz, M, sink, window, L, q_pos, idx, count,
                              stream=None):
    """lsa_bucket_select with the library's static 8 MiB scratch (for callers that cannot allocate)."""
    B, H_I, d_I = q_idx.shape
    st = load_library().lsa_bucket_select_noalloc(_ptr(q_idx), None, _ptr(w), _dtype_code(q_idx), B, H_I, d_I,
                                                  _ptr(centroids), centroids.shape[0], _ptr(members), bsz, M, sink,
                                                  window, L, _ptr(q_pos), _ptr(idx), idx.stride(0), _ptr(count),
                                                  _stream(stream))
    _check("lsa_bucket_select_noalloc", st)


def lsa_sparse_attn(q, kv, idx, count, scale, out, lse=None, ws=None, stream=None):
    """out[b,h] = softmax_{s in S_b}(scale q[b,h].kv[s]) kv[s,:512] over the selected latent rows."""
    B, H, d_qk = q.shape
    d_v = out.shape[-1]
    st = load_library().lsa_sparse_attn(_ptr(q), _ptr(kv), kv.shape[0], _ptr(idx), idx.stride(0), _ptr(count), B, H,
                                        d_qk, d_v, float(scale), _ptr(out), _ptr(lse), _ptr(ws),
                                        0 if ws is None else ws.numel() * ws.element_size(), _stream(stream))
    _check("lsa_sparse_attn", st)


def lsa_hybrid_attn(q, kv, idx, count, sink, window, q_pos, scale, out, lse=None, ws=None, stream=None):
    """lsa_sparse_attn over sink | sparse | window rows, the fixed part on a second stream, merged by LSE."""
    B, H, d_qk = q.shape
    d_v = out.shape[-1]
    st = load_library().lsa_hybrid_attn(_ptr(q), _ptr(kv), kv.shape[0], _ptr(idx), idx.stride(0), _ptr(count), B, H,
                                        d_qk, d_v, sink, window, _ptr(q_pos), float(scale), _ptr(out), _ptr(lse),
                                        _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                        _stream(stream))
    _check("lsa_hybrid_attn", st)


def lsa_msa_workspace_size(B, L, G, KB):
    return load_library().lsa_msa_workspace_size(B, L, G, KB)


def lsa_msa_select(q_idx, w, k_idx, G, KB, q_pos, idx, gmask, count, ws, stream=None):
    """Group-wise block selection: per group of index heads, top-KB 128-token blocks by max-pooled score."""
    B, H_I, d_I = q_idx.shape
    st = load_library().lsa_msa_select(_ptr(q_idx), _ptr(w), _ptr(k_idx), B, H_I, d_I, k_idx.shape[0], G, KB,
                                       _ptr(q_pos), _ptr(idx), _ptr(gmask), idx.stride(0), _ptr(count), _ptr(ws),
                                       0 if ws is None else ws.numel() * ws.element_size(), _stream(stream))
    _check("lsa_msa_select", st)


def lsa_msa_attn_workspace_size(B, idx_ld, G):
    return load_library().lsa_msa_attn_workspace_size(B, idx_ld, G)


def lsa_msa_attn(q, kv, idx, gmask, count, G, scale, out, lse=None, ws=None, stream=None):
    """Attention over a group-wise selection: head h attends to the rows its group kept."""
    B, H, d_qk = q.shape
    d_v = out.shape[-1]
    st = load_library().lsa_msa_attn(_ptr(q), _ptr(kv), kv.shape[0], _ptr(idx), _ptr(gmask), idx.stride(0),
                                     _ptr(count), B, H, d_qk, d_v, G, float(scale), _ptr(out), _ptr(lse), _ptr(ws),
                                     0 if ws is None else ws.numel() * ws.element_size(), _stream(stream))
    _check("lsa_msa_attn", st)


# The calls below take a few microseconds on the GPU in a decode step, so they are written to cost little: one test a
# tensor, messages formed on failure only, the stream asked for as a number (a Stream object costs 3 us), the arguments
# packed into the C struct of the *_packed forms (22 converted arguments cost 2.8 us, the struct 0.6).
# (0Q: a C struct is padded to its widest field.)
_NORM_ROPE = struct.Struct("@QQqqqQQQQQqqQQ7i2f0Q")
_CACHE_APPEND = struct.Struct("@QQqqQQQQQqQqQQQQQ8i3f0Q")
_PREFIX_ATTN = struct.Struct("@QQqQqQqQqQQQQQQ4if0Q")


def _bad(fn: str, what: str):
    raise LsaError(fn, -1, what)


def _refuse(fn: str, name: str, t, dtype, shape, dev: int):
    _bad(fn, f"{name}: contiguous {dtype} {tuple(shape)} on cuda:{dev} wanted, got {t.dtype} {tuple(t.shape)} on {t.device}")


def _ten(fn: str, name: str, t, dtype, shape, dev: int):
    """Address of a contiguous tensor of this dtype and shape on GPU `dev`."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    _refuse(fn, name, t, dtype, shape, dev)


def _vec(fn: str, name: str, t, dtype, n: int, dev: int):
    """Address of n contiguous elements, or 0 for None."""
    if t is None:
        return 0
    if t.dtype is dtype and t.numel() == n and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    _refuse(fn, name, t, dtype, (n,), dev)


def _code(fn: str, name: str, table: dict, key) -> int:
    c = table.get(key)
    if c is None:
        _bad(fn, f"{name} must be one of {', '.join(table)}, got {key!r}")
    return c


_get_device = getattr(torch._C, "_cuda_getDevice", None)
_get_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _off_device(dev: int) -> bool:
    """Whether the call has to make the tensors' GPU the current one first."""
    return dev != _get_device()


def lsa_rope_freqs(R, base=10000.0, scaling="none", factor=1.0, original_len=4096, beta_fast=32.0, beta_slow=1.0,
                   device="cuda"):
    """Angular frequencies of the position rotation (fp64 [R / 2] on `device`) and the factor of cos and sin."""
    freqs, mul = torch.empty(max(int(R) // 2, 1), dtype=torch.float64), ctypes.c_float(0.0)
    st = load_library().lsa_rope_freqs(int(R), float(base), _code("lsa_rope_freqs", "scaling", _SCALINGS, scaling),
                                       float(factor), int(original_len), float(beta_fast), float(beta_slow),
                                       freqs.data_ptr(), ctypes.byref(mul))
    _check("lsa_rope_freqs", st)
    return freqs.to(device), mul.value


def lsa_norm_rope(x, y, pos=None, freqs=None, norm="none", weight=None, bias=None, eps=1e-6, rope_off=0,
                  layout="interleaved", mul=1.0, y_scale=None, stream=None):
    """y[t, h] = norm of x[t, h] with dims [rope_off, rope_off + 2 len(freqs)) rotated by pos[t]; x bf16 [T, H, D] with
    any token and head strides, y bf16 (it may be x) or, with y_scale [T, H], e4m3 codes."""
    fn = "lsa_norm_rope"
    if x.dim() != 3 or not x.is_cuda or x.dtype is not _bf16:
        _bad(fn, "x: bf16 [T, H, D] on a GPU wanted")
    dev = x.get_device()
    if _off_device(dev):
        with torch.cuda.device(x.device):
            return lsa_norm_rope(x, y, pos, freqs, norm, weight, bias, eps, rope_off, layout, mul, y_scale, stream)
    T, H, D = shape = x.shape
    if y.shape != shape or y.get_device() != dev:
        _bad(fn, "y: the shape and device of x wanted")
    (xt, xh, xd), (yt, yh, yd) = x.stride(), y.stride()
    if (xd != 1 or yd != 1) and D != 1:
        _bad(fn, "x, y: the last axis must be contiguous")
    if T == 1:  # an axis of length one has no stride that matters
        xt = yt = 0
    elif yt == 0:
        _bad(fn, "y: a broadcast output")
    if H == 1:
        xh = yh = 0
    elif yh == 0:
        _bad(fn, "y: a broadcast output")
    R = 0
    if freqs is not None:
        if pos is None or freqs.dim() != 1:
            _bad(fn, "freqs [rotary dims / 2] and pos belong together")
        R = 2 * freqs.shape[0]
    elif pos is not None:
        _bad(fn, "pos without freqs")
    st = (_lib or load_library()).lsa_norm_rope_packed(_NORM_ROPE.pack(
        _NORM_ROPE.size, x.data_ptr(), xt, xh, T, _vec(fn, "weight", weight, _f32, D, dev),
        _vec(fn, "bias", bias, _f32, D, dev), _vec(fn, "freqs", freqs, _f64, R // 2, dev),
        _vec(fn, "pos", pos, _i64, T, dev), y.data_ptr(), yt, yh,
        0 if y_scale is None else _ten(fn, "y_scale", y_scale, _f32, (T, H), dev),
        _get_stream(dev) if stream is None else stream.cuda_stream, H, D, _code(fn, "norm", _NORMS, norm), rope_off, R,
        _code(fn, "layout", _LAYOUTS, layout), _dtype_code(y), eps, mul))
    if st:
        _check(fn, st)


def _rows(fn: str, name: str, t, T, D, dev: int) -> int:
    """Row stride of bf16 [T, D] with contiguous rows."""
    if t.shape == (T, D) and t.dtype is _bf16 and t.get_device() == dev:
        st, sd = t.stride()
        if sd == 1:
            return st if T > 1 else 0
    raise LsaError(fn, -1, f"{name}: bf16 [{T}, {D}] on cuda:{dev} with contiguous rows wanted")


def lsa_cache_append(a, kv, slot, pos=None, freqs=None, kv_weight=None, kv_eps=1e-6, layout="interleaved", mul=1.0,
                     k=None, k_cache=None, k_scale=None, k_norm="none", k_weight=None, k_bias=None, k_eps=1e-6,
                     k_rope_off=-1, k_layout="half", stream=None):
    """kv[slot[t]] = a[t] with its first 512 dims RMS-normed (kv_weight given) and its last 64 rotated by pos[t]; with k,
    the index keys normed, rotated and written to k_cache[slot[t]] too (bf16, or e4m3 codes with k_scale)."""
    fn = "lsa_cache_append"
    if not a.is_cuda or slot.dim() != 1 or kv.dim() != 2:
        _bad(fn, "a [T, 576], kv [slots, 576] and slot [T] on a GPU wanted")
    dev = a.get_device()
    if _off_device(dev):
        with torch.cuda.device(a.device):
            return lsa_cache_append(a, kv, slot, pos, freqs, kv_weight, kv_eps, layout, mul, k, k_cache, k_scale, k_norm,
                                    k_weight, k_bias, k_eps, k_rope_off, k_layout, stream)
    T, n = slot.shape[0], kv.shape[0]
    if (freqs is None) != (pos is None) or (k is None) != (k_cache is None):
        _bad(fn, "freqs and pos, and k and k_cache, belong together")
    a_ld = _rows(fn, "a", a, T, 576, dev)
    k_p = k_ld = d_I = k_dtype = kc_p = 0
    if k is not None:
        if k.dim() != 2:
            _bad(fn, "k [T, d_I] wanted")
        d_I, k_dtype = k.shape[1], _dtype_code(k_cache)
        k_p, k_ld = k.data_ptr(), _rows(fn, "k", k, T, d_I, dev)
        kc_p = _ten(fn, "k_cache", k_cache, k_cache.dtype, (n, d_I), dev)
    else:
        k_rope_off = -1
    st = (_lib or load_library()).lsa_cache_append_packed(_CACHE_APPEND.pack(
        _CACHE_APPEND.size, a.data_ptr(), a_ld, T, _vec(fn, "kv_weight", kv_weight, _f32, 512, dev),
        _vec(fn, "freqs", freqs, _f64, 32, dev), _vec(fn, "pos", pos, _i64, T, dev), _vec(fn, "slot", slot, _i64, T, dev),
        _ten(fn, "kv", kv, _bf16, (n, 576), dev), n, k_p, k_ld, _vec(fn, "k_weight", k_weight, _f32, d_I, dev),
        _vec(fn, "k_bias", k_bias, _f32, d_I, dev), kc_p, _vec(fn, "k_scale", k_scale, _f32, n, dev),
        _get_stream(dev) if stream is None else stream.cuda_stream, 576, 512, _code(fn, "layout", _LAYOUTS, layout), d_I,
        _code(fn, "k_norm", _NORMS, k_norm), k_rope_off, _code(fn, "k_layout", _LAYOUTS, k_layout), k_dtype, kv_eps, mul,
        k_eps))
    if st:
        _check(fn, st)


def lsa_prefix_attn_workspace_size(B, H):
    return load_library().lsa_prefix_attn_workspace_size(B, H)


def lsa_prefix_attn(q, prefix, scale, out, lse=None, pages=None, table=None, own_len=None, ws=None, stream=None):
    """out[b, h] = softmax over the rows of `prefix` (None: no prefix) and the query's own own_len[b] rows in `pages`
    ([n_pages, page, 576], found through table [B, cols]) of scale q.k, times the rows' first 512 dims."""
    fn = "lsa_prefix_attn"
    if q.dim() != 3 or not q.is_cuda or out.dim() != 3:
        _bad(fn, "q [B, H, 576] and out [B, H, 512] on a GPU wanted")
    dev = q.get_device()
    if _off_device(dev):
        with torch.cuda.device(q.device):
            return lsa_prefix_attn(q, prefix, scale, out, lse, pages, table, own_len, ws, stream)
    B, H, d_qk = q_shape = q.shape
    d_v, Lp, prefix_p = out.shape[2], 0, 0
    if prefix is not None:
        Lp = prefix.shape[0]
        prefix_p = _ten(fn, "prefix", prefix, _bf16, (Lp, d_qk), dev)
    n_pages = page = cols = 0
    pages_p = table_p = 0
    if own_len is not None:
        if pages is None or table is None or pages.dim() != 3 or table.dim() != 2:
            _bad(fn, "pages [n_pages, page, 576] and table [B, cols] wanted with own_len")
        n_pages, page, _ = pages.shape
        cols = table.shape[1]
        pages_p, table_p = _ten(fn, "pages", pages, _bf16, (n_pages, page, d_qk), dev), _ten(fn, "table", table, _i32, (B, cols), dev)
    elif pages is not None or table is not None:
        _bad(fn, "pages and table without own_len")
    ws_p = ws_n = 0
    if ws is not None:
        if ws.get_device() != dev or not ws.is_contiguous():
            _bad(fn, "ws: contiguous bytes on the GPU of q wanted")
        ws_p, ws_n = ws.data_ptr(), ws.numel() * ws.element_size()
    st = (_lib or load_library()).lsa_prefix_attn_packed(_PREFIX_ATTN.pack(
        _PREFIX_ATTN.size, _ten(fn, "q", q, _bf16, q_shape, dev), B, prefix_p, Lp, pages_p, n_pages, table_p, cols,
        _vec(fn, "own_len", own_len, _i32, B, dev), _ten(fn, "out", out, _bf16, (B, H, d_v), dev),
        0 if lse is None else _ten(fn, "lse", lse, _f32, (B, H), dev), ws_p, ws_n,
        _get_stream(dev) if stream is None else stream.cuda_stream, H, d_qk, d_v, page, scale))
    if st:
        _check(fn, st)


def workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """Caller-owned scratch buffer (256-byte aligned by the CUDA caching allocator)."""
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
