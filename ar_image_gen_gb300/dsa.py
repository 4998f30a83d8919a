"""Thin ctypes binding over libdsa.so (include/dsa.h).

The module-level functions carry the C names and only marshal arguments:
torch tensors become device pointers, torch streams become cudaStream_t.
Every step of the decode path runs in the library's CUDA kernels; there is
no fallback.  Importing this module raises if libdsa.so has not been built.

Method: "Understanding and Exploiting Diagonal Attention Sparsity in
Autoregressive Image Generation" (arXiv 2609.19702), section 4, Algorithm 1.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

from .build import LIB as _BUILT_LIB

# DSA_LIB may point at another build of the same library (e.g. a variant with
# a different pipeline shape); the default is the in-tree build.
LIB = os.environ.get("DSA_LIB", _BUILT_LIB)

if not os.path.exists(LIB):
    raise ImportError(f"libdsa.so is not built ({LIB}); run ar_image_gen_gb300.build.build()")

_L = ctypes.CDLL(LIB)

DSA_OK = 0
DSA_ERR_ARG = -1
DSA_ERR_STATE = -2
DSA_ERR_OOM = -3
DSA_ERR_CUDA = -4
DSA_ERR_TIMEOUT = -5
DSA_ERR_DEVICE_CHECK = -6
DSA_BF16 = 0
DSA_F32 = 1
DSA_FP8_E4M3 = 2
DTYPES = {"bf16": DSA_BF16, "f32": DSA_F32, "fp8e4m3": DSA_FP8_E4M3}

STATUS_NAMES = {0: "DSA_OK", -1: "DSA_ERR_ARG", -2: "DSA_ERR_STATE", -3: "DSA_ERR_OOM", -4: "DSA_ERR_CUDA",
                -5: "DSA_ERR_TIMEOUT", -6: "DSA_ERR_DEVICE_CHECK"}

EXPORTS = ["dsa_create", "dsa_create_ex", "dsa_prefill", "dsa_decode_step", "dsa_destroy", "dsa_get_step",
           "dsa_get_skip_mask", "dsa_get_last_selection", "dsa_sync_status", "dsa_last_error",
           "dsa_state_bytes", "dsa_plan_step", "dsa_plan_query", "dsa_set_kv_scales", "dsa_set_splits", "dsa_set_pipeline",
           "dsa_set_merge", "dsa_set_wait_limit", "dsa_debug_copy_state", "dsa_debug_set_step",
           "dsa_debug_fail_alloc_after", "dsa_decode_step_noalloc", "dsa_decode_step_noalloc_status", "dsa_diag_trace", "dsa_set_graph_mode",
           "dsa_sync_step",
           "dsa_proj_create", "dsa_proj_destroy", "dsa_qkv_rope", "dsa_decode_step_fused", "dsa_proj_sync_status",
           "dsa_proj_set_wait_limit", "dsa_pol_create", "dsa_pol_destroy", "dsa_pol_prefill", "dsa_pol_decode_step",
           "dsa_pol_get_positions", "dsa_pol_get_last_eviction", "dsa_pol_sync_status", "dsa_pol_set_wait_limit",
           "dsa_pol_set_shape", "dsa_rope_create", "dsa_rope_destroy", "dsa_rope_apply", "dsa_paged_create",
           "dsa_paged_destroy", "dsa_paged_append", "dsa_paged_attend", "dsa_paged_sync_status",
           "dsa_paged_set_wait_limit"]


class dsa_step_plan(ctypes.Structure):
    _fields_ = [("phase", ctypes.c_int), ("t_inner", ctypes.c_int), ("n_prefix", ctypes.c_int),
                ("n_decode", ctypes.c_int), ("select", ctypes.c_int), ("nsplit", ctypes.c_int),
                ("chunk", ctypes.c_int), ("grid", ctypes.c_int), ("pipeline", ctypes.c_int),
                ("algo_bytes", ctypes.c_ulonglong), ("cta_merge", ctypes.c_int)]


_P = ctypes.c_void_p
_I = ctypes.c_int
_L.dsa_create.argtypes = [_I] * 6 + [ctypes.POINTER(_P)]
_L.dsa_create_ex.argtypes = [_I] * 7 + [ctypes.POINTER(_P)]
_L.dsa_prefill.argtypes = [_P, _P, _P, _P]
_L.dsa_decode_step.argtypes = [_P, _P, _P, _P, _P, _P]
_L.dsa_destroy.argtypes = [_P]
_L.dsa_get_step.argtypes = [_P, ctypes.POINTER(_I)]
_L.dsa_get_skip_mask.argtypes = [_P, _P, _P]
_L.dsa_get_last_selection.argtypes = [_P, _P, _P]
_L.dsa_sync_status.argtypes = [_P, _P]
_L.dsa_last_error.restype = ctypes.c_char_p
_L.dsa_state_bytes.argtypes = [_I] * 6
_L.dsa_state_bytes.restype = ctypes.c_size_t
_L.dsa_plan_step.argtypes = [_P, _I, ctypes.POINTER(dsa_step_plan)]
_L.dsa_plan_query.argtypes = [_I] * 9 + [_P, _P, ctypes.POINTER(dsa_step_plan)]
_L.dsa_set_splits.argtypes = [_P, _I]
_L.dsa_set_kv_scales.argtypes = [_P, _P, _P]
_L.dsa_debug_copy_state.argtypes = [_P, _P, _P]
_L.dsa_debug_set_step.argtypes = [_P, _I, _P]
_L.dsa_set_pipeline.argtypes = [_P, _I]
_L.dsa_set_merge.argtypes = [_P, _I]
_L.dsa_set_wait_limit.argtypes = [_P, ctypes.c_uint32]
_L.dsa_debug_fail_alloc_after.argtypes = [_I]
_L.dsa_set_graph_mode.argtypes = [_P, _I]
_L.dsa_sync_step.argtypes = [_P, _P]
_L.dsa_decode_step_noalloc.argtypes = [_I] * 8 + [_P] * 9
_L.dsa_decode_step_noalloc_status.argtypes = [_P]
_L.dsa_diag_trace.argtypes = [_I] * 5 + [_P] * 3 + [_I] + [_P] * 6
_L.dsa_proj_create.argtypes = [_I] * 4 + [ctypes.POINTER(_P)]
_L.dsa_proj_destroy.argtypes = [_P]
_L.dsa_qkv_rope.argtypes = [_P, _P, _P, _I, _P, _P, _P, _P]
_L.dsa_decode_step_fused.argtypes = [_P] * 6
_L.dsa_proj_sync_status.argtypes = [_P, _P]
_L.dsa_proj_set_wait_limit.argtypes = [_P, ctypes.c_uint32]
_L.dsa_pol_create.argtypes = [_I] * 6 + [ctypes.POINTER(_P)]
_L.dsa_pol_destroy.argtypes = [_P]
_L.dsa_pol_prefill.argtypes = [_P] * 4
_L.dsa_pol_decode_step.argtypes = [_P] * 6
_L.dsa_pol_get_positions.argtypes = [_P] * 3
_L.dsa_pol_get_last_eviction.argtypes = [_P] * 3
_L.dsa_pol_sync_status.argtypes = [_P] * 2
_L.dsa_pol_set_wait_limit.argtypes = [_P, ctypes.c_uint32]
_L.dsa_pol_set_shape.argtypes = [_P, _I]
_Q = ctypes.c_int64
_L.dsa_rope_create.argtypes = [_I, _I, _P, _I, ctypes.c_double, ctypes.POINTER(_P)]
_L.dsa_rope_destroy.argtypes = [_P]
_L.dsa_rope_apply.argtypes = [_P, _I, _I, _I, _P, _P, _Q, _P, _Q, _I, _P]
_L.dsa_paged_create.argtypes = [_I] * 6 + [_P, _P, ctypes.POINTER(_P)]
_L.dsa_paged_destroy.argtypes = [_P]
_L.dsa_paged_append.argtypes = [_P, _I, _I, _P, _P, _P, _I, _P, _P, _P, _Q, _P, _Q, _P, _Q, _P, _P]
_L.dsa_paged_attend.argtypes = [_P, _I, _I, _I, _P, _P, _P, _I, _P, _P, _P]
_L.dsa_paged_sync_status.argtypes = [_P, _P]
_L.dsa_paged_set_wait_limit.argtypes = [_P, ctypes.c_uint32]
DSA_POLICY_TOVA = 1
DSA_POLICY_H2O = 2
POLICIES = {"tova": DSA_POLICY_TOVA, "h2o": DSA_POLICY_H2O}


class DSAError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {STATUS_NAMES.get(code, code)}: {dsa_last_error()}")


def _check(code: int, what: str) -> int:
    if code != DSA_OK:
        raise DSAError(code, what)
    return code


def _ptr(x) -> int | None:
    """Device (or host) address of a tensor / ndarray / int, None for None."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    if isinstance(x, np.ndarray):
        return x.ctypes.data
    raise TypeError(f"cannot take the address of {type(x)}")


def _stream(stream) -> int | None:
    if stream is None:
        try:
            import torch
            return torch.cuda.current_stream().cuda_stream
        except Exception:
            return None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


_raw_stream = None
_current_device = None


def _stream_of(device: int, stream) -> int:
    """The given stream, or torch's current one of the device, without the
    Stream object that torch.cuda.current_stream() makes."""
    global _raw_stream
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    if _raw_stream is None:
        import torch

        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda d: torch.cuda.current_stream(d).cuda_stream)
    return _raw_stream(device)


def _on_current_device(device: int):
    """The library launches on the current device: tensors of another are refused."""
    global _current_device
    if _current_device is None:
        import torch

        _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    if device != _current_device():
        raise ValueError(f"the tensors are on CUDA device {device}, the current device is {_current_device()}")


def library_path() -> str:
    return LIB


# ---- C names ---------------------------------------------------------------

def dsa_last_error() -> str:
    return (_L.dsa_last_error() or b"").decode()


def dsa_create(heads, head_dim, L_p, N_r, N_att, sink=0):
    h = _P()
    return _L.dsa_create(heads, head_dim, L_p, N_r, N_att, sink, ctypes.byref(h)), h


def dsa_create_ex(heads, head_dim, L_p, N_r, N_att, sink, dtype):
    h = _P()
    return _L.dsa_create_ex(heads, head_dim, L_p, N_r, N_att, sink, dtype, ctypes.byref(h)), h


def dsa_prefill(h, K, V, stream=None) -> int:
    return _L.dsa_prefill(h, _ptr(K), _ptr(V), _stream(stream))


def dsa_decode_step(h, q, k_new, v_new, out, stream=None) -> int:
    return _L.dsa_decode_step(h, _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(out), _stream(stream))


def dsa_destroy(h) -> int:
    return _L.dsa_destroy(h)


def dsa_get_step(h):
    t = _I()
    return _L.dsa_get_step(h, ctypes.byref(t)), t.value


def dsa_get_skip_mask(h, host_dst: np.ndarray, stream=None) -> int:
    assert host_dst.dtype == np.uint32 and host_dst.flags["C_CONTIGUOUS"]
    return _L.dsa_get_skip_mask(h, host_dst.ctypes.data, _stream(stream))


def dsa_get_last_selection(h, host_dst: np.ndarray, stream=None) -> int:
    assert host_dst.dtype == np.int32 and host_dst.flags["C_CONTIGUOUS"]
    return _L.dsa_get_last_selection(h, host_dst.ctypes.data, _stream(stream))


def dsa_sync_status(h, stream=None) -> int:
    return _L.dsa_sync_status(h, _stream(stream))


def dsa_state_bytes(heads, head_dim, L_p, N_r, sink=0, dtype=DSA_BF16) -> int:
    return int(_L.dsa_state_bytes(heads, head_dim, L_p, N_r, sink, dtype))


def dsa_plan_step(h, t):
    p = dsa_step_plan()
    return _L.dsa_plan_step(h, t, ctypes.byref(p)), p


def dsa_plan_query(heads, head_dim, L_p, N_r, N_att, sink, dtype, t, sm_count, ctas_per_sm, cta_merge_ok=None):
    """Host-only plan of step t for a state of these sizes on a device of
    `sm_count` SMs with the given resident CTAs per SM of the 4 launch
    pipelines (and where the in-CTA merge fits); returns (status, plan)."""
    ctas = (ctypes.c_int * 4)(*[int(c) for c in ctas_per_sm])
    ok = None if cta_merge_ok is None else (ctypes.c_int * 4)(*[int(c) for c in cta_merge_ok])
    p = dsa_step_plan()
    code = _L.dsa_plan_query(heads, head_dim, L_p, N_r, N_att, sink, dtype, t, sm_count, ctas, ok, ctypes.byref(p))
    return code, p


def dsa_set_kv_scales(h, k_scale: np.ndarray, v_scale: np.ndarray) -> int:
    k = np.ascontiguousarray(k_scale, dtype=np.float32)
    v = np.ascontiguousarray(v_scale, dtype=np.float32)
    return _L.dsa_set_kv_scales(h, k.ctypes.data, v.ctypes.data)


def dsa_debug_copy_state(h, host_prefix: np.ndarray | None, host_ring: np.ndarray | None) -> int:
    return _L.dsa_debug_copy_state(h, None if host_prefix is None else host_prefix.ctypes.data,
                                   None if host_ring is None else host_ring.ctypes.data)


def dsa_debug_set_step(h, t, stream=None) -> int:
    return _L.dsa_debug_set_step(h, t, _stream(stream))


def dsa_set_splits(h, nsplit) -> int:
    return _L.dsa_set_splits(h, nsplit)


def dsa_set_pipeline(h, pipeline) -> int:
    return _L.dsa_set_pipeline(h, pipeline)


def dsa_set_merge(h, mode) -> int:
    return _L.dsa_set_merge(h, mode)


def dsa_set_wait_limit(h, limit) -> int:
    return _L.dsa_set_wait_limit(h, limit)


def dsa_debug_fail_alloc_after(n) -> int:
    return _L.dsa_debug_fail_alloc_after(n)


def dsa_set_graph_mode(h, on) -> int:
    return _L.dsa_set_graph_mode(h, 1 if on else 0)


def dsa_sync_step(h, stream=None) -> int:
    return _L.dsa_sync_step(h, _stream(stream))


def dsa_decode_step_noalloc(heads, head_dim, L_p, N_r, N_att, sink, dtype, t, prefix, ring, mask, last_sel,
                            q, k_new, v_new, out, stream=None) -> int:
    return _L.dsa_decode_step_noalloc(heads, head_dim, L_p, N_r, N_att, sink, dtype, t, _ptr(prefix), _ptr(ring),
                                      _ptr(mask), _ptr(last_sel), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(out),
                                      _stream(stream))


def dsa_decode_step_noalloc_status(stream=None) -> int:
    return _L.dsa_decode_step_noalloc_status(_stream(stream))


def dsa_diag_trace(heads, head_dim, L_p, L_dec, dtype, Q, Kp, Kd, dist: np.ndarray, step_mass, mass_mean: np.ndarray,
                   vertical: np.ndarray, diagonal: np.ndarray, stream=None) -> int:
    return _L.dsa_diag_trace(heads, head_dim, L_p, L_dec, dtype, _ptr(Q), _ptr(Kp), _ptr(Kd), len(dist), _ptr(dist),
                             _ptr(step_mass), _ptr(mass_mean), _ptr(vertical), _ptr(diagonal), _stream(stream))


def diag_trace(Q, Kp, Kd, dists, step_mass=None, stream=None):
    """Fig. 8 / Fig. 10 diagnostics of a dense decode trace (include/dsa_diag.h).
    Q, Kd: [heads, L_dec, d], Kp: [heads, L_p, d] device tensors (bf16 or fp32).
    Returns (mass_mean [3], vertical [n], diagonal [n]) as numpy arrays;
    step_mass, if given, is a device float tensor [heads, L_dec, 3] to fill."""
    import torch

    heads, L_dec, d = Q.shape
    L_p = Kp.shape[1] if Kp is not None else 0
    dtype = {torch.bfloat16: DSA_BF16, torch.float32: DSA_F32}[Q.dtype]
    dist = np.ascontiguousarray(dists, dtype=np.int32)
    mass = np.zeros(3)
    vert = np.zeros(len(dist))
    diag = np.zeros(len(dist))
    _check(dsa_diag_trace(heads, d, L_p, L_dec, dtype, Q, Kp if L_p > 0 else None, Kd, dist, step_mass, mass, vert,
                          diag, stream), "dsa_diag_trace")
    return mass, vert, diag


def dsa_proj_create(batch, heads, head_dim, hidden):
    p = _P()
    return _L.dsa_proj_create(batch, heads, head_dim, hidden, ctypes.byref(p)), p


def dsa_proj_destroy(p) -> int:
    return _L.dsa_proj_destroy(p)


def dsa_qkv_rope(p, x, W, pos, q, k, v, stream=None) -> int:
    return _L.dsa_qkv_rope(p, _ptr(x), _ptr(W), pos, _ptr(q), _ptr(k), _ptr(v), _stream(stream))


def dsa_decode_step_fused(h, p, x, W, out, stream=None) -> int:
    return _L.dsa_decode_step_fused(h, p, _ptr(x), _ptr(W), _ptr(out), _stream(stream))


def dsa_proj_sync_status(p, stream=None) -> int:
    return _L.dsa_proj_sync_status(p, _stream(stream))


def dsa_proj_set_wait_limit(p, limit) -> int:
    return _L.dsa_proj_set_wait_limit(p, limit)


def dsa_pol_create(heads, head_dim, L_p, N_att, policy, dtype):
    h = _P()
    return _L.dsa_pol_create(heads, head_dim, L_p, N_att, policy, dtype, ctypes.byref(h)), h


def dsa_pol_destroy(h) -> int:
    return _L.dsa_pol_destroy(h)


def dsa_pol_prefill(h, K, V, stream=None) -> int:
    return _L.dsa_pol_prefill(h, _ptr(K), _ptr(V), _stream(stream))


def dsa_pol_decode_step(h, q, k_new, v_new, out, stream=None) -> int:
    return _L.dsa_pol_decode_step(h, _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(out), _stream(stream))


def dsa_pol_get_positions(h, host_dst: np.ndarray, stream=None) -> int:
    assert host_dst.dtype == np.int32 and host_dst.flags["C_CONTIGUOUS"]
    return _L.dsa_pol_get_positions(h, host_dst.ctypes.data, _stream(stream))


def dsa_pol_get_last_eviction(h, host_dst: np.ndarray, stream=None) -> int:
    assert host_dst.dtype == np.int32 and host_dst.flags["C_CONTIGUOUS"]
    return _L.dsa_pol_get_last_eviction(h, host_dst.ctypes.data, _stream(stream))


def dsa_pol_sync_status(h, stream=None) -> int:
    return _L.dsa_pol_sync_status(h, _stream(stream))


def dsa_pol_set_wait_limit(h, limit) -> int:
    return _L.dsa_pol_set_wait_limit(h, limit)


def dsa_pol_set_shape(h, shape) -> int:
    return _L.dsa_pol_set_shape(h, shape)


def dsa_rope_create(head_dim, pairs, restart=False, base=10000.0):
    r = _P()
    n = np.ascontiguousarray(pairs, dtype=np.int32)
    return _L.dsa_rope_create(head_dim, n.size, n.ctypes.data, 1 if restart else 0, base, ctypes.byref(r)), r


def dsa_rope_destroy(r) -> int:
    return _L.dsa_rope_destroy(r)


def dsa_rope_apply(r, tokens, heads, dtype, pos, x, x_stride, y, y_stride, inverse=False, stream=None) -> int:
    return _L.dsa_rope_apply(r, tokens, heads, dtype, _ptr(pos), _ptr(x), x_stride, _ptr(y), y_stride,
                             1 if inverse else 0, _stream(stream))


def dsa_paged_create(q_heads, kv_heads, head_dim, page_size, num_pages, dtype, pages, scales):
    h = _P()
    return _L.dsa_paged_create(q_heads, kv_heads, head_dim, page_size, num_pages, dtype, _ptr(pages), _ptr(scales),
                               ctypes.byref(h)), h


def dsa_paged_destroy(h) -> int:
    return _L.dsa_paged_destroy(h)


def dsa_paged_append(h, n_seqs, n_tokens, cu, lens, table, table_width, rope, pos, q, q_stride, k, k_stride, v,
                     v_stride, q_out, stream=None) -> int:
    return _L.dsa_paged_append(h, n_seqs, n_tokens, _ptr(cu), _ptr(lens), _ptr(table), table_width, rope, _ptr(pos),
                               _ptr(q), q_stride, _ptr(k), k_stride, _ptr(v), v_stride, _ptr(q_out), _stream(stream))


def dsa_paged_attend(h, n_seqs, n_tokens, max_new, cu, lens, table, table_width, q, out, stream=None) -> int:
    return _L.dsa_paged_attend(h, n_seqs, n_tokens, max_new, _ptr(cu), _ptr(lens), _ptr(table), table_width, _ptr(q),
                               _ptr(out), _stream(stream))


def dsa_paged_sync_status(h, stream=None) -> int:
    return _L.dsa_paged_sync_status(h, _stream(stream))


def dsa_paged_set_wait_limit(h, limit) -> int:
    return _L.dsa_paged_set_wait_limit(h, limit)


# ---- convenience wrappers --------------------------------------------------

def _rows(name, x, tokens, heads, head_dim, dtype, device):
    """Row stride of a device tensor [tokens, heads, head_dim] whose heads lie side by side."""
    if x.shape != (tokens, heads, head_dim) or x.dtype is not dtype or x.get_device() != device:
        raise ValueError(f"{name} must be a tensor [{tokens}, {heads}, {head_dim}] of {dtype} on CUDA device {device}, "
                         f"got {tuple(x.shape)} of {x.dtype} on {x.device}")
    if x.is_contiguous():
        return heads * head_dim
    st = x.stride()
    if st[2] != 1 or (st[1] != head_dim and heads > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous (strides {st})")
    # the row stride of a single token is never used
    return st[0] if tokens > 1 else heads * head_dim


def _packed(name, x, shape, dtype, device):
    if x.shape != shape or x.dtype is not dtype or x.get_device() != device or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor {shape} of {dtype} on CUDA device {device}, "
                         f"got {tuple(x.shape)} of {x.dtype} on {x.device}")
    return x.data_ptr()


class Rope:
    """A rotation plan over several position axes (include/dsa_rope.h):
    `pairs[a]` pairs of every head turn with axis a."""

    _types = None

    def __init__(self, head_dim, pairs, base=10000.0, restart=False):
        code, r = dsa_rope_create(head_dim, pairs, restart, base)
        _check(code, "dsa_rope_create")
        self.r = r
        self.head_dim, self.axes = head_dim, len(pairs)

    def close(self):
        if getattr(self, "r", None):
            dsa_rope_destroy(self.r)
            self.r = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def apply(self, x, pos, out, inverse=False, stream=None):
        """out = x rotated ([tokens, heads, head_dim] bf16 or fp32, `out` may
        be x) at pos [tokens, axes] int32; inverse: by the negative angles,
        the gradient of the rotation."""
        if self._types is None:
            import torch

            self._types = {torch.bfloat16: DSA_BF16, torch.float32: DSA_F32}, torch.int32
        codes, int32 = self._types
        n, heads, d = x.shape
        dtype, device = x.dtype, x.get_device()
        if dtype not in codes or device < 0:
            raise ValueError(f"x must be a bfloat16 or float32 tensor on a GPU, got {dtype} on {x.device}")
        _on_current_device(device)
        xs = _rows("x", x, n, heads, self.head_dim, dtype, device)
        ys = _rows("out", out, n, heads, self.head_dim, dtype, device)
        _check(_L.dsa_rope_apply(self.r, n, heads, codes[dtype], _packed("pos", pos, (n, self.axes), int32, device),
                                 x.data_ptr(), xs, out.data_ptr(), ys, 1 if inverse else 0,
                                 _stream_of(device, stream)), "dsa_rope_apply")


class PagedKV:
    """A paged KV cache of one layer (include/dsa_paged.h).  `pages`
    [num_pages, kv_heads, page_size, 2, head_dim] (bfloat16 or float8_e4m3fn)
    and, for "fp8e4m3", `scales` [num_pages, kv_heads, 2] float32 are the
    caller's tensors, or are allocated here."""

    def __init__(self, q_heads, kv_heads, head_dim, page_size, num_pages, dtype="bf16", pages=None, scales=None):
        import torch

        eight = DTYPES[dtype] == DSA_FP8_E4M3
        want = torch.float8_e4m3fn if eight else torch.bfloat16
        shape = (num_pages, kv_heads, page_size, 2, head_dim)
        if pages is None:
            pages = torch.empty(shape, dtype=want, device="cuda")
        if scales is None and eight:
            scales = torch.ones((num_pages, kv_heads, 2), dtype=torch.float32, device="cuda")
        if tuple(pages.shape) != shape or pages.dtype != want or not pages.is_cuda or not pages.is_contiguous():
            raise ValueError(f"pages must be a contiguous CUDA tensor {shape} of {want}")
        if eight and (tuple(scales.shape) != (num_pages, kv_heads, 2) or scales.dtype != torch.float32
                      or not scales.is_cuda or not scales.is_contiguous()):
            raise ValueError(f"scales must be a contiguous CUDA float32 tensor {(num_pages, kv_heads, 2)}")
        # the handle, its workspace and its kernels are the current device's
        _on_current_device(pages.get_device())
        if eight and scales.get_device() != pages.get_device():
            raise ValueError(f"pages are on CUDA device {pages.get_device()}, scales on {scales.get_device()}")
        code, h = dsa_paged_create(q_heads, kv_heads, head_dim, page_size, num_pages, DTYPES[dtype], pages, scales)
        _check(code, "dsa_paged_create")
        self.h, self.pages, self.scales, self.device = h, pages, scales, pages.get_device()
        self._bf16, self._int32 = torch.bfloat16, torch.int32
        self.q_heads, self.kv_heads, self.head_dim, self.page_size = q_heads, kv_heads, head_dim, page_size

    def close(self):
        if getattr(self, "h", None):
            dsa_paged_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def append(self, q, k, v, cu, lens, table, q_out=None, rope=None, pos=None, stream=None):
        """Writes rows k, v [tokens, kv_heads, head_dim] bf16 of the new
        tokens into their pages, rotated (k) by `rope` at pos [tokens, axes];
        q [tokens, q_heads, head_dim] (or None), rotated, goes to q_out."""
        if (rope is None) != (pos is None):
            raise ValueError("rope and pos go together")
        if (q is None) != (q_out is None):
            raise ValueError("q and q_out go together")
        bf, i32, dev, Hk, d = self._bf16, self._int32, self.device, self.kv_heads, self.head_dim
        n = k.shape[0]
        n_seqs, width = table.shape
        ks = _rows("k", k, n, Hk, d, bf, dev)
        vs = _rows("v", v, n, Hk, d, bf, dev)
        qs, qp, op = 0, None, None
        if q is not None:
            qs, qp = _rows("q", q, n, self.q_heads, d, bf, dev), q.data_ptr()
            op = _packed("q_out", q_out, (n, self.q_heads, d), bf, dev)
        r, pp = None, None
        if rope is not None:
            r, pp = rope.r, _packed("pos", pos, (n, rope.axes), i32, dev)
            if not r:
                raise ValueError("the rotation plan is closed")
        _check(_L.dsa_paged_append(self.h, n_seqs, n, _packed("cu", cu, (n_seqs + 1,), i32, dev),
                                   _packed("lens", lens, (n_seqs,), i32, dev),
                                   _packed("table", table, (n_seqs, width), i32, dev), width, r, pp, qp, qs,
                                   k.data_ptr(), ks, v.data_ptr(), vs, op, _stream_of(dev, stream)), "dsa_paged_append")

    def attend(self, q, cu, lens, table, out, max_new=None, stream=None):
        """out = causal attention of q [tokens, q_heads, head_dim] bf16 (the
        new tokens, already appended) over their sequences; `max_new`: the
        most new tokens of a sequence (a hint for the launch; without it the
        mean, the rows of q per sequence: of a prompt all, of a decode step
        one)."""
        bf, i32, dev = self._bf16, self._int32, self.device
        n = q.shape[0]
        n_seqs, width = table.shape
        if max_new is None:
            max_new = max(1, -(-n // max(1, n_seqs)))
        shape = (n, self.q_heads, self.head_dim)
        _check(_L.dsa_paged_attend(self.h, n_seqs, n, max_new, _packed("cu", cu, (n_seqs + 1,), i32, dev),
                                   _packed("lens", lens, (n_seqs,), i32, dev),
                                   _packed("table", table, (n_seqs, width), i32, dev), width,
                                   _packed("q", q, shape, bf, dev), _packed("out", out, shape, bf, dev),
                                   _stream_of(dev, stream)), "dsa_paged_attend")

    def sync_status(self, stream=None) -> int:
        return dsa_paged_sync_status(self.h, stream)

    def set_wait_limit(self, limit: int):
        _check(dsa_paged_set_wait_limit(self.h, limit), "dsa_paged_set_wait_limit")


class Policy:
    """A score-based eviction baseline handle (include/dsa_policy.h):
    `heads` streams, `policy` "tova" or "h2o", N_att attended decode
    entries, bf16 or f32 rows."""

    def __init__(self, heads, head_dim, L_p, N_att, policy, dtype="bf16"):
        code, h = dsa_pol_create(heads, head_dim, L_p, N_att, POLICIES[policy], DTYPES[dtype])
        _check(code, "dsa_pol_create")
        self.h = h
        self.heads, self.head_dim, self.L_p, self.N_att, self.policy = heads, head_dim, L_p, N_att, policy

    def close(self):
        if getattr(self, "h", None):
            dsa_pol_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def prefill(self, K, V, stream=None):
        _check(dsa_pol_prefill(self.h, K, V, stream), "dsa_pol_prefill")

    def decode_step(self, q, k_new, v_new, out, stream=None):
        _check(dsa_pol_decode_step(self.h, q, k_new, v_new, out, stream), "dsa_pol_decode_step")

    def positions(self, stream=None) -> np.ndarray:
        dst = np.zeros((self.heads, self.N_att), dtype=np.int32)
        _check(dsa_pol_get_positions(self.h, dst, stream), "dsa_pol_get_positions")
        return dst

    def last_eviction(self, stream=None) -> np.ndarray:
        dst = np.zeros(self.heads, dtype=np.int32)
        _check(dsa_pol_get_last_eviction(self.h, dst, stream), "dsa_pol_get_last_eviction")
        return dst

    def sync_status(self, stream=None) -> int:
        return dsa_pol_sync_status(self.h, stream)

    def set_wait_limit(self, limit: int):
        _check(dsa_pol_set_wait_limit(self.h, limit), "dsa_pol_set_wait_limit")

    def set_shape(self, shape: int):
        _check(dsa_pol_set_shape(self.h, shape), "dsa_pol_set_shape")


class Proj:
    """A QKV projection context (include/dsa_proj.h): `batch` tokens, `heads`
    heads of `head_dim`, `hidden` input features."""

    def __init__(self, batch, heads, head_dim, hidden):
        code, p = dsa_proj_create(batch, heads, head_dim, hidden)
        _check(code, "dsa_proj_create")
        self.p = p
        self.batch, self.heads, self.head_dim, self.hidden = batch, heads, head_dim, hidden

    def close(self):
        if getattr(self, "p", None):
            dsa_proj_destroy(self.p)
            self.p = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def qkv_rope(self, x, W, pos, q, k, v, stream=None):
        _check(dsa_qkv_rope(self.p, x, W, pos, q, k, v, stream), "dsa_qkv_rope")

    def sync_status(self, stream=None) -> int:
        return dsa_proj_sync_status(self.p, stream)

    def set_wait_limit(self, limit: int):
        _check(dsa_proj_set_wait_limit(self.p, limit), "dsa_proj_set_wait_limit")


class DSA:
    """One handle: `heads` streams of one layer stepping together."""

    def __init__(self, heads, head_dim, L_p, N_r, N_att, sink=0, dtype="bf16"):
        self.dtype_code = DTYPES[dtype]
        code, h = dsa_create_ex(heads, head_dim, L_p, N_r, N_att, sink, self.dtype_code)
        _check(code, "dsa_create_ex")
        self.h = h
        self.heads, self.head_dim, self.L_p, self.N_r, self.N_att, self.sink = heads, head_dim, L_p, N_r, N_att, sink
        self.mask_words = (N_r - sink + 31) // 32

    def close(self):
        if getattr(self, "h", None):
            dsa_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def prefill(self, K, V, stream=None):
        _check(dsa_prefill(self.h, K, V, stream), "dsa_prefill")

    def decode_step(self, q, k_new, v_new, out, stream=None):
        _check(dsa_decode_step(self.h, q, k_new, v_new, out, stream), "dsa_decode_step")

    def decode_step_fused(self, proj: "Proj", x, W, out, stream=None):
        """Projection of x by W (position L_p + t) and the decode step on it."""
        _check(dsa_decode_step_fused(self.h, proj.p, x, W, out, stream), "dsa_decode_step_fused")

    @property
    def t(self) -> int:
        code, t = dsa_get_step(self.h)
        _check(code, "dsa_get_step")
        return t

    def skip_mask(self, stream=None) -> np.ndarray:
        dst = np.zeros((self.heads, self.mask_words), dtype=np.uint32)
        _check(dsa_get_skip_mask(self.h, dst, stream), "dsa_get_skip_mask")
        return dst

    def last_selection(self, stream=None) -> np.ndarray:
        dst = np.zeros(self.heads, dtype=np.int32)
        _check(dsa_get_last_selection(self.h, dst, stream), "dsa_get_last_selection")
        return dst

    def sync_status(self, stream=None) -> int:
        return dsa_sync_status(self.h, stream)

    def state_bytes(self) -> int:
        """Device bytes of the handle's KV state (prefix, ring, skip mask)."""
        return dsa_state_bytes(self.heads, self.head_dim, self.L_p, self.N_r, self.sink, self.dtype_code)

    def plan(self, t: int | None = None) -> dsa_step_plan:
        code, p = dsa_plan_step(self.h, self.t if t is None else t)
        _check(code, "dsa_plan_step")
        return p

    def set_kv_scales(self, k_scale, v_scale):
        """Per-stream FP8 scales (host arrays of `heads` floats); a prefill must follow."""
        _check(dsa_set_kv_scales(self.h, k_scale, v_scale), "dsa_set_kv_scales")

    def copy_state(self):
        """(prefix, ring) as uint8 arrays [heads, rows, 2, head_dim * element bytes]."""
        eb = {DSA_BF16: 2, DSA_F32: 4, DSA_FP8_E4M3: 1}[self.dtype_code]
        pre = np.zeros((self.heads, self.L_p + self.sink, 2, self.head_dim * eb), dtype=np.uint8)
        ring = np.zeros((self.heads, self.N_r - self.sink, 2, self.head_dim * eb), dtype=np.uint8)
        _check(dsa_debug_copy_state(self.h, pre, ring), "dsa_debug_copy_state")
        return pre, ring

    def set_splits(self, nsplit: int):
        _check(dsa_set_splits(self.h, nsplit), "dsa_set_splits")

    def debug_set_step(self, t: int, stream=None):
        """N_att == N_r handles only, right after prefill: jump to step t
        (the skipped-over decode entries read as zero rows)."""
        _check(dsa_debug_set_step(self.h, t, stream), "dsa_debug_set_step")

    def set_pipeline(self, pipeline: int):
        _check(dsa_set_pipeline(self.h, pipeline), "dsa_set_pipeline")

    def set_merge(self, mode: int):
        """0: split streams merged inside the CTA where possible; 1: always by the merge launch."""
        _check(dsa_set_merge(self.h, mode), "dsa_set_merge")

    def set_wait_limit(self, limit: int):
        _check(dsa_set_wait_limit(self.h, limit), "dsa_set_wait_limit")

    def set_graph_mode(self, on: bool):
        """Steady-state steps replayable from a CUDA graph (the step lives on the device)."""
        _check(dsa_set_graph_mode(self.h, on), "dsa_set_graph_mode")

    def sync_step(self, stream=None):
        _check(dsa_sync_step(self.h, stream), "dsa_sync_step")
