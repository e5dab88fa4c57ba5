"""GB300 (sm_103a) decode hot path of TokenSwift-style ultra-long generation.

Thin Python binding over the C-ABI library libtokenswift_gb300.so (see
include/tokenswift_gb300.h).  The functions carry the C names and only
marshal arguments: torch tensors supply device memory and the current CUDA
stream; every step of the computation runs in the library's CUDA kernels.
There is no CPU fallback: if the library is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

from ._build import LIB_PATH, build  # noqa: F401

__all__ = [
    "TsError", "lib", "build", "ts_status_string", "ts_last_error", "ts_version",
    "ts_set_wait_limit",
    "ts_verify_workspace_bytes", "ts_verify_attention", "ts_importance_softmax",
    "ts_select_workspace_bytes", "ts_partial_kv_select_gather", "ts_partial_kv_select_gather_noalloc",
    "ts_select_batched_workspace_bytes", "ts_partial_kv_select_gather_batched", "layer_pointer_table",
    "ts_refresh_workspace_bytes", "ts_partial_kv_refresh_incremental",
    "ts_partial_kv_refresh_incremental_batched",
    "ts_sample_workspace_bytes", "ts_penalized_sample_accept", "ts_kv_commit",
    "ts_kv_commit_batched", "commit_pointer_table", "ts_kv_append_batched",
    "ts_reject_workspace_bytes", "ts_rejection_sample_accept",
    "ts_rope_frequencies", "ts_paged_rope_append",
    "ts_paged_attention_workspace_bytes", "ts_paged_attention",
    "ts_paged_select_workspace_bytes", "ts_paged_select_pages",
    "ts_paged_selected_workspace_bytes", "ts_paged_attention_selected",
    "ts_paged_tree_attention_workspace_bytes", "ts_paged_tree_attention", "ts_paged_kv_commit",
    "ts_token_counts", "ts_logits_process",
]

TS_OK, TS_ERR_INVALID_ARG, TS_ERR_UNSUPPORTED, TS_ERR_CUDA, TS_ERR_TIMEOUT, TS_ERR_WORKSPACE = range(6)
TS_VERIFY_V_FP16 = 1     # ts_verify_attention_flags: the V cache holds fp16
TS_KV_V_FP16 = 1         # ts_kv_append_batched_flags: write V rows into fp16 caches

_c_void_p, _i32, _i64, _sz, _f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
_f64 = ctypes.c_double

_SIGNATURES = {
    "ts_status_string": (ctypes.c_char_p, [_i32]),
    "ts_last_error": (ctypes.c_char_p, []),
    "ts_version": (_i32, []),
    "ts_set_wait_limit": (_i32, [_i64]),
    "ts_verify_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32, _i64]),
    "ts_verify_attention": (_i32, [_c_void_p, _c_void_p, _c_void_p, _i64, _i64, _c_void_p,
                                   _i32, _i32, _i32, _i32, _i32, _c_void_p, _c_void_p, _c_void_p,
                                   _c_void_p, _sz, _c_void_p, _c_void_p]),
    "ts_verify_attention_flags": (_i32, [_c_void_p, _c_void_p, _c_void_p, _i64, _i64, _c_void_p,
                                         _i32, _i32, _i32, _i32, _i32, _c_void_p, _c_void_p,
                                         _c_void_p, _c_void_p, _sz, _i32, _c_void_p, _c_void_p]),
    "ts_select_workspace_bytes": (_sz, [_i32, _i64]),
    "ts_importance_softmax": (_i32, [_c_void_p, _c_void_p, _c_void_p, _i64, _i64, _i32, _i32, _i32,
                                     _i32, _i32, _c_void_p, _c_void_p, _c_void_p]),
    "ts_partial_kv_select_gather": (_i32, [_c_void_p, _c_void_p, _c_void_p, _i64, _i64, _i32, _i32,
                                           _i32, _i32, _i32, _c_void_p, _c_void_p, _c_void_p,
                                           ctypes.POINTER(_i64), _c_void_p, _sz, _c_void_p,
                                           _c_void_p]),
    "ts_partial_kv_select_gather_noalloc": (_i32, [_c_void_p, _c_void_p, _c_void_p, _i64, _i64,
                                                   _i32, _i32, _i32, _i32, _i32, _c_void_p,
                                                   _c_void_p, _c_void_p, ctypes.POINTER(_i64),
                                                   _c_void_p, _c_void_p]),
    "ts_select_batched_workspace_bytes": (_sz, [_i32, _i32, _i64]),
    "ts_partial_kv_select_gather_batched": (_i32, [_i32, _c_void_p, _c_void_p, _c_void_p, _i64, _i64,
                                                   _i32, _i32, _i32, _i32, _i32, _c_void_p,
                                                   _c_void_p, _c_void_p, ctypes.POINTER(_i64),
                                                   _c_void_p, _sz, _c_void_p, _c_void_p]),
    "ts_sample_workspace_bytes": (_sz, [_i32, _i32]),
    "ts_refresh_workspace_bytes": (_sz, [_i32, _i32, _i64, _i64]),
    "ts_partial_kv_refresh_incremental": (_i32, [_c_void_p, _c_void_p, _c_void_p, _i64, _i64, _i32,
                                                 _i32, _i32, _i32, _i32, _c_void_p, _c_void_p,
                                                 _c_void_p, _i64, _i64, ctypes.POINTER(_i64),
                                                 _c_void_p, _c_void_p, _sz, _c_void_p, _c_void_p]),
    "ts_partial_kv_refresh_incremental_batched": (_i32, [_i32, _c_void_p, _c_void_p, _c_void_p,
                                                         _i64, _i64, _i32, _i32, _i32, _i32, _i32,
                                                         _c_void_p, _c_void_p, _c_void_p, _i64,
                                                         _i64, ctypes.POINTER(_i64), _c_void_p,
                                                         _c_void_p, _sz, _c_void_p, _c_void_p]),
    "ts_penalized_sample_accept": (_i32, [_c_void_p, _c_void_p, _c_void_p, _i32, _c_void_p, _i32,
                                          _i32, _i32, _f32, _f32, _f32, _f32, _c_void_p,
                                          _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                          _c_void_p, _sz, _c_void_p, _c_void_p]),
    "ts_penalized_sample_accept_flags": (_i32, [_c_void_p, _c_void_p, _c_void_p, _i32, _c_void_p,
                                                _i32, _i32, _i32, _f32, _f32, _f32, _f32,
                                                _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                                _c_void_p, _c_void_p, _sz, _i32, _c_void_p,
                                                _c_void_p]),
    "ts_penalized_sample_accept_eta": (_i32, [_c_void_p, _c_void_p, _c_void_p, _i32, _c_void_p,
                                              _i32, _i32, _i32, _f32, _f32, _f32, _f32,
                                              _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                              _c_void_p, _c_void_p, _sz, _c_void_p, _c_void_p]),
    "ts_kv_commit": (_i32, [_c_void_p, _c_void_p, _i64, _i64, _i32, _i32, _i32, _c_void_p,
                            _c_void_p, _c_void_p, _c_void_p]),
    "ts_ngram_table_bytes": (_sz, [_i32, _i32]),
    "ts_kv_commit_batched": (_i32, [_i32, _c_void_p, _c_void_p, _i64, _i64, _i32, _i32, _i32,
                                    _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "ts_kv_append_batched": (_i32, [_i32, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _i64, _i64,
                                    _i32, _i32, _i32, _c_void_p]),
    "ts_kv_append_batched_flags": (_i32, [_i32, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _i64,
                                          _i64, _i32, _i32, _i32, _i32, _c_void_p, _c_void_p]),
    "ts_reject_workspace_bytes": (_sz, [_i32]),
    "ts_rejection_sample_accept": (_i32, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _i32,
                                          _c_void_p, _i32, _i32, _i32, _f32, _f32, _f32, _f32,
                                          _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                          _c_void_p, _sz, _i32, _c_void_p, _c_void_p]),
    "ts_ngram_insert": (_i32, [_c_void_p, _i32, _i32, _c_void_p, _i32, _i32, _c_void_p,
                               _c_void_p]),
    "ts_ngram_build_tree": (_i32, [_c_void_p, _i32, _i32, _c_void_p, _c_void_p, _i32, _i32, _i32,
                                   _c_void_p, _i32, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                   _c_void_p]),
    "ts_rope_frequencies": (_i32, [_i32, _f64, _i32, _f64, _f64, _f64, _f64,
                                   ctypes.POINTER(_f64), ctypes.POINTER(_f32)]),
    "ts_paged_rope_append": (_i32, [_c_void_p, _c_void_p, _c_void_p, _i64, _i64, _i64, _i32, _i32,
                                    _i32, _i32, _c_void_p, _c_void_p, _i32, _c_void_p, _i32, _i32,
                                    _i64, _c_void_p, _c_void_p, _i32, _f32, _c_void_p, _c_void_p,
                                    _c_void_p, _c_void_p, _c_void_p, _i32, _c_void_p, _c_void_p]),
    "ts_paged_attention_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
                                                 _i64]),
    "ts_paged_attention": (_i32, [_c_void_p, _c_void_p, _c_void_p, _i32, _i32, _i32, _i32,
                                  _c_void_p, _c_void_p, _i32, _c_void_p, _i32, _i32, _i64, _i32,
                                  _i64, _c_void_p, _c_void_p, _c_void_p, _sz, _i32, _c_void_p,
                                  _c_void_p]),
    "ts_paged_select_workspace_bytes": (_sz, [_i32, _i32, _i32]),
    "ts_paged_select_pages": (_i32, [_c_void_p, _c_void_p, _c_void_p, _i32, _i32, _i32, _i32,
                                     _c_void_p, _c_void_p, _i32, _c_void_p, _i32, _i32, _i64, _i32,
                                     _i32, _i32, _c_void_p, _c_void_p, _c_void_p, _sz, _i32,
                                     _c_void_p, _c_void_p]),
    "ts_paged_selected_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32]),
    "ts_paged_attention_selected": (_i32, [_c_void_p, _c_void_p, _c_void_p, _i32, _i32, _i32, _i32,
                                           _c_void_p, _c_void_p, _i32, _c_void_p, _i32, _i32, _i64,
                                           _c_void_p, _c_void_p, _i32, _c_void_p, _c_void_p,
                                           _c_void_p, _sz, _i32, _c_void_p, _c_void_p]),
    "ts_paged_tree_attention_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32, _i32,
                                                      _i32, _i64]),
    "ts_paged_tree_attention": (_i32, [_c_void_p, _c_void_p, _c_void_p, _i32, _i32, _i32, _i32,
                                       _c_void_p, _c_void_p, _i32, _c_void_p, _i32, _i32, _i64,
                                       _c_void_p, _i32, _i64, _c_void_p, _c_void_p, _c_void_p, _sz,
                                       _i32, _c_void_p, _c_void_p]),
    "ts_paged_kv_commit": (_i32, [_i32, _c_void_p, _c_void_p, _i32, _i32, _c_void_p, _c_void_p,
                                  _i32, _c_void_p, _i32, _i32, _i64, _c_void_p, _i32, _c_void_p,
                                  _c_void_p, _c_void_p, _c_void_p, _i32, _c_void_p, _c_void_p]),
    "ts_token_counts": (_i32, [_c_void_p, _i32, _c_void_p, _i32, _i32, _c_void_p, _c_void_p, _i32,
                               _c_void_p, _c_void_p]),
    "ts_logits_process": (_i32, [_c_void_p, _i64, _i32, _i32, _c_void_p, _i32, _c_void_p,
                                 _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                 _c_void_p, _c_void_p, _i32, _c_void_p, _i32, _c_void_p, _f32,
                                 _c_void_p, _i64, _i32, _c_void_p, _c_void_p]),
}

_LIB = None


class TsError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"[{code}] {msg}")
        self.code = code


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{os.path.basename(LIB_PATH)} is not built: call "
                               "self_speculative_ultra_gb300.build() first")
        h = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(h, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = h
    return _LIB


def ts_status_string(code: int) -> str:
    return lib().ts_status_string(code).decode()


def ts_last_error() -> str:
    return lib().ts_last_error().decode()


def ts_version() -> int:
    return lib().ts_version()


def ts_set_wait_limit(cycles: int) -> None:
    """Limit of one bounded device wait (SM clocks) for later launches;
    cycles <= 0 restores the default (~1 s)."""
    _check(lib().ts_set_wait_limit(int(cycles)))


def _check(rc: int):
    if rc != TS_OK:
        raise TsError(rc, f"{ts_status_string(rc)}: {ts_last_error()}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# a V cache holds bf16 or fp16 values (fp16: the precision of the P.V product)
_V_DTYPES = (torch.bfloat16, torch.float16)


def _dev(t, dtype, name, shape=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _workspace(nbytes, device, workspace):
    if nbytes == 0:
        return None, 0
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    if workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError(f"workspace too small: {nbytes} bytes needed")
    return workspace, workspace.numel() * workspace.element_size()


def ts_verify_workspace_bytes(T, Hq, Hkv, d, L) -> int:
    return lib().ts_verify_workspace_bytes(T, Hq, Hkv, d, L)


def ts_verify_attention(q, k, v, L, parents, n_imp=0, o=None, lse=None, imp=None,
                        want_lse=True, want_imp=True, workspace=None, status=None, stream=None):
    """Tree verification attention + importance.  q [T,Hq,d] bf16, k
    [Hkv,L_cap,d] bf16, v [Hkv,L_cap,d] bf16 or fp16 (an fp16 V cache skips the
    kernel's per-tile conversion), parents [T] int32.  Returns (o, lse, imp)."""
    T, Hq, d = q.shape
    Hkv, L_cap = k.shape[0], k.shape[1]
    _dev(q, torch.bfloat16, "q")
    _dev(k, torch.bfloat16, "k", (Hkv, L_cap, d))
    _dev(v, _V_DTYPES, "v", (Hkv, L_cap, d))
    _dev(parents, torch.int32, "parents", (T,))
    dev = q.device
    if o is None:
        o = torch.empty((T, Hq, d), dtype=torch.float32, device=dev)
    if lse is None and want_lse:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=dev)
    if imp is None and want_imp:
        imp = torch.empty((Hkv, L), dtype=torch.float32, device=dev)
    ws, nb = _workspace(ts_verify_workspace_bytes(T, Hq, Hkv, d, L), dev, workspace)
    flags = TS_VERIFY_V_FP16 if v.dtype == torch.float16 else 0
    rc = lib().ts_verify_attention_flags(_ptr(q), _ptr(k), _ptr(v), L, L_cap, _ptr(parents), T, Hq,
                                         Hkv, d, n_imp, _ptr(o), _ptr(lse), _ptr(imp), _ptr(ws), nb,
                                         flags, _ptr(status), _stream(stream))
    _check(rc)
    return o, lse, imp


def ts_importance_softmax(q, k, L, lse, n_imp=0, imp=None, status=None, stream=None):
    """Softmax-weighted importance of cache positions [0, L): for each KV head
    the attention probability its positions receive from the group's last
    n_imp tree queries.  q [T,Hq,d] bf16, k [Hkv,L_cap,d] bf16, lse [T,Hq]
    fp32 (from ts_verify_attention).  Returns imp [Hkv, L] fp32."""
    T, Hq, d = q.shape
    Hkv, L_cap = k.shape[0], k.shape[1]
    _dev(q, torch.bfloat16, "q")
    _dev(k, torch.bfloat16, "k", (Hkv, L_cap, d))
    _dev(lse, torch.float32, "lse", (T, Hq))
    if imp is None:
        imp = torch.empty((Hkv, L), dtype=torch.float32, device=q.device)
    rc = lib().ts_importance_softmax(_ptr(q), _ptr(k), _ptr(lse), L, L_cap, T, Hq, Hkv, d, n_imp,
                                     _ptr(imp), _ptr(status), _stream(stream))
    _check(rc)
    return imp


def ts_select_workspace_bytes(Hkv, L) -> int:
    return lib().ts_select_workspace_bytes(Hkv, L)


def ts_partial_kv_select_gather(imp, k, v, L, B, S, R, idx=None, kd=None, vd=None,
                                workspace=None, status=None, stream=None):
    """Top-B + sinks + recent selection and gather.  Returns (idx, kd, vd)."""
    Hkv, L_cap, d = k.shape
    _dev(imp, torch.float32, "imp", (Hkv, L))
    _dev(k, torch.bfloat16, "k")
    _dev(v, _V_DTYPES, "v", (Hkv, L_cap, d))
    N = min(L, S + B + R)
    dev = k.device
    if idx is None:
        idx = torch.empty((Hkv, N), dtype=torch.int32, device=dev)
    if kd is None:
        kd = torch.empty((Hkv, N, d), dtype=torch.bfloat16, device=dev)
    if vd is None:
        vd = torch.empty((Hkv, N, d), dtype=v.dtype, device=dev)
    ws, nb = _workspace(ts_select_workspace_bytes(Hkv, L), dev, workspace)
    n_out = _i64(0)
    rc = lib().ts_partial_kv_select_gather(_ptr(imp), _ptr(k), _ptr(v), L, L_cap, Hkv, d, B, S, R,
                                           _ptr(idx), _ptr(kd), _ptr(vd), ctypes.byref(n_out),
                                           _ptr(ws), nb, _ptr(status), _stream(stream))
    _check(rc)
    assert n_out.value == N
    return idx, kd, vd


def ts_partial_kv_select_gather_noalloc(imp, k, v, L, B, S, R, idx, kd, vd, status=None,
                                        stream=None):
    """Selection + gather without a workspace, for callers that may not
    allocate device memory: the library keeps its scratch in a fixed device
    array (see the C header for the size limit and the sharing rules).  The
    outputs idx [Hkv,N] int32, kd/vd [Hkv,N,d] bf16 are the caller's."""
    Hkv, L_cap, d = k.shape
    _dev(imp, torch.float32, "imp", (Hkv, L))
    _dev(k, torch.bfloat16, "k")
    _dev(v, _V_DTYPES, "v", (Hkv, L_cap, d))
    N = min(L, S + B + R)
    _dev(idx, torch.int32, "idx", (Hkv, N))
    _dev(kd, torch.bfloat16, "kd", (Hkv, N, d))
    _dev(vd, v.dtype, "vd", (Hkv, N, d))
    n_out = _i64(0)
    rc = lib().ts_partial_kv_select_gather_noalloc(_ptr(imp), _ptr(k), _ptr(v), L, L_cap, Hkv, d,
                                                   B, S, R, _ptr(idx), _ptr(kd), _ptr(vd),
                                                   ctypes.byref(n_out), _ptr(status),
                                                   _stream(stream))
    _check(rc)
    return idx, kd, vd


def ts_select_batched_workspace_bytes(n_layers, Hkv, L) -> int:
    return lib().ts_select_batched_workspace_bytes(n_layers, Hkv, L)


def layer_pointer_table(imps, ks, vs, idxs, kds, vds):
    """Device table [6, n_layers] of the per-layer tensor addresses the batched
    selection reads (build it once and reuse it while the tensors live)."""
    rows = [imps, ks, vs, idxs, kds, vds]
    n = len(imps)
    if any(len(r) != n for r in rows):
        raise ValueError("every per-layer list must have n_layers entries")
    host = torch.tensor([[t.data_ptr() for t in r] for r in rows], dtype=torch.int64)
    return host.to(imps[0].device)


def ts_partial_kv_select_gather_batched(imps, ks, vs, L, B, S, R, idxs, kds, vds, table=None,
                                        workspace=None, status=None, stream=None):
    """Selection + gather for several layers in one pipeline of launches.
    Lists of per-layer tensors with the single-layer shapes."""
    n = len(imps)
    Hkv, L_cap, d = ks[0].shape
    for i in range(n):
        _dev(imps[i], torch.float32, "imp", (Hkv, L))
        _dev(ks[i], torch.bfloat16, "k", (Hkv, L_cap, d))
        _dev(vs[i], _V_DTYPES, "v", (Hkv, L_cap, d))
    if table is None:
        table = layer_pointer_table(imps, ks, vs, idxs, kds, vds)
    ws, nb = _workspace(ts_select_batched_workspace_bytes(n, Hkv, L), ks[0].device, workspace)
    n_out = _i64(0)
    row = lambda r: ctypes.c_void_p(table[r].data_ptr())  # noqa: E731
    rc = lib().ts_partial_kv_select_gather_batched(n, row(0), row(1), row(2), L, L_cap, Hkv, d, B,
                                                   S, R, row(3), row(4), row(5), ctypes.byref(n_out),
                                                   _ptr(ws), nb, _ptr(status), _stream(stream))
    _check(rc)
    return idxs, kds, vds


def ts_refresh_workspace_bytes(n_layers, Hkv, L, N_cap) -> int:
    return lib().ts_refresh_workspace_bytes(n_layers, Hkv, L, N_cap)


def ts_partial_kv_refresh_incremental(imp, k, v, L, B, S, R, idx, kd, vd, N_prev, n_written=None,
                                      workspace=None, status=None, stream=None):
    """Update one layer's compact cache in place: slots whose position stays
    selected keep their row, newly selected positions fill the freed slots
    (then the new ones while the cache grows).  idx [Hkv, N_cap] int32,
    kd/vd [Hkv, N_cap, d] bf16 hold the previous state in slots [0, N_prev).
    Returns N_new (the slots now valid)."""
    Hkv, L_cap, d = k.shape
    _dev(imp, torch.float32, "imp", (Hkv, L))
    _dev(k, torch.bfloat16, "k")
    _dev(v, _V_DTYPES, "v", (Hkv, L_cap, d))
    N_cap = idx.shape[1]
    _dev(idx, torch.int32, "idx", (Hkv, N_cap))
    _dev(kd, torch.bfloat16, "kd", (Hkv, N_cap, d))
    _dev(vd, v.dtype, "vd", (Hkv, N_cap, d))
    ws, nb = _workspace(ts_refresh_workspace_bytes(1, Hkv, L, N_cap), k.device, workspace)
    n_out = _i64(0)
    rc = lib().ts_partial_kv_refresh_incremental(_ptr(imp), _ptr(k), _ptr(v), L, L_cap, Hkv, d, B,
                                                 S, R, _ptr(idx), _ptr(kd), _ptr(vd), N_cap,
                                                 N_prev, ctypes.byref(n_out), _ptr(n_written),
                                                 _ptr(ws), nb, _ptr(status), _stream(stream))
    _check(rc)
    return n_out.value


def ts_partial_kv_refresh_incremental_batched(imps, ks, vs, L, B, S, R, idxs, kds, vds, N_prev,
                                              table=None, n_written=None, workspace=None,
                                              status=None, stream=None):
    """The incremental refresh of several layers in one pipeline of launches
    (per-layer lists with the single-layer shapes).  Returns N_new."""
    n = len(imps)
    Hkv, L_cap, d = ks[0].shape
    N_cap = idxs[0].shape[1]
    for i in range(n):
        _dev(imps[i], torch.float32, "imp", (Hkv, L))
        _dev(ks[i], torch.bfloat16, "k", (Hkv, L_cap, d))
        _dev(vs[i], _V_DTYPES, "v", (Hkv, L_cap, d))
        _dev(idxs[i], torch.int32, "idx", (Hkv, N_cap))
        _dev(kds[i], torch.bfloat16, "kd", (Hkv, N_cap, d))
        _dev(vds[i], vs[i].dtype, "vd", (Hkv, N_cap, d))
    if table is None:
        table = layer_pointer_table(imps, ks, vs, idxs, kds, vds)
    ws, nb = _workspace(ts_refresh_workspace_bytes(n, Hkv, L, N_cap), ks[0].device, workspace)
    n_out = _i64(0)
    row = lambda r: ctypes.c_void_p(table[r].data_ptr())  # noqa: E731
    rc = lib().ts_partial_kv_refresh_incremental_batched(
        n, row(0), row(1), row(2), L, L_cap, Hkv, d, B, S, R, row(3), row(4), row(5), N_cap, N_prev,
        ctypes.byref(n_out), _ptr(n_written), _ptr(ws), nb, _ptr(status), _stream(stream))
    _check(rc)
    return n_out.value


def ts_sample_workspace_bytes(T, V) -> int:
    return lib().ts_sample_workspace_bytes(T, V)


TS_PENALTY_CTRL_LITERAL = 1


def ts_penalized_sample_accept(logits, tree_tokens, parents, prior, W, penalty, temperature,
                               top_p, min_p, uniforms, sampled=None, path=None, n_path=None,
                               bonus=None, workspace=None, status=None, stream=None,
                               literal=False):
    """Penalised top-p/min-p draw at every node + exact-match acceptance
    (literal=True: the literal CTRL penalty, every windowed logit divided).
    Returns (sampled [T], path [T], n_path [1], bonus [1]) device int32."""
    T, V = logits.shape
    _dev(logits, torch.float32, "logits")
    _dev(tree_tokens, torch.int32, "tree_tokens", (T,))
    _dev(parents, torch.int32, "parents", (T,))
    _dev(prior, torch.int32, "prior")
    _dev(uniforms, torch.float32, "uniforms", (T,))
    dev = logits.device
    mk = lambda n: torch.empty(n, dtype=torch.int32, device=dev)  # noqa: E731
    sampled = mk(T) if sampled is None else sampled
    path = mk(T) if path is None else path
    n_path = mk(1) if n_path is None else n_path
    bonus = mk(1) if bonus is None else bonus
    ws, nb = _workspace(ts_sample_workspace_bytes(T, V), dev, workspace)
    rc = lib().ts_penalized_sample_accept_flags(
        _ptr(logits), _ptr(tree_tokens), _ptr(parents), T, _ptr(prior), prior.numel(), W, V,
        penalty, temperature, top_p, min_p, _ptr(uniforms), _ptr(sampled), _ptr(path),
        _ptr(n_path), _ptr(bonus), _ptr(ws), nb, TS_PENALTY_CTRL_LITERAL if literal else 0,
        _ptr(status), _stream(stream))
    _check(rc)
    return sampled, path, n_path, bonus


def ts_penalized_sample_accept_eta(logits, tree_tokens, parents, prior, W, penalty, temperature,
                                   eta_epsilon, eta_alpha, uniforms, sampled=None, path=None,
                                   n_path=None, bonus=None, workspace=None, status=None,
                                   stream=None):
    """Penalised eta-sampling draw at every node + exact-match acceptance.
    Returns (sampled [T], path [T], n_path [1], bonus [1]) device int32."""
    T, V = logits.shape
    _dev(logits, torch.float32, "logits")
    _dev(tree_tokens, torch.int32, "tree_tokens", (T,))
    _dev(parents, torch.int32, "parents", (T,))
    _dev(prior, torch.int32, "prior")
    _dev(uniforms, torch.float32, "uniforms", (T,))
    dev = logits.device
    mk = lambda n: torch.empty(n, dtype=torch.int32, device=dev)  # noqa: E731
    sampled = mk(T) if sampled is None else sampled
    path = mk(T) if path is None else path
    n_path = mk(1) if n_path is None else n_path
    bonus = mk(1) if bonus is None else bonus
    ws, nb = _workspace(ts_sample_workspace_bytes(T, V), dev, workspace)
    rc = lib().ts_penalized_sample_accept_eta(_ptr(logits), _ptr(tree_tokens), _ptr(parents), T,
                                              _ptr(prior), prior.numel(), W, V, penalty,
                                              temperature, eta_epsilon, eta_alpha, _ptr(uniforms),
                                              _ptr(sampled), _ptr(path), _ptr(n_path), _ptr(bonus),
                                              _ptr(ws), nb, _ptr(status), _stream(stream))
    _check(rc)
    return sampled, path, n_path, bonus


def ts_kv_commit(k, v, L, T, path, n_path, status=None, stream=None):
    """Move the accepted tree rows L+path[t] to L+t (in place)."""
    Hkv, L_cap, d = k.shape
    _dev(k, torch.bfloat16, "k")
    _dev(v, _V_DTYPES, "v", (Hkv, L_cap, d))
    rc = lib().ts_kv_commit(_ptr(k), _ptr(v), L, L_cap, Hkv, d, T, _ptr(path), _ptr(n_path),
                            _ptr(status), _stream(stream))
    _check(rc)


def commit_pointer_table(ks, vs):
    """Device table [2, n_layers] of the per-layer K and V cache addresses the
    batched commit reads (build it once and reuse it while the caches live)."""
    if len(ks) != len(vs):
        raise ValueError("ks and vs must have one entry per layer")
    host = torch.tensor([[t.data_ptr() for t in ks], [t.data_ptr() for t in vs]],
                        dtype=torch.int64)
    return host.to(ks[0].device)


def ts_kv_commit_batched(ks, vs, L, T, path, n_path, table=None, status=None, stream=None):
    """ts_kv_commit for every layer in one launch (lists of per-layer caches
    [Hkv, L_cap, d] bf16)."""
    Hkv, L_cap, d = ks[0].shape
    for x, y in zip(ks, vs):
        _dev(x, torch.bfloat16, "k", (Hkv, L_cap, d))
        _dev(y, _V_DTYPES, "v", (Hkv, L_cap, d))
    if table is None:
        table = commit_pointer_table(ks, vs)
    rc = lib().ts_kv_commit_batched(len(ks), ctypes.c_void_p(table[0].data_ptr()),
                                    ctypes.c_void_p(table[1].data_ptr()), L, L_cap, Hkv, d, T,
                                    _ptr(path), _ptr(n_path), _ptr(status), _stream(stream))
    _check(rc)


def ts_kv_append_batched(ks, vs, k_rows, v_rows, L, table=None, status=None, stream=None):
    """Write the tree's K/V rows [L, L+T) into every layer's cache in one
    launch.  k_rows, v_rows [n_layers, Hkv, T, d] bf16 (contiguous); fp16 V
    caches receive the V rows rounded to fp16."""
    Hkv, L_cap, d = ks[0].shape
    n, T = len(ks), k_rows.shape[2]
    _dev(k_rows, torch.bfloat16, "k_rows", (n, Hkv, T, d))
    _dev(v_rows, torch.bfloat16, "v_rows", (n, Hkv, T, d))
    for x, y in zip(ks, vs):
        _dev(x, torch.bfloat16, "k", (Hkv, L_cap, d))
        _dev(y, _V_DTYPES, "v", (Hkv, L_cap, d))
    if table is None:
        table = commit_pointer_table(ks, vs)
    if len({y.dtype for y in vs}) != 1:
        raise TypeError("every layer's V cache must have the same dtype")
    flags = TS_KV_V_FP16 if vs[0].dtype == torch.float16 else 0
    rc = lib().ts_kv_append_batched_flags(n, ctypes.c_void_p(table[0].data_ptr()),
                                          ctypes.c_void_p(table[1].data_ptr()), _ptr(k_rows),
                                          _ptr(v_rows), L, L_cap, Hkv, d, T, flags, _ptr(status),
                                          _stream(stream))
    _check(rc)


def ts_reject_workspace_bytes(V) -> int:
    return lib().ts_reject_workspace_bytes(V)


def ts_rejection_sample_accept(logits, q, tree_tokens, parents, prior, W, penalty, temperature,
                               top_p, min_p, u_accept, u_draw, path=None, n_path=None, bonus=None,
                               workspace=None, status=None, stream=None, literal=False):
    """Speculative-sampling acceptance over the draft tree: children tried in
    index order against the draft distributions q [T, V].  Returns
    (path [T], n_path [1], bonus [1]) device int32."""
    T, V = logits.shape
    _dev(logits, torch.float32, "logits")
    _dev(q, torch.float32, "q", (T, V))
    _dev(tree_tokens, torch.int32, "tree_tokens", (T,))
    _dev(parents, torch.int32, "parents", (T,))
    _dev(prior, torch.int32, "prior")
    _dev(u_accept, torch.float32, "u_accept", (T,))
    _dev(u_draw, torch.float32, "u_draw", (T,))
    dev = logits.device
    mk = lambda n: torch.empty(n, dtype=torch.int32, device=dev)  # noqa: E731
    path = mk(T) if path is None else path
    n_path = mk(1) if n_path is None else n_path
    bonus = mk(1) if bonus is None else bonus
    ws, nb = _workspace(ts_reject_workspace_bytes(V), dev, workspace)
    rc = lib().ts_rejection_sample_accept(
        _ptr(logits), _ptr(q), _ptr(tree_tokens), _ptr(parents), T, _ptr(prior), prior.numel(), W,
        V, penalty, temperature, top_p, min_p, _ptr(u_accept), _ptr(u_draw), _ptr(path),
        _ptr(n_path), _ptr(bonus), _ptr(ws), nb, TS_PENALTY_CTRL_LITERAL if literal else 0,
        _ptr(status), _stream(stream))
    _check(rc)
    return path, n_path, bonus


def ts_ngram_table_bytes(V, cap) -> int:
    return lib().ts_ngram_table_bytes(V, cap)


def ngram_table(V, cap, device="cuda"):
    """A zeroed (empty) 4-gram table: int32 device buffer."""
    nb = ts_ngram_table_bytes(V, cap)
    if nb == 0:
        raise ValueError(f"unsupported table shape V={V}, cap={cap}")
    return torch.zeros(nb // 4, dtype=torch.int32, device=device)


def ts_ngram_insert(table, V, cap, tokens, start, n_tokens=None, status=None, stream=None):
    """Insert the 4-grams ending at positions start .. n_tokens-1 of tokens."""
    _dev(table, torch.int32, "table")
    _dev(tokens, torch.int32, "tokens")
    n = tokens.numel() if n_tokens is None else n_tokens
    _check(lib().ts_ngram_insert(_ptr(table), V, cap, _ptr(tokens), n, start, _ptr(status),
                                 _stream(stream)))


def ts_ngram_build_tree(table, V, cap, root_token, head_topk, k, rand_keys, T_max,
                        parents=None, tokens=None, n_nodes=None, status=None, stream=None):
    """Draft tree from the heads' candidates [n_heads, head_k] and the root's
    retrieved continuations.  Returns (parents [T_max], tokens [T_max],
    n_nodes [1]) device int32; entries past n_nodes are untouched."""
    _dev(table, torch.int32, "table")
    _dev(root_token, torch.int32, "root_token", (1,))
    _dev(head_topk, torch.int32, "head_topk")
    _dev(rand_keys, torch.int32, "rand_keys", (cap,))
    n_heads, head_k = head_topk.shape
    dev = table.device
    if parents is None:
        parents = torch.full((T_max,), -2, dtype=torch.int32, device=dev)
    if tokens is None:
        tokens = torch.full((T_max,), -2, dtype=torch.int32, device=dev)
    if n_nodes is None:
        n_nodes = torch.zeros(1, dtype=torch.int32, device=dev)
    _check(lib().ts_ngram_build_tree(_ptr(table), V, cap, _ptr(root_token), _ptr(head_topk),
                                     n_heads, head_k, k, _ptr(rand_keys), T_max, _ptr(parents),
                                     _ptr(tokens), _ptr(n_nodes), _ptr(status), _stream(stream)))
    return parents, tokens, n_nodes


# ---------------------------------------------------------------------------
# the paged cache
# ---------------------------------------------------------------------------
TS_PAGED_FP16 = 1
TS_ROPE_INTERLEAVED = 2
_ROPE_SCALINGS = {"plain": 0, "linear": 1, "base": 2, "wavelength": 3, "ramp": 4}


def ts_rope_frequencies(rot_dim, base=10000.0, scaling="plain", factor=1.0, original_len=0.0,
                        low=1.0, high=32.0, device="cuda"):
    """Rotary frequencies [rot_dim / 2] fp64 (radians a position) on `device`
    and the factor rotated rows carry, for scaling "plain", "linear", "base",
    "wavelength" or "ramp" (formulas in the C header).  Make it once a model."""
    if scaling not in _ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_ROPE_SCALINGS)}")
    host = (_f64 * max(rot_dim // 2, 1))()
    scale = _f32(0.0)
    _check(lib().ts_rope_frequencies(rot_dim, base, _ROPE_SCALINGS[scaling], factor, original_len,
                                     low, high, host, ctypes.byref(scale)))
    return torch.tensor(list(host), dtype=torch.float64).to(device), scale.value


# the current stream's handle without building a Stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_raw_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_PAGED_DTYPES = (torch.bfloat16, torch.float16)


def _need(t, dtype, shape, dev, name):
    """The address of tensor `t` after its checks (None stays None)."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _dev(t, dtype, name, shape)
    raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")


def _paged_q(q):
    """(n, Hq, d, type, device index, flags) of a call's queries."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise TypeError("q must be a CUDA tensor")
    dt = q.dtype
    if dt not in _PAGED_DTYPES:
        raise TypeError(f"q must be {_PAGED_DTYPES}, got {dt}")
    if q.dim() != 3:
        raise ValueError(f"q has shape {tuple(q.shape)}, expected (n, Hq, d)")
    n, Hq, d = q.shape
    return n, Hq, d, dt, q.get_device(), TS_PAGED_FP16 if dt is torch.float16 else 0


def _paged_batch(cu_q, seq_lens, page_table, dev):
    """(n_seq, max_pages, the three addresses) of a call's batch."""
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be a tensor [n_seq, pages]")
    n_seq, max_pages = shape = page_table.shape
    i32 = torch.int32
    return (n_seq, max_pages, _need(cu_q, i32, (n_seq + 1,), dev, "cu_q"),
            _need(seq_lens, i32, (n_seq,), dev, "seq_lens"),
            _need(page_table, i32, shape, dev, "page_table"))


def _alloc(shape, dtype, device, stream):
    """Memory of a call on `stream` (None: the current one), from that stream's own
    blocks: what was freed on the current stream may still be read by kernels that
    are queued there, and nothing holds `stream` back until they are done."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _alloc_like(t, dtype, stream):
    """_alloc of t's shape, dense (half of torch.empty's host time)."""
    if stream is None:
        return torch.empty_like(t, dtype=dtype, memory_format=torch.contiguous_format)
    with torch.cuda.stream(stream):
        return torch.empty_like(t, dtype=dtype, memory_format=torch.contiguous_format)


def _paged_call(fn, dev, stream, outputs, args):
    """One library call with the tensors' device current.  `outputs`: what the binding
    allocated for the caller, who may read it on the current stream (after waiting for
    `stream`): once freed, it is not used again before those readers are done."""
    if _raw_device() == dev:
        rc = fn(*args, _raw_stream(dev) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(dev) if stream is None else stream.cuda_stream)
    if stream is not None and outputs:
        here = torch.cuda.current_stream(dev)
        for t in outputs:
            t.record_stream(here)
    if rc:
        _check(rc)


def _given_workspace(workspace, nbytes, dev):
    """(address, bytes) of a caller's workspace."""
    if workspace.get_device() != dev:
        raise ValueError(f"workspace is on {workspace.device}, q is on cuda:{dev}")
    if not workspace.is_contiguous():      # an expanded one has fewer bytes than its shape says
        raise ValueError("workspace must be contiguous")
    have = workspace.numel() * workspace.element_size()
    if have < nbytes:
        raise ValueError(f"workspace too small: {nbytes} bytes needed")
    return workspace.data_ptr(), have


def _new_rows(t, name, n, heads, d, dt, dev):
    """(address, token stride) of a strided [n, heads, d] input of the append."""
    try:
        if t.dtype is dt and t.shape == (n, heads, d) and t.get_device() == dev:
            row, head, one = t.stride()
            if n == 0 or (one == 1 and (head == d or heads == 1)):
                # a single token's stride is never walked; a view may report any
                return t.data_ptr(), row if n > 1 else heads * d
            raise ValueError(f"{name}: the heads of a token must be dense")
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype is not dt:
        raise TypeError(f"{name} must be {dt}, got {t.dtype}")
    raise ValueError(f"{name} has shape {tuple(t.shape)} on {t.device}, expected {(n, heads, d)} "
                     f"on cuda:{dev}")


def ts_paged_rope_append(q, k, v, cu_q, seq_lens, page_table, k_pages, v_pages, freqs,
                         positions=None, rope_scale=1.0, interleaved=False, key_min=None,
                         key_max=None, q_out=None, status=None, stream=None):
    """Rotate new queries and keys and write keys and values into a paged
    cache.  q [n, Hq, d], k, v [n, Hkv, d] bf16 or fp16 (any token stride that
    is a multiple of 8 elements; the heads dense), k_pages, v_pages [n_pages,
    Hkv, page_size, d], freqs [rot_dim / 2] fp64 (see ts_rope_frequencies).
    key_min, key_max [n_pages, Hkv, d]: the pages' key bounds, updated.
    Returns the rotated queries [n, Hq, d]."""
    n, Hq, d, dt, dev, flags = _paged_q(q)
    n_pages, Hkv, ps, _ = pool = k_pages.shape
    qp, q_stride = _new_rows(q, "q", n, Hq, d, dt, dev)
    kr, k_stride = _new_rows(k, "k", n, Hkv, d, dt, dev)
    vr, v_stride = _new_rows(v, "v", n, Hkv, d, dt, dev)
    if interleaved:
        flags |= TS_ROPE_INTERLEAVED
    n_seq, max_pages, cu, lens, table = _paged_batch(cu_q, seq_lens, page_table, dev)
    if pool[3] != d:
        raise ValueError(f"k_pages has shape {tuple(pool)}, expected head dim {d}")
    kp = _need(k_pages, dt, pool, dev, "k_pages")
    vp = _need(v_pages, dt, pool, dev, "v_pages")
    fr = _need(freqs, torch.float64, freqs.shape, dev, "freqs")
    pos = mn = mx = st = None
    if positions is not None:
        pos = _need(positions, torch.int32, (n,), dev, "positions")
    if key_min is not None:
        mn = _need(key_min, dt, (n_pages, Hkv, d), dev, "key_min")
    if key_max is not None:
        mx = _need(key_max, dt, (n_pages, Hkv, d), dev, "key_max")
    if status is not None:
        st = _need(status, torch.int32, status.shape, dev, "status")
    outputs = ()
    if q_out is None:
        q_out = _alloc((n, Hq, d), dt, q.device, stream)
        out, outputs = q_out.data_ptr(), (q_out,)
    else:
        out = _need(q_out, dt, (n, Hq, d), dev, "q_out")
    _paged_call(lib().ts_paged_rope_append, dev, stream, outputs, (
        qp, kr, vr, q_stride, k_stride, v_stride, n, Hq, Hkv, d, cu, lens, n_seq, table, max_pages,
        ps, n_pages, pos, fr, 2 * freqs.numel(), rope_scale, out, kp, vp, mn, mx, flags, st))
    return q_out


@functools.lru_cache(maxsize=4096)
def ts_paged_attention_workspace_bytes(n, n_seq, Hq, Hkv, d, max_pages, page_size, max_q,
                                       max_kv=0) -> int:
    return lib().ts_paged_attention_workspace_bytes(n, n_seq, Hq, Hkv, d, max_pages, page_size,
                                                    max_q, max_kv)


def _attend(fn, q, pools, o, lse, want_lse, nbytes, workspace, status, stream, head):
    """Outputs, workspace and launch that the two attention calls share; head: the
    arguments in front of (o, lse, workspace, bytes, flags, status, stream)."""
    n, Hq, d, dt, dev, flags = pools
    outputs = []
    if o is None:
        o = _alloc_like(q, dt, stream)
        out = o.data_ptr()
        outputs.append(o)
    else:
        out = _need(o, dt, (n, Hq, d), dev, "o")
    ls = None
    if lse is not None:
        ls = _need(lse, torch.float32, (n, Hq), dev, "lse")
    elif want_lse:
        lse = _alloc((n, Hq), torch.float32, q.device, stream)
        ls = lse.data_ptr()
        outputs.append(lse)
    ws, nb = None, nbytes
    if workspace is not None:
        ws, nb = _given_workspace(workspace, nbytes, dev)
    elif nbytes:
        scratch = _alloc(nbytes, torch.uint8, q.device, stream)
        ws = scratch.data_ptr()
    st = None if status is None else _need(status, torch.int32, status.shape, dev, "status")
    _paged_call(fn, dev, stream, outputs, head + (out, ls, ws, nb, flags, st))
    return o, lse


def ts_paged_attention(q, k_pages, v_pages, cu_q, seq_lens, page_table, max_q, max_kv=0, o=None,
                       lse=None, want_lse=True, workspace=None, status=None, stream=None):
    """Causal attention of new tokens (prompts, chunks, single tokens) over a
    paged cache that holds their rows already.  q [n, Hq, d] bf16 or fp16,
    k_pages, v_pages [n_pages, Hkv, page_size, d]; max_q bounds the sequences'
    new tokens, max_kv (0: the page table's width) is the longest sequence as
    far as the host knows.  Returns (o [n, Hq, d], lse [n, Hq] fp32)."""
    n, Hq, d, dt, dev, _ = what = _paged_q(q)
    n_pages, Hkv, ps, _ = k_pages.shape
    pool = (n_pages, Hkv, ps, d)
    n_seq, max_pages, cu, lens, table = _paged_batch(cu_q, seq_lens, page_table, dev)
    return _attend(
        lib().ts_paged_attention, q, what, o, lse, want_lse,
        ts_paged_attention_workspace_bytes(n, n_seq, Hq, Hkv, d, max_pages, ps, max_q, max_kv),
        workspace, status, stream,
        (_need(q, dt, (n, Hq, d), dev, "q"), _need(k_pages, dt, pool, dev, "k_pages"),
         _need(v_pages, dt, pool, dev, "v_pages"), n, Hq, Hkv, d, cu, lens, n_seq, table,
         max_pages, ps, n_pages, max_q, max_kv))


@functools.lru_cache(maxsize=4096)
def ts_paged_select_workspace_bytes(n, Hkv, max_pages) -> int:
    return lib().ts_paged_select_workspace_bytes(n, Hkv, max_pages)


def ts_paged_select_pages(q, key_min, key_max, cu_q, seq_lens, page_table, page_size, n_top,
                          n_sink, n_recent, pages=None, counts=None, workspace=None, status=None,
                          stream=None):
    """Choose each new token's pages by the bound their key bounds put on its
    scores: the first n_sink, the last n_recent and the n_top best between.
    q [n, Hq, d] rotated, key_min, key_max [n_pages, Hkv, d].  Returns
    (pages [n, Hkv, n_sink + n_top + n_recent], counts [n, Hkv]) int32:
    ascending positions in the page table's row, -1 behind the last."""
    n, Hq, d, dt, dev, flags = _paged_q(q)
    n_pages, Hkv, _ = key_min.shape
    bounds = (n_pages, Hkv, d)
    n_seq, max_pages, cu, lens, table = _paged_batch(cu_q, seq_lens, page_table, dev)
    qp = _need(q, dt, (n, Hq, d), dev, "q")
    mn = _need(key_min, dt, bounds, dev, "key_min")
    mx = _need(key_max, dt, bounds, dev, "key_max")
    n_sel = max(n_sink + n_top + n_recent, 0)
    outputs = []
    if pages is None:
        pages = _alloc((n, Hkv, n_sel), torch.int32, q.device, stream)
        pg = pages.data_ptr()
        outputs.append(pages)
    else:
        pg = _need(pages, torch.int32, (n, Hkv, n_sel), dev, "pages")
    if counts is None:
        counts = _alloc((n, Hkv), torch.int32, q.device, stream)
        ct = counts.data_ptr()
        outputs.append(counts)
    else:
        ct = _need(counts, torch.int32, (n, Hkv), dev, "counts")
    nb = ts_paged_select_workspace_bytes(n, Hkv, max_pages)
    ws = None
    if workspace is not None:
        ws, nb = _given_workspace(workspace, nb, dev)
    elif nb:
        scratch = _alloc(nb, torch.uint8, q.device, stream)
        ws = scratch.data_ptr()
    st = None if status is None else _need(status, torch.int32, status.shape, dev, "status")
    _paged_call(lib().ts_paged_select_pages, dev, stream, outputs, (
        qp, mn, mx, n, Hq, Hkv, d, cu, lens, n_seq, table, max_pages, page_size, n_pages, n_top,
        n_sink, n_recent, pg, ct, ws, nb, flags, st))
    return pages, counts


@functools.lru_cache(maxsize=4096)
def ts_paged_selected_workspace_bytes(n, Hq, Hkv, d, page_size, n_sel) -> int:
    return lib().ts_paged_selected_workspace_bytes(n, Hq, Hkv, d, page_size, n_sel)


def ts_paged_attention_selected(q, k_pages, v_pages, cu_q, seq_lens, page_table, pages, counts,
                                o=None, lse=None, want_lse=True, workspace=None, status=None,
                                stream=None):
    """ts_paged_attention over each token's chosen pages (pages [n, Hkv,
    n_sel], counts [n, Hkv] int32, as ts_paged_select_pages returns them).
    Returns (o [n, Hq, d], lse [n, Hq] fp32)."""
    n, Hq, d, dt, dev, _ = what = _paged_q(q)
    n_pages, Hkv, ps, _ = k_pages.shape
    pool = (n_pages, Hkv, ps, d)
    n_seq, max_pages, cu, lens, table = _paged_batch(cu_q, seq_lens, page_table, dev)
    n_sel = pages.shape[-1]
    return _attend(
        lib().ts_paged_attention_selected, q, what, o, lse, want_lse,
        ts_paged_selected_workspace_bytes(n, Hq, Hkv, d, ps, n_sel), workspace, status, stream,
        (_need(q, dt, (n, Hq, d), dev, "q"), _need(k_pages, dt, pool, dev, "k_pages"),
         _need(v_pages, dt, pool, dev, "v_pages"), n, Hq, Hkv, d, cu, lens, n_seq, table,
         max_pages, ps, n_pages, _need(pages, torch.int32, (n, Hkv, n_sel), dev, "pages"),
         _need(counts, torch.int32, (n, Hkv), dev, "counts"), n_sel))


@functools.lru_cache(maxsize=4096)
def ts_paged_tree_attention_workspace_bytes(n, n_seq, Hq, Hkv, d, max_pages, page_size, max_q,
                                            max_kv=0) -> int:
    return lib().ts_paged_tree_attention_workspace_bytes(n, n_seq, Hq, Hkv, d, max_pages,
                                                         page_size, max_q, max_kv)


def ts_paged_tree_attention(q, k_pages, v_pages, cu_q, seq_lens, page_table, parents, max_q,
                            max_kv=0, o=None, lse=None, want_lse=True, workspace=None, status=None,
                            stream=None):
    """Attention of the nodes of several streams' draft trees over a paged
    cache that holds their rows already: each node sees the rows in front of
    its tree, its ancestors' and its own.  q [n, Hq, d] bf16 or fp16, parents
    [n] int32 (within each tree, -1 of its first node), max_q (at most 64)
    bounds the trees' nodes; the rest as in ts_paged_attention.  Returns
    (o [n, Hq, d], lse [n, Hq] fp32)."""
    n, Hq, d, dt, dev, _ = what = _paged_q(q)
    n_pages, Hkv, ps, _ = k_pages.shape
    pool = (n_pages, Hkv, ps, d)
    n_seq, max_pages, cu, lens, table = _paged_batch(cu_q, seq_lens, page_table, dev)
    return _attend(
        lib().ts_paged_tree_attention, q, what, o, lse, want_lse,
        ts_paged_tree_attention_workspace_bytes(n, n_seq, Hq, Hkv, d, max_pages, ps, max_q,
                                                max_kv),
        workspace, status, stream,
        (_need(q, dt, (n, Hq, d), dev, "q"), _need(k_pages, dt, pool, dev, "k_pages"),
         _need(v_pages, dt, pool, dev, "v_pages"), n, Hq, Hkv, d, cu, lens, n_seq, table,
         max_pages, ps, n_pages, _need(parents, torch.int32, (n,), dev, "parents"), max_q, max_kv))


def _layers(x, name, dt, shape, dev):
    """The number of layers of per-layer tensors of one shape: a list of them, or
    one tensor with the layers in front."""
    if isinstance(x, torch.Tensor):
        at = _need(x, dt, (x.shape[0], *shape), dev, name)
        n = x.shape[0]
    else:
        at = 0
        for t in x:
            at |= _need(t, dt, shape, dev, name)
        n = len(x)
    if at & 15:                            # the kernel reads the addresses from a table
        raise ValueError(f"{name}: a layer is not 16-byte aligned")
    return n


def ts_paged_kv_commit(k_pages, v_pages, cu_q, seq_lens, page_table, path, n_path, key_min=None,
                       key_max=None, new_lens=None, table=None, bounds_table=None, status=None,
                       stream=None):
    """Move the accepted rows of several streams' draft trees to the end of
    their sequences, in every layer's pages and in place.  k_pages, v_pages: a
    list of the layers' pools [n_pages, Hkv, page_size, d], or one tensor
    [n_layers, n_pages, Hkv, page_size, d]; path [n_seq, T], n_path [n_seq]
    int32 (node indices, root first); key_min, key_max: the layers' key bounds
    likewise.  table = commit_pointer_table(k_pages, v_pages), bounds_table =
    commit_pointer_table(key_min, key_max): make them once and reuse them while
    the pools live.  Returns the new lengths [n_seq] int32."""
    first = k_pages if isinstance(k_pages, torch.Tensor) else k_pages[0] if len(k_pages) else None
    if first is None or first.shape[0] == 0:
        raise ValueError("at least one layer is needed")
    if not isinstance(first, torch.Tensor) or not first.is_cuda:
        raise TypeError("k_pages must be CUDA tensors")
    dt, dev, pool = first.dtype, first.get_device(), first.shape[-4:]
    if dt not in _PAGED_DTYPES:
        raise TypeError(f"k_pages must be {_PAGED_DTYPES}, got {dt}")
    if len(pool) != 4:
        raise ValueError("a layer's pool has shape [n_pages, Hkv, page_size, d]")
    n_pages, Hkv, ps, d = pool
    n_layers = _layers(k_pages, "k_pages", dt, pool, dev)
    if _layers(v_pages, "v_pages", dt, pool, dev) != n_layers:
        raise ValueError("k_pages and v_pages must have one entry per layer")
    n_seq, max_pages, cu, lens, pt = _paged_batch(cu_q, seq_lens, page_table, dev)
    i32 = torch.int32
    T = path.shape[-1]
    made = []
    if table is None:
        table = commit_pointer_table(k_pages, v_pages)
        made.append(table)
    at = _need(table, torch.int64, (2, n_layers), dev, "table")
    mn = mx = st = None
    if key_min is not None or key_max is not None:
        if key_min is None or key_max is None:
            raise ValueError("key_min and key_max go together")
        bounds = (n_pages, Hkv, d)
        if _layers(key_min, "key_min", dt, bounds, dev) != n_layers or \
                _layers(key_max, "key_max", dt, bounds, dev) != n_layers:
            raise ValueError("key_min and key_max must have one entry per layer")
        if bounds_table is None:
            bounds_table = commit_pointer_table(key_min, key_max)
            made.append(bounds_table)
        mn = _need(bounds_table, torch.int64, (2, n_layers), dev, "bounds_table")
        mx = mn + 8 * n_layers
    outputs = ()
    if new_lens is None:
        new_lens = _alloc_like(seq_lens, i32, stream)
        new, outputs = new_lens.data_ptr(), (new_lens,)
    else:
        new = _need(new_lens, i32, (n_seq,), dev, "new_lens")
    if status is not None:
        st = _need(status, i32, status.shape, dev, "status")
    _paged_call(lib().ts_paged_kv_commit, dev, stream, outputs, (
        n_layers, at, at + 8 * n_layers, Hkv, d, cu, lens, n_seq, pt, max_pages, ps, n_pages,
        _need(path, i32, (n_seq, T), dev, "path"), T, _need(n_path, i32, (n_seq,), dev, "n_path"),
        mn, mx, new, TS_PAGED_FP16 if dt is torch.float16 else 0, st))
    if stream is not None:
        for t in made:                     # from the current stream's memory, read on `stream`
            t.record_stream(stream)
    return new_lens


# ---------------------------------------------------------------------------
# logits of a batch's rows
# ---------------------------------------------------------------------------
TS_COUNTS_RESET, TS_COUNTS_PROMPT = 1, 2
_LOGITS_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def ts_token_counts(tokens, lens, V, seen, counts=None, reset=False, prompt=False, status=None,
                    stream=None):
    """Add tokens[s, :lens[s]] to what the sequences have met: their bits in
    seen [n_seq, ceil(V / 32)] and, except with prompt=True, counts [n_seq, V]
    (None: only the bits are kept), all int32.  reset=True starts over with
    these tokens."""
    if not isinstance(tokens, torch.Tensor) or not tokens.is_cuda:
        raise TypeError("tokens must be a CUDA tensor")
    if tokens.dim() != 2:
        raise ValueError(f"tokens has shape {tuple(tokens.shape)}, expected (n_seq, m)")
    dev, i32 = tokens.get_device(), torch.int32
    n_seq, m = shape = tokens.shape
    st = None if status is None else _need(status, i32, status.shape, dev, "status")
    _paged_call(lib().ts_token_counts, dev, stream, (), (
        _need(tokens, i32, shape, dev, "tokens"), m, _need(lens, i32, (n_seq,), dev, "lens"), n_seq,
        V, _need(counts, i32, (n_seq, V), dev, "counts"),
        _need(seen, i32, (n_seq, (V + 31) // 32), dev, "seen"),
        (TS_COUNTS_RESET if reset else 0) | (TS_COUNTS_PROMPT if prompt else 0), st))


def _row_stride(t, n, V, name):
    """Elements between the rows of a [n, V] tensor whose rows are dense."""
    row, one = t.stride()
    if (one != 1 and V > 1) or (row < V and n > 1):
        raise ValueError(f"{name}: a row's values must be dense")
    return row if n > 1 else V


def ts_logits_process(logits, cu_q, seen=None, counts=None, repetition=None, frequency=None,
                      presence=None, tree_tokens=None, parents=None, bias_ids=None, bias=None,
                      mask=None, mask_rows=None, masked_value=float("-inf"), out=None, status=None,
                      stream=None):
    """Logits [n, V] (fp32, bf16 or fp16; any row stride) of the sequences' rows
    (cu_q [n_seq + 1]) under biases, penalties for the tokens met and masks:
    fp32 [n, V].  seen, counts: the state of ts_token_counts; repetition,
    frequency, presence [n_seq] fp32; tree_tokens, parents [n]: the rows are
    nodes of draft trees, whose paths are met too; bias_ids, bias [n_seq, m];
    mask [n_masks, ceil(V / 32)] int32 bits of the tokens allowed, mask_rows [n]
    (None: row t has mask t; -1: none).  out may be logits itself if fp32."""
    if not isinstance(logits, torch.Tensor) or not logits.is_cuda:
        raise TypeError("logits must be a CUDA tensor")
    kind = _LOGITS_TYPES.get(logits.dtype)
    if kind is None:
        raise TypeError(f"logits must be {tuple(_LOGITS_TYPES)}, got {logits.dtype}")
    if logits.dim() != 2:
        raise ValueError(f"logits has shape {tuple(logits.shape)}, expected (n, V)")
    n, V = shape = logits.shape
    dev, i32, f32 = logits.get_device(), torch.int32, torch.float32
    stride = _row_stride(logits, n, V, "logits")
    if not isinstance(cu_q, torch.Tensor) or cu_q.dim() != 1 or cu_q.shape[0] < 1:
        raise ValueError("cu_q must be a tensor [n_seq + 1]")
    n_seq, words = cu_q.shape[0] - 1, (V + 31) // 32
    per_row, per_seq = (n,), (n_seq,)
    tok = par = cnt = sn = rep = frq = prs = ids = bv = mk = rows = st = None
    n_bias = n_masks = 0
    if tree_tokens is not None:
        tok = _need(tree_tokens, i32, per_row, dev, "tree_tokens")
    if parents is not None:
        par = _need(parents, i32, per_row, dev, "parents")
    if counts is not None:
        cnt = _need(counts, i32, (n_seq, V), dev, "counts")
    if seen is not None:
        sn = _need(seen, i32, (n_seq, words), dev, "seen")
    if repetition is not None:
        rep = _need(repetition, f32, per_seq, dev, "repetition")
    if frequency is not None:
        frq = _need(frequency, f32, per_seq, dev, "frequency")
    if presence is not None:
        prs = _need(presence, f32, per_seq, dev, "presence")
    if bias_ids is not None or bias is not None:
        if bias_ids is None or bias is None:
            raise ValueError("bias_ids and bias go together")
        n_bias = bias_ids.shape[-1]
        ids = _need(bias_ids, i32, (n_seq, n_bias), dev, "bias_ids")
        bv = _need(bias, f32, (n_seq, n_bias), dev, "bias")
    if mask is not None:
        n_masks = mask.shape[0]
        mk = _need(mask, i32, (n_masks, words), dev, "mask")
    if mask_rows is not None:
        rows = _need(mask_rows, i32, per_row, dev, "mask_rows")
    if status is not None:
        st = _need(status, i32, status.shape, dev, "status")
    outputs = ()
    if out is None:
        out = _alloc_like(logits, f32, stream)
        outputs, out_stride = (out,), V
    else:
        if not isinstance(out, torch.Tensor) or out.dtype is not f32 or out.shape != shape or \
                out.get_device() != dev:
            raise ValueError(f"out must be a float32 tensor {tuple(shape)} on cuda:{dev}")
        out_stride = _row_stride(out, n, V, "out")
    _paged_call(lib().ts_logits_process, dev, stream, outputs, (
        logits.data_ptr(), stride, n, V, _need(cu_q, i32, (n_seq + 1,), dev, "cu_q"), n_seq, tok,
        par, cnt, sn, rep, frq, prs, ids, bv, n_bias, mk, n_masks, rows, masked_value,
        out.data_ptr(), out_stride, kind, st))
    return out
