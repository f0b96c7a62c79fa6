"""Python binding of the MI355X KDA library (``libkda.so``, C ABI in include/kda.h).

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI.  PyTorch provides device memory and the stream.
The library must have been built (``python gated_delta_rule_03_amd/build.py``);
importing the binding without it raises ImportError -- there is no fallback.

Entry points (same names as the C ABI):
  kda_prefill(cfg, q, k, v, alpha, b, ...)          B equal-length sequences
  kda_varlen_prefill(cfg, cu_seqlens, q, ...)       packed sequences
  kda_decode_step(cfg, q, k, v, alpha, b, state, conv_state, o=None)
  kda_decode_multi(cfg, q, ..., state_pool, conv_pool, slots=, n_commit=)
  kda_decode_step_gated / kda_decode_multi_gated   the same, output epilogue fused
  kda_output_gate(cfg, o, gate, o_norm_weight)     the output epilogue alone
  kda_add_rmsnorm(cfg, x, residual, weight)        the norm in front of a layer, and its residual's addition
  kda_add_rmsnorm_fp8 / kda_output_gate_fp8        the norm / the epilogue with e4m3 rows and block scales
  kda_add_rmsnorm_backward / kda_output_gate_backward
  kda_fp8_matmul(cfg, a, a_scale, w, w_scale)      a projection of e4m3 rows
  kda_qk_norm_rope(cfg, rope, q, k, ...)           norm and rotation of query and key heads; kda_qk_norm_rope_backward
  kda_append_kv(cfg, cache, ...) / kda_read_kv     a paged 4-bit cache of keys and values
  kda_paged_attention(cfg, cache, q, ...)          attention of the newest tokens over it
  kda_prefill_workspace_bytes / kda_varlen_workspace_bytes / kda_prefill_slab_workspace_bytes
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
from dataclasses import dataclass, field
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkda.so")

KDA_OK = 0
KDA_ERR_INVALID_ARGUMENT = 1
KDA_ERR_UNSUPPORTED = 2
KDA_ERR_WORKSPACE_TOO_SMALL = 3
KDA_ERR_HIP = 4

KDA_BF16 = 0
KDA_FP32 = 1

FLAG_SKIP_CONV = 1 << 0
FLAG_SKIP_L2NORM = 1 << 1
FLAG_RAW_GATE = 1 << 2
FLAG_RAW_BETA = 1 << 3
FLAG_BETA_X2 = 1 << 4

STAGES = ("chunk_table", "chunk_prep", "chunk_scan", "conv_state", "decode", "output_gate", "backward", "norm",
          "matmul", "rope", "cache", "attention")
NUM_STAGES = len(STAGES)

EXPORTED = ("kda_version", "kda_status_string", "kda_prefill_workspace_bytes", "kda_prefill",
            "kda_varlen_workspace_bytes", "kda_varlen_prefill", "kda_decode_step", "kda_decode_multi",
            "kda_decode_step_gated", "kda_decode_multi_gated", "kda_output_gate", "kda_varlen_prefill_noalloc",
            "kda_varlen_backward_workspace_bytes", "kda_varlen_backward", "kda_prefill_slab_workspace_bytes",
            "kda_add_rmsnorm", "kda_add_rmsnorm_fp8", "kda_add_rmsnorm_backward_workspace_bytes",
            "kda_add_rmsnorm_backward", "kda_output_gate_fp8", "kda_output_gate_backward_workspace_bytes",
            "kda_output_gate_backward", "kda_fp8_matmul", "kda_qk_norm_rope",
            "kda_qk_norm_rope_backward_workspace_bytes", "kda_qk_norm_rope_backward", "kda_append_kv", "kda_read_kv",
            "kda_paged_attention_workspace_bytes", "kda_paged_attention")

# consecutive values of an e4m3 row that share a scale
SCALE_BLOCK = 128

# the fixed scratch behind kda_varlen_prefill_noalloc (KDA_NOALLOC_SCRATCH_BYTES)
NOALLOC_SCRATCH_BYTES = 256 << 20


class KdaError(RuntimeError):
    def __init__(self, status: int, name: str):
        super().__init__(f"{name} returned {status_string(status)} ({status})")
        self.status = status


class KdaConfigC(ctypes.Structure):
    _fields_ = [
        ("num_heads", ctypes.c_int32),
        ("head_k_dim", ctypes.c_int32),
        ("head_v_dim", ctypes.c_int32),
        ("io_dtype", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("gate_lower_bound", ctypes.c_float),
        ("l2norm_eps", ctypes.c_float),
        ("chunk_size", ctypes.c_int32),
        ("flags", ctypes.c_uint32),
        ("A_log", ctypes.c_void_p),
        ("dt_bias", ctypes.c_void_p),
        ("conv_w_q", ctypes.c_void_p),
        ("conv_w_k", ctypes.c_void_p),
        ("conv_w_v", ctypes.c_void_p),
        ("stage_events", ctypes.c_void_p),
    ]


class KdaRopeC(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("num_axes", ctypes.c_int32),
                ("inv_freq", ctypes.c_void_p), ("axis", ctypes.c_void_p)]


class KdaKvCacheC(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("page_table", ctypes.c_void_p),
                ("lengths", ctypes.c_void_p), ("cu_seqlens", ctypes.c_void_p)]


def _load_library():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"KDA HIP library not built: {LIB_PATH} is missing "
                          "(run `python gated_delta_rule_03_amd/build.py`)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    cfgp = ctypes.POINTER(KdaConfigC)
    lib.kda_version.restype = i32
    lib.kda_version.argtypes = []
    lib.kda_status_string.restype = ctypes.c_char_p
    lib.kda_status_string.argtypes = [ctypes.c_int]
    lib.kda_prefill_workspace_bytes.restype = sz
    lib.kda_prefill_workspace_bytes.argtypes = [cfgp, i32, i32]
    lib.kda_varlen_workspace_bytes.restype = sz
    lib.kda_varlen_workspace_bytes.argtypes = [cfgp, i32, i32]
    lib.kda_prefill_slab_workspace_bytes.restype = sz
    lib.kda_prefill_slab_workspace_bytes.argtypes = [cfgp, i32, i32]
    lib.kda_prefill.restype = ctypes.c_int
    lib.kda_prefill.argtypes = [cfgp, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.kda_varlen_prefill.restype = ctypes.c_int
    lib.kda_varlen_prefill.argtypes = [cfgp, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.kda_varlen_prefill_noalloc.restype = ctypes.c_int
    lib.kda_varlen_prefill_noalloc.argtypes = [cfgp, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.kda_varlen_backward_workspace_bytes.restype = sz
    lib.kda_varlen_backward_workspace_bytes.argtypes = [cfgp, i32, i32]
    lib.kda_varlen_backward.restype = ctypes.c_int
    lib.kda_varlen_backward.argtypes = [cfgp, i32, i32] + [vp] * 23 + [sz, vp]
    lib.kda_decode_step.restype = ctypes.c_int
    lib.kda_decode_step.argtypes = [cfgp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.kda_decode_multi.restype = ctypes.c_int
    lib.kda_decode_multi.argtypes = [cfgp, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.kda_decode_step_gated.restype = ctypes.c_int
    lib.kda_decode_step_gated.argtypes = [cfgp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_float, vp, vp]
    lib.kda_decode_multi_gated.restype = ctypes.c_int
    lib.kda_decode_multi_gated.argtypes = [cfgp, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                           ctypes.c_float, vp, vp, vp]
    lib.kda_output_gate.restype = ctypes.c_int
    lib.kda_output_gate.argtypes = [cfgp, ctypes.c_int64, vp, vp, vp, ctypes.c_float, vp, vp]
    i64, f32 = ctypes.c_int64, ctypes.c_float
    lib.kda_add_rmsnorm.restype = ctypes.c_int
    lib.kda_add_rmsnorm.argtypes = [cfgp, i64, i32, vp, vp, vp, f32, vp, vp, vp]
    lib.kda_add_rmsnorm_fp8.restype = ctypes.c_int
    lib.kda_add_rmsnorm_fp8.argtypes = [cfgp, i64, i32, vp, vp, vp, f32, vp, vp, vp, vp]
    lib.kda_add_rmsnorm_backward_workspace_bytes.restype = sz
    lib.kda_add_rmsnorm_backward_workspace_bytes.argtypes = [cfgp, i64, i32]
    lib.kda_add_rmsnorm_backward.restype = ctypes.c_int
    lib.kda_add_rmsnorm_backward.argtypes = [cfgp, i64, i32, vp, vp, f32, vp, vp, vp, vp, vp, sz, vp]
    lib.kda_output_gate_fp8.restype = ctypes.c_int
    lib.kda_output_gate_fp8.argtypes = [cfgp, i64, vp, vp, vp, f32, vp, vp, vp]
    lib.kda_output_gate_backward_workspace_bytes.restype = sz
    lib.kda_output_gate_backward_workspace_bytes.argtypes = [cfgp, i64]
    lib.kda_output_gate_backward.restype = ctypes.c_int
    lib.kda_output_gate_backward.argtypes = [cfgp, i64, vp, vp, vp, f32, vp, vp, vp, vp, vp, sz, vp]
    lib.kda_fp8_matmul.restype = ctypes.c_int
    lib.kda_fp8_matmul.argtypes = [cfgp, i64, i32, i32, vp, vp, vp, vp, vp, vp]
    ropep, cachep = ctypes.POINTER(KdaRopeC), ctypes.POINTER(KdaKvCacheC)
    lib.kda_qk_norm_rope.restype = ctypes.c_int
    lib.kda_qk_norm_rope.argtypes = [cfgp, ropep, i64, i32, vp, i64, vp, i64, vp, vp, f32, vp, vp, vp, vp]
    lib.kda_qk_norm_rope_backward_workspace_bytes.restype = sz
    lib.kda_qk_norm_rope_backward_workspace_bytes.argtypes = [cfgp, i64, i32]
    lib.kda_qk_norm_rope_backward.restype = ctypes.c_int
    lib.kda_qk_norm_rope_backward.argtypes = [cfgp, ropep, i64, i32, vp, i64, vp, i64, vp, vp, f32] + [vp] * 7 + [sz, vp]
    lib.kda_append_kv.restype = ctypes.c_int
    lib.kda_append_kv.argtypes = [cfgp, ropep, cachep, i32, i64, vp, i64, vp, i64, vp, f32, vp, vp]
    lib.kda_read_kv.restype = ctypes.c_int
    lib.kda_read_kv.argtypes = [cfgp, cachep, i32, i64, vp, vp, vp]
    lib.kda_paged_attention_workspace_bytes.restype = sz
    lib.kda_paged_attention_workspace_bytes.argtypes = [cfgp, i32, i32, i64, i32]
    lib.kda_paged_attention.restype = ctypes.c_int
    lib.kda_paged_attention.argtypes = [cfgp, cachep, i32, i64, i32, vp, f32, vp, vp, vp, sz, vp]
    return lib


_lib = _load_library()


def library():
    """The loaded ctypes library handle."""
    return _lib


def status_string(status: int) -> str:
    return _lib.kda_status_string(int(status)).decode()


def version() -> int:
    return int(_lib.kda_version())


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return KDA_BF16
    if dt == torch.float32:
        return KDA_FP32
    raise ValueError(f"unsupported dtype {dt}")


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


@dataclass
class Config:
    """Per-layer parameters and numerics of the KDA core (device tensors)."""
    A_log: torch.Tensor          # [H] fp32
    dt_bias: torch.Tensor        # [H*dk] fp32
    conv_w_q: torch.Tensor       # [H*dk, 4] io dtype
    conv_w_k: torch.Tensor       # [H*dk, 4]
    conv_w_v: torch.Tensor       # [H*dv, 4]
    num_heads: int
    head_k_dim: int
    head_v_dim: int
    io_dtype: torch.dtype = torch.bfloat16
    out_dtype: torch.dtype = torch.bfloat16
    scale: float = 1.0
    gate_lower_bound: float = -5.0
    l2norm_eps: float = 1e-6
    chunk_size: int = 64
    flags: int = 0
    stage_events: Optional[object] = None   # ctypes array of 2*NUM_STAGES hipEvent_t, or None
    _c: Optional[KdaConfigC] = field(default=None, repr=False)

    def c_struct(self) -> KdaConfigC:
        c = KdaConfigC()
        c.num_heads = self.num_heads
        c.head_k_dim = self.head_k_dim
        c.head_v_dim = self.head_v_dim
        c.io_dtype = _dtype_code(self.io_dtype)
        c.out_dtype = _dtype_code(self.out_dtype)
        c.scale = self.scale
        c.gate_lower_bound = self.gate_lower_bound
        c.l2norm_eps = self.l2norm_eps
        c.chunk_size = self.chunk_size
        c.flags = self.flags
        for name in ("A_log", "dt_bias", "conv_w_q", "conv_w_k", "conv_w_v"):
            t = getattr(self, name)
            setattr(c, name, None if t is None else t.data_ptr())
        c.stage_events = None if self.stage_events is None else ctypes.cast(self.stage_events, ctypes.c_void_p)
        self._c = c   # keep alive
        return c

    @property
    def ctot(self) -> int:
        return self.num_heads * (2 * self.head_k_dim + self.head_v_dim)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(status: int, name: str):
    if status != KDA_OK:
        raise KdaError(status, name)


def kda_prefill_workspace_bytes(cfg: Config, B: int, T: int) -> int:
    return int(_lib.kda_prefill_workspace_bytes(ctypes.byref(cfg.c_struct()), B, T))


def kda_varlen_workspace_bytes(cfg: Config, N: int, total_T: int) -> int:
    return int(_lib.kda_varlen_workspace_bytes(ctypes.byref(cfg.c_struct()), N, total_T))


def kda_prefill_slab_workspace_bytes(cfg: Config, N: int, slab_tokens: int) -> int:
    """Workspace for the chunked prefill of N sequences run in slabs of
    slab_tokens positions; passing a workspace of this size (smaller than
    the one-pass size) to kda_prefill / kda_varlen_prefill runs them in slabs."""
    return int(_lib.kda_prefill_slab_workspace_bytes(ctypes.byref(cfg.c_struct()), N, slab_tokens))


def _workspace(nbytes: int, device, workspace: Optional[torch.Tensor]) -> torch.Tensor:
    if workspace is not None:
        return workspace
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


def kda_prefill(cfg: Config, q, k, v, alpha, b, initial_state=None, conv_state_in=None, *,
                o=None, final_state=None, conv_state_out=None, workspace=None, stream=None):
    """q, k [B, T, H*dk]; v [B, T, H*dv]; alpha [B, T, H, dk]; b [B, T, H].
    Returns (o [B, T, H, dv], final_state or None, conv_state_out or None)."""
    B, T = q.shape[0], q.shape[1]
    H, dv = cfg.num_heads, cfg.head_v_dim
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=cfg.out_dtype, device=q.device)
    nbytes = kda_prefill_workspace_bytes(cfg, B, T)
    ws = _workspace(nbytes, q.device, workspace)
    st = _lib.kda_prefill(ctypes.byref(cfg.c_struct()), B, T, _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(b),
                          _ptr(initial_state), _ptr(conv_state_in), _ptr(o), _ptr(final_state),
                          _ptr(conv_state_out), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "kda_prefill")
    return o, final_state, conv_state_out


def kda_varlen_prefill(cfg: Config, cu_seqlens, q, k, v, alpha, b, initial_state=None, conv_state_in=None, *,
                       o=None, final_state=None, conv_state_out=None, workspace=None, stream=None):
    """cu_seqlens int32 [N+1] on the device; q, k [total_T, H*dk]; v [total_T, H*dv];
    alpha [total_T, H, dk]; b [total_T, H].  Returns (o, final_state, conv_state_out)."""
    N = cu_seqlens.numel() - 1
    total = q.shape[0]
    H, dv = cfg.num_heads, cfg.head_v_dim
    if cu_seqlens.dtype != torch.int32:
        raise ValueError("cu_seqlens must be int32")
    if o is None:
        o = torch.empty((total, H, dv), dtype=cfg.out_dtype, device=q.device)
    nbytes = kda_varlen_workspace_bytes(cfg, N, total)
    ws = _workspace(nbytes, q.device, workspace)
    st = _lib.kda_varlen_prefill(ctypes.byref(cfg.c_struct()), N, total, _ptr(cu_seqlens), _ptr(q), _ptr(k),
                                 _ptr(v), _ptr(alpha), _ptr(b), _ptr(initial_state), _ptr(conv_state_in),
                                 _ptr(o), _ptr(final_state), _ptr(conv_state_out), _ptr(ws),
                                 ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "kda_varlen_prefill")
    return o, final_state, conv_state_out


def kda_varlen_prefill_noalloc(cfg: Config, cu_seqlens, q, k, v, alpha, b, initial_state=None, conv_state_in=None,
                               *, o, final_state=None, conv_state_out=None, stream=None):
    """kda_varlen_prefill on the library's fixed per-GPU scratch: no workspace
    argument and no allocation (o must be passed in).  Batches whose
    workspace exceeds NOALLOC_SCRATCH_BYTES raise KdaError
    (KDA_ERR_WORKSPACE_TOO_SMALL).  Returns (o, final_state, conv_state_out)."""
    N = cu_seqlens.numel() - 1
    if cu_seqlens.dtype != torch.int32:
        raise ValueError("cu_seqlens must be int32")
    st = _lib.kda_varlen_prefill_noalloc(ctypes.byref(cfg.c_struct()), N, q.shape[0], _ptr(cu_seqlens), _ptr(q),
                                         _ptr(k), _ptr(v), _ptr(alpha), _ptr(b), _ptr(initial_state),
                                         _ptr(conv_state_in), _ptr(o), _ptr(final_state), _ptr(conv_state_out),
                                         _stream(stream))
    _check(st, "kda_varlen_prefill_noalloc")
    return o, final_state, conv_state_out


def kda_varlen_backward_workspace_bytes(cfg: Config, N: int, total_T: int) -> int:
    return int(_lib.kda_varlen_backward_workspace_bytes(ctypes.byref(cfg.c_struct()), N, total_T))


def kda_varlen_backward(cfg: Config, cu_seqlens, q, k, v, alpha, b, initial_state=None, conv_state_in=None, *,
                        d_o, d_final_state=None, want_initial_state=True, want_conv_state=True, workspace=None,
                        stream=None):
    """Gradient of a loss through o and the final state of kda_varlen_prefill
    with respect to every input and parameter.  d_o [total_T, H, dv] (out
    dtype), d_final_state [N, H, dk, dv] fp32 or None.  Returns a dict of
    fp32 tensors: dq, dk [total_T, H*dk], dv [total_T, H*dv], dalpha
    [total_T, H, dk], db [total_T, H], dS0 [N, H, dk, dv] (or None), dconv
    [N, 3, Ctot] (or None), dw_q, dw_k [H*dk, 4], dw_v [H*dv, 4], ddt_bias
    [H*dk], dA_log [H]."""
    N = cu_seqlens.numel() - 1
    total = q.shape[0]
    H, dk, dv = cfg.num_heads, cfg.head_k_dim, cfg.head_v_dim
    if cu_seqlens.dtype != torch.int32:
        raise ValueError("cu_seqlens must be int32")
    dev = q.device
    f = lambda *shape: torch.empty(shape, dtype=torch.float32, device=dev)
    g = {"dq": f(total, H * dk), "dk": f(total, H * dk), "dv": f(total, H * dv), "dalpha": f(total, H, dk),
         "db": f(total, H), "dS0": f(N, H, dk, dv) if want_initial_state else None,
         "dconv": f(N, 3, cfg.ctot) if want_conv_state else None, "dw_q": f(H * dk, 4), "dw_k": f(H * dk, 4),
         "dw_v": f(H * dv, 4), "ddt_bias": f(H * dk), "dA_log": f(H)}
    nbytes = kda_varlen_backward_workspace_bytes(cfg, N, total)
    ws = _workspace(nbytes, dev, workspace)
    st = _lib.kda_varlen_backward(ctypes.byref(cfg.c_struct()), N, total, _ptr(cu_seqlens), _ptr(q), _ptr(k),
                                  _ptr(v), _ptr(alpha), _ptr(b), _ptr(initial_state), _ptr(conv_state_in),
                                  _ptr(d_o), _ptr(d_final_state), _ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]),
                                  _ptr(g["dalpha"]), _ptr(g["db"]), _ptr(g["dS0"]), _ptr(g["dconv"]),
                                  _ptr(g["dw_q"]), _ptr(g["dw_k"]), _ptr(g["dw_v"]), _ptr(g["ddt_bias"]),
                                  _ptr(g["dA_log"]), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "kda_varlen_backward")
    return g


def kda_decode_step(cfg: Config, q, k, v, alpha, b, state, conv_state, *, o=None, stream=None):
    """One token for each of N sequences: q, k [N, H*dk]; v [N, H*dv];
    alpha [N, H, dk]; b [N, H]; state [N, H, dk, dv] fp32 and conv_state
    [N, 3, Ctot] are updated in place.  Returns o [N, H, dv]."""
    N = q.shape[0]
    if o is None:
        o = torch.empty((N, cfg.num_heads, cfg.head_v_dim), dtype=cfg.out_dtype, device=q.device)
    st = _lib.kda_decode_step(ctypes.byref(cfg.c_struct()), N, _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(b),
                              _ptr(state), _ptr(conv_state), _ptr(o), _stream(stream))
    _check(st, "kda_decode_step")
    return o


def kda_decode_multi(cfg: Config, q, k, v, alpha, b, state_pool, conv_pool, *, slots=None, n_commit=None, o=None,
                     stream=None):
    """K tokens for each of N sequences through state / conv-history pools:
    q, k [N, K, H*dk]; v [N, K, H*dv]; alpha [N, K, H, dk]; b [N, K, H];
    state_pool [P, H, dk, dv] fp32 and conv_pool [P, 3, Ctot] are updated in
    place (rows slots[n], after the first n_commit[n] tokens).  slots and
    n_commit are int32 device tensors [N] or None.  Returns o [N, K, H, dv]."""
    N, K = q.shape[0], q.shape[1]
    for t in (slots, n_commit):
        if t is not None and (t.dtype != torch.int32 or t.numel() != N):
            raise ValueError("slots and n_commit must be int32 tensors of N entries")
    if o is None:
        o = torch.empty((N, K, cfg.num_heads, cfg.head_v_dim), dtype=cfg.out_dtype, device=q.device)
    st = _lib.kda_decode_multi(ctypes.byref(cfg.c_struct()), N, K, _ptr(slots), _ptr(q), _ptr(k), _ptr(v),
                               _ptr(alpha), _ptr(b), _ptr(state_pool), _ptr(conv_pool), _ptr(o), _ptr(n_commit),
                               _stream(stream))
    _check(st, "kda_decode_multi")
    return o


def kda_decode_step_gated(cfg: Config, q, k, v, alpha, b, state, conv_state, gate, o_norm_weight,
                          eps: float = 1e-6, *, y=None, stream=None):
    """kda_decode_step with the output epilogue fused: gate [N, H, dv] (io
    dtype), o_norm_weight [dv] fp32.  Returns y [N, H, dv] (out dtype) =
    o / sqrt(mean(o^2) + eps) * o_norm_weight * sigmoid(gate) per row."""
    N = q.shape[0]
    if y is None:
        y = torch.empty((N, cfg.num_heads, cfg.head_v_dim), dtype=cfg.out_dtype, device=q.device)
    st = _lib.kda_decode_step_gated(ctypes.byref(cfg.c_struct()), N, _ptr(q), _ptr(k), _ptr(v), _ptr(alpha),
                                    _ptr(b), _ptr(state), _ptr(conv_state), _ptr(gate), _ptr(o_norm_weight),
                                    float(eps), _ptr(y), _stream(stream))
    _check(st, "kda_decode_step_gated")
    return y


def kda_decode_multi_gated(cfg: Config, q, k, v, alpha, b, state_pool, conv_pool, gate, o_norm_weight,
                           eps: float = 1e-6, *, slots=None, n_commit=None, y=None, stream=None):
    """kda_decode_multi with the output epilogue fused: gate [N, K, H, dv]
    (io dtype), o_norm_weight [dv] fp32.  Returns y [N, K, H, dv]."""
    N, K = q.shape[0], q.shape[1]
    for t in (slots, n_commit):
        if t is not None and (t.dtype != torch.int32 or t.numel() != N):
            raise ValueError("slots and n_commit must be int32 tensors of N entries")
    if y is None:
        y = torch.empty((N, K, cfg.num_heads, cfg.head_v_dim), dtype=cfg.out_dtype, device=q.device)
    st = _lib.kda_decode_multi_gated(ctypes.byref(cfg.c_struct()), N, K, _ptr(slots), _ptr(q), _ptr(k), _ptr(v),
                                     _ptr(alpha), _ptr(b), _ptr(state_pool), _ptr(conv_pool), _ptr(gate),
                                     _ptr(o_norm_weight), float(eps), _ptr(y), _ptr(n_commit), _stream(stream))
    _check(st, "kda_decode_multi_gated")
    return y


def kda_output_gate(cfg: Config, o, gate, o_norm_weight, eps: float = 1e-6, *, y=None, stream=None):
    """The output epilogue: y = o / sqrt(mean(o^2) + eps) * o_norm_weight * sigmoid(gate)
    per (token, head) row.  o [..., H, dv] out_dtype; gate the same shape in
    io_dtype; o_norm_weight [dv] fp32.  y defaults to a new tensor; pass
    y=o to work in place.  Returns y."""
    if o.shape != gate.shape or o.shape[-1] != cfg.head_v_dim or o.shape[-2] != cfg.num_heads:
        raise ValueError("o and gate must both be [..., num_heads, head_v_dim]")
    n_tokens = o.numel() // (cfg.num_heads * cfg.head_v_dim) if o.numel() else 0
    if y is None:
        y = torch.empty_like(o)
    st = _lib.kda_output_gate(ctypes.byref(cfg.c_struct()), n_tokens, _ptr(o), _ptr(gate), _ptr(o_norm_weight),
                              float(eps), _ptr(y), _stream(stream))
    _check(st, "kda_output_gate")
    return y


# ---- the operators around the core -----------------------------------------
# These take their device and default stream from their tensors, check shapes
# and types, and allocate what they return on the stream that they run on.
# They are called once a token and layer, so the binding's own time counts: it
# does each step once (a kernel launch is ~4 us, the binding 3 to 6).

def _on_stream(device, stream, again):
    """again() with the tensors' device current, and `stream` if there is one:
    what it allocates and launches is that stream's."""
    if device.type != "cuda":
        raise ValueError("tensors must be on the GPU")
    if stream is None:
        with torch.cuda.device(device):
            return again()
    if stream.device != device:
        raise ValueError("the stream belongs to another device than the tensors")
    with torch.cuda.stream(stream):
        return again()


def _elsewhere(device, stream):
    """Whether a call has to change the current device or stream first."""
    return stream is not None or device.type != "cuda" or device.index != torch._C._cuda_getDevice()


def _at(name, t, shape, dtype, device):
    """The address of a tensor that has to be of this shape and type, or None for None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.device != device:
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)} on {device}, "
                         f"not {t.dtype} of shape {tuple(t.shape)} on {t.device}")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _workspace_at(nbytes, device, workspace):
    """(tensor, address, bytes) of the caller's workspace, or of a new one."""
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


@functools.lru_cache(maxsize=64)
def _op_fields(num_heads, head_v_dim, io_dtype, out_dtype):
    """The struct of these values (never written afterwards, so calls share it)."""
    c = KdaConfigC()
    c.num_heads = _int32(num_heads)
    c.head_v_dim = _int32(head_v_dim)
    c.io_dtype = _dtype_code(io_dtype)
    c.out_dtype = _dtype_code(out_dtype)
    return c


def _op_struct(cfg: Config):
    """The fields of the config that these operators read."""
    c = _op_fields(cfg.num_heads, cfg.head_v_dim, cfg.io_dtype, cfg.out_dtype)
    if cfg.stage_events is not None:
        c = KdaConfigC.from_buffer_copy(c)
        c.stage_events = ctypes.cast(cfg.stage_events, ctypes.c_void_p)
    return ctypes.byref(c)


# ctypes cuts an integer to its argument's width: a size beyond that is passed as
# one that the library refuses
_INT32_MAX = 2**31 - 1


def _int32(n: int) -> int:
    return max(-1, min(n, _INT32_MAX))


def _int64(n: int) -> int:
    return max(-1, min(n, 2**63 - 1))


def _scale_blocks(k: int) -> int:
    return (k + SCALE_BLOCK - 1) // SCALE_BLOCK


def kda_add_rmsnorm(cfg: Config, x, residual, weight, eps: float = 1e-6, *, h=None, y=None, stream=None):
    """h = x + residual and y = h / sqrt(mean(h^2) + eps) * weight per row:
    x, residual [..., hidden] io dtype (residual may be None), weight [hidden]
    fp32.  Returns (y, h), y in the out dtype, h in the io dtype (x itself
    without a residual or h).  h=x or h=residual works in place; so does y=x
    without either, which leaves no h: None is returned for it."""
    shape, dev = x.shape, x.device
    hidden = min(shape[-1], _INT32_MAX)
    xp, rp = _at("x", x, shape, cfg.io_dtype, dev), _at("residual", residual, shape, cfg.io_dtype, dev)
    wp = _at("weight", weight, (hidden,), torch.float32, dev)
    hp, yp = _at("h", h, shape, cfg.io_dtype, dev), _at("y", y, shape, cfg.out_dtype, dev)
    if _elsewhere(dev, stream):
        return _on_stream(dev, stream, lambda: kda_add_rmsnorm(cfg, x, residual, weight, eps, h=h, y=y))
    st = torch._C._cuda_getCurrentRawStream(dev.index)
    h_ = torch.empty_like(x) if h is None and residual is not None else h
    y_ = torch.empty_like(x, dtype=cfg.out_dtype) if y is None else y
    _check(_lib.kda_add_rmsnorm(_op_struct(cfg), x.numel() // hidden if hidden else 0, hidden, xp, rp, wp, eps,
                                hp if h_ is h else h_.data_ptr(), yp if y_ is y else y_.data_ptr(), st),
           "kda_add_rmsnorm")
    if h_ is None and not (yp and yp == xp):   # (y over x: x no longer holds h)
        h_ = x
    return y_, h_


def kda_add_rmsnorm_fp8(cfg: Config, x, residual, weight, eps: float = 1e-6, *, h=None, y=None, y_scale=None,
                        stream=None):
    """kda_add_rmsnorm with y as e4m3 rows.  Returns (y, y_scale, h): y
    [..., hidden] float8_e4m3fn, y_scale [..., ceil(hidden / 128)] fp32."""
    shape, dev = x.shape, x.device
    hidden = min(shape[-1], _INT32_MAX)
    blocks = (*shape[:-1], _scale_blocks(hidden))
    xp, rp = _at("x", x, shape, cfg.io_dtype, dev), _at("residual", residual, shape, cfg.io_dtype, dev)
    wp = _at("weight", weight, (hidden,), torch.float32, dev)
    hp, yp = _at("h", h, shape, cfg.io_dtype, dev), _at("y", y, shape, torch.float8_e4m3fn, dev)
    sp = _at("y_scale", y_scale, blocks, torch.float32, dev)
    if _elsewhere(dev, stream):
        return _on_stream(dev, stream, lambda: kda_add_rmsnorm_fp8(cfg, x, residual, weight, eps, h=h, y=y,
                                                                    y_scale=y_scale))
    st = torch._C._cuda_getCurrentRawStream(dev.index)
    h_ = torch.empty_like(x) if h is None and residual is not None else h
    y_ = torch.empty_like(x, dtype=torch.float8_e4m3fn) if y is None else y
    s_ = torch.empty(*blocks, dtype=torch.float32, device=dev) if y_scale is None else y_scale
    _check(_lib.kda_add_rmsnorm_fp8(_op_struct(cfg), x.numel() // hidden if hidden else 0, hidden, xp, rp, wp, eps,
                                    hp if h_ is h else h_.data_ptr(), yp if y_ is y else y_.data_ptr(),
                                    sp if s_ is y_scale else s_.data_ptr(), st), "kda_add_rmsnorm_fp8")
    return y_, s_, x if h_ is None else h_


def kda_add_rmsnorm_backward_workspace_bytes(cfg: Config, n_tokens: int, hidden: int) -> int:
    """Bytes of workspace; 0 for sizes that the library refuses."""
    return int(_lib.kda_add_rmsnorm_backward_workspace_bytes(_op_struct(cfg), _int64(n_tokens), _int32(hidden)))


def kda_add_rmsnorm_backward(cfg: Config, h, weight, dy, d_h=None, eps: float = 1e-6, *, dx=None, workspace=None,
                             stream=None):
    """Gradients of kda_add_rmsnorm: h as it returned it, dy [..., hidden] in
    the out dtype, d_h the gradient that reaches h otherwise (fp32) or None.
    Returns (dx [..., hidden], dweight [hidden]), fp32; dx is the gradient of x
    and of residual alike.  dx=d_h works in place."""
    shape, dev = h.shape, h.device
    hidden = min(shape[-1], _INT32_MAX)
    n = h.numel() // hidden if hidden else 0
    hp, wp = _at("h", h, shape, cfg.io_dtype, dev), _at("weight", weight, (hidden,), torch.float32, dev)
    dyp, dhp = _at("dy", dy, shape, cfg.out_dtype, dev), _at("d_h", d_h, shape, torch.float32, dev)
    dxp = _at("dx", dx, shape, torch.float32, dev)
    if _elsewhere(dev, stream):
        return _on_stream(dev, stream, lambda: kda_add_rmsnorm_backward(cfg, h, weight, dy, d_h, eps, dx=dx,
                                                                         workspace=workspace))
    st = torch._C._cuda_getCurrentRawStream(dev.index)
    dx_ = torch.empty_like(h, dtype=torch.float32) if dx is None else dx
    dw = torch.empty_like(weight)
    c = _op_struct(cfg)
    ws, wsp, size = _workspace_at(_lib.kda_add_rmsnorm_backward_workspace_bytes(c, n, hidden), dev, workspace)
    _check(_lib.kda_add_rmsnorm_backward(c, n, hidden, hp, wp, eps, dyp, dhp,
                                         dxp if dx_ is dx else dx_.data_ptr(), dw.data_ptr(), wsp, size, st),
           "kda_add_rmsnorm_backward")
    return dx_, dw


def _gate_args(cfg, o, gate, o_norm_weight):
    """(leading axes, n_tokens, addresses) of the output epilogue's inputs."""
    H, dv, dev = cfg.num_heads, cfg.head_v_dim, o.device
    lead = o.shape[:-2]
    full = (*lead, H, dv)
    return (lead, full, o.numel() // max(H * dv, 1), _at("o", o, full, cfg.out_dtype, dev),
            _at("gate", gate, full, cfg.io_dtype, dev), _at("o_norm_weight", o_norm_weight, (dv,), torch.float32, dev))


def kda_output_gate_fp8(cfg: Config, o, gate, o_norm_weight, eps: float = 1e-6, *, y=None, y_scale=None, stream=None):
    """kda_output_gate with its output as e4m3 rows: o [..., H, dv] out dtype,
    gate the same shape in the io dtype.  Returns (y [..., H * dv]
    float8_e4m3fn, y_scale [..., ceil(H * dv / 128)] fp32)."""
    dev = o.device
    lead, _, n, op, gp, wp = _gate_args(cfg, o, gate, o_norm_weight)
    row = cfg.num_heads * cfg.head_v_dim
    rows, blocks = (*lead, row), (*lead, _scale_blocks(row))
    yp, sp = _at("y", y, rows, torch.float8_e4m3fn, dev), _at("y_scale", y_scale, blocks, torch.float32, dev)
    if _elsewhere(dev, stream):
        return _on_stream(dev, stream, lambda: kda_output_gate_fp8(cfg, o, gate, o_norm_weight, eps, y=y,
                                                                    y_scale=y_scale))
    st = torch._C._cuda_getCurrentRawStream(dev.index)
    y_ = torch.empty(*rows, dtype=torch.float8_e4m3fn, device=dev) if y is None else y
    s_ = torch.empty(*blocks, dtype=torch.float32, device=dev) if y_scale is None else y_scale
    _check(_lib.kda_output_gate_fp8(_op_struct(cfg), n, op, gp, wp, eps,
                                    yp if y_ is y else y_.data_ptr(), sp if s_ is y_scale else s_.data_ptr(), st),
           "kda_output_gate_fp8")
    return y_, s_


def kda_output_gate_backward_workspace_bytes(cfg: Config, n_tokens: int) -> int:
    """Bytes of workspace; 0 for sizes that the library refuses."""
    return int(_lib.kda_output_gate_backward_workspace_bytes(_op_struct(cfg), _int64(n_tokens)))


def kda_output_gate_backward(cfg: Config, o, gate, o_norm_weight, dy, eps: float = 1e-6, *, workspace=None,
                             stream=None):
    """Gradients of kda_output_gate: o, dy [..., H, dv] out dtype, gate the
    same shape in the io dtype.  Returns (d_o in the out dtype, as
    kda_varlen_backward takes it, d_gate fp32, d_weight [dv] fp32)."""
    dev = o.device
    _, full, n, op, gp, wp = _gate_args(cfg, o, gate, o_norm_weight)
    dyp = _at("dy", dy, full, cfg.out_dtype, dev)
    if _elsewhere(dev, stream):
        return _on_stream(dev, stream, lambda: kda_output_gate_backward(cfg, o, gate, o_norm_weight, dy, eps,
                                                                         workspace=workspace))
    st = torch._C._cuda_getCurrentRawStream(dev.index)
    d_o, d_gate = torch.empty_like(o), torch.empty_like(gate, dtype=torch.float32)
    dw = torch.empty_like(o_norm_weight)
    c = _op_struct(cfg)
    ws, wsp, size = _workspace_at(_lib.kda_output_gate_backward_workspace_bytes(c, n), dev, workspace)
    _check(_lib.kda_output_gate_backward(c, n, op, gp, wp, eps, dyp, d_o.data_ptr(), d_gate.data_ptr(),
                                         dw.data_ptr(), wsp, size, st), "kda_output_gate_backward")
    return d_o, d_gate, dw


def kda_fp8_matmul(cfg: Config, a, a_scale, w, w_scale, *, y=None, stream=None):
    """y = a w^T of e4m3 operands: a [..., K] float8_e4m3fn with a_scale
    [..., ceil(K / 128)] fp32 (as kda_add_rmsnorm_fp8 and kda_output_gate_fp8
    return them), w [N, K] float8_e4m3fn with w_scale [ceil(N / 128),
    ceil(K / 128)] fp32.  Returns y [..., N] in the out dtype."""
    (N, K), dev, lead = w.shape, a.device, a.shape[:-1]
    kb, f8 = _scale_blocks(K), torch.float8_e4m3fn
    ap, sp = _at("a", a, (*lead, K), f8, dev), _at("a_scale", a_scale, (*lead, kb), torch.float32, dev)
    wp, wsp = _at("w", w, (N, K), f8, dev), _at("w_scale", w_scale, (_scale_blocks(N), kb), torch.float32, dev)
    shape = (*lead, N)
    yp = _at("y", y, shape, cfg.out_dtype, dev)
    if _elsewhere(dev, stream):
        return _on_stream(dev, stream, lambda: kda_fp8_matmul(cfg, a, a_scale, w, w_scale, y=y))
    st = torch._C._cuda_getCurrentRawStream(dev.index)
    y_ = torch.empty(*shape, dtype=cfg.out_dtype, device=dev) if y is None else y
    _check(_lib.kda_fp8_matmul(_op_struct(cfg), math.prod(lead), min(N, _INT32_MAX), min(K, _INT32_MAX), ap, sp, wp, wsp,
                               yp if y_ is y else y_.data_ptr(), st), "kda_fp8_matmul")
    return y_


# ---- the full-attention layers ----------------------------------------------

# channels of a head that share a scale in the cache, and the page sizes it can have
KV_BLOCK = 32
PAGE_SIZES = (32, 64, 128, 256)


@dataclass(frozen=True, eq=False)
class Rope:
    """A rotation of the first 2 * len(inv_freq) channels of a head: pair i
    turns by positions[axis[i]] * inv_freq[i] (axis None: one axis).  Pair i is
    channels (i, i + len(inv_freq)), or (2 i, 2 i + 1) when interleaved."""
    inv_freq: torch.Tensor                    # [pairs] fp32, on the GPU; pairs a multiple of 8
    axis: Optional[torch.Tensor] = None       # [pairs] int32
    num_axes: int = 1
    interleaved: bool = False

    def __post_init__(self):
        n, dev = self.inv_freq.numel(), self.inv_freq.device
        c = KdaRopeC(2 * n, int(self.interleaved), _int32(self.num_axes), _at("inv_freq", self.inv_freq, (n,), torch.float32, dev),
                     _at("axis", self.axis, (n,), torch.int32, dev))
        # (frozen: the tensors it points to stay)
        object.__setattr__(self, "_c", c)
        object.__setattr__(self, "_ref", ctypes.byref(c))
        object.__setattr__(self, "_device", dev)

    @classmethod
    def build(cls, rotary_dim: int, theta: float = 10000.0, sections=None, interleaved: bool = False, device="cuda"):
        """The usual frequencies theta^(-2 i / rotary_dim).  sections: pairs of
        each position axis, in order (their sum is rotary_dim / 2)."""
        half = rotary_dim // 2
        inv_freq = (float(theta) ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))).float().to(device)
        if sections is None:
            return cls(inv_freq, interleaved=interleaved)
        if sum(sections) != half:
            raise ValueError("the sections have to add up to rotary_dim / 2 pairs")
        axis = torch.repeat_interleave(torch.arange(len(sections), dtype=torch.int32), torch.tensor(list(sections)))
        return cls(inv_freq, axis.to(device), len(sections), interleaved)


@dataclass(frozen=True, eq=False)
class KvCache:
    """A paged cache of 4-bit keys and values (layout in include/kda.h)."""
    k: torch.Tensor          # [num_pages, num_kv_heads, page_size, d / 2] uint8
    k_scale: torch.Tensor    # [num_pages, num_kv_heads, d / 32, page_size] uint8
    v: torch.Tensor
    v_scale: torch.Tensor

    def __post_init__(self):
        dev, u8 = self.k.device, torch.uint8
        if self.k.dim() != 4 or self.k.shape[3] % (KV_BLOCK // 2):
            raise ValueError("k must be [num_pages, num_kv_heads, page_size, d / 2]")
        pages, heads, size, half = self.k.shape
        scales = (pages, heads, 2 * half // KV_BLOCK, size)
        c = KdaKvCacheC(_at("k", self.k, self.k.shape, u8, dev), _at("k_scale", self.k_scale, scales, u8, dev),
                        _at("v", self.v, self.k.shape, u8, dev), _at("v_scale", self.v_scale, scales, u8, dev),
                        _int32(pages), _int32(size), _int32(heads))
        object.__setattr__(self, "_c", c)

    @classmethod
    def empty(cls, num_pages: int, num_kv_heads: int, head_dim: int, page_size: int = 64, device="cuda"):
        """A cache of zeros."""
        t = lambda *shape: torch.zeros((num_pages, num_kv_heads, *shape), dtype=torch.uint8, device=device)
        return cls(t(page_size, head_dim // 2), t(head_dim // KV_BLOCK, page_size),
                   t(page_size, head_dim // 2), t(head_dim // KV_BLOCK, page_size))


@functools.lru_cache(maxsize=64)
def _attention_fields(num_heads, head_k_dim, head_v_dim, io_dtype, out_dtype):
    c = KdaConfigC()
    c.num_heads, c.head_k_dim, c.head_v_dim = _int32(num_heads), _int32(head_k_dim), _int32(head_v_dim)
    c.io_dtype, c.out_dtype = _dtype_code(io_dtype), _dtype_code(out_dtype)
    return c


def _attention_struct(cfg: Config):
    """The fields of the config that these operators read."""
    c = _attention_fields(cfg.num_heads, cfg.head_k_dim, cfg.head_v_dim, cfg.io_dtype, cfg.out_dtype)
    if cfg.stage_events is not None:
        c = KdaConfigC.from_buffer_copy(c)
        c.stage_events = ctypes.cast(cfg.stage_events, ctypes.c_void_p)
    return ctypes.byref(c)


def _rows_at(name, t, shape, dtype, device):
    """(address, row stride) of a tensor whose rows are contiguous: its leading axis may be strided."""
    if t.dtype is not dtype or t.shape != shape or t.device != device:
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)} on {device}, "
                         f"not {t.dtype} of shape {tuple(t.shape)} on {t.device}")
    row = shape[1] * shape[2]
    if t.is_contiguous():
        return t.data_ptr(), row
    s = t.stride()
    if (s[2] != 1 and shape[2] > 1) or (s[1] != shape[2] and shape[1] > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return t.data_ptr(), s[0]


def _rope_at(rope, positions, n, device):
    """(pointer to the struct or None, address of the positions)."""
    if rope is None:
        return None, None
    if rope._device != device:
        raise ValueError(f"rope must be on {device}")
    shape = (n,) if rope.num_axes == 1 and positions is not None and positions.dim() == 1 else (rope.num_axes, n)
    return rope._ref, _at("positions", positions, shape, torch.int32, device)


def kda_qk_norm_rope(cfg: Config, rope: Optional[Rope], q, k, q_weight=None, k_weight=None, positions=None,
                     eps: float = 1e-6, *, q_out=None, k_out=None, stream=None):
    """y = rotate(x / sqrt(mean(x^2) + eps) * weight) per head: q [n, num_heads,
    d], k [n, kv heads, d] or None, io dtype (their tokens may be strided:
    views into a wider projection); weights [d] fp32 (of a zero-centred norm 1 +
    its weight) or None (no norm); rope None rotates nothing; positions int32 [num_axes, n] (or [n]).  Returns
    (q_out, k_out), out dtype.  q_out=q and k_out=k work in place for
    contiguous tensors of one type."""
    dev, d, H = q.device, cfg.head_k_dim, cfg.num_heads
    n = q.shape[0]
    heads = 0 if k is None else k.shape[1]
    qp, qs = _rows_at("q", q, (n, H, d), cfg.io_dtype, dev)
    kp, ks = (None, 0) if k is None else _rows_at("k", k, (n, heads, d), cfg.io_dtype, dev)
    f32, out = torch.float32, cfg.out_dtype
    wp, vp = _at("q_weight", q_weight, (d,), f32, dev), _at("k_weight", k_weight, (d,), f32, dev)
    rp, pp = _rope_at(rope, positions, n, dev)
    qo, ko = _at("q_out", q_out, (n, H, d), out, dev), _at("k_out", k_out, (n, heads, d), out, dev)
    if _elsewhere(dev, stream):
        return _on_stream(dev, stream, lambda: kda_qk_norm_rope(cfg, rope, q, k, q_weight, k_weight, positions, eps,
                                                                 q_out=q_out, k_out=k_out))
    st = torch._C._cuda_getCurrentRawStream(dev.index)
    y = torch.empty((n, H, d), dtype=out, device=dev) if q_out is None else q_out
    z = torch.empty((n, heads, d), dtype=out, device=dev) if k_out is None and k is not None else k_out
    _check(_lib.kda_qk_norm_rope(_attention_struct(cfg), rp, n, heads, qp, qs, kp, ks, wp, vp, eps, pp,
                                 qo or y.data_ptr(), ko or (z.data_ptr() if z is not None else None), st),
           "kda_qk_norm_rope")
    return y, z


def kda_qk_norm_rope_backward_workspace_bytes(cfg: Config, n_tokens: int, num_kv_heads: int) -> int:
    """Bytes of workspace; 0 for sizes that the library refuses."""
    return int(_lib.kda_qk_norm_rope_backward_workspace_bytes(_attention_struct(cfg), _int64(n_tokens), _int32(num_kv_heads)))


def kda_qk_norm_rope_backward(cfg: Config, rope: Optional[Rope], q, k, q_weight, k_weight, positions, dq_out, dk_out,
                              eps: float = 1e-6, *, workspace=None, stream=None):
    """Gradients of kda_qk_norm_rope: its inputs, dq_out [n, num_heads, d] and
    dk_out (None with k) in the out dtype.  Returns (dq, dk, dq_weight,
    dk_weight), fp32; a weight that is None has a gradient of zeros, k None a
    dk of None."""
    dev, d, H = q.device, cfg.head_k_dim, cfg.num_heads
    n = q.shape[0]
    heads = 0 if k is None else k.shape[1]
    if (k is None) != (dk_out is None):
        raise ValueError("k and dk_out come together")
    qp, qs = _rows_at("q", q, (n, H, d), cfg.io_dtype, dev)
    kp, ks = (None, 0) if k is None else _rows_at("k", k, (n, heads, d), cfg.io_dtype, dev)
    f32, out = torch.float32, cfg.out_dtype
    wp, vp = _at("q_weight", q_weight, (d,), f32, dev), _at("k_weight", k_weight, (d,), f32, dev)
    rp, pp = _rope_at(rope, positions, n, dev)
    gp, hp = _at("dq_out", dq_out, (n, H, d), out, dev), _at("dk_out", dk_out, (n, heads, d), out, dev)
    if _elsewhere(dev, stream):
        return _on_stream(dev, stream, lambda: kda_qk_norm_rope_backward(
            cfg, rope, q, k, q_weight, k_weight, positions, dq_out, dk_out, eps, workspace=workspace))
    st = torch._C._cuda_getCurrentRawStream(dev.index)
    dq = torch.empty((n, H, d), dtype=f32, device=dev)
    dk = None if k is None else torch.empty((n, heads, d), dtype=f32, device=dev)
    dw = torch.empty((2, d), dtype=f32, device=dev)
    c = _attention_struct(cfg)
    ws, wsp, size = _workspace_at(_lib.kda_qk_norm_rope_backward_workspace_bytes(c, n, heads), dev, workspace)
    _check(_lib.kda_qk_norm_rope_backward(c, rp, n, heads, qp, qs, kp, ks, wp, vp, eps, pp, gp, hp, dq.data_ptr(),
                                          None if dk is None else dk.data_ptr(), dw.data_ptr(), wsp, size, st),
           "kda_qk_norm_rope_backward")
    return dq, dk, dw[0], dw[1]


def _cache_at(cfg, cache, cu_seqlens, page_table, lengths):
    """(struct of the cache and the call's sequences in it, N, device)."""
    dev = cache.k.device
    if 2 * cache.k.shape[3] != cfg.head_k_dim:
        raise ValueError("the cache's heads are not head_k_dim wide")
    N = lengths.numel()
    i32 = torch.int32
    if page_table.dim() != 2:
        raise ValueError("page_table must be [N, max_pages]")
    c = KdaKvCacheC.from_buffer_copy(cache._c)
    c.max_pages = _int32(page_table.shape[1])
    c.page_table = _at("page_table", page_table, (N, page_table.shape[1]), i32, dev)
    c.lengths = _at("lengths", lengths, (N,), i32, dev)
    c.cu_seqlens = _at("cu_seqlens", cu_seqlens, (N + 1,), i32, dev)
    return c, N, dev


def kda_append_kv(cfg: Config, cache: KvCache, cu_seqlens, page_table, lengths, k, v, k_weight=None,
                  eps: float = 1e-6, *, rope: Optional[Rope] = None, positions=None, stream=None):
    """Appends keys and values [n_tokens, kv heads, d] (io dtype; their tokens
    may be strided): token j of the q_n tokens of sequence n goes to position
    lengths[n] - q_n + j of page_table's pages.  cu_seqlens [N + 1], page_table
    [N, max_pages], lengths [N], int32; cu_seqlens None: one token each.  Keys
    are normed and rotated on the way as in kda_qk_norm_rope; positions None:
    the cache positions."""
    c, N, dev = _cache_at(cfg, cache, cu_seqlens, page_table, lengths)
    n, shape = k.shape[0], (k.shape[0], cache.k.shape[1], cfg.head_k_dim)
    kp, ks = _rows_at("k", k, shape, cfg.io_dtype, dev)
    vp, vs = _rows_at("v", v, shape, cfg.io_dtype, dev)
    wp = _at("k_weight", k_weight, (cfg.head_k_dim,), torch.float32, dev)
    rp, pp = _rope_at(rope, positions, n, dev)
    if _elsewhere(dev, stream):
        return _on_stream(dev, stream, lambda: kda_append_kv(cfg, cache, cu_seqlens, page_table, lengths, k, v, k_weight,
                                                              eps, rope=rope, positions=positions))
    _check(_lib.kda_append_kv(_attention_struct(cfg), rp, ctypes.byref(c), N, n, kp, ks, vp, vs, wp, eps, pp,
                              torch._C._cuda_getCurrentRawStream(dev.index)), "kda_append_kv")


def kda_read_kv(cfg: Config, cache: KvCache, cu_seqlens, page_table, lengths, n_tokens: int, *, k=None, v=None,
                stream=None):
    """The last cu_seqlens[n + 1] - cu_seqlens[n] rows of each sequence, as
    kda_append_kv left them.  Returns (k, v) [n_tokens, kv heads, d], out dtype;
    rows that are not held are 0, rows behind cu_seqlens[N] are not written."""
    c, N, dev = _cache_at(cfg, cache, cu_seqlens, page_table, lengths)
    shape, out = (n_tokens, cache.k.shape[1], cfg.head_k_dim), cfg.out_dtype
    kp, vp = _at("k", k, shape, out, dev), _at("v", v, shape, out, dev)
    if _elsewhere(dev, stream):
        return _on_stream(dev, stream, lambda: kda_read_kv(cfg, cache, cu_seqlens, page_table, lengths, n_tokens, k=k, v=v))
    st = torch._C._cuda_getCurrentRawStream(dev.index)
    k_ = torch.empty(shape, dtype=out, device=dev) if k is None else k
    v_ = torch.empty(shape, dtype=out, device=dev) if v is None else v
    _check(_lib.kda_read_kv(_attention_struct(cfg), ctypes.byref(c), N, n_tokens, kp or k_.data_ptr(),
                            vp or v_.data_ptr(), st), "kda_read_kv")
    return k_, v_


def kda_paged_attention_workspace_bytes(cfg: Config, num_kv_heads: int, N: int, n_tokens: int, max_q: int = 0) -> int:
    """Bytes of workspace; 0 for sizes that the library refuses."""
    return int(_lib.kda_paged_attention_workspace_bytes(_attention_struct(cfg), _int32(num_kv_heads), _int32(N),
                                                        _int64(n_tokens), _int32(max_q)))


def kda_paged_attention(cfg: Config, cache: KvCache, q, cu_seqlens, page_table, lengths, scale: Optional[float] = None,
                        *, max_q: int = 0, o=None, lse=None, workspace=None, stream=None):
    """Attention of each sequence's newest tokens, q [n_tokens, num_heads, d]
    (io dtype), over its cache (their own keys and values among it), causal:
    token j of q_n sees positions up to lengths[n] - q_n + j.  scale: 1 /
    sqrt(d) by default; max_q: at least the most tokens of one sequence (0: not
    known, the kernel is then chosen by the mean; cu_seqlens None: one each).  lse: fp32 [n_tokens, num_heads], filled
    with the log of the sum of exponentials.  Returns o, out dtype; rows behind
    cu_seqlens[N] are not written."""
    c, N, dev = _cache_at(cfg, cache, cu_seqlens, page_table, lengths)
    d, H, heads = cfg.head_k_dim, cfg.num_heads, cache.k.shape[1]
    n = q.shape[0]
    qp, op = _at("q", q, (n, H, d), cfg.io_dtype, dev), _at("o", o, (n, H, d), cfg.out_dtype, dev)
    lp = _at("lse", lse, (n, H), torch.float32, dev)
    if _elsewhere(dev, stream):
        return _on_stream(dev, stream, lambda: kda_paged_attention(cfg, cache, q, cu_seqlens, page_table, lengths, scale,
                                                                    max_q=max_q, o=o, lse=lse, workspace=workspace))
    st = torch._C._cuda_getCurrentRawStream(dev.index)
    o_ = torch.empty((n, H, d), dtype=cfg.out_dtype, device=dev) if o is None else o
    cs = _attention_struct(cfg)
    max_q = 1 if cu_seqlens is None else _int32(max_q)
    ws, wsp, size = _workspace_at(_lib.kda_paged_attention_workspace_bytes(cs, heads, N, n, max_q), dev, workspace)
    _check(_lib.kda_paged_attention(cs, ctypes.byref(c), N, n, max_q, qp, d ** -0.5 if scale is None else scale,
                                    op or o_.data_ptr(), lp, wsp, size, st), "kda_paged_attention")
    return o_
