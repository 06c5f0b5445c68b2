"""Thin Python binding of libgdn (include/gdn.h), same names as the C ABI.

Only argument marshalling lives here: torch allocates device memory (outputs and the
workspace) and provides the stream; every step of the recurrence runs in the CUDA kernels of
libgdn.so.  There is no CPU fallback: if the library is missing or a tensor is not on a CUDA
device, the call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib.util
import os
from typing import Dict, Optional, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgdn.so")

GDN_BF16, GDN_F32 = 0, 1
_STATUS = {0: "GDN_OK", 1: "GDN_ERR_INVALID_ARG", 2: "GDN_ERR_UNSUPPORTED", 3: "GDN_ERR_CUDA",
           4: "GDN_ERR_WORKSPACE", 5: "GDN_ERR_TIMEOUT"}

P = ctypes.c_void_p
I64 = ctypes.c_int64
I32 = ctypes.c_int32
F32 = ctypes.c_float


class Strides(ctypes.Structure):
    """gdn_strides: token strides in elements (0 = dense)."""
    _fields_ = [("q", I64), ("k", I64), ("v", I64), ("alpha", I64), ("b", I64), ("w", I64), ("z", I64)]


class FwdArgs(ctypes.Structure):
    _fields_ = [("q", P), ("k", P), ("v", P), ("alpha", P), ("b", P), ("w", P), ("h0", P),
                ("z", P), ("o", P), ("ht", P), ("head_map", P),
                ("B", I64), ("T", I64), ("Hk", I64), ("Hv", I64), ("dk", I64), ("dv", I64),
                ("scale", F32), ("alpha_per_channel", I32), ("gates_per_channel", I32),
                ("dtype", I32), ("gate_dtype", I32), ("out_f32", I32),
                ("bwd_cache", P), ("bwd_cache_bytes", ctypes.c_size_t), ("gate_logits", I32),
                ("alpha_scale", P), ("strides", Strides)]


class BwdArgs(ctypes.Structure):
    _fields_ = [("q", P), ("k", P), ("v", P), ("alpha", P), ("b", P), ("w", P), ("h0", P),
                ("head_map", P), ("grad_o", P), ("grad_ht", P), ("grad_q", P), ("grad_k", P),
                ("grad_v", P), ("grad_alpha", P), ("grad_b", P), ("grad_w", P), ("grad_h0", P),
                ("B", I64), ("T", I64), ("Hk", I64), ("Hv", I64), ("dk", I64), ("dv", I64),
                ("scale", F32), ("alpha_per_channel", I32), ("gates_per_channel", I32),
                ("dtype", I32), ("gate_dtype", I32),
                ("fwd_cache", P), ("fwd_cache_bytes", ctypes.c_size_t), ("gate_logits", I32),
                ("alpha_scale", P), ("grad_alpha_scale", P), ("grads_in_dtype", I32), ("strides", Strides)]


class DecodeArgs(ctypes.Structure):
    _fields_ = [("q", P), ("k", P), ("v", P), ("alpha", P), ("b", P), ("w", P), ("state", P),
                ("o", P), ("head_map", P), ("conv_state", P), ("conv_w", P), ("z", P),
                ("N", I64), ("Hk", I64), ("Hv", I64), ("dk", I64), ("dv", I64),
                ("scale", F32), ("alpha_per_channel", I32), ("gates_per_channel", I32),
                ("dtype", I32), ("gate_dtype", I32), ("out_f32", I32), ("gate_logits", I32),
                ("alpha_scale", P), ("strides", Strides)]


class LayerArgs(ctypes.Structure):
    _fields_ = [("xq", P), ("xk", P), ("xv", P), ("conv_w", P), ("alpha", P), ("b", P), ("w", P),
                ("z", P), ("h0", P), ("y", P), ("ht", P), ("conv_state_out", P), ("head_map", P),
                ("B", I64), ("T", I64), ("Hk", I64), ("Hv", I64), ("dk", I64), ("dv", I64),
                ("scale", F32), ("alpha_per_channel", I32), ("gates_per_channel", I32),
                ("dtype", I32), ("gate_dtype", I32), ("out_f32", I32), ("bwd_cache", P),
                ("bwd_cache_bytes", ctypes.c_size_t), ("norm_w", P), ("norm_eps", F32), ("gate_logits", I32),
                ("alpha_scale", P), ("strides", Strides)]


class LayerBwdArgs(ctypes.Structure):
    _fields_ = [("xq", P), ("xk", P), ("xv", P), ("conv_w", P), ("alpha", P), ("b", P), ("w", P),
                ("z", P), ("h0", P), ("head_map", P), ("grad_y", P), ("grad_ht", P),
                ("grad_xq", P), ("grad_xk", P), ("grad_xv", P), ("grad_conv_w", P), ("grad_alpha", P),
                ("grad_b", P), ("grad_w", P), ("grad_z", P), ("grad_h0", P),
                ("B", I64), ("T", I64), ("Hk", I64), ("Hv", I64), ("dk", I64), ("dv", I64),
                ("scale", F32), ("alpha_per_channel", I32), ("gates_per_channel", I32),
                ("dtype", I32), ("gate_dtype", I32), ("fwd_cache", P), ("fwd_cache_bytes", ctypes.c_size_t),
                ("norm_w", P), ("norm_eps", F32), ("grad_norm_w", P), ("gate_logits", I32),
                ("alpha_scale", P), ("grad_alpha_scale", P), ("strides", Strides)]


class QkNorm(ctypes.Structure):
    _fields_ = [("q_norm_w", P), ("k_norm_w", P), ("inv_freq", P), ("rot_dim", I64), ("interleaved", I32),
                ("norm_eps", F32), ("rot_scale", F32)]


class QkFwdArgs(ctypes.Structure):
    _fields_ = [("q", P), ("k", P), ("positions", P), ("q_out", P), ("k_out", P), ("T", I64), ("Hq", I64),
                ("Hk", I64), ("d", I64), ("dtype", I32), ("norm", QkNorm), ("strides", Strides)]


class QkBwdArgs(ctypes.Structure):
    _fields_ = [("q", P), ("k", P), ("positions", P), ("grad_q_out", P), ("grad_k_out", P), ("grad_q", P),
                ("grad_k", P), ("grad_q_norm_w", P), ("grad_k_norm_w", P), ("T", I64), ("Hq", I64), ("Hk", I64),
                ("d", I64), ("dtype", I32), ("norm", QkNorm), ("strides", Strides)]


class AttnFwdArgs(ctypes.Structure):
    _fields_ = [("q", P), ("k", P), ("v", P), ("cu_seqlens", P), ("o", P), ("T", I64), ("nseq", I64), ("Hq", I64),
                ("Hk", I64), ("d", I64), ("window", I64), ("scale", F32), ("dtype", I32), ("bwd_cache", P),
                ("bwd_cache_bytes", ctypes.c_size_t), ("strides", Strides)]


class AttnBwdArgs(ctypes.Structure):
    _fields_ = [("q", P), ("k", P), ("v", P), ("cu_seqlens", P), ("o", P), ("grad_o", P), ("grad_q", P),
                ("grad_k", P), ("grad_v", P), ("T", I64), ("nseq", I64), ("Hq", I64), ("Hk", I64), ("d", I64),
                ("window", I64), ("scale", F32), ("dtype", I32), ("fwd_cache", P),
                ("fwd_cache_bytes", ctypes.c_size_t), ("strides", Strides)]


class KvAppendArgs(ctypes.Structure):
    _fields_ = [("q", P), ("k", P), ("v", P), ("cu_seqlens", P), ("context_lens", P), ("block_table", P),
                ("q_out", P), ("k_out", P), ("k_cache", P), ("v_cache", P), ("T", I64), ("nseq", I64), ("Hq", I64),
                ("Hk", I64), ("d", I64), ("num_pages", I64), ("page_size", I64), ("max_pages", I64),
                ("dtype", I32), ("norm", QkNorm), ("strides", Strides)]


class AttnDecodeArgs(ctypes.Structure):
    _fields_ = [("q", P), ("k_cache", P), ("v_cache", P), ("block_table", P), ("context_lens", P), ("o", P),
                ("N", I64), ("Hq", I64), ("Hk", I64), ("d", I64), ("num_pages", I64), ("page_size", I64),
                ("max_pages", I64), ("max_context", I64), ("window", I64), ("scale", F32), ("dtype", I32),
                ("strides", Strides)]


EXPORTED = ["gdn_chunk_fwd_cache_size", "gdn_chunk_fwd_workspace_size", "gdn_chunk_fwd", "gdn_chunk_fwd_noalloc",
            "gdn_chunk_fwd_noalloc_status", "gdn_chunk_bwd_workspace_size",
            "gdn_chunk_bwd", "gdn_decode_step", "gdn_layer_core_fwd_cache_size", "gdn_layer_core_fwd_workspace_size",
            "gdn_layer_core_fwd", "gdn_layer_core_bwd_workspace_size", "gdn_layer_core_bwd",
            "gdn_segment_map_workspace_size", "gdn_segment_map", "gdn_state_compose",
            "gdn_qk_norm_rope_fwd", "gdn_qk_norm_rope_bwd_workspace_size", "gdn_qk_norm_rope_bwd",
            "gdn_attn_fwd_cache_size", "gdn_attn_fwd_workspace_size", "gdn_attn_fwd",
            "gdn_attn_bwd_workspace_size", "gdn_attn_bwd", "gdn_kv_append",
            "gdn_attn_decode_workspace_size", "gdn_attn_decode",
            "gdn_workspace_status", "gdn_last_error", "gdn_kernel_launches", "gdn_version"]

_lib = None


class GdnError(RuntimeError):
    pass


def load(path: str = LIB_PATH):
    """Load libgdn.so and declare its C signatures.  Raises if the library is missing."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise GdnError(f"{path} is missing: build it with `python -m gated_delta_rule_76_b200.build`")
    lib = ctypes.CDLL(path)
    lib.gdn_chunk_fwd_cache_size.argtypes = [ctypes.POINTER(FwdArgs)]
    lib.gdn_chunk_fwd_cache_size.restype = ctypes.c_size_t
    lib.gdn_chunk_fwd_workspace_size.argtypes = [ctypes.POINTER(FwdArgs)]
    lib.gdn_chunk_fwd_workspace_size.restype = ctypes.c_size_t
    lib.gdn_chunk_fwd.argtypes = [ctypes.POINTER(FwdArgs), P, ctypes.c_size_t, P]
    lib.gdn_chunk_fwd.restype = ctypes.c_int
    lib.gdn_chunk_fwd_noalloc.argtypes = [ctypes.POINTER(FwdArgs), P]
    lib.gdn_chunk_fwd_noalloc.restype = ctypes.c_int
    lib.gdn_chunk_fwd_noalloc_status.argtypes = [P]
    lib.gdn_chunk_fwd_noalloc_status.restype = ctypes.c_int
    lib.gdn_chunk_bwd_workspace_size.argtypes = [ctypes.POINTER(BwdArgs)]
    lib.gdn_chunk_bwd_workspace_size.restype = ctypes.c_size_t
    lib.gdn_chunk_bwd.argtypes = [ctypes.POINTER(BwdArgs), P, ctypes.c_size_t, P]
    lib.gdn_chunk_bwd.restype = ctypes.c_int
    lib.gdn_decode_step.argtypes = [ctypes.POINTER(DecodeArgs), P]
    lib.gdn_decode_step.restype = ctypes.c_int
    lib.gdn_layer_core_fwd_cache_size.argtypes = [ctypes.POINTER(LayerArgs)]
    lib.gdn_layer_core_fwd_cache_size.restype = ctypes.c_size_t
    lib.gdn_layer_core_fwd_workspace_size.argtypes = [ctypes.POINTER(LayerArgs)]
    lib.gdn_layer_core_fwd_workspace_size.restype = ctypes.c_size_t
    lib.gdn_layer_core_fwd.argtypes = [ctypes.POINTER(LayerArgs), P, ctypes.c_size_t, P]
    lib.gdn_layer_core_fwd.restype = ctypes.c_int
    lib.gdn_layer_core_bwd_workspace_size.argtypes = [ctypes.POINTER(LayerBwdArgs)]
    lib.gdn_layer_core_bwd_workspace_size.restype = ctypes.c_size_t
    lib.gdn_layer_core_bwd.argtypes = [ctypes.POINTER(LayerBwdArgs), P, ctypes.c_size_t, P]
    lib.gdn_layer_core_bwd.restype = ctypes.c_int
    lib.gdn_segment_map_workspace_size.argtypes = [ctypes.POINTER(FwdArgs)]
    lib.gdn_segment_map_workspace_size.restype = ctypes.c_size_t
    lib.gdn_segment_map.argtypes = [ctypes.POINTER(FwdArgs), P, P, ctypes.c_size_t, P]
    lib.gdn_segment_map.restype = ctypes.c_int
    lib.gdn_state_compose.argtypes = [P, P, P, P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int32, P]
    lib.gdn_state_compose.restype = ctypes.c_int
    lib.gdn_qk_norm_rope_fwd.argtypes = [ctypes.POINTER(QkFwdArgs), P]
    lib.gdn_qk_norm_rope_fwd.restype = ctypes.c_int
    lib.gdn_kv_append.argtypes = [ctypes.POINTER(KvAppendArgs), P]
    lib.gdn_kv_append.restype = ctypes.c_int
    for name, struct in (("gdn_qk_norm_rope_bwd", QkBwdArgs), ("gdn_attn_fwd", AttnFwdArgs),
                         ("gdn_attn_bwd", AttnBwdArgs), ("gdn_attn_decode", AttnDecodeArgs)):
        size, call = getattr(lib, name + "_workspace_size"), getattr(lib, name)
        size.argtypes = [ctypes.POINTER(struct)]
        size.restype = ctypes.c_size_t
        call.argtypes = [ctypes.POINTER(struct), P, ctypes.c_size_t, P]
        call.restype = ctypes.c_int
    lib.gdn_attn_fwd_cache_size.argtypes = [ctypes.POINTER(AttnFwdArgs)]
    lib.gdn_attn_fwd_cache_size.restype = ctypes.c_size_t
    lib.gdn_workspace_status.argtypes = [P, P]
    lib.gdn_workspace_status.restype = ctypes.c_int
    lib.gdn_last_error.argtypes = []
    lib.gdn_last_error.restype = ctypes.c_char_p
    lib.gdn_kernel_launches.argtypes = []
    lib.gdn_kernel_launches.restype = ctypes.c_longlong
    lib.gdn_version.argtypes = []
    lib.gdn_version.restype = ctypes.c_int
    if path == LIB_PATH:
        _lib = lib
    return lib


def kernel_launches() -> int:
    """Kernels launched by libgdn in this process so far."""
    return int(load().gdn_kernel_launches())


def check(status: int, what: str):
    if status != 0:
        msg = load().gdn_last_error().decode(errors="replace")
        raise GdnError(f"{what}: {_STATUS.get(status, status)}: {msg}")


# ---------------------------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------------------------
def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise GdnError("libgdn takes CUDA tensors only (there is no CPU path)")
    if not t.is_contiguous():
        raise GdnError("libgdn takes contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _tok(t: Optional[torch.Tensor], lead: int = 2):
    """A token-major input as (pointer, token stride in elements, 0 when dense).  Besides a
    contiguous tensor it takes a view whose heads and channels are dense and whose tokens are
    evenly spaced, such as a slice of a fused projection [B, T, C] viewed as [B, T, H, d].
    ``lead`` is the number of token dimensions (2: [B, T, ...]; 1: the decode step's [N, ...])."""
    if t is None:
        return None, 0
    if t.is_contiguous():
        return _ptr(t), 0
    if not t.is_cuda:
        raise GdnError("libgdn takes CUDA tensors only (there is no CPU path)")
    return ctypes.c_void_p(t.data_ptr()), _token_stride(tuple(t.shape), tuple(t.stride()), lead)


def _token_stride(shape, strides, lead: int) -> int:
    """The token stride, in elements, of a tensor of this shape and these strides (0 when its
    tokens are dense); its first ``lead`` dimensions index tokens."""
    row = 1
    for dim in range(len(shape) - 1, lead - 1, -1):
        if shape[dim] != 1 and strides[dim] != row:
            raise GdnError("libgdn takes token-major tensors whose heads and channels are dense")
        row *= shape[dim]
    dims = [d for d in range(lead) if shape[d] != 1]
    s = strides[dims[-1]] if dims else row
    if len(dims) == 2 and strides[dims[0]] != shape[dims[1]] * s:
        raise GdnError("libgdn takes token-major tensors whose tokens are evenly spaced")
    if s < row:
        raise GdnError(f"token stride {s} is below the {row} elements of a token")
    return 0 if s == row else s


def _inputs(lead: int, q, k, v, alpha, b, w, z=None):
    """Pointers and gdn_strides of a call's token-major inputs."""
    ptrs, strides = {}, {}
    for name, t in (("q", q), ("k", k), ("v", v), ("alpha", alpha), ("b", b), ("w", w), ("z", z)):
        ptrs[name], strides[name] = _tok(t, lead)
    return ptrs, Strides(**strides)


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return GDN_BF16
    if t.dtype == torch.float32:
        return GDN_F32
    raise GdnError(f"unsupported dtype {t.dtype}")


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _workspace(nbytes: int, device, workspace: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    if nbytes == 0:
        return None
    if workspace is not None and workspace.numel() * workspace.element_size() >= nbytes:
        return workspace
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _gates(alpha, b, w, beta):
    if beta is not None:
        if b is not None or w is not None:
            raise GdnError("give either beta or (b, w)")
        return beta, None, 0
    if b is None or w is None:
        raise GdnError("channel gates need both b and w")
    return b, w, 1


def _head_map(head_map, device, Hk: int):
    """The value-head -> key-head map as an int32 device array.  A map given on the host (a list
    or a CPU tensor) is checked before it is uploaded: every entry must be in [0, Hk).  A map
    already on the device is passed through unchecked (checking it would synchronise)."""
    if head_map is None:
        return None
    if not torch.is_tensor(head_map):
        head_map = torch.tensor(head_map, dtype=torch.int32)
    if head_map.device.type == "cpu" and head_map.numel():
        lo, hi = int(head_map.min()), int(head_map.max())
        if lo < 0 or hi >= Hk:
            raise GdnError(f"head_map entries must be in [0, {Hk}); got [{lo}, {hi}]")
    return head_map.to(device=device, dtype=torch.int32).contiguous()


# ---------------------------------------------------------------------------------------------
# public calls
#
# Token-major inputs (q, k, v, the gates, z; xq, xk, xv for the layer calls) may be views whose
# tokens are evenly spaced and whose heads and channels are dense, such as column slices of one
# fused projection buffer viewed as [B, T, H, d]: they are passed with their token stride
# (gdn_strides), without a copy here.  Every other tensor must be contiguous.
# ---------------------------------------------------------------------------------------------
def fwd_args(q, k, v, alpha, b=None, w=None, beta=None, h0=None, z=None, head_map=None,
             scale: float = 1.0, o=None, ht=None, bwd_cache=None, alpha_scale=None) -> Tuple[FwdArgs, list]:
    """Build the gdn_fwd_args struct (the returned list keeps referenced tensors alive).
    ``alpha_scale`` [Hv] fp32: the gates are logits (alpha = exp(-alpha_scale softplus(x)),
    b, w, beta = sigmoid(x))."""
    bb, ww, gpc = _gates(alpha, b, w, beta)
    B, T, Hk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    hm = _head_map(head_map, q.device, q.shape[-2])
    tp, ts = _inputs(2, q, k, v, alpha, bb, ww, z)
    a = FwdArgs(q=tp["q"], k=tp["k"], v=tp["v"], alpha=tp["alpha"], b=tp["b"], w=tp["w"],
                h0=_ptr(h0), z=tp["z"], o=_ptr(o), ht=_ptr(ht), head_map=_ptr(hm),
                B=B, T=T, Hk=Hk, Hv=Hv, dk=dk, dv=dv, scale=scale,
                alpha_per_channel=int(alpha.dim() == 4), gates_per_channel=gpc,
                dtype=_dt(q), gate_dtype=_dt(alpha),
                out_f32=int(o is not None and o.dtype == torch.float32 and q.dtype != torch.float32),
                bwd_cache=_ptr(bwd_cache),
                bwd_cache_bytes=0 if bwd_cache is None else bwd_cache.numel() * bwd_cache.element_size(),
                gate_logits=int(alpha_scale is not None), alpha_scale=_ptr(alpha_scale), strides=ts)
    return a, [q, k, v, alpha, bb, ww, h0, z, o, ht, hm, bwd_cache, alpha_scale]


def gdn_chunk_fwd_cache_size(q, k, v, alpha, b=None, w=None, beta=None, h0=None, head_map=None,
                             scale: float = 1.0, alpha_scale=None) -> int:
    """Bytes of the forward cache gdn_chunk_fwd(..., bwd_cache=) can fill for a later backward
    (0: this problem runs on the CUDA-core path, which keeps none)."""
    B, T, Hk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    a, keep = fwd_args(q, k, v, alpha, b, w, beta, h0, None, head_map, scale, alpha_scale=alpha_scale)
    return int(load().gdn_chunk_fwd_cache_size(ctypes.byref(a)))


def gdn_chunk_fwd(q, k, v, alpha, b=None, w=None, beta=None, h0=None, z=None, head_map=None,
                  scale: float = 1.0, *, o=None, ht=None, want_ht: bool = True, out_f32: bool = False,
                  bwd_cache: Optional[torch.Tensor] = None, alpha_scale: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None):
    """Chunkwise forward.  Returns (o [B,T,Hv,dv], ht [B,Hv,dk,dv] or None).
    ``out_f32`` writes o in fp32 (the unrounded accumulator) instead of the input dtype.
    ``bwd_cache``: a device byte tensor of gdn_chunk_fwd_cache_size() bytes that the forward fills
    for gdn_chunk_bwd(..., fwd_cache=) over the same inputs."""
    B, T, Hk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    if o is None:
        o = torch.empty((B, T, Hv, dv), dtype=torch.float32 if out_f32 else q.dtype, device=q.device)
    if ht is None and want_ht:
        ht = torch.empty((B, Hv, dk, dv), dtype=torch.float32, device=q.device)
    lib = load()
    a, keep = fwd_args(q, k, v, alpha, b, w, beta, h0, z, head_map, scale, o, ht, bwd_cache, alpha_scale)
    need = lib.gdn_chunk_fwd_workspace_size(ctypes.byref(a))
    ws = _workspace(need, q.device, workspace)
    check(lib.gdn_chunk_fwd(ctypes.byref(a), _ptr(ws), need, _stream(stream)), "gdn_chunk_fwd")
    return o, ht


def gdn_chunk_fwd_noalloc(q, k, v, alpha, b=None, w=None, beta=None, h0=None, z=None, head_map=None,
                          scale: float = 1.0, *, o=None, ht=None, want_ht: bool = True, out_f32: bool = False,
                          stream=None):
    """gdn_chunk_fwd with the library's built-in 16 MiB scratch instead of a workspace (calls on one
    device must not overlap in time).  Returns (o, ht)."""
    B, T, Hk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    if o is None:
        o = torch.empty((B, T, Hv, dv), dtype=torch.float32 if out_f32 else q.dtype, device=q.device)
    if ht is None and want_ht:
        ht = torch.empty((B, Hv, dk, dv), dtype=torch.float32, device=q.device)
    lib = load()
    a, keep = fwd_args(q, k, v, alpha, b, w, beta, h0, z, head_map, scale, o, ht)
    check(lib.gdn_chunk_fwd_noalloc(ctypes.byref(a), _stream(stream)), "gdn_chunk_fwd_noalloc")
    return o, ht


def gdn_chunk_fwd_noalloc_status(stream=None) -> int:
    """The status word of the built-in scratch after gdn_chunk_fwd_noalloc calls (synchronises
    ``stream``): 0, or GDN_ERR_TIMEOUT (5) if a bounded wait inside a kernel expired."""
    return int(load().gdn_chunk_fwd_noalloc_status(_stream(stream)))


def gdn_segment_map(q, k, v, alpha, b=None, w=None, beta=None, head_map=None, *, want_o: bool = False,
                    workspace: Optional[torch.Tensor] = None, stream=None):
    """The affine map of this segment of every sequence on the state: returns (M [B,Hv,dk,dk],
    N [B,Hv,dk,dv]) with state_after = M state_before + N, plus the segment's output from a zero
    entering state when ``want_o`` (then (M, N, o))."""
    B, T, Hk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    M = torch.empty((B, Hv, dk, dk), dtype=torch.float32, device=q.device)
    N = torch.empty((B, Hv, dk, dv), dtype=torch.float32, device=q.device)
    o = torch.empty((B, T, Hv, dv), dtype=q.dtype, device=q.device) if want_o else None
    lib = load()
    a, keep = fwd_args(q, k, v, alpha, b, w, beta, None, None, head_map, 1.0, o, N)
    need = lib.gdn_segment_map_workspace_size(ctypes.byref(a))
    ws = _workspace(need, q.device, workspace)
    check(lib.gdn_segment_map(ctypes.byref(a), _ptr(M), _ptr(ws), need, _stream(stream)), "gdn_segment_map")
    return (M, N, o) if want_o else (M, N)


def gdn_state_compose(M, N, S, *, transpose: bool = False, out: Optional[torch.Tensor] = None, stream=None):
    """op(M) S + N per (sequence, head) on the device, op = transpose or identity.  M [..., dk, dk],
    N and S [..., dk, dv] fp32 (S or N may be None: zero).  Returns the result (``out`` if given)."""
    ref = S if S is not None else N
    dk, dv = M.shape[-1], ref.shape[-1]
    pairs = M.numel() // (dk * dk)
    if out is None:
        out = torch.empty(ref.shape, dtype=torch.float32, device=M.device)
    check(load().gdn_state_compose(_ptr(M), _ptr(N), _ptr(S), _ptr(out), pairs, dk, dv, int(transpose),
                                   _stream(stream)), "gdn_state_compose")
    return out


def bwd_args(q, k, v, alpha, b=None, w=None, beta=None, h0=None, head_map=None, scale=1.0,
             grad_o=None, grad_ht=None, grads=None, fwd_cache=None, alpha_scale=None,
             grads_in_dtype: bool = False) -> Tuple[BwdArgs, list]:
    bb, ww, gpc = _gates(alpha, b, w, beta)
    B, T, Hk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    hm = _head_map(head_map, q.device, q.shape[-2])
    g = grads
    tp, ts = _inputs(2, q, k, v, alpha, bb, ww)
    a = BwdArgs(q=tp["q"], k=tp["k"], v=tp["v"], alpha=tp["alpha"], b=tp["b"], w=tp["w"],
                h0=_ptr(h0), head_map=_ptr(hm), grad_o=_ptr(grad_o), grad_ht=_ptr(grad_ht),
                grad_q=_ptr(g["dq"]), grad_k=_ptr(g["dk"]), grad_v=_ptr(g["dv"]),
                grad_alpha=_ptr(g["dalpha"]), grad_b=_ptr(g["db"] if gpc else g["dbeta"]),
                grad_w=_ptr(g.get("dw")), grad_h0=_ptr(g.get("dh0")),
                B=B, T=T, Hk=Hk, Hv=Hv, dk=dk, dv=dv, scale=scale,
                alpha_per_channel=int(alpha.dim() == 4), gates_per_channel=gpc,
                dtype=_dt(q), gate_dtype=_dt(alpha), fwd_cache=_ptr(fwd_cache),
                fwd_cache_bytes=0 if fwd_cache is None else fwd_cache.numel() * fwd_cache.element_size(),
                gate_logits=int(alpha_scale is not None), alpha_scale=_ptr(alpha_scale),
                grad_alpha_scale=_ptr(g.get("dalpha_scale")), grads_in_dtype=int(grads_in_dtype), strides=ts)
    return a, [q, k, v, alpha, bb, ww, h0, hm, grad_o, grad_ht, g, fwd_cache, alpha_scale]


def gdn_chunk_bwd(q, k, v, alpha, b=None, w=None, beta=None, h0=None, head_map=None,
                  scale: float = 1.0, *, grad_o, grad_ht=None, want_dh0: bool = True,
                  fwd_cache: Optional[torch.Tensor] = None, alpha_scale: Optional[torch.Tensor] = None,
                  grads_in_dtype: bool = False, workspace: Optional[torch.Tensor] = None,
                  stream=None) -> Dict[str, torch.Tensor]:
    """Chunkwise backward.  Returns dq, dk, dv, dalpha and db/dw (or dbeta) in fp32, or with
    ``grads_in_dtype`` in the dtypes of q and of the gates; dh0 in fp32.
    ``fwd_cache``: the cache a gdn_chunk_fwd(..., bwd_cache=) call filled with these same inputs
    (the forward is then not recomputed).  With ``alpha_scale`` the gates are logits: dalpha, db,
    dw, dbeta are the gradients of the logits, and dalpha_scale [Hv] that of alpha_scale."""
    bb, ww, gpc = _gates(alpha, b, w, beta)
    like = lambda t: torch.empty(t.shape, dtype=t.dtype if grads_in_dtype else torch.float32, device=t.device)
    grads = {"dq": like(q), "dk": like(k), "dv": like(v), "dalpha": like(alpha)}
    if gpc:
        grads["db"] = like(b)
        grads["dw"] = like(w)
    else:
        grads["dbeta"] = like(beta)
    if want_dh0:
        B, T, Hk, dk = q.shape
        Hv, dv = v.shape[2], v.shape[3]
        grads["dh0"] = torch.empty((B, Hv, dk, dv), dtype=torch.float32, device=q.device)
    if alpha_scale is not None:
        grads["dalpha_scale"] = torch.empty(tuple(alpha_scale.shape), dtype=torch.float32, device=q.device)
    lib = load()
    a, keep = bwd_args(q, k, v, alpha, b, w, beta, h0, head_map, scale, grad_o, grad_ht, grads, fwd_cache,
                       alpha_scale, grads_in_dtype)
    need = lib.gdn_chunk_bwd_workspace_size(ctypes.byref(a))
    ws = _workspace(need, q.device, workspace)
    check(lib.gdn_chunk_bwd(ctypes.byref(a), _ptr(ws), need, _stream(stream)), "gdn_chunk_bwd")
    return grads


def gdn_decode_step(state, q, k, v, alpha, b=None, w=None, beta=None, head_map=None,
                    scale: float = 1.0, *, conv_state=None, conv_w=None, z=None, o=None,
                    out_f32: bool = False, alpha_scale=None, stream=None):
    """One token for N sequences; ``state`` [N,Hv,dk,dv] fp32 is updated in place.  Returns o."""
    bb, ww, gpc = _gates(alpha, b, w, beta)
    N, Hk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    if o is None:
        o = torch.empty((N, Hv, dv), dtype=torch.float32 if out_f32 else q.dtype, device=q.device)
    hm = _head_map(head_map, q.device, q.shape[-2])
    tp, ts = _inputs(1, q, k, v, alpha, bb, ww, z)
    a = DecodeArgs(q=tp["q"], k=tp["k"], v=tp["v"], alpha=tp["alpha"], b=tp["b"], w=tp["w"],
                   state=_ptr(state), o=_ptr(o), head_map=_ptr(hm), conv_state=_ptr(conv_state),
                   conv_w=_ptr(conv_w), z=tp["z"], N=N, Hk=Hk, Hv=Hv, dk=dk, dv=dv, scale=scale,
                   alpha_per_channel=int(alpha.dim() == 3), gates_per_channel=gpc,
                   dtype=_dt(q), gate_dtype=_dt(alpha),
                   out_f32=int(o.dtype == torch.float32 and q.dtype != torch.float32),
                   gate_logits=int(alpha_scale is not None), alpha_scale=_ptr(alpha_scale), strides=ts)
    check(load().gdn_decode_step(ctypes.byref(a), _stream(stream)), "gdn_decode_step")
    return o


NORM_EPS = 1e-6  # the output norm's epsilon when the caller gives none


def _layer_args(xq, xk, xv, conv_w, alpha, z, b, w, beta, h0, head_map, scale, y=None, ht=None, cs=None,
                out_f32=0, bwd_cache=None, norm_w=None, norm_eps=NORM_EPS, alpha_scale=None):
    bb, ww, gpc = _gates(alpha, b, w, beta)
    B, T, Hk, dk = xq.shape
    Hv, dv = xv.shape[2], xv.shape[3]
    hm = _head_map(head_map, xq.device, xq.shape[-2])
    tp, ts = _inputs(2, xq, xk, xv, alpha, bb, ww, z)
    a = LayerArgs(xq=tp["q"], xk=tp["k"], xv=tp["v"], conv_w=_ptr(conv_w), alpha=tp["alpha"],
                  b=tp["b"], w=tp["w"], z=tp["z"], h0=_ptr(h0), y=_ptr(y), ht=_ptr(ht),
                  conv_state_out=_ptr(cs), head_map=_ptr(hm), B=B, T=T, Hk=Hk, Hv=Hv, dk=dk,
                  dv=dv, scale=scale, alpha_per_channel=int(alpha.dim() == 4),
                  gates_per_channel=gpc, dtype=_dt(xq), gate_dtype=_dt(alpha), out_f32=out_f32,
                  bwd_cache=_ptr(bwd_cache), bwd_cache_bytes=bwd_cache.numel() if bwd_cache is not None else 0,
                  norm_w=_ptr(norm_w), norm_eps=norm_eps, gate_logits=int(alpha_scale is not None),
                  alpha_scale=_ptr(alpha_scale), strides=ts)
    return a, hm


def gdn_layer_core_fwd_cache_size(xq, xk, xv, conv_w, alpha, z, b=None, w=None, beta=None, h0=None,
                                  head_map=None, scale: float = 1.0, norm_w=None) -> int:
    """Bytes of the layer forward's optional backward cache (0 where it cannot keep one)."""
    a, _ = _layer_args(xq, xk, xv, conv_w, alpha, z, b, w, beta, h0, head_map, scale, norm_w=norm_w)
    return int(load().gdn_layer_core_fwd_cache_size(ctypes.byref(a)))


def gdn_layer_core_fwd(xq, xk, xv, conv_w, alpha, z, b=None, w=None, beta=None, h0=None,
                       head_map=None, scale: float = 1.0, *, want_ht: bool = True,
                       want_conv_state: bool = False, y=None, out_f32: bool = False,
                       bwd_cache: Optional[torch.Tensor] = None, norm_w=None, norm_eps: float = NORM_EPS,
                       alpha_scale=None, workspace: Optional[torch.Tensor] = None, stream=None):
    """GQA layer core forward.  Returns (y, ht or None, conv_state or None).  ``bwd_cache``: a
    uint8 device tensor of gdn_layer_core_fwd_cache_size() bytes that a later
    gdn_layer_core_bwd(..., fwd_cache=) over the same inputs reads.  ``norm_w`` [dv] (the layer's
    dtype): the output norm before the gate, y = RMSNorm(o) * norm_w * swish(z)."""
    B, T, Hk, dk = xq.shape
    Hv, dv = xv.shape[2], xv.shape[3]
    if y is None:
        y = torch.empty((B, T, Hv, dv), dtype=torch.float32 if out_f32 else xq.dtype, device=xq.device)
    ht = torch.empty((B, Hv, dk, dv), dtype=torch.float32, device=xq.device) if want_ht else None
    cs = (torch.empty((B, 2 * Hk * dk + Hv * dv, 3), dtype=xq.dtype, device=xq.device)
          if want_conv_state else None)
    a, hm = _layer_args(xq, xk, xv, conv_w, alpha, z, b, w, beta, h0, head_map, scale, y=y, ht=ht, cs=cs,
                        out_f32=int(y.dtype == torch.float32 and xq.dtype != torch.float32), bwd_cache=bwd_cache,
                        norm_w=norm_w, norm_eps=norm_eps, alpha_scale=alpha_scale)
    lib = load()
    need = lib.gdn_layer_core_fwd_workspace_size(ctypes.byref(a))
    ws = _workspace(need, xq.device, workspace)
    check(lib.gdn_layer_core_fwd(ctypes.byref(a), _ptr(ws), need, _stream(stream)),
          "gdn_layer_core_fwd")
    return y, ht, cs


def gdn_layer_core_bwd(xq, xk, xv, conv_w, alpha, z, grad_y, b=None, w=None, beta=None, h0=None,
                       grad_ht=None, head_map=None, scale: float = 1.0, *, want_h0_grad: bool = True,
                       fwd_cache: Optional[torch.Tensor] = None, norm_w=None, norm_eps: float = NORM_EPS,
                       alpha_scale=None, workspace: Optional[torch.Tensor] = None,
                       stream=None) -> Dict[str, torch.Tensor]:
    """GQA layer core backward (reverse mode of gdn_layer_core_fwd).  Returns a dict of fp32
    gradients: dxq, dxk, dxv, dconv_w, dalpha, dz, dh0 (or None), db/dw or dbeta, and dnorm_w
    with the output norm (``norm_w``).
    ``fwd_cache``: the cache a gdn_layer_core_fwd(..., bwd_cache=) call filled with these inputs."""
    bb, ww, gpc = _gates(alpha, b, w, beta)
    B, T, Hk, dk = xq.shape
    Hv, dv = xv.shape[2], xv.shape[3]
    dev = xq.device
    f32 = dict(dtype=torch.float32, device=dev)
    out = {"dxq": torch.empty((B, T, Hk, dk), **f32), "dxk": torch.empty((B, T, Hk, dk), **f32),
           "dxv": torch.empty((B, T, Hv, dv), **f32), "dconv_w": torch.empty(tuple(conv_w.shape), **f32),
           "dalpha": torch.empty(tuple(alpha.shape), **f32), "dz": torch.empty((B, T, Hv, dv), **f32),
           "dh0": torch.empty((B, Hv, dk, dv), **f32) if want_h0_grad else None}
    if gpc:
        out["db"] = torch.empty(tuple(bb.shape), **f32)
        out["dw"] = torch.empty(tuple(ww.shape), **f32)
        gb, gw = out["db"], out["dw"]
    else:
        out["dbeta"] = torch.empty(tuple(bb.shape), **f32)
        gb, gw = out["dbeta"], None
    if norm_w is not None:
        out["dnorm_w"] = torch.empty((dv,), **f32)
    if alpha_scale is not None:
        out["dalpha_scale"] = torch.empty(tuple(alpha_scale.shape), **f32)
    hm = _head_map(head_map, dev, Hk)
    tp, ts = _inputs(2, xq, xk, xv, alpha, bb, ww, z)
    a = LayerBwdArgs(xq=tp["q"], xk=tp["k"], xv=tp["v"], conv_w=_ptr(conv_w), alpha=tp["alpha"],
                     b=tp["b"], w=tp["w"], z=tp["z"], h0=_ptr(h0), head_map=_ptr(hm), grad_y=_ptr(grad_y),
                     grad_ht=_ptr(grad_ht), grad_xq=_ptr(out["dxq"]), grad_xk=_ptr(out["dxk"]),
                     grad_xv=_ptr(out["dxv"]), grad_conv_w=_ptr(out["dconv_w"]), grad_alpha=_ptr(out["dalpha"]),
                     grad_b=_ptr(gb), grad_w=_ptr(gw), grad_z=_ptr(out["dz"]), grad_h0=_ptr(out["dh0"]),
                     B=B, T=T, Hk=Hk, Hv=Hv, dk=dk, dv=dv, scale=scale,
                     alpha_per_channel=int(alpha.dim() == 4), gates_per_channel=gpc, dtype=_dt(xq),
                     gate_dtype=_dt(alpha), fwd_cache=_ptr(fwd_cache),
                     fwd_cache_bytes=fwd_cache.numel() if fwd_cache is not None else 0,
                     norm_w=_ptr(norm_w), norm_eps=norm_eps, grad_norm_w=_ptr(out.get("dnorm_w")),
                     gate_logits=int(alpha_scale is not None), alpha_scale=_ptr(alpha_scale),
                     grad_alpha_scale=_ptr(out.get("dalpha_scale")), strides=ts)
    lib = load()
    need = lib.gdn_layer_core_bwd_workspace_size(ctypes.byref(a))
    ws = _workspace(need, dev, workspace)
    check(lib.gdn_layer_core_bwd(ctypes.byref(a), _ptr(ws), need, _stream(stream)), "gdn_layer_core_bwd")
    return out


# ---------------------------------------------------------------------------------------------
# the softmax-attention layer of hybrid stacks
#
# Serving calls these once a token and layer, on kernels of a few microseconds.  They are marshalled natively where
# their arguments are plain (csrc/binding/attn_calls.cpp: 5 to 8 us a call instead of 13 to 17); the marshalling below
# takes every other case.
# ---------------------------------------------------------------------------------------------
def _find_native():
    """The native module, calling the library that load() has opened; None where it is not built: every call then goes the
    general way.  Not looked for on import: a program that reads the package's inputs, or builds the library, maps none of it."""
    global _native
    from .build import binding
    lib, native, path = load(), None, binding()
    if os.path.exists(path):
        spec = importlib.util.spec_from_file_location(f"{__package__}._attn_calls", path)
        try:
            native = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(native)
        except ImportError:  # against other libraries than this host's
            native = None
        else:
            native.bind({name: ctypes.cast(getattr(lib, name), P).value for name in native.entries()})
    _native = native
    return native


def __getattr__(name):  # _native before the first call
    if name == "_native":
        return _find_native()
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")


def _native_calls():
    try:
        return _native
    except NameError:
        return _find_native()


_AS_IS = contextlib.nullcontext()
# what torch.cuda.current_device and current_stream come down to once CUDA is up, as it is where a CUDA tensor exists
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _on(t: torch.Tensor, stream):
    """The context the calls below run in: their tensors' device, whichever is current, and the given
    stream, so that what they allocate (results, workspace) belongs to the stream they run on."""
    if not t.is_cuda:
        raise GdnError("libgdn takes CUDA tensors only (there is no CPU path)")
    if stream is None:
        return _AS_IS if t.get_device() == _current_device() else torch.cuda.device(t.device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=t.device)
    if stream.device != t.device:
        raise GdnError(f"a stream of {stream.device} for tensors on {t.device}")
    return torch.cuda.stream(stream)


def _unexpected(name, t, shape, dtype, device):
    return GdnError(f"{name} is {tuple(t.shape)} {t.dtype} on {t.device}: expected "
                    f"{'' if shape is None else tuple(shape)} {dtype} on cuda:{device}")


def _dense(name: str, t: Optional[torch.Tensor], shape, dtype, device: int):
    """The address of a contiguous tensor of this shape (None: any), dtype and device, or None."""
    if t is None:
        return None
    if (shape is not None and t.shape != shape) or t.dtype != dtype or t.get_device() != device:
        raise _unexpected(name, t, shape, dtype, device)
    if not t.is_contiguous():
        raise GdnError("libgdn takes contiguous tensors")
    return t.data_ptr()


def _result(name: str, t: Optional[torch.Tensor], like: torch.Tensor, dtype, device: int):
    """(the caller's buffer for a result laid out like `like`, or a new one; its address)."""
    if t is None:
        t = torch.empty_like(like, memory_format=torch.contiguous_format)
        return t, t.data_ptr()
    return t, _dense(name, t, like.shape, dtype, device)


def _first(name: str, t: torch.Tensor):
    """(device, dtype, T, heads, d, token stride) of the packed tokens [T, heads, d] that the others go by."""
    shape = t.shape
    if len(shape) != 3:
        raise GdnError(f"{name} has shape {tuple(shape)}: expected [tokens, heads, channels]")
    return (t.get_device(), t.dtype, *shape, 0 if t.is_contiguous() else _token_stride(shape, t.stride(), 1))


def _packed(name: str, t: torch.Tensor, T: int, d: int, dtype, device: int):
    """(heads, token stride) of packed tokens [T, heads, d]."""
    shape = t.shape
    if len(shape) != 3 or shape[0] != T or shape[2] != d or t.dtype != dtype or t.get_device() != device:
        raise _unexpected(name, t, (T, "heads", d), dtype, device)
    return shape[1], 0 if t.is_contiguous() else _token_stride(shape, t.stride(), 1)


def _bytes(nbytes: int, like: torch.Tensor, workspace: Optional[torch.Tensor]):
    """(address, the tensor that holds it) of a workspace of nbytes: the caller's where it is large enough."""
    if nbytes == 0:
        return None, None
    if workspace is None or workspace.numel() * workspace.element_size() < nbytes:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=like.device)
    elif workspace.get_device() != like.get_device() or not workspace.is_contiguous():
        raise GdnError(f"the workspace must be contiguous and on {like.device}")
    return workspace.data_ptr(), workspace


def _cu_seqlens(cu, device: int, T: int):
    """cu_seqlens as (address, number of sequences, the int32 device array).  One given on the host (a
    list or a CPU tensor) is checked before it is uploaded; one on the device is passed through
    (checking it would synchronise)."""
    if not torch.is_tensor(cu):
        cu = torch.tensor(cu, dtype=torch.int64)
    if cu.dim() != 1 or cu.numel() < 1:
        raise GdnError("cu_seqlens needs nseq + 1 entries")
    if not cu.is_cuda:
        x = cu.tolist()
        if any(b < a for a, b in zip(x, x[1:])) or x[0] < 0 or x[-1] > T:
            raise GdnError(f"cu_seqlens must ascend from >= 0 to <= {T} tokens")
        cu = cu.to(device=f"cuda:{device}", dtype=torch.int32)
    return _dense("cu_seqlens", cu, None, torch.int32, device), cu.numel() - 1, cu


def _qk_norm(d, dtype, device, inv_freq, q_norm_w, k_norm_w, norm_eps, interleaved, rot_scale) -> QkNorm:
    rot = 0
    if inv_freq is not None:
        if inv_freq.dim() != 1:
            raise GdnError("inv_freq is a vector of fp32 frequencies")
        rot = 2 * inv_freq.numel()
    return QkNorm(_dense("q_norm_w", q_norm_w, (d,), dtype, device), _dense("k_norm_w", k_norm_w, (d,), dtype, device),
                  _dense("inv_freq", inv_freq, None, torch.float32, device), rot, int(interleaved), norm_eps, rot_scale)


def _qk_inputs(q, k):
    """(device, dtype, T, Hq, Hk, d, q's address, k's, Strides) of packed q and k (or None)."""
    dev, dtype, T, Hq, d, sq = _first("q", q)
    if k is None:
        return dev, dtype, T, Hq, 0, d, q.data_ptr(), None, Strides(sq)
    Hk, sk = _packed("k", k, T, d, dtype, dev)
    return dev, dtype, T, Hq, Hk, d, q.data_ptr(), k.data_ptr(), Strides(sq, sk)


def gdn_qk_norm_rope_fwd(q, k, positions=None, inv_freq=None, *, q_norm_w=None, k_norm_w=None,
                         norm_eps: float = NORM_EPS, interleaved: bool = False, rot_scale: float = 1.0,
                         q_out=None, k_out=None, stream=None):
    """Per-head RMS norm of q [T,Hq,d] and k [T,Hk,d] (or None) and the rotation of their first
    ``2 * len(inv_freq)`` channels by ``positions`` [T] int32.  Returns (q_out, k_out)."""
    if stream is None and q_out is None and k_out is None and (native := _native_calls()) is not None:
        r = native.qk_norm_rope_fwd(q, k, positions, inv_freq, q_norm_w, k_norm_w, norm_eps, interleaved, rot_scale)
        if r is not None:
            return r if type(r) is tuple else check(r, "gdn_qk_norm_rope_fwd")
    with _on(q, stream):
        dev, dtype, T, Hq, Hk, d, pq, pk, strides = _qk_inputs(q, k)
        q_out, pqo = _result("q_out", q_out, q, dtype, dev)
        pko = None
        if k is not None:
            k_out, pko = _result("k_out", k_out, k, dtype, dev)
        elif k_out is not None:
            raise GdnError("k_out needs k")
        a = QkFwdArgs(pq, pk, _dense("positions", positions, (T,), torch.int32, dev), pqo, pko, T, Hq, Hk, d, _dt(q),
                      _qk_norm(d, dtype, dev, inv_freq, q_norm_w, k_norm_w, norm_eps, interleaved, rot_scale), strides)
        check(load().gdn_qk_norm_rope_fwd(ctypes.byref(a), _raw_stream(dev)), "gdn_qk_norm_rope_fwd")
    return q_out, k_out


def gdn_qk_norm_rope_bwd(q, k, positions=None, inv_freq=None, *, grad_q, grad_k=None, q_norm_w=None, k_norm_w=None,
                         norm_eps: float = NORM_EPS, interleaved: bool = False, rot_scale: float = 1.0,
                         workspace: Optional[torch.Tensor] = None, stream=None) -> Dict[str, torch.Tensor]:
    """Reverse mode of gdn_qk_norm_rope_fwd for the gradients ``grad_q``, ``grad_k`` of its results.
    Returns dq, dk in the inputs' dtype and dq_norm_w, dk_norm_w [d] fp32 (those that apply)."""
    if stream is None and workspace is None and (native := _native_calls()) is not None:
        r = native.qk_norm_rope_bwd(q, k, positions, inv_freq, q_norm_w, k_norm_w, norm_eps, interleaved, rot_scale, grad_q, grad_k)
        if r is not None:
            names = ("dq", "dk", "dq_norm_w", "dk_norm_w")
            return {n: t for n, t in zip(names, r) if t is not None} if type(r) is tuple else check(r, "gdn_qk_norm_rope_bwd")
    with _on(q, stream):
        dev, dtype, T, Hq, Hk, d, pq, pk, strides = _qk_inputs(q, k)
        out = {"dq": _result("dq", None, q, dtype, dev)[0]}
        if k is not None:
            out["dk"] = _result("dk", None, k, dtype, dev)[0]
        for name, w in (("dq_norm_w", q_norm_w), ("dk_norm_w", k_norm_w)):
            if w is not None:
                out[name] = torch.empty(d, dtype=torch.float32, device=q.device)
        ptr = {name: t.data_ptr() for name, t in out.items()}
        a = QkBwdArgs(pq, pk, _dense("positions", positions, (T,), torch.int32, dev),
                      _dense("grad_q", grad_q, q.shape, dtype, dev),
                      _dense("grad_k", grad_k, None if k is None else k.shape, dtype, dev), ptr["dq"], ptr.get("dk"),
                      ptr.get("dq_norm_w"), ptr.get("dk_norm_w"), T, Hq, Hk, d, _dt(q),
                      _qk_norm(d, dtype, dev, inv_freq, q_norm_w, k_norm_w, norm_eps, interleaved, rot_scale), strides)
        lib = load()
        need = lib.gdn_qk_norm_rope_bwd_workspace_size(ctypes.byref(a))
        ws, keep = _bytes(need, q, workspace)
        check(lib.gdn_qk_norm_rope_bwd(ctypes.byref(a), ws, need, _raw_stream(dev)), "gdn_qk_norm_rope_bwd")
    return out


def gdn_attn_fwd_cache_size(q, k, v, cu_seqlens) -> int:
    """Bytes of the cache gdn_attn_fwd(..., bwd_cache=) fills for gdn_attn_bwd."""
    T, Hq, d = q.shape
    nseq = (cu_seqlens.numel() if torch.is_tensor(cu_seqlens) else len(cu_seqlens)) - 1
    a = AttnFwdArgs(T=T, nseq=nseq, Hq=Hq, Hk=k.shape[1], d=d)
    return int(load().gdn_attn_fwd_cache_size(ctypes.byref(a)))


def _qkv(q, k, v):
    """(device, dtype, T, Hq, Hk, d, addresses of q, k, v, Strides) of packed q, k, v."""
    dev, dtype, T, Hq, d, sq = _first("q", q)
    Hk, sk = _packed("k", k, T, d, dtype, dev)
    Hv, sv = _packed("v", v, T, d, dtype, dev)
    if Hv != Hk:
        raise _unexpected("v", v, k.shape, dtype, dev)
    return dev, dtype, T, Hq, Hk, d, q.data_ptr(), k.data_ptr(), v.data_ptr(), Strides(sq, sk, sv)


def gdn_attn_fwd(q, k, v, cu_seqlens, *, scale: Optional[float] = None, window: int = 0, o=None,
                 bwd_cache: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Causal attention over packed sequences: q [T,Hq,d], k and v [T,Hk,d] bf16, ``cu_seqlens``
    [nseq + 1] (int32 on the device, or a list or CPU tensor, which is checked).  ``scale``: d ** -0.5
    unless given; ``window``: 0, or how many tokens, itself included, a token sees.  Returns o; rows
    outside every sequence stay as they were (unset in an ``o`` made here)."""
    if stream is None and o is None and workspace is None and (native := _native_calls()) is not None:
        r = native.attn_fwd(q, k, v, cu_seqlens, scale, window, bwd_cache)
        if r is not None:
            return r if type(r) is not int else check(r, "gdn_attn_fwd")
    with _on(q, stream):
        dev, dtype, T, Hq, Hk, d, pq, pk, pv, strides = _qkv(q, k, v)
        pcu, nseq, cu = _cu_seqlens(cu_seqlens, dev, T)
        o, po = _result("o", o, q, dtype, dev)
        a = AttnFwdArgs(pq, pk, pv, pcu, po, T, nseq, Hq, Hk, d, window,
                        d ** -0.5 if scale is None else scale, _dt(q),
                        _dense("bwd_cache", bwd_cache, None, torch.uint8, dev),
                        0 if bwd_cache is None else bwd_cache.numel(), strides)
        lib = load()
        need = lib.gdn_attn_fwd_workspace_size(ctypes.byref(a))
        ws, keep = _bytes(need, q, workspace)
        check(lib.gdn_attn_fwd(ctypes.byref(a), ws, need, _raw_stream(dev)), "gdn_attn_fwd")
    return o


def gdn_attn_bwd(q, k, v, cu_seqlens, o, *, grad_o, fwd_cache: torch.Tensor, scale: Optional[float] = None,
                 window: int = 0, dq=None, dk=None, dv=None, workspace: Optional[torch.Tensor] = None,
                 stream=None) -> Dict[str, torch.Tensor]:
    """Reverse mode of gdn_attn_fwd from its output ``o`` and the cache it filled.  Returns dq, dk, dv
    in bf16 (``dq``, ``dk``, ``dv``: buffers to fill; rows outside every sequence stay as they were)."""
    if stream is None and dq is None and dk is None and dv is None and workspace is None and (native := _native_calls()) is not None:
        r = native.attn_bwd(q, k, v, cu_seqlens, scale, window, o, grad_o, fwd_cache)
        if r is not None:
            return dict(zip(("dq", "dk", "dv"), r)) if type(r) is tuple else check(r, "gdn_attn_bwd")
    with _on(q, stream):
        dev, dtype, T, Hq, Hk, d, pq, pk, pv, strides = _qkv(q, k, v)
        pcu, nseq, cu = _cu_seqlens(cu_seqlens, dev, T)
        dq, pdq = _result("dq", dq, q, dtype, dev)
        dk, pdk = _result("dk", dk, k, dtype, dev)
        dv, pdv = _result("dv", dv, v, dtype, dev)
        a = AttnBwdArgs(pq, pk, pv, pcu, _dense("o", o, q.shape, dtype, dev), _dense("grad_o", grad_o, q.shape, dtype, dev),
                        pdq, pdk, pdv, T, nseq, Hq, Hk, d, window,
                        d ** -0.5 if scale is None else scale, _dt(q),
                        _dense("fwd_cache", fwd_cache, None, torch.uint8, dev), fwd_cache.numel(), strides)
        lib = load()
        need = lib.gdn_attn_bwd_workspace_size(ctypes.byref(a))
        ws, keep = _bytes(need, q, workspace)
        check(lib.gdn_attn_bwd(ctypes.byref(a), ws, need, _raw_stream(dev)), "gdn_attn_bwd")
    return {"dq": dq, "dk": dk, "dv": dv}


def _cache_args(k_cache, v_cache, block_table, context_lens, nseq, Hk, d, dtype, dev):
    """Addresses of (k_cache, v_cache, block_table, context_lens), and (num_pages, page_size, max_pages),
    of a paged cache [num_pages, page_size, Hk, d]."""
    if k_cache.dim() != 4 or k_cache.shape[2:] != (Hk, d):
        raise GdnError(f"k_cache has shape {tuple(k_cache.shape)}: expected [num_pages, page_size, {Hk}, {d}]")
    if block_table.dim() != 2 or block_table.shape[0] != nseq:
        raise GdnError(f"block_table has shape {tuple(block_table.shape)}: expected [{nseq}, max_pages]")
    return ((_dense("k_cache", k_cache, None, dtype, dev), _dense("v_cache", v_cache, k_cache.shape, dtype, dev),
             _dense("block_table", block_table, None, torch.int32, dev),
             _dense("context_lens", context_lens, (nseq,), torch.int32, dev)),
            (k_cache.shape[0], k_cache.shape[1], block_table.shape[1]))


def gdn_kv_append(k, v, k_cache, v_cache, block_table, context_lens, *, cu_seqlens=None, q=None, inv_freq=None,
                  q_norm_w=None, k_norm_w=None, norm_eps: float = NORM_EPS, interleaved: bool = False,
                  rot_scale: float = 1.0, q_out=None, k_out=None, want_k: bool = False, stream=None):
    """Appends the new tokens' k (normalised and rotated at its cache position) and v [T,Hk,d] to the
    paged caches [num_pages, page_size, Hk, d], in place.  ``context_lens`` [nseq] int32: tokens cached
    before (unchanged); ``cu_seqlens``: the sequences' new tokens, None for one each.  With ``q``
    [T,Hq,d], the same norm and rotation of q.  Returns (q_out or None, k_out or None: the keys as
    cached, with ``want_k``)."""
    if stream is None and q_out is None and k_out is None and (native := _native_calls()) is not None:
        r = native.kv_append(k, v, k_cache, v_cache, block_table, context_lens, cu_seqlens, q, inv_freq, q_norm_w, k_norm_w,
                              norm_eps, interleaved, rot_scale, want_k)
        if r is not None:
            return r if type(r) is tuple else check(r, "gdn_kv_append")
    with _on(k, stream):
        dev, dtype, T, Hk, d, sk = _first("k", k)
        Hv, sv = _packed("v", v, T, d, dtype, dev)
        if Hv != Hk:
            raise _unexpected("v", v, k.shape, dtype, dev)
        pcu, nseq, cu = (None, T, None) if cu_seqlens is None else _cu_seqlens(cu_seqlens, dev, T)
        (pkc, pvc, ptab, pctx), pages = _cache_args(k_cache, v_cache, block_table, context_lens, nseq, Hk, d, dtype, dev)
        pq, pqo, pko, sq, Hq = None, None, None, 0, 0
        if q is not None:
            Hq, sq = _packed("q", q, T, d, dtype, dev)
            pq = q.data_ptr()
            q_out, pqo = _result("q_out", q_out, q, dtype, dev)
        elif q_out is not None:
            raise GdnError("q_out needs q")
        if want_k or k_out is not None:
            k_out, pko = _result("k_out", k_out, k, dtype, dev)
        a = KvAppendArgs(pq, k.data_ptr(), v.data_ptr(), pcu, pctx, ptab, pqo, pko, pkc, pvc, T, nseq, Hq, Hk, d, *pages, _dt(k),
                         _qk_norm(d, dtype, dev, inv_freq, q_norm_w, k_norm_w, norm_eps, interleaved, rot_scale),
                         Strides(sq, sk, sv))
        check(load().gdn_kv_append(ctypes.byref(a), _raw_stream(dev)), "gdn_kv_append")
    return q_out, k_out


def gdn_attn_decode(q, k_cache, v_cache, block_table, context_lens, *, scale: Optional[float] = None, window: int = 0,
                    max_context: int = 0, o=None, workspace: Optional[torch.Tensor] = None, stream=None):
    """One query token for N sequences, q [N,Hq,d], over the paged caches: ``context_lens`` [N] int32
    tokens each, this one's included.  ``max_context``: a bound on the lengths that the caller knows
    (0: the block table's reach, by which the work is then split: give it where the table is much wider).  Returns o [N,Hq,d]."""
    if stream is None and o is None and workspace is None and (native := _native_calls()) is not None:
        r = native.attn_decode(q, k_cache, v_cache, block_table, context_lens, scale, window, max_context)
        if r is not None:
            return r if type(r) is not int else check(r, "gdn_attn_decode")
    with _on(q, stream):
        dev, dtype, N, Hq, d, sq = _first("q", q)
        Hk = k_cache.shape[2] if k_cache.dim() == 4 else 0
        (pkc, pvc, ptab, pctx), pages = _cache_args(k_cache, v_cache, block_table, context_lens, N, Hk, d, dtype, dev)
        o, po = _result("o", o, q, dtype, dev)
        a = AttnDecodeArgs(q.data_ptr(), pkc, pvc, ptab, pctx, po, N, Hq, Hk, d, *pages,
                           max_context, window, d ** -0.5 if scale is None else scale, _dt(q), Strides(sq))
        lib = load()
        need = lib.gdn_attn_decode_workspace_size(ctypes.byref(a))
        ws, keep = _bytes(need, q, workspace)
        check(lib.gdn_attn_decode(ctypes.byref(a), ws, need, _raw_stream(dev)), "gdn_attn_decode")
    return o
