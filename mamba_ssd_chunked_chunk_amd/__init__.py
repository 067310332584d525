"""Mamba-2 SSD selective-state-space scan on AMD MI355X (gfx950).

Thin Python binding over libssd.so (include/ssd.h).  Every step of the scan
runs in the library's HIP kernels; this module only checks and marshals
arguments.  torch supplies device memory and the current HIP stream.

    y = chunk_scan(x, dt, A, B, C, D, chunk_size=256)
    y, final = chunk_scan(..., initial_state=h0, return_final_state=True)
    y = step(state, x_t, dt_t, A, B_t, C_t, D)        # state updated in place

Tensor contract (nnterp guide, "Mamba-2" page, section "The values"):
x [b, l, h, p], dt [b, l, h], B and C [b, l, g, n], states [b, h, n, p]
(fp32), A, D, dt_bias [h] (fp32).  x, dt, B, C share one io dtype
(torch.float32 or torch.bfloat16); y has that dtype.
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import Optional, Tuple

from . import _lib
from ._lib import LibraryMissing, load, status_string  # noqa: F401

__all__ = ["chunk_scan", "chunk_scan_noalloc", "chunk_scan_bwd", "step", "conv1d_silu", "gated_norm",
           "mixer_forward", "mixer_workspace_bytes",
           "segment_log_decay", "combine_segments",
           "linear", "linear_bwd", "linear_workspace_bytes", "linear_bwd_workspace_bytes",
           "gated_scan", "gated_scan_bwd", "gated_step", "gated_scan_workspace_bytes",
           "gated_scan_bwd_workspace_bytes",
           "layer_norm", "layer_norm_bwd", "layer_norm_bwd_workspace_bytes",
           "delta_scan", "delta_scan_bwd", "delta_step", "delta_scan_workspace_bytes",
           "delta_scan_bwd_workspace_bytes",
           "workspace_bytes", "state_chunks", "abi_version",
           "LibraryMissing", "SsdError"]


class SsdError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__("%s failed: %s (status %d)" % (fn, status_string(code), code))
        self.code = code


def _torch():
    import torch
    return torch


def _io_code(dtype) -> int:
    torch = _torch()
    if dtype == torch.float32:
        return _lib.SSD_F32
    if dtype == torch.bfloat16:
        return _lib.SSD_BF16
    raise ValueError("io dtype must be torch.float32 or torch.bfloat16, got %s" % (dtype,))


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _check(name, t, dtype=None, shape=None, device=None):
    if t is None:
        return
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must have dtype %s, got %s" % (name, dtype, t.dtype))
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))


def abi_version() -> int:
    return int(load().ssd_abi_version())


def workspace_bytes(batch, seqlen, heads, head_dim, state_dim, groups, chunk) -> int:
    return int(load().ssd_chunk_scan_workspace_bytes(batch, seqlen, heads, head_dim,
                                                     state_dim, groups, chunk))


def state_chunks(batch, seqlen, heads, head_dim, state_dim, groups, chunk, io="bf16",
                 with_chunk_states=False) -> int:
    """Chunks per sequence whose boundary states a chunk_scan call with these
    sizes stores on the current device (ssd_chunk_scan_state_chunks)."""
    code = {"f32": 0, "bf16": 1}[io]
    v = int(load().ssd_chunk_scan_state_chunks(batch, seqlen, heads, head_dim, state_dim,
                                                 groups, chunk, code, int(bool(with_chunk_states))))
    if v < 0:
        raise SsdError("ssd_chunk_scan_state_chunks", v)
    return v


def chunk_scan(x, dt, A, B, C, D=None, chunk_size: int = 256, dt_bias=None,
               dt_softplus: bool = True, dt_limit: Tuple[float, float] = (0.0, math.inf),
               initial_state=None, return_final_state: bool = False, out=None,
               final_out=None, workspace=None, seq_idx=None,
               return_chunk_states: bool = False, chunk_states_out=None, kernel_events=None):
    """The chunked SSD scan of a whole sequence (ssd_chunk_scan_ex).

    Returns y, followed by final_state when return_final_state and by the
    state after every chunk [b, ceil(l / chunk_size), h, n, p] when
    return_chunk_states (a tuple when either is asked for).  seq_idx
    [b, l] int32: packed documents, a zero state wherever the index changes
    from one token to the next.  `out`, `final_out`, `chunk_states_out` and
    `workspace` (uint8, at least workspace_bytes(...)) may be given to avoid
    allocations; final_out may alias initial_state.  kernel_events: None, or
    8 raw hipEvent_t handles (ints; 0 for none) that receive the start and
    end of the call's kernel in each slot of _lib.EVENT_SLOTS.
    """
    torch = _torch()
    lib = load()
    if x.dim() != 4:
        raise ValueError("x must be [batch, seqlen, heads, head_dim]")
    b, l, h, p = x.shape
    if B.dim() != 4:
        raise ValueError("B must be [batch, seqlen, groups, state_dim]")
    g, n = B.shape[2], B.shape[3]
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("x must be a GPU tensor")
    io = x.dtype
    _io_code(io)
    _check("x", x, io)
    _check("dt", dt, io, (b, l, h), dev)
    _check("B", B, io, (b, l, g, n), dev)
    _check("C", C, io, (b, l, g, n), dev)
    _check("A", A, torch.float32, (h,), dev)
    _check("D", D, torch.float32, (h,), dev)
    _check("dt_bias", dt_bias, torch.float32, (h,), dev)
    _check("initial_state", initial_state, torch.float32, (b, h, n, p), dev)
    _check("seq_idx", seq_idx, torch.int32, (b, l), dev)
    y = torch.empty_like(x) if out is None else out
    _check("out", y, io, (b, l, h, p), dev)
    fin = None
    if return_final_state:
        fin = torch.empty((b, h, n, p), dtype=torch.float32, device=dev) \
            if final_out is None else final_out
        _check("final_out", fin, torch.float32, (b, h, n, p), dev)
    states = None
    if return_chunk_states:
        nck = -(-l // int(chunk_size)) if chunk_size > 0 else 0
        states = torch.empty((b, nck, h, n, p), dtype=torch.float32, device=dev) \
            if chunk_states_out is None else chunk_states_out
        _check("chunk_states_out", states, torch.float32, (b, nck, h, n, p), dev)
    wsb = int(lib.ssd_chunk_scan_workspace_bytes(b, l, h, p, n, g, int(chunk_size)))
    ws = workspace
    if ws is None:
        ws = torch.empty(max(wsb, 256), dtype=torch.uint8, device=dev)
    _check("workspace", ws, torch.uint8, None, dev)
    ev = None
    if kernel_events is not None:
        if len(kernel_events) != 2 * len(_lib.EVENT_SLOTS):
            raise ValueError("kernel_events must hold %d handles" % (2 * len(_lib.EVENT_SLOTS)))
        ev = (ctypes.c_void_p * len(kernel_events))(*[int(e) or None for e in kernel_events])
    stream = torch.cuda.current_stream(dev).cuda_stream
    rc = lib.ssd_chunk_scan_ex(
        _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(dt_bias),
        int(bool(dt_softplus)), float(dt_limit[0]), float(dt_limit[1]),
        _ptr(initial_state), _ptr(seq_idx), _ptr(y), _ptr(fin), _ptr(states), b, l, h, p, n,
        g, int(chunk_size), _io_code(io), _ptr(ws), ws.numel() * ws.element_size(), stream, ev)
    if rc != 0:
        raise SsdError("ssd_chunk_scan_ex", rc)
    if not return_final_state and not return_chunk_states:
        return y
    return (y,) + ((fin,) if return_final_state else ()) + \
        ((states,) if return_chunk_states else ())


def chunk_scan_noalloc(x, dt, A, B, C, y, D=None, chunk_size: int = 256, dt_bias=None,
                       dt_softplus: bool = True, dt_limit: Tuple[float, float] = (0.0, math.inf),
                       initial_state=None, final_state=None, seq_idx=None, chunk_states=None):
    """chunk_scan on the library's static device scratch (ssd_chunk_scan_noalloc):
    no workspace, and nothing allocated here either -- the caller passes the
    outputs y, and optionally final_state [b, h, n, p] and chunk_states
    [b, ceil(l / chunk_size), h, n, p] (fp32).  Sizes whose workspace_bytes
    exceed SSD_SCRATCH_BYTES raise SsdError (SSD_ERR_SCRATCH).  Calls that
    overlap on one GPU race on its scratch."""
    torch = _torch()
    lib = load()
    b, l, h, p = x.shape
    g, n = B.shape[2], B.shape[3]
    dev = x.device
    io = x.dtype
    _check("x", x, io)
    _check("dt", dt, io, (b, l, h), dev)
    _check("B", B, io, (b, l, g, n), dev)
    _check("C", C, io, (b, l, g, n), dev)
    _check("y", y, io, (b, l, h, p), dev)
    _check("A", A, torch.float32, (h,), dev)
    _check("D", D, torch.float32, (h,), dev)
    _check("dt_bias", dt_bias, torch.float32, (h,), dev)
    _check("initial_state", initial_state, torch.float32, (b, h, n, p), dev)
    _check("final_state", final_state, torch.float32, (b, h, n, p), dev)
    _check("seq_idx", seq_idx, torch.int32, (b, l), dev)
    nck = -(-l // int(chunk_size)) if chunk_size > 0 else 0
    _check("chunk_states", chunk_states, torch.float32, (b, nck, h, n, p), dev)
    stream = torch.cuda.current_stream(dev).cuda_stream
    rc = lib.ssd_chunk_scan_noalloc(
        _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(dt_bias),
        int(bool(dt_softplus)), float(dt_limit[0]), float(dt_limit[1]),
        _ptr(initial_state), _ptr(seq_idx), _ptr(y), _ptr(final_state), _ptr(chunk_states),
        b, l, h, p, n, g, int(chunk_size), _io_code(io), stream, None)
    if rc != 0:
        raise SsdError("ssd_chunk_scan_noalloc", rc)
    return y


def chunk_scan_bwd(x, dt, A, B, C, dy, D=None, chunk_size: int = 256, dt_bias=None,
                   initial_state=None, d_final=None, dt_softplus: bool = True,
                   dt_limit: Tuple[float, float] = (0.0, math.inf), seq_idx=None,
                   workspace=None):
    """Gradients of chunk_scan's y (cotangent dy) and final state (d_final)
    with respect to every input (ssd_chunk_scan_bwd), deterministic.
    Returns a dict: dx, ddt, dB, dC (io dtype), dA, and dD, d_dt_bias,
    d_init (fp32) for the inputs that were given."""
    torch = _torch()
    lib = load()
    b, l, h, p = x.shape
    g, n = B.shape[2], B.shape[3]
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("x must be a GPU tensor")
    io = x.dtype
    _io_code(io)
    _check("x", x, io)
    _check("dt", dt, io, (b, l, h), dev)
    _check("B", B, io, (b, l, g, n), dev)
    _check("C", C, io, (b, l, g, n), dev)
    _check("dy", dy, io, (b, l, h, p), dev)
    _check("A", A, torch.float32, (h,), dev)
    _check("D", D, torch.float32, (h,), dev)
    _check("dt_bias", dt_bias, torch.float32, (h,), dev)
    _check("initial_state", initial_state, torch.float32, (b, h, n, p), dev)
    _check("d_final", d_final, torch.float32, (b, h, n, p), dev)
    _check("seq_idx", seq_idx, torch.int32, (b, l), dev)
    out = dict(dx=torch.empty_like(x), ddt=torch.empty_like(dt),
               dA=torch.empty((h,), dtype=torch.float32, device=dev),
               dB=torch.empty_like(B), dC=torch.empty_like(C))
    if D is not None:
        out["dD"] = torch.empty((h,), dtype=torch.float32, device=dev)
    if dt_bias is not None:
        out["d_dt_bias"] = torch.empty((h,), dtype=torch.float32, device=dev)
    if initial_state is not None:
        out["d_init"] = torch.empty((b, h, n, p), dtype=torch.float32, device=dev)
    wsb = int(lib.ssd_chunk_scan_bwd_workspace_bytes(b, l, h, p, n, g, int(chunk_size),
                                                     _io_code(io)))
    ws = workspace if workspace is not None else torch.empty(max(wsb, 1), dtype=torch.uint8,
                                                             device=dev)
    _check("workspace", ws, torch.uint8, None, dev)
    stream = torch.cuda.current_stream(dev).cuda_stream
    rc = lib.ssd_chunk_scan_bwd(
        _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(dt_bias),
        int(bool(dt_softplus)), float(dt_limit[0]), float(dt_limit[1]), _ptr(initial_state),
        _ptr(seq_idx), _ptr(dy), _ptr(d_final), _ptr(out["dx"]), _ptr(out["ddt"]),
        _ptr(out["dA"]), _ptr(out["dB"]), _ptr(out["dC"]), _ptr(out.get("dD")),
        _ptr(out.get("d_dt_bias")), _ptr(out.get("d_init")), b, l, h, p, n, g,
        int(chunk_size), _io_code(io), _ptr(ws), ws.numel() * ws.element_size(), stream)
    if rc != 0:
        raise SsdError("ssd_chunk_scan_bwd", rc)
    return out


def segment_log_decay(dt, A, dt_bias=None, dt_softplus: bool = True,
                      dt_limit: Tuple[float, float] = (0.0, math.inf), seq_idx=None):
    """Total log decay [b, h] of a segment (ssd_segment_log_decay)."""
    torch = _torch()
    lib = load()
    b, l, h = dt.shape
    dev = dt.device
    _check("dt", dt, dt.dtype)
    _check("A", A, torch.float32, (h,), dev)
    _check("dt_bias", dt_bias, torch.float32, (h,), dev)
    _check("seq_idx", seq_idx, torch.int32, (b, l), dev)
    out = torch.empty((b, h), dtype=torch.float32, device=dev)
    stream = torch.cuda.current_stream(dev).cuda_stream
    rc = lib.ssd_segment_log_decay(_ptr(dt), _ptr(A), _ptr(dt_bias), int(bool(dt_softplus)),
                                   float(dt_limit[0]), float(dt_limit[1]), _ptr(seq_idx),
                                   _ptr(out), b, l, h, _io_code(dt.dtype), stream)
    if rc != 0:
        raise SsdError("ssd_segment_log_decay", rc)
    return out


def combine_segments(log_decay, seg_states, initial_state=None, starts_document=None):
    """Entry states [K, b, h, n, p] of K segments and the final state
    [b, h, n, p] from their log decays [K, b, h] and zero-start final
    states [K, b, h, n, p] (ssd_combine_segments)."""
    torch = _torch()
    lib = load()
    K, b, h, n, p = seg_states.shape
    dev = seg_states.device
    _check("log_decay", log_decay, torch.float32, (K, b, h), dev)
    _check("seg_states", seg_states, torch.float32)
    _check("initial_state", initial_state, torch.float32, (b, h, n, p), dev)
    _check("starts_document", starts_document, torch.int32, (K, b), dev)
    entry = torch.empty_like(seg_states)
    fin = torch.empty((b, h, n, p), dtype=torch.float32, device=dev)
    stream = torch.cuda.current_stream(dev).cuda_stream
    rc = lib.ssd_combine_segments(_ptr(log_decay), _ptr(seg_states), _ptr(initial_state),
                                  _ptr(starts_document), _ptr(entry), _ptr(fin), K, b, h, p, n,
                                  stream)
    if rc != 0:
        raise SsdError("ssd_combine_segments", rc)
    return entry, fin


def step(state, x, dt, A, B, C, D=None, dt_bias=None, dt_softplus: bool = True,
         dt_limit: Tuple[float, float] = (0.0, math.inf), out=None):
    """One decode step (ssd_step): updates `state` [b,h,n,p] in place, returns y."""
    torch = _torch()
    lib = load()
    if x.dim() != 3:
        raise ValueError("x must be [batch, heads, head_dim]")
    b, h, p = x.shape
    g, n = B.shape[1], B.shape[2]
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("x must be a GPU tensor")
    io = x.dtype
    _io_code(io)
    _check("state", state, torch.float32, (b, h, n, p), dev)
    _check("x", x, io)
    _check("dt", dt, io, (b, h), dev)
    _check("B", B, io, (b, g, n), dev)
    _check("C", C, io, (b, g, n), dev)
    _check("A", A, torch.float32, (h,), dev)
    _check("D", D, torch.float32, (h,), dev)
    _check("dt_bias", dt_bias, torch.float32, (h,), dev)
    y = torch.empty_like(x) if out is None else out
    _check("out", y, io, (b, h, p), dev)
    stream = torch.cuda.current_stream(dev).cuda_stream
    rc = lib.ssd_step(_ptr(state), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                      _ptr(dt_bias), int(bool(dt_softplus)), float(dt_limit[0]),
                      float(dt_limit[1]), _ptr(y), b, h, p, n, g, _io_code(io), stream)
    if rc != 0:
        raise SsdError("ssd_step", rc)
    return y


def conv1d_silu(xbc, weight, heads, head_dim, state_dim, groups, bias=None, conv_init=None,
                seq_idx=None, apply_silu: bool = True, return_conv_state: bool = False, out=None):
    """Causal depthwise conv1d + bias + SiLU over the packed x | B | C
    channels xbc [b, l, ch], split into the scan's inputs (ssd_conv1d_silu).
    weight [ch, width] fp32; conv_init [b, width-1, ch] fp32.  Returns
    (x, B, C), plus the final conv state [b, width-1, ch] when asked for.
    `out` may pass preallocated (x, B, C)."""
    torch = _torch()
    lib = load()
    if xbc.dim() != 3:
        raise ValueError("xbc must be [batch, seqlen, channels]")
    b, l, ch = xbc.shape
    dev = xbc.device
    if dev.type != "cuda":
        raise ValueError("xbc must be a GPU tensor")
    io = xbc.dtype
    h, p, n, g = int(heads), int(head_dim), int(state_dim), int(groups)
    if ch != h * p + 2 * g * n:
        raise ValueError("xbc has %d channels, expected heads*head_dim + 2*groups*state_dim = %d"
                         % (ch, h * p + 2 * g * n))
    K = int(weight.shape[1]) if weight.dim() == 2 else -1
    _check("xbc", xbc, io)
    _check("weight", weight, torch.float32, (ch, K), dev)
    _check("bias", bias, torch.float32, (ch,), dev)
    _check("conv_init", conv_init, torch.float32, (b, K - 1, ch), dev)
    _check("seq_idx", seq_idx, torch.int32, (b, l), dev)
    if out is None:
        x = torch.empty((b, l, h, p), dtype=io, device=dev)
        B = torch.empty((b, l, g, n), dtype=io, device=dev)
        C = torch.empty((b, l, g, n), dtype=io, device=dev)
    else:
        x, B, C = out
    _check("x", x, io, (b, l, h, p), dev)
    _check("B", B, io, (b, l, g, n), dev)
    _check("C", C, io, (b, l, g, n), dev)
    fin = None
    if return_conv_state:
        fin = torch.empty((b, K - 1, ch), dtype=torch.float32, device=dev)
    stream = torch.cuda.current_stream(dev).cuda_stream
    rc = lib.ssd_conv1d_silu(_ptr(xbc), _ptr(weight), _ptr(bias), _ptr(conv_init), _ptr(seq_idx),
                             _ptr(x), _ptr(B), _ptr(C), _ptr(fin), b, l, h, p, n, g, K,
                             int(bool(apply_silu)), _io_code(io), stream)
    if rc != 0:
        raise SsdError("ssd_conv1d_silu", rc)
    return (x, B, C, fin) if return_conv_state else (x, B, C)


def gated_norm(y, z=None, weight=None, group_size: Optional[int] = None, eps: float = 1e-5,
               normalize: bool = True, out=None):
    """y * silu(z), then an RMS norm over groups of `group_size` channels of
    the last axis times `weight` (ssd_gated_norm).  y [..., dim] in the io
    dtype; z like y or None; weight [dim] fp32 or None.  `out` may be y."""
    torch = _torch()
    lib = load()
    dev = y.device
    if dev.type != "cuda":
        raise ValueError("y must be a GPU tensor")
    io = y.dtype
    dim = int(y.shape[-1])
    rows = y.numel() // dim if dim else 0
    G = dim if group_size is None else int(group_size)
    _check("y", y, io)
    _check("z", z, io, tuple(y.shape), dev)
    _check("weight", weight, torch.float32, (dim,), dev)
    o = torch.empty_like(y) if out is None else out
    _check("out", o, io, tuple(y.shape), dev)
    stream = torch.cuda.current_stream(dev).cuda_stream
    rc = lib.ssd_gated_norm(_ptr(y), _ptr(z), _ptr(weight), _ptr(o), rows, dim, G, float(eps),
                            int(bool(normalize)), _io_code(io), stream)
    if rc != 0:
        raise SsdError("ssd_gated_norm", rc)
    return o


def mixer_workspace_bytes(batch, seqlen, heads, head_dim, state_dim, groups, chunk,
                          io="bf16") -> int:
    """Workspace bytes of one mixer_forward call (ssd_mixer_workspace_bytes)."""
    code = _lib.SSD_BF16 if io == "bf16" else _lib.SSD_F32
    return int(load().ssd_mixer_workspace_bytes(batch, seqlen, heads, head_dim, state_dim,
                                                groups, chunk, code))


def mixer_forward(xbc, dt, A, conv_weight, heads, head_dim, state_dim, groups, z=None,
                  conv_bias=None, conv_init=None, D=None, dt_bias=None,
                  dt_softplus: bool = True, dt_limit: Tuple[float, float] = (0.0, math.inf),
                  initial_state=None, seq_idx=None, norm_weight=None,
                  norm_group: Optional[int] = None, eps: float = 1e-5, normalize: bool = True,
                  chunk_size: int = 256, return_final_state: bool = False,
                  return_conv_state: bool = False, out=None, workspace=None):
    """The mixer between its projections in one call (ssd_mixer_forward):
    conv1d + SiLU + split of xbc [b, l, h*p + 2*g*n], the chunk scan, and
    the silu(z)-gated RMS norm over groups of norm_group channels (default:
    all h*p).  Returns out [b, l, h, p], followed by the final state and/or
    the final conv state [b, width-1, ch] when asked for."""
    torch = _torch()
    lib = load()
    if xbc.dim() != 3:
        raise ValueError("xbc must be [batch, seqlen, channels]")
    b, l, ch = xbc.shape
    dev = xbc.device
    if dev.type != "cuda":
        raise ValueError("xbc must be a GPU tensor")
    io = xbc.dtype
    code = _io_code(io)
    h, p, n, g = int(heads), int(head_dim), int(state_dim), int(groups)
    if ch != h * p + 2 * g * n:
        raise ValueError("xbc has %d channels, expected heads*head_dim + 2*groups*state_dim = %d"
                         % (ch, h * p + 2 * g * n))
    K = int(conv_weight.shape[1]) if conv_weight.dim() == 2 else -1
    _check("xbc", xbc, io)
    _check("dt", dt, io, (b, l, h), dev)
    _check("z", z, io, (b, l, h * p), dev)
    _check("conv_weight", conv_weight, torch.float32, (ch, K), dev)
    _check("conv_bias", conv_bias, torch.float32, (ch,), dev)
    _check("conv_init", conv_init, torch.float32, (b, K - 1, ch), dev)
    _check("A", A, torch.float32, (h,), dev)
    _check("D", D, torch.float32, (h,), dev)
    _check("dt_bias", dt_bias, torch.float32, (h,), dev)
    _check("initial_state", initial_state, torch.float32, (b, h, n, p), dev)
    _check("seq_idx", seq_idx, torch.int32, (b, l), dev)
    _check("norm_weight", norm_weight, torch.float32, (h * p,), dev)
    y = torch.empty((b, l, h, p), dtype=io, device=dev) if out is None else out
    _check("out", y, io, (b, l, h, p), dev)
    fin = torch.empty((b, h, n, p), dtype=torch.float32, device=dev) \
        if return_final_state else None
    cfin = torch.empty((b, K - 1, ch), dtype=torch.float32, device=dev) \
        if return_conv_state else None
    wsb = int(lib.ssd_mixer_workspace_bytes(b, l, h, p, n, g, int(chunk_size), code))
    ws = workspace
    if ws is None:
        ws = torch.empty(max(wsb, 256), dtype=torch.uint8, device=dev)
    _check("workspace", ws, torch.uint8, None, dev)
    G = h * p if norm_group is None else int(norm_group)
    stream = torch.cuda.current_stream(dev).cuda_stream
    rc = lib.ssd_mixer_forward(
        _ptr(xbc), _ptr(z), _ptr(dt), _ptr(conv_weight), _ptr(conv_bias), K, _ptr(conv_init),
        _ptr(cfin), _ptr(A), _ptr(D), _ptr(dt_bias), int(bool(dt_softplus)),
        float(dt_limit[0]), float(dt_limit[1]), _ptr(initial_state), _ptr(fin), _ptr(seq_idx),
        _ptr(norm_weight), G, float(eps), int(bool(normalize)), _ptr(y), b, l, h, p, n, g,
        int(chunk_size), code, _ptr(ws), ws.numel() * ws.element_size(), stream)
    if rc != 0:
        raise SsdError("ssd_mixer_forward", rc)
    if not return_final_state and not return_conv_state:
        return y
    return (y,) + ((fin,) if return_final_state else ()) + \
        ((cfin,) if return_conv_state else ())


def _activation(name) -> int:
    try:
        return _lib.ACTIVATIONS[name]
    except KeyError:
        raise ValueError("activation must be one of %s, got %r"
                         % (", ".join(sorted(_lib.ACTIVATIONS)), name)) from None


def _fit(name, t, dtype, shape, device):
    """_check with everything given, at the cost of four comparisons where all
    is well (a decode step makes several such checks per launch)."""
    if t is None or (t.dtype is dtype and t.shape == shape and t.device == device
                     and t.is_contiguous()):
        return
    _check(name, t, dtype, shape, device)


def _raw_stream(index: int) -> int:
    """The current stream's handle on device `index`; torch's own accessor of
    the bare handle where it has one (building a Stream object costs as much
    as half a launch)."""
    torch = _torch()
    get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return get(index) if get is not None else torch.cuda.current_stream(index).cuda_stream


def _launch(name, dev, *args) -> None:
    """Calls the library's `name` on the current stream of `dev` (its last
    argument), with `dev` the current device, and raises its errors."""
    cuda = _torch().cuda
    fn = getattr(load(), name)
    if dev.index == cuda.current_device():
        rc = fn(*args, _raw_stream(dev.index))
    else:
        with cuda.device(dev):
            rc = fn(*args, _raw_stream(dev.index))
    if rc != 0:
        raise SsdError(name, rc)


@functools.lru_cache(maxsize=1024)
def _query(name, *sizes) -> int:
    """A workspace query of the library: a pure function of the sizes."""
    return int(getattr(load(), name)(*sizes))


def _scratch(workspace, nbytes, dev):
    """The caller's workspace, or one of nbytes from torch's allocator."""
    torch = _torch()
    if workspace is None:
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)
    _check("workspace", workspace, torch.uint8, None, dev)
    return workspace


def _io_name(io) -> int:
    try:
        return {"f32": _lib.SSD_F32, "bf16": _lib.SSD_BF16}[io]
    except KeyError:
        raise ValueError("io must be f32 or bf16, got %r" % (io,)) from None


def linear_workspace_bytes(rows, in_dim, out_dim, io="bf16") -> int:
    """Workspace bytes of one linear call (ssd_linear_workspace_bytes)."""
    return int(load().ssd_linear_workspace_bytes(rows, in_dim, out_dim, _io_name(io)))


def linear_bwd_workspace_bytes(rows, in_dim, out_dim, activation="none", io="bf16") -> int:
    """Workspace bytes of one linear_bwd call (ssd_linear_bwd_workspace_bytes)."""
    return int(load().ssd_linear_bwd_workspace_bytes(rows, in_dim, out_dim,
                                                     _activation(activation), _io_name(io)))


def linear(x, weight, bias=None, activation: str = "none", residual=None,
           return_pre: bool = False, out=None, pre_out=None, workspace=None):
    """out = act(x W^T + bias) + residual in one product (ssd_linear).

    x [..., in_dim] and weight [out_dim, in_dim] in the io dtype, bias
    [out_dim] fp32, residual [..., out_dim] in the io dtype; activation
    "none", "silu", "gelu" (erf) or "sigmoid".  Returns out [..., out_dim],
    and with return_pre also the pre-activation in the io dtype, which
    linear_bwd takes.  `out` may be the residual."""
    torch = _torch()
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("x must be a GPU tensor")
    io = x.dtype
    code = _io_code(io)
    act = _activation(activation)
    if x.dim() < 1 or weight.dim() != 2:
        raise ValueError("x must be [..., in_dim] and weight [out_dim, in_dim]")
    n, k = weight.shape
    shape = tuple(x.shape[:-1]) + (n,)
    _check("x", x, io, tuple(x.shape[:-1]) + (k,))
    _check("weight", weight, io, None, dev)
    _fit("bias", bias, torch.float32, (n,), dev)
    _fit("residual", residual, io, shape, dev)
    o = torch.empty(shape, dtype=io, device=dev) if out is None else out
    _fit("out", o, io, shape, dev)
    pre = None
    if return_pre:
        pre = torch.empty(shape, dtype=io, device=dev) if pre_out is None else pre_out
        _fit("pre_out", pre, io, shape, dev)
    m = x.numel() // k if k else 0
    wsb = _query("ssd_linear_workspace_bytes", m, k, n, code)
    ws = _scratch(workspace, wsb, dev) if wsb or workspace is not None else None
    _launch("ssd_linear", dev, _ptr(x), _ptr(weight), _ptr(bias), _ptr(residual), _ptr(o),
            _ptr(pre), act, m, k, n, code, _ptr(ws), 0 if ws is None else ws.numel())
    return (o, pre) if return_pre else o


def linear_bwd(dy, x, weight, pre=None, activation: str = "none", bias: bool = False,
               workspace=None):
    """Gradients of linear's out (cotangent dy [..., out_dim]) with respect to
    x, weight and, with `bias`, the bias (ssd_linear_bwd), deterministic.
    pre: the pre-activation that linear returned (not needed for "none").
    Returns a dict: dx, dweight (io dtype), dbias (fp32); the residual's
    gradient is dy."""
    torch = _torch()
    dev = dy.device
    if dev.type != "cuda":
        raise ValueError("dy must be a GPU tensor")
    io = dy.dtype
    code = _io_code(io)
    act = _activation(activation)
    if dy.dim() < 1 or weight.dim() != 2:
        raise ValueError("dy must be [..., out_dim] and weight [out_dim, in_dim]")
    n, k = weight.shape
    lead = tuple(dy.shape[:-1])
    _check("dy", dy, io, lead + (n,))
    _fit("x", x, io, lead + (k,), dev)
    _check("weight", weight, io, None, dev)
    if act and pre is None:
        raise ValueError("pre is needed for the gradient of %s" % activation)
    _fit("pre", pre, io, lead + (n,), dev)
    res = dict(dx=torch.empty_like(x), dweight=torch.empty_like(weight))
    if bias:
        res["dbias"] = torch.empty((n,), dtype=torch.float32, device=dev)
    m = dy.numel() // n if n else 0
    ws = _scratch(workspace, _query("ssd_linear_bwd_workspace_bytes", m, k, n, act, code), dev)
    _launch("ssd_linear_bwd", dev, _ptr(dy), _ptr(x), _ptr(weight), _ptr(pre), act,
            _ptr(res["dx"]), _ptr(res["dweight"]), _ptr(res.get("dbias")), m, k, n, code,
            _ptr(ws), ws.numel())
    return res


def gated_scan_workspace_bytes(batch, seqlen, dim) -> int:
    """Workspace bytes of one gated_scan call (ssd_gated_scan_workspace_bytes)."""
    return int(load().ssd_gated_scan_workspace_bytes(batch, seqlen, dim))


def gated_scan_bwd_workspace_bytes(batch, seqlen, dim) -> int:
    """Workspace bytes of one gated_scan_bwd call (ssd_gated_scan_bwd_workspace_bytes)."""
    return int(load().ssd_gated_scan_bwd_workspace_bytes(batch, seqlen, dim))


def gated_scan(x, gates, lam, scale: float = 8.0, initial_state=None, seq_idx=None,
               return_final_state: bool = False, return_states: bool = False, out=None,
               final_out=None, states_out=None, workspace=None):
    """The gated linear recurrence over a whole sequence (ssd_gated_scan):
    h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t per channel, with
    a_t = exp(-scale softplus(lam) sigmoid(r_t)).

    x [b, l, d] and gates [b, l, 2d] (r | i, before their sigmoids) in the io
    dtype, lam [d] fp32, initial_state [b, d] fp32, seq_idx [b, l] int32.
    Returns y [b, l, d], followed by the final state [b, d] and by the states
    after every 64 tokens [b, ceil(l / 64), d] (fp32, for gated_scan_bwd) when
    asked for.  final_out may be initial_state."""
    torch = _torch()
    if x.dim() != 3:
        raise ValueError("x must be [batch, seqlen, dim]")
    b, l, d = x.shape
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("x must be a GPU tensor")
    io = x.dtype
    code = _io_code(io)
    _check("x", x, io)
    _fit("gates", gates, io, (b, l, 2 * d), dev)
    _fit("lam", lam, torch.float32, (d,), dev)
    _fit("initial_state", initial_state, torch.float32, (b, d), dev)
    _fit("seq_idx", seq_idx, torch.int32, (b, l), dev)
    y = torch.empty_like(x) if out is None else out
    _fit("out", y, io, (b, l, d), dev)
    fin = states = None
    if return_final_state:
        fin = torch.empty((b, d), dtype=torch.float32, device=dev) \
            if final_out is None else final_out
        _fit("final_out", fin, torch.float32, (b, d), dev)
    if return_states:
        ns = -(-l // _lib.SSD_GATED_CHUNK)
        states = torch.empty((b, ns, d), dtype=torch.float32, device=dev) \
            if states_out is None else states_out
        _fit("states_out", states, torch.float32, (b, ns, d), dev)
    ws = _scratch(workspace, _query("ssd_gated_scan_workspace_bytes", b, l, d), dev)
    _launch("ssd_gated_scan", dev, _ptr(x), _ptr(gates), _ptr(lam), float(scale),
            _ptr(initial_state), _ptr(seq_idx), _ptr(y), _ptr(fin), _ptr(states), b, l, d,
            code, _ptr(ws), ws.numel())
    if not return_final_state and not return_states:
        return y
    return (y,) + ((fin,) if return_final_state else ()) + ((states,) if return_states else ())


def gated_scan_bwd(x, gates, lam, dy, scale: float = 8.0, initial_state=None, d_final=None,
                   seq_idx=None, states=None, workspace=None):
    """Gradients of gated_scan's y (cotangent dy) and final state (d_final)
    with respect to every input (ssd_gated_scan_bwd), deterministic.  states:
    what gated_scan returned for these inputs (None: computed again).
    Returns a dict: dx, dgates (io dtype), dlam, and d_init (fp32) if
    initial_state was given."""
    torch = _torch()
    if x.dim() != 3:
        raise ValueError("x must be [batch, seqlen, dim]")
    b, l, d = x.shape
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("x must be a GPU tensor")
    io = x.dtype
    code = _io_code(io)
    _check("x", x, io)
    _fit("gates", gates, io, (b, l, 2 * d), dev)
    _fit("lam", lam, torch.float32, (d,), dev)
    _fit("dy", dy, io, (b, l, d), dev)
    _fit("initial_state", initial_state, torch.float32, (b, d), dev)
    _fit("d_final", d_final, torch.float32, (b, d), dev)
    _fit("seq_idx", seq_idx, torch.int32, (b, l), dev)
    _fit("states", states, torch.float32, (b, -(-l // _lib.SSD_GATED_CHUNK), d), dev)
    res = dict(dx=torch.empty_like(x), dgates=torch.empty_like(gates), dlam=torch.empty_like(lam))
    if initial_state is not None:
        res["d_init"] = torch.empty_like(initial_state)
    ws = _scratch(workspace, _query("ssd_gated_scan_bwd_workspace_bytes", b, l, d), dev)
    _launch("ssd_gated_scan_bwd", dev, _ptr(x), _ptr(gates), _ptr(lam), float(scale),
            _ptr(initial_state), _ptr(seq_idx), _ptr(states), _ptr(dy), _ptr(d_final),
            _ptr(res["dx"]), _ptr(res["dgates"]), _ptr(res["dlam"]),
            _ptr(res.get("d_init")), b, l, d, code, _ptr(ws), ws.numel())
    return res


def gated_step(state, x, gates, lam, scale: float = 8.0, out=None):
    """One token of gated_scan (ssd_gated_step): updates `state` [b, d] (fp32)
    in place, returns y [b, d].  x [b, d], gates [b, 2d] in the io dtype."""
    torch = _torch()
    if x.dim() != 2:
        raise ValueError("x must be [batch, dim]")
    b, d = x.shape
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("x must be a GPU tensor")
    io = x.dtype
    code = _io_code(io)
    _fit("state", state, torch.float32, (b, d), dev)
    _check("x", x, io)
    _fit("gates", gates, io, (b, 2 * d), dev)
    _fit("lam", lam, torch.float32, (d,), dev)
    y = torch.empty_like(x) if out is None else out
    _fit("out", y, io, (b, d), dev)
    _launch("ssd_gated_step", dev, _ptr(state), _ptr(x), _ptr(gates), _ptr(lam), float(scale),
            _ptr(y), b, d, code)
    return y


def layer_norm_bwd_workspace_bytes(rows, dim) -> int:
    """Workspace bytes of one layer_norm_bwd call (ssd_layer_norm_bwd_workspace_bytes)."""
    return int(load().ssd_layer_norm_bwd_workspace_bytes(rows, dim))


def layer_norm(x, weight=None, bias=None, residual=None, eps: float = 1e-5,
               return_stats: bool = False, out=None, sum_out=None):
    """Layer norm over the last axis (ssd_layer_norm): (x - mean) rstd weight
    + bias, with `residual` of x + residual, rounded to the io dtype.

    x [..., dim] and residual in the io dtype, weight and bias [dim] fp32.
    Returns y, followed by the sum (with `residual`) and by the row statistics
    [2, rows] fp32 (mean, 1 / deviation; return_stats), which layer_norm_bwd
    takes.  `sum_out` may be x or residual, `out` either where the sum is
    another tensor."""
    torch = _torch()
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("x must be a GPU tensor")
    io = x.dtype
    code = _io_code(io)
    if x.dim() < 1:
        raise ValueError("x must be [..., dim]")
    dim, shape = x.shape[-1], x.shape
    _check("x", x, io)
    _fit("residual", residual, io, shape, dev)
    _fit("weight", weight, torch.float32, (dim,), dev)
    _fit("bias", bias, torch.float32, (dim,), dev)
    y = torch.empty_like(x) if out is None else out
    _fit("out", y, io, shape, dev)
    total = None
    if residual is not None:
        total = torch.empty_like(x) if sum_out is None else sum_out
        _fit("sum_out", total, io, shape, dev)
    elif sum_out is not None:
        raise ValueError("sum_out is the output of x + residual, and there is no residual")
    rows = x.numel() // dim if dim else 0
    stats = torch.empty((2, rows), dtype=torch.float32, device=dev) if return_stats else None
    _launch("ssd_layer_norm", dev, _ptr(x), _ptr(residual), _ptr(weight), _ptr(bias), float(eps),
            _ptr(y), _ptr(total), _ptr(stats), rows, dim, code)
    if total is None and stats is None:
        return y
    return (y,) + (() if total is None else (total,)) + (() if stats is None else (stats,))


def layer_norm_bwd(dy, x, stats, weight=None, bias: bool = False, d_sum=None, out=None,
                   workspace=None):
    """Gradients of layer_norm's y (cotangent dy) with respect to its input,
    weight and, with `bias`, the bias (ssd_layer_norm_bwd), deterministic.

    x: what was normalised (the sum, where there was a residual); stats: what
    layer_norm returned; d_sum: the gradient that reaches the sum from
    elsewhere, added to dx.  Returns a dict: dx (io dtype; also the residual's
    gradient), dweight (fp32, with `weight`) and dbias (fp32).  `out` (for dx)
    may be dy or d_sum."""
    torch = _torch()
    dev = dy.device
    if dev.type != "cuda":
        raise ValueError("dy must be a GPU tensor")
    io = dy.dtype
    code = _io_code(io)
    if dy.dim() < 1:
        raise ValueError("dy must be [..., dim]")
    dim, shape = dy.shape[-1], dy.shape
    rows = dy.numel() // dim if dim else 0
    _check("dy", dy, io)
    _fit("x", x, io, shape, dev)
    _fit("stats", stats, torch.float32, (2, rows), dev)
    _fit("weight", weight, torch.float32, (dim,), dev)
    _fit("d_sum", d_sum, io, shape, dev)
    dx = torch.empty_like(dy) if out is None else out
    _fit("out", dx, io, shape, dev)
    res = dict(dx=dx)
    if weight is not None:
        res["dweight"] = torch.empty((dim,), dtype=torch.float32, device=dev)
    if bias:
        res["dbias"] = torch.empty((dim,), dtype=torch.float32, device=dev)
    need = _query("ssd_layer_norm_bwd_workspace_bytes", rows, dim) if len(res) > 1 else 0
    ws = _scratch(workspace, need, dev) if need or workspace is not None else None
    _launch("ssd_layer_norm_bwd", dev, _ptr(dy), _ptr(x), _ptr(stats), _ptr(weight), _ptr(d_sum),
            _ptr(dx), _ptr(res.get("dweight")), _ptr(res.get("dbias")), rows, dim, code, _ptr(ws),
            0 if ws is None else ws.numel())
    return res


def delta_scan_workspace_bytes(batch, seqlen, heads, value_dim, key_dim, groups, io="bf16") -> int:
    """Workspace bytes of one delta_scan call (ssd_delta_scan_workspace_bytes)."""
    return int(load().ssd_delta_scan_workspace_bytes(batch, seqlen, heads, value_dim, key_dim,
                                                     groups, _io_name(io)))


def delta_scan_bwd_workspace_bytes(batch, seqlen, heads, value_dim, key_dim, groups, io="bf16",
                                   with_states: bool = True) -> int:
    """Workspace bytes of one delta_scan_bwd call (ssd_delta_scan_bwd_workspace_bytes)."""
    return int(load().ssd_delta_scan_bwd_workspace_bytes(batch, seqlen, heads, value_dim, key_dim,
                                                         groups, _io_name(io),
                                                         int(bool(with_states))))


def _delta_inputs(lead, q, k, v, dt, A, beta, dt_bias):
    """The checks that delta_scan, its gradient and its step share; lead is the
    number of axes in front of the heads.  Returns io dtype, code, device, the
    leading sizes and heads, value_dim, key_dim, groups."""
    torch = _torch()
    names = "[batch, seqlen, " if lead == 2 else "[batch, "
    if v.dim() != lead + 2:
        raise ValueError("v must be %sheads, value_dim]" % names)
    if k.dim() != lead + 2:
        raise ValueError("k must be %sgroups, key_dim]" % names)
    dev = v.device
    if dev.type != "cuda":
        raise ValueError("v must be a GPU tensor")
    io = v.dtype
    code = _io_code(io)
    lead = tuple(v.shape[:lead])
    h, p = v.shape[-2:]
    g, n = k.shape[-2:]
    _check("v", v, io)
    _fit("k", k, io, lead + (g, n), dev)
    _fit("q", q, io, lead + (g, n), dev)
    _fit("dt", dt, io, lead + (h,), dev)
    _fit("beta", beta, io, lead + (h,), dev)
    _fit("A", A, torch.float32, (h,), dev)
    _fit("dt_bias", dt_bias, torch.float32, (h,), dev)
    return io, code, dev, lead, h, p, n, g


def _delta_rule(q, k, v, dt, A, beta, dt_bias, dt_softplus, dt_limit, scale, normalize, norm_eps, n):
    """The arguments from q to norm_eps of the library's calls."""
    return (_ptr(q), _ptr(k), _ptr(v), _ptr(dt), _ptr(A), _ptr(dt_bias), int(bool(dt_softplus)),
            float(dt_limit[0]), float(dt_limit[1]), _ptr(beta),
            float(n) ** -0.5 if scale is None else float(scale), int(bool(normalize)),
            float(norm_eps))


def delta_scan(q, k, v, dt, A, beta, dt_bias=None, dt_softplus: bool = True,
               dt_limit: Tuple[float, float] = (0.0, math.inf), scale: Optional[float] = None,
               normalize: bool = False, norm_eps: float = 1e-6, initial_state=None, seq_idx=None,
               return_final_state: bool = False, return_states: bool = False, out=None,
               final_out=None, states_out=None, workspace=None):
    """The gated delta rule over a whole sequence (ssd_delta_scan): per head,
    with a state S [n, p] and d = clamp(softplus(dt + dt_bias)),

        P_t = exp(A d_t) S_{t-1},  u_t = beta_t (v_t - P_t^T k_t)
        S_t = P_t + k_t u_t^T,     y_t = scale S_t^T q_t

    v [b, l, h, p], q and k [b, l, g, n], dt and beta [b, l, h] in the io
    dtype, A and dt_bias [h] fp32, initial_state [b, h, n, p] fp32, seq_idx
    [b, l] int32.  scale: 1 / sqrt(n) by default.  normalize: q and k are
    divided by sqrt(|.|^2 + norm_eps) first.  Returns y [b, l, h, p], followed
    by the final state [b, h, n, p] and by the states after every 64 tokens
    [b, ceil(l / 64), h, n, p] (fp32, for delta_scan_bwd) when asked for.
    final_out may be initial_state."""
    torch = _torch()
    io, code, dev, (b, l), h, p, n, g = _delta_inputs(2, q, k, v, dt, A, beta, dt_bias)
    _fit("initial_state", initial_state, torch.float32, (b, h, n, p), dev)
    _fit("seq_idx", seq_idx, torch.int32, (b, l), dev)
    y = torch.empty_like(v) if out is None else out
    _fit("out", y, io, (b, l, h, p), dev)
    fin = states = None
    if return_final_state:
        fin = torch.empty((b, h, n, p), dtype=torch.float32, device=dev) \
            if final_out is None else final_out
        _fit("final_out", fin, torch.float32, (b, h, n, p), dev)
    if return_states:
        shape = (b, -(-l // _lib.SSD_DELTA_CHUNK), h, n, p)
        states = torch.empty(shape, dtype=torch.float32, device=dev) \
            if states_out is None else states_out
        _fit("states_out", states, torch.float32, shape, dev)
    ws = _scratch(workspace, _query("ssd_delta_scan_workspace_bytes", b, l, h, p, n, g, code), dev)
    _launch("ssd_delta_scan", dev,
            *_delta_rule(q, k, v, dt, A, beta, dt_bias, dt_softplus, dt_limit, scale, normalize,
                         norm_eps, n),
            _ptr(initial_state), _ptr(seq_idx), _ptr(y), _ptr(fin), _ptr(states), b, l, h, p, n, g,
            code, _ptr(ws), ws.numel())
    if not return_final_state and not return_states:
        return y
    return (y,) + ((fin,) if return_final_state else ()) + ((states,) if return_states else ())


def delta_scan_bwd(q, k, v, dt, A, beta, dy, dt_bias=None, dt_softplus: bool = True,
                   dt_limit: Tuple[float, float] = (0.0, math.inf),
                   scale: Optional[float] = None, normalize: bool = False,
                   norm_eps: float = 1e-6, initial_state=None, d_final=None, seq_idx=None,
                   states=None, workspace=None):
    """Gradients of delta_scan's y (cotangent dy) and final state (d_final)
    with respect to every input (ssd_delta_scan_bwd), deterministic.  states:
    what delta_scan returned for these inputs (None: computed again).
    Returns a dict: dq, dk, dv, ddt, dbeta (io dtype), dA, ddt_bias (with
    dt_bias) and d_init (with initial_state) in fp32."""
    torch = _torch()
    io, code, dev, (b, l), h, p, n, g = _delta_inputs(2, q, k, v, dt, A, beta, dt_bias)
    _fit("dy", dy, io, (b, l, h, p), dev)
    _fit("initial_state", initial_state, torch.float32, (b, h, n, p), dev)
    _fit("d_final", d_final, torch.float32, (b, h, n, p), dev)
    _fit("seq_idx", seq_idx, torch.int32, (b, l), dev)
    _fit("states", states, torch.float32, (b, -(-l // _lib.SSD_DELTA_CHUNK), h, n, p), dev)
    res = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
               ddt=torch.empty_like(dt), dbeta=torch.empty_like(beta), dA=torch.empty_like(A))
    if dt_bias is not None:
        res["ddt_bias"] = torch.empty_like(dt_bias)
    if initial_state is not None:
        res["d_init"] = torch.empty_like(initial_state)
    ws = _scratch(workspace, _query("ssd_delta_scan_bwd_workspace_bytes", b, l, h, p, n, g, code,
                                    int(states is not None)), dev)
    _launch("ssd_delta_scan_bwd", dev,
            *_delta_rule(q, k, v, dt, A, beta, dt_bias, dt_softplus, dt_limit, scale, normalize,
                         norm_eps, n),
            _ptr(initial_state), _ptr(seq_idx), _ptr(states), _ptr(dy), _ptr(d_final),
            _ptr(res["dq"]), _ptr(res["dk"]), _ptr(res["dv"]), _ptr(res["ddt"]),
            _ptr(res["dbeta"]), _ptr(res["dA"]), _ptr(res.get("ddt_bias")),
            _ptr(res.get("d_init")), b, l, h, p, n, g, code, _ptr(ws), ws.numel())
    return res


def delta_step(state, q, k, v, dt, A, beta, dt_bias=None, dt_softplus: bool = True,
               dt_limit: Tuple[float, float] = (0.0, math.inf), scale: Optional[float] = None,
               normalize: bool = False, norm_eps: float = 1e-6, out=None):
    """One token of delta_scan (ssd_delta_step): updates `state` [b, h, n, p]
    (fp32) in place, returns y [b, h, p].  v [b, h, p], q and k [b, g, n], dt
    and beta [b, h] in the io dtype."""
    torch = _torch()
    io, code, dev, (b,), h, p, n, g = _delta_inputs(1, q, k, v, dt, A, beta, dt_bias)
    _fit("state", state, torch.float32, (b, h, n, p), dev)
    if state is None:
        raise ValueError("state is needed")
    y = torch.empty_like(v) if out is None else out
    _fit("out", y, io, (b, h, p), dev)
    _launch("ssd_delta_step", dev, _ptr(state),
            *_delta_rule(q, k, v, dt, A, beta, dt_bias, dt_softplus, dt_limit, scale, normalize,
                         norm_eps, n),
            _ptr(y), b, h, p, n, g, code)
    return y
