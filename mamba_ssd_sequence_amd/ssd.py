"""Thin Python binding of libssd.so (ctypes).

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI of include/ssd.h.  PyTorch supplies device memory and
the current HIP stream.  There is no fallback: if the library is missing or a
call fails, an exception is raised.

    dt, a_cs, a_chunk = prep(dt_proj, dt_bias, A_log, chunk)
    y = forward(q, k, v, dt, a_cs, order=2, chunk=64)
    y = decode_step(q, k, v, dt_proj, dt_bias, A_log, state, norm_state, order=2)
    y = decode_step_amask(q, k, v, A_proj, dt_proj, state, norm_state, order=2)
    y = decode_step_conv(q, k, v, conv_w, conv_b, conv_state, state, norm_state, order=2, A_proj=A_proj)
    state_p, norm_p = state_pack(state, norm_state)
    dq, dk, dv, ddt, da = backward(q, k, v, dt, a_cs, y, den, dy, order=2, chunk=64)
    d_dt_proj, d_dt_bias, d_A_log = prep_backward(dt_proj, dt_bias, A_log, da, ddt)

The gated linear recurrence, and the norms, gate and residual scale around a mixer block:

    y = gated_scan(x, A_proj, I_proj, scale=SSD_INPUT_UNIT)
    state = gated_scan_step(x, A_proj, I_proj, state, scale=SSD_INPUT_UNIT)
    dx, dA_proj, dI_proj, dh0 = gated_scan_backward(x, A_proj, I_proj, y, dy, scale=SSD_INPUT_UNIT)
    residual, u = norm_in(residual, branch, branch_scale, weight, eps)
    d_residual, d_branch, d_weight, d_scale = norm_in_backward(du, d_residual, residual, branch, branch_scale, weight, eps)
    o = norm_out(y, z, weight, eps, groups=1, gate_first=True)
    dy, dz, d_weight = norm_out_backward(do, y, z, weight, eps, groups=1, gate_first=True)
"""
from __future__ import annotations

import ctypes
import functools
import os
import re

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libssd.so")
HEADER = os.path.join(os.path.dirname(PKG), "include", "ssd.h")

SSD_OK = 0
SSD_F32 = 0
SSD_BF16 = 1
SSD_STATE_FULL = 0
SSD_STATE_PACKED = 1
SSD_INPUT_PLAIN = 0
SSD_INPUT_CONVEX = 1
SSD_INPUT_UNIT = 2
SSD_NOALLOC_SCRATCH_BYTES = 64 << 20  # include/ssd.h
STATUS = ["SSD_OK", "SSD_ERR_NULL", "SSD_ERR_SHAPE", "SSD_ERR_UNSUPPORTED", "SSD_ERR_ALIGN",
          "SSD_ERR_ALIAS", "SSD_ERR_WORKSPACE", "SSD_ERR_HIP"]

_lib = None


class SSDError(RuntimeError):
    def __init__(self, status: int, msg: str):
        name = STATUS[status] if 0 <= status < len(STATUS) else str(status)
        super().__init__(f"{name}: {msg}")
        self.status = status


def _declare(lib):
    i64, vp, fp, i32, sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.ssd_abi_version.restype = ctypes.c_int
    lib.ssd_abi_version.argtypes = []
    lib.ssd_status_str.restype = ctypes.c_char_p
    lib.ssd_status_str.argtypes = [ctypes.c_int]
    lib.ssd_last_error.restype = ctypes.c_char_p
    lib.ssd_last_error.argtypes = []
    lib.ssd_prep.restype = ctypes.c_int
    lib.ssd_prep.argtypes = [fp, fp, fp, i64, i64, i64, i64, fp, fp, fp, vp]
    lib.ssd_prep_amask.restype = ctypes.c_int
    lib.ssd_prep_amask.argtypes = [fp, fp, i64, i64, i64, i64, fp, fp, fp, vp]
    lib.ssd_forward_workspace_size.restype = sz
    lib.ssd_forward_workspace_size.argtypes = [i64, i64, i64, i64, i32, i64, i32]
    lib.ssd_forward.restype = ctypes.c_int
    lib.ssd_forward.argtypes = [vp, vp, vp, fp, fp, fp, fp, i64, i64, i64, i64, i32, i64, i32,
                                fp, fp, fp, fp, vp, sz, vp]
    lib.ssd_forward_noalloc.restype = ctypes.c_int
    lib.ssd_forward_noalloc.argtypes = [vp, vp, vp, fp, fp, fp, fp, i64, i64, i64, i64, i32, i64, i32,
                                        fp, fp, fp, fp, vp]
    lib.ssd_set_timing_events.restype = ctypes.c_int
    lib.ssd_set_timing_events.argtypes = [vp, ctypes.c_int]
    lib.ssd_timing_count.restype = ctypes.c_int
    lib.ssd_timing_count.argtypes = []
    lib.ssd_decode_step.restype = ctypes.c_int
    lib.ssd_decode_step.argtypes = [vp, vp, vp, fp, fp, fp, i64, i64, i64, i32, i32, i32, fp, fp, fp, vp]
    lib.ssd_decode_step_amask.restype = ctypes.c_int
    lib.ssd_decode_step_amask.argtypes = [vp, vp, vp, fp, fp, i64, i64, i64, i32, i32, i32, fp, fp, fp, vp]
    lib.ssd_decode_step_conv.restype = ctypes.c_int
    lib.ssd_decode_step_conv.argtypes = [vp, vp, vp, fp, fp, i32, vp, fp, fp, fp, fp, i64, i64, i64, i32,
                                         i32, i32, fp, fp, fp, vp]
    lib.ssd_state_pack.restype = ctypes.c_int
    lib.ssd_state_pack.argtypes = [fp, fp, i64, i64, fp, fp, vp]
    lib.ssd_state_unpack.restype = ctypes.c_int
    lib.ssd_state_unpack.argtypes = [fp, fp, i64, i64, fp, fp, vp]
    lib.ssd_backward_workspace_size.restype = sz
    lib.ssd_backward_workspace_size.argtypes = [i64, i64, i64, i64, i32, i64, i32]
    lib.ssd_backward.restype = ctypes.c_int
    lib.ssd_backward.argtypes = [vp, vp, vp, fp, fp, fp, fp, fp, i64, i64, i64, i64, i32, i64, i32,
                                 fp, fp, fp, fp, fp, vp, sz, vp]
    lib.ssd_prep_backward.restype = ctypes.c_int
    lib.ssd_prep_backward.argtypes = [fp, fp, fp, fp, fp, i64, i64, i64, fp, fp, fp, vp]
    lib.ssd_prep_amask_backward.restype = ctypes.c_int
    lib.ssd_prep_amask_backward.argtypes = [fp, fp, fp, fp, i64, i64, i64, fp, fp, vp]
    f32 = ctypes.c_float
    lib.ssd_gated_scan_workspace_size.restype = sz
    lib.ssd_gated_scan_workspace_size.argtypes = [i64, i64, i64, i64]
    lib.ssd_gated_scan.restype = ctypes.c_int
    lib.ssd_gated_scan.argtypes = [vp, vp, vp, fp, i64, i64, i64, i64, i32, i32, fp, fp, vp, sz, vp]
    lib.ssd_gated_scan_step.restype = ctypes.c_int
    lib.ssd_gated_scan_step.argtypes = [vp, vp, vp, fp, i64, i64, i64, i32, i32, fp, vp]
    lib.ssd_gated_scan_backward_workspace_size.restype = sz
    lib.ssd_gated_scan_backward_workspace_size.argtypes = [i64, i64, i64, i64]
    lib.ssd_gated_scan_backward.restype = ctypes.c_int
    lib.ssd_gated_scan_backward.argtypes = [vp, vp, vp, fp, fp, fp, fp, i64, i64, i64, i64, i32, i32,
                                            fp, fp, fp, fp, vp, sz, vp]
    lib.ssd_norm_in.restype = ctypes.c_int
    lib.ssd_norm_in.argtypes = [fp, vp, fp, fp, i64, i64, f32, i32, fp, vp, vp]
    lib.ssd_norm_in_backward_workspace_size.restype = sz
    lib.ssd_norm_in_backward_workspace_size.argtypes = [i64, i64]
    lib.ssd_norm_in_backward.restype = ctypes.c_int
    lib.ssd_norm_in_backward.argtypes = [vp, fp, fp, vp, fp, fp, i64, i64, f32, i32, fp, fp, fp, fp, vp, sz, vp]
    lib.ssd_norm_out.restype = ctypes.c_int
    lib.ssd_norm_out.argtypes = [fp, vp, fp, i64, i64, i64, i64, i64, i32, f32, i32, vp, vp]
    lib.ssd_norm_out_backward_workspace_size.restype = sz
    lib.ssd_norm_out_backward_workspace_size.argtypes = [i64, i64, i64, i64, i64]
    lib.ssd_norm_out_backward.restype = ctypes.c_int
    lib.ssd_norm_out_backward.argtypes = [vp, fp, vp, fp, i64, i64, i64, i64, i64, i32, f32, i32, fp, fp, fp,
                                          vp, sz, vp]
    return lib


def lib():
    """Load libssd.so (built in-tree by ``python -m mamba_ssd_sequence_amd.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m mamba_ssd_sequence_amd.build` (no fallback path exists)")
        _lib = _declare(ctypes.CDLL(LIB_PATH))
    return _lib


def header_functions() -> list[str]:
    """Names of the functions declared in include/ssd.h."""
    with open(HEADER) as f:
        txt = f.read()
    return sorted(set(re.findall(r"^\s*(?:ssd_status|size_t|int|const char\*)\s+(ssd_\w+)\s*\(", txt, re.M)))


def _check(status: int):
    if status != SSD_OK:
        raise SSDError(status, lib().ssd_last_error().decode())


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device):
    torch = _torch()
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _require(t, name, dtype=None, device=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _qkv_dtype(t):
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return SSD_BF16
    if t.dtype == torch.float32:
        return SSD_F32
    raise ValueError(f"q/k/v must be bfloat16 or float32, got {t.dtype}")


def prep(dt_proj, dt_bias, A_log, chunk: int, out=None):
    """ssd_prep: returns (dt [B,H,N], a_cs [B,H,N], a_chunk [B,H,ceil(N/chunk)])."""
    torch = _torch()
    f32 = torch.float32
    _require(dt_proj, "dt_proj", f32)
    dev = dt_proj.device
    _require(dt_bias, "dt_bias", f32, dev)
    _require(A_log, "A_log", f32, dev)
    B, H, N = dt_proj.shape
    if dt_bias.shape != (H,) or A_log.shape != (H,):
        raise ValueError("dt_bias and A_log must have shape [H]")
    nc = -(-N // chunk)
    if out is None:
        out = (torch.empty_like(dt_proj), torch.empty_like(dt_proj),
               torch.empty((B, H, nc), dtype=f32, device=dev))
    dt, a_cs, a_chunk = out
    _check(lib().ssd_prep(_ptr(dt_proj), _ptr(dt_bias), _ptr(A_log), B, H, N, chunk,
                          _ptr(dt), _ptr(a_cs), _ptr(a_chunk), _stream(dev)))
    return dt, a_cs, a_chunk


def prep_amask(A_proj, dt_proj, chunk: int, out=None):
    """ssd_prep_amask (the A-mask of Algorithms 4 and 5): returns (dt or None,
    a_cs, a_chunk); dt_proj None means no dt (plain value operand)."""
    torch = _torch()
    f32 = torch.float32
    _require(A_proj, "A_proj", f32)
    dev = A_proj.device
    if dt_proj is not None:
        _require(dt_proj, "dt_proj", f32, dev)
        if dt_proj.shape != A_proj.shape:
            raise ValueError("dt_proj must have the shape of A_proj")
    B, H, N = A_proj.shape
    nc = -(-N // chunk)
    if out is None:
        out = (torch.empty_like(A_proj) if dt_proj is not None else None, torch.empty_like(A_proj),
               torch.empty((B, H, nc), dtype=f32, device=dev))
    dt, a_cs, a_chunk = out
    _check(lib().ssd_prep_amask(_ptr(A_proj), _ptr(dt_proj), B, H, N, chunk, _ptr(dt), _ptr(a_cs),
                                _ptr(a_chunk), _stream(dev)))
    return dt, a_cs, a_chunk


def workspace_size(B, H, N, d_h, order, chunk, dtype) -> int:
    return int(lib().ssd_forward_workspace_size(B, H, N, d_h, order, chunk, dtype))


def forward(q, k, v, dt, a_cs, order: int, chunk: int, *, y=None, den=None,
            final_state=None, final_norm=None, workspace=None, initial_state=None,
            initial_norm=None):
    """ssd_forward: y [B,H,N,d_h] fp32 (den and final states optional outputs;
    initial states optional inputs).  workspace: a uint8 device tensor, None
    (one is allocated), or "noalloc" for ssd_forward_noalloc (the library's
    per-device scratch; sizes up to SSD_NOALLOC_SCRATCH_BYTES of workspace)."""
    torch = _torch()
    _require(q, "q")
    dev = q.device
    dtype = _qkv_dtype(q)
    for name, t in (("k", k), ("v", v)):
        _require(t, name, q.dtype, dev)
        if t.shape != q.shape:
            raise ValueError(f"{name} shape {tuple(t.shape)} != q shape {tuple(q.shape)}")
    B, H, N, d_h = q.shape
    if dt is not None:
        _require(dt, "dt", torch.float32, dev)
    _require(a_cs, "a_cs", torch.float32, dev)
    if y is None:
        y = torch.empty((B, H, N, d_h), dtype=torch.float32, device=dev)
    for name, t in (("y", y), ("den", den), ("final_state", final_state), ("final_norm", final_norm),
                    ("initial_state", initial_state), ("initial_norm", initial_norm)):
        if t is not None:
            _require(t, name, torch.float32, dev)
    if workspace == "noalloc":
        # ssd_forward_noalloc: the library's own per-device scratch, no workspace
        _check(lib().ssd_forward_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(dt), _ptr(a_cs), _ptr(initial_state),
                                         _ptr(initial_norm), B, H, N, d_h, order, chunk, dtype, _ptr(y),
                                         _ptr(den), _ptr(final_state), _ptr(final_norm), _stream(dev)))
        return y
    need = workspace_size(B, H, N, d_h, order, chunk, dtype)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().ssd_forward(_ptr(q), _ptr(k), _ptr(v), _ptr(dt), _ptr(a_cs), _ptr(initial_state),
                             _ptr(initial_norm), B, H, N, d_h, order,
                             chunk, dtype, _ptr(y), _ptr(den), _ptr(final_state), _ptr(final_norm),
                             _ptr(workspace), wbytes, _stream(dev)))
    return y


class KernelTimer:
    """Per-kernel HIP-event timing of one ssd_forward call (events recorded by
    the library on its own stream, between its kernel launches)."""

    N_EVENTS = 8

    def __init__(self):
        torch = _torch()
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(self.N_EVENTS)]
        for e in self.events:  # materialise the underlying hipEvent_t
            e.record()
        self._arr = (ctypes.c_void_p * self.N_EVENTS)(*[e.cuda_event for e in self.events])
        self.count = 0

    def arm(self):
        _check(lib().ssd_set_timing_events(self._arr, self.N_EVENTS))

    def collect(self):
        """After ssd_forward: remember how many kernels were bracketed."""
        self.count = lib().ssd_timing_count()

    def durations_ms(self):
        """Per-kernel durations (call after synchronising)."""
        return [self.events[i].elapsed_time(self.events[i + 1]) for i in range(self.count)]


def _decode_common(q, k, v, params, state, norm_state, order, y, packed):
    torch = _torch()
    _require(q, "q")
    dev = q.device
    dtype = _qkv_dtype(q)
    for name, t in (("k", k), ("v", v)):
        _require(t, name, q.dtype, dev)
    S, H, d_h = q.shape
    for name, t in params + (("state", state), ("norm_state", norm_state)):
        if t is not None:
            _require(t, name, torch.float32, dev)
    if y is None:
        y = torch.empty((S, H, d_h), dtype=torch.float32, device=dev)
    layout = SSD_STATE_PACKED if packed else SSD_STATE_FULL
    return dev, dtype, S, H, d_h, layout, y


def decode_step(q, k, v, dt_proj, dt_bias, A_log, state, norm_state, order: int, *, y=None,
                packed=False):
    """ssd_decode_step: updates state/norm_state in place, returns y [S,H,d_h] fp32.
    packed: the order-2 states are in the packed layout (rows a <= b)."""
    dev, dtype, S, H, d_h, layout, y = _decode_common(
        q, k, v, (("dt_proj", dt_proj), ("dt_bias", dt_bias), ("A_log", A_log)), state, norm_state,
        order, y, packed)
    _check(lib().ssd_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(dt_proj), _ptr(dt_bias), _ptr(A_log),
                                 S, H, d_h, order, dtype, layout, _ptr(state), _ptr(norm_state), _ptr(y),
                                 _stream(dev)))
    return y


def decode_step_amask(q, k, v, A_proj, dt_proj, state, norm_state, order: int, *, y=None,
                      packed=False):
    """ssd_decode_step_amask (Algorithm 6 as printed): decay exp(-softplus(A_P));
    value operand v softplus(dt_P), or plain v when dt_proj is None."""
    dev, dtype, S, H, d_h, layout, y = _decode_common(
        q, k, v, (("A_proj", A_proj), ("dt_proj", dt_proj)), state, norm_state, order, y, packed)
    _check(lib().ssd_decode_step_amask(_ptr(q), _ptr(k), _ptr(v), _ptr(A_proj),
                                       _ptr(dt_proj) if dt_proj is not None else None,
                                       S, H, d_h, order, dtype, layout, _ptr(state), _ptr(norm_state),
                                       _ptr(y), _stream(dev)))
    return y


def decode_step_conv(q, k, v, conv_w, conv_b, conv_state, state, norm_state, order: int, *,
                     A_proj=None, dt_proj=None, dt_bias=None, A_log=None, act=False, y=None,
                     packed=False):
    """ssd_decode_step_conv: Algorithm 6's window-2 convolution of the raw q, k,
    v [S,H,d_h] (conv_w [3,H,d_h,2], conv_b [3,H,d_h] or None, SiLU if act)
    with the previous raw token held in conv_state [S,3,H,d_h] (updated in
    place), then the decode step: the A-mask with A_proj (optional dt_proj),
    else the Mamba-2 discretisation (dt_proj, dt_bias, A_log)."""
    dev, dtype, S, H, d_h, layout, y = _decode_common(
        q, k, v, (("A_proj", A_proj), ("dt_proj", dt_proj), ("dt_bias", dt_bias), ("A_log", A_log),
                  ("conv_w", conv_w), ("conv_b", conv_b)), state, norm_state, order, y, packed)
    _require(conv_state, "conv_state", q.dtype, dev)
    if tuple(conv_state.shape) != (S, 3, H, d_h) or tuple(conv_w.shape) != (3, H, d_h, 2):
        raise ValueError(f"conv_state {tuple(conv_state.shape)} / conv_w {tuple(conv_w.shape)} do not match "
                         f"[{S},3,{H},{d_h}] / [3,{H},{d_h},2]")
    if conv_b is not None and tuple(conv_b.shape) != (3, H, d_h):
        raise ValueError(f"conv_b {tuple(conv_b.shape)} does not match [3,{H},{d_h}]")
    _check(lib().ssd_decode_step_conv(_ptr(q), _ptr(k), _ptr(v), _ptr(conv_w), _ptr(conv_b), 1 if act else 0,
                                      _ptr(conv_state), _ptr(A_proj), _ptr(dt_proj), _ptr(dt_bias),
                                      _ptr(A_log), S, H, d_h, order, dtype, layout, _ptr(state),
                                      _ptr(norm_state), _ptr(y), _stream(dev)))
    return y


def _state_layout(fn, src_S, src_z, to_packed, out):
    torch = _torch()
    _require(src_S, "state", torch.float32)
    dev = src_S.device
    _require(src_z, "norm", torch.float32, dev)
    lead = src_S.shape[:-2]
    d_h = src_S.shape[-1]
    BH = 1
    for n in lead:
        BH *= n
    src_rows = d_h * d_h if to_packed else d_h * (d_h + 1) // 2
    if src_S.shape[-2] != src_rows or tuple(src_z.shape) != tuple(lead) + (src_rows,):
        raise ValueError(f"state shape {tuple(src_S.shape)} / norm shape {tuple(src_z.shape)} "
                         f"do not match {src_rows} rows of width {d_h}")
    rows = d_h * (d_h + 1) // 2 if to_packed else d_h * d_h
    if out is None:
        out = (torch.empty(lead + (rows, d_h), dtype=torch.float32, device=dev),
               torch.empty(lead + (rows,), dtype=torch.float32, device=dev))
    _check(fn(_ptr(src_S), _ptr(src_z), BH, d_h, _ptr(out[0]), _ptr(out[1]), _stream(dev)))
    return out


def state_pack(state, norm_state, out=None):
    """ssd_state_pack: full order-2 states [..., d_h^2, d_h], [..., d_h^2] ->
    packed [..., d_h(d_h+1)/2, d_h], [..., d_h(d_h+1)/2]."""
    return _state_layout(lib().ssd_state_pack, state, norm_state, True, out)


def state_unpack(state_p, norm_p, out=None):
    """ssd_state_unpack: packed order-2 states -> the full layout."""
    return _state_layout(lib().ssd_state_unpack, state_p, norm_p, False, out)


def backward(q, k, v, dt, a_cs, y, den, dy, order: int, chunk: int, *, workspace=None):
    """ssd_backward: returns dq, dk, dv, ddt (None when dt is None), da."""
    torch = _torch()
    _require(q, "q")
    dev = q.device
    dtype = _qkv_dtype(q)
    for name, t in (("k", k), ("v", v)):
        _require(t, name, q.dtype, dev)
    B, H, N, d_h = q.shape
    for name, t in (("a_cs", a_cs), ("y", y), ("den", den), ("dy", dy)) + ((("dt", dt),) if dt is not None else ()):
        _require(t, name, torch.float32, dev)
    dq, dk, dv = (torch.empty((B, H, N, d_h), dtype=torch.float32, device=dev) for _ in range(3))
    da = torch.empty((B, H, N), dtype=torch.float32, device=dev)
    ddt = torch.empty((B, H, N), dtype=torch.float32, device=dev) if dt is not None else None
    need = lib().ssd_backward_workspace_size(B, H, N, d_h, order, chunk, dtype)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    wptr = _ptr(workspace) if workspace is not None else None
    wbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    opt = lambda t: _ptr(t) if t is not None else None
    _check(lib().ssd_backward(_ptr(q), _ptr(k), _ptr(v), opt(dt), _ptr(a_cs), _ptr(y), _ptr(den), _ptr(dy),
                              B, H, N, d_h, order, chunk, dtype, _ptr(dq), _ptr(dk), _ptr(dv), opt(ddt),
                              _ptr(da), wptr, wbytes, _stream(dev)))
    return dq, dk, dv, ddt, da


def prep_backward(dt_proj, dt_bias, A_log, da, ddt=None):
    """ssd_prep_backward: returns d_dt_proj [B,H,N], d_dt_bias [H], d_A_log [H]."""
    torch = _torch()
    _require(dt_proj, "dt_proj", torch.float32)
    dev = dt_proj.device
    for name, t in (("dt_bias", dt_bias), ("A_log", A_log), ("da", da)) + ((("ddt", ddt),) if ddt is not None else ()):
        _require(t, name, torch.float32, dev)
    B, H, N = dt_proj.shape
    d_dt_proj = torch.empty_like(dt_proj)
    d_bias = torch.empty((H,), dtype=torch.float32, device=dev)
    d_alog = torch.empty((H,), dtype=torch.float32, device=dev)
    _check(lib().ssd_prep_backward(_ptr(dt_proj), _ptr(dt_bias), _ptr(A_log), _ptr(da),
                                   _ptr(ddt) if ddt is not None else None, B, H, N, _ptr(d_dt_proj),
                                   _ptr(d_bias), _ptr(d_alog), _stream(dev)))
    return d_dt_proj, d_bias, d_alog


def prep_amask_backward(A_proj, dt_proj, da, ddt=None):
    """ssd_prep_amask_backward: returns d_A_proj and d_dt_proj (None without dt_proj)."""
    torch = _torch()
    _require(A_proj, "A_proj", torch.float32)
    dev = A_proj.device
    _require(da, "da", torch.float32, dev)
    if (dt_proj is None) != (ddt is None):
        raise ValueError("dt_proj and ddt go together")
    if dt_proj is not None:
        _require(dt_proj, "dt_proj", torch.float32, dev)
        _require(ddt, "ddt", torch.float32, dev)
    B, H, N = A_proj.shape
    d_A = torch.empty_like(A_proj)
    d_dt = torch.empty_like(A_proj) if dt_proj is not None else None
    opt = lambda t: _ptr(t) if t is not None else None
    _check(lib().ssd_prep_amask_backward(_ptr(A_proj), opt(dt_proj), _ptr(da), opt(ddt), B, H, N,
                                         _ptr(d_A), opt(d_dt), _stream(dev)))
    return d_A, d_dt


# ---- the gated linear recurrence and the norms around a mixer block ----
#
# The shortest of these calls take a few microseconds on the GPU, so what a call
# costs on the host counts: tensors are checked by one condition each (the
# message is made only when it fails), and the stream is taken as a number.


def _refuse(t, name, dtype, shape, index):
    """Why a tensor was refused."""
    _require(t, name, dtype, _torch().device("cuda", index))
    raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _at(t, name, dtype, shape, index):
    """The address of a call's tensor after its checks (None for None)."""
    if t is None:
        return None
    try:
        if t.get_device() == index and t.dtype is dtype and t.shape == shape and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, dtype, shape, index)


def _first(t, name):
    """The checks of a tensor that sets a call's sizes; returns its element type and device index."""
    try:
        index, kind = t.get_device(), _kinds().get(t.dtype)
        if index >= 0 and kind is not None and t.is_contiguous():
            return kind, index
    except AttributeError:
        pass
    _require(t, name)
    raise ValueError(f"{name} must be bfloat16 or float32, got {t.dtype}")


@functools.lru_cache(maxsize=1)
def _kinds():
    torch = _torch()
    return {torch.bfloat16: SSD_BF16, torch.float32: SSD_F32}


@functools.lru_cache(maxsize=1)
def _current():
    """Functions for the current device's index and a device's current stream as a number."""
    torch = _torch()
    device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return device, stream or (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(fn, index, *args):
    """fn(*args, stream) on the arrays' device and its current stream (the
    library launches on the current device)."""
    device, stream = _current()
    if index == device():
        status = fn(*args, stream(index))
    else:
        with _torch().cuda.device(index):
            status = fn(*args, stream(index))
    if status != SSD_OK:
        _check(status)


@functools.lru_cache(maxsize=256)
def _scratch_size(name, *sizes):
    return int(getattr(lib(), name)(*sizes))


def _scratch(workspace, need, like):
    """A call's workspace: (address, bytes, tensor); one is allocated on like's device when None is given."""
    if workspace is None:
        if not need:
            return None, 0, None
        workspace = _torch().empty(need, dtype=_torch().uint8, device=like.device)
        return workspace.data_ptr(), need, workspace
    _require(workspace, "workspace", None, like.device)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def gated_scan(x, A_proj, I_proj=None, *, scale: int, initial_state=None, final_state=None, y=None,
               workspace=None):
    """ssd_gated_scan: h_t = a_t h_{t-1} + beta_t g_t x_t with a = sigmoid(-A_proj), g = sigmoid(I_proj)
    (or 1) and beta by scale (SSD_INPUT_PLAIN, _CONVEX, _UNIT).  x, A_proj, I_proj [B,H,N,d_h] bf16 or
    fp32, states [B,H,d_h] fp32 (final_state is written when given); returns y [B,H,N,d_h] fp32."""
    torch = _torch()
    kind, i = _first(x, "x")
    f32, xt, shape = torch.float32, x.dtype, x.shape
    B, H, N, d_h = shape
    state = (B, H, d_h)
    if y is None:
        y = torch.empty_like(x, dtype=f32)
    ws, nbytes, keep = _scratch(workspace, _scratch_size("ssd_gated_scan_workspace_size", B, H, N, d_h), x)
    _call(lib().ssd_gated_scan, i, x.data_ptr(), _at(A_proj, "A_proj", xt, shape, i),
          _at(I_proj, "I_proj", xt, shape, i), _at(initial_state, "initial_state", f32, state, i), B, H, N, d_h,
          scale, kind, _at(y, "y", f32, shape, i), _at(final_state, "final_state", f32, state, i), ws, nbytes)
    return y


def gated_scan_step(x, A_proj, I_proj, state, *, scale: int, new_state=None):
    """ssd_gated_scan_step: one token of S sequences, x, A_proj, I_proj (or None) [S,H,d_h], state
    [S,H,d_h] fp32.  The state is updated in place unless new_state is given; returns the new state,
    which is the step's output."""
    kind, i = _first(x, "x")
    f32, xt, shape = _torch().float32, x.dtype, x.shape
    S, H, d_h = shape
    if new_state is None:
        new_state = state
    _call(lib().ssd_gated_scan_step, i, x.data_ptr(), _at(A_proj, "A_proj", xt, shape, i),
          _at(I_proj, "I_proj", xt, shape, i), _at(state, "state", f32, shape, i), S, H, d_h, scale, kind,
          _at(new_state, "new_state", f32, shape, i))
    return new_state


def gated_scan_backward(x, A_proj, I_proj, y, dy, *, scale: int, initial_state=None, d_final_state=None,
                        workspace=None):
    """ssd_gated_scan_backward: returns dx, dA_proj, dI_proj (None without I_proj) and d_initial_state
    (None without initial_state), all fp32.  y: gated_scan's output; dy, d_final_state (or None): the
    gradients with respect to y and the final state."""
    torch = _torch()
    kind, i = _first(x, "x")
    f32, xt, shape = torch.float32, x.dtype, x.shape
    B, H, N, d_h = shape
    state = (B, H, d_h)
    py, ph0 = _at(y, "y", f32, shape, i), _at(initial_state, "initial_state", f32, state, i)
    if y is None:
        raise TypeError("y must be a torch.Tensor")
    dx, dA = torch.empty_like(y), torch.empty_like(y)
    dI = torch.empty_like(y) if I_proj is not None else None
    dh0 = torch.empty_like(initial_state) if initial_state is not None else None
    ws, nbytes, keep = _scratch(workspace, _scratch_size("ssd_gated_scan_backward_workspace_size", B, H, N, d_h), x)
    _call(lib().ssd_gated_scan_backward, i, x.data_ptr(), _at(A_proj, "A_proj", xt, shape, i),
          _at(I_proj, "I_proj", xt, shape, i), ph0, py, _at(dy, "dy", f32, shape, i),
          _at(d_final_state, "d_final_state", f32, state, i), B, H, N, d_h, scale, kind, dx.data_ptr(),
          dA.data_ptr(), dI.data_ptr() if dI is not None else None, dh0.data_ptr() if dh0 is not None else None,
          ws, nbytes)
    return dx, dA, dI, dh0


def norm_in(residual, branch, branch_scale, weight, eps: float, *, dtype=None, residual_out=None, out=None):
    """ssd_norm_in: r' = residual + branch_scale branch, u = weight r' / sqrt(mean r'^2 + eps) over the last
    dimension.  residual [..,E] fp32; branch [..,E] bf16 or fp32, or None (then r' is residual, and dtype
    is u's type); branch_scale [E] fp32 or None (1).  Returns (r' fp32, u of branch's type, which dtype,
    if given, has to be)."""
    torch = _torch()
    f32 = torch.float32
    i = _first(residual, "residual")[1]
    shape = residual.shape
    E = shape[-1]
    at = _at(residual, "residual", f32, shape, i)
    if branch is not None:
        if dtype is not None and dtype is not branch.dtype:
            raise ValueError(f"dtype {dtype} with a branch of {branch.dtype}: the result has the branch's type")
        dtype = branch.dtype
        if residual_out is None:
            residual_out = torch.empty_like(residual)
    if out is None:
        out = torch.empty_like(residual, dtype=dtype)
    kind, dtype = _qkv_dtype(out), (out.dtype if dtype is None else dtype)
    rows = residual.numel() // E if E else 0
    _call(lib().ssd_norm_in, i, at, _at(branch, "branch", dtype, shape, i),
          _at(branch_scale, "branch_scale", f32, (E,), i), _at(weight, "weight", f32, (E,), i), rows, E,
          eps, kind, _at(residual_out, "residual_out", f32, shape, i), _at(out, "out", dtype, shape, i))
    return (residual if branch is None else residual_out), out


def norm_in_backward(d_out, d_residual_out, residual_out, branch, branch_scale, weight, eps: float, *,
                     workspace=None):
    """ssd_norm_in_backward: returns d_residual [..,E], d_branch [..,E], d_weight [E], d_branch_scale [E], all
    fp32.  Without branch_scale the branch's gradient is d_residual itself and d_branch_scale is None; branch
    is then not read.  d_residual_out: fp32, or None (zero); residual_out: the r' of norm_in."""
    torch = _torch()
    f32 = torch.float32
    kind, i = _first(d_out, "d_out")
    shape = d_out.shape
    E = shape[-1]
    if branch_scale is not None and branch is None:
        raise ValueError("branch_scale without branch")
    if branch_scale is None:
        branch = None
    rows = d_out.numel() // E if E else 0
    pr, pw = _at(residual_out, "residual_out", f32, shape, i), _at(weight, "weight", f32, (E,), i)
    if residual_out is None or weight is None:
        raise TypeError("residual_out and weight must be torch.Tensors")
    d_residual, d_weight = torch.empty_like(residual_out), torch.empty_like(weight)
    d_branch = torch.empty_like(residual_out) if branch is not None else None
    d_scale = torch.empty_like(weight) if branch is not None else None
    ws, nbytes, keep = _scratch(workspace, _scratch_size("ssd_norm_in_backward_workspace_size", rows, E), d_out)
    _call(lib().ssd_norm_in_backward, i, d_out.data_ptr(), _at(d_residual_out, "d_residual_out", f32, shape, i), pr,
          _at(branch, "branch", d_out.dtype, shape, i), _at(branch_scale, "branch_scale", f32, (E,), i), pw, rows, E,
          eps, kind, d_residual.data_ptr(),
          d_branch.data_ptr() if branch is not None else None, d_weight.data_ptr(),
          d_scale.data_ptr() if branch is not None else None, ws, nbytes)
    return d_residual, (d_residual if d_branch is None else d_branch), d_weight, d_scale


def norm_out(y, z, weight, eps: float, *, groups: int = 1, gate_first: bool = True, out=None):
    """ssd_norm_out: the mixer's y [B,H,N,d_h] fp32, gated by silu(z) and normalised over `groups` groups of a
    token's channels, in token order: z and the result [B,N,H d_h] bf16 or fp32, weight [H d_h] fp32."""
    torch = _torch()
    kind, i = _first(z, "z")
    zt = z.dtype
    py = _at(y, "y", torch.float32, y.shape, i)
    B, H, N, d_h = y.shape
    shape = (B, N, H * d_h)
    if out is None:
        out = torch.empty_like(z)
    _call(lib().ssd_norm_out, i, py, _at(z, "z", zt, shape, i),
          _at(weight, "weight", torch.float32, (H * d_h,), i), B, H, N, d_h, groups, 1 if gate_first else 0, eps,
          kind, _at(out, "out", zt, shape, i))
    return out


def norm_out_backward(d_out, y, z, weight, eps: float, *, groups: int = 1, gate_first: bool = True,
                      workspace=None):
    """ssd_norm_out_backward: returns dy [B,H,N,d_h], dz [B,N,H d_h], d_weight [H d_h], all fp32."""
    torch = _torch()
    f32 = torch.float32
    kind, i = _first(z, "z")
    zt = z.dtype
    py = _at(y, "y", f32, y.shape, i)
    B, H, N, d_h = y.shape
    shape = (B, N, H * d_h)
    pw = _at(weight, "weight", f32, (H * d_h,), i)
    if weight is None:
        raise TypeError("weight must be a torch.Tensor")
    dy, dz, d_weight = torch.empty_like(y), torch.empty_like(z, dtype=f32), torch.empty_like(weight)
    ws, nbytes, keep = _scratch(workspace,
                                _scratch_size("ssd_norm_out_backward_workspace_size", B, H, N, d_h, groups), z)
    _call(lib().ssd_norm_out_backward, i, _at(d_out, "d_out", zt, shape, i), py, _at(z, "z", zt, shape, i), pw, B, H,
          N, d_h, groups, 1 if gate_first else 0, eps, kind, dy.data_ptr(), dz.data_ptr(), d_weight.data_ptr(), ws,
          nbytes)
    return dy, dz, d_weight
