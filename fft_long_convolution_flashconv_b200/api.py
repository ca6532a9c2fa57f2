"""PyTorch-facing wrappers over the C ABI (argument marshalling only: every
step runs in the CUDA library; torch only provides device memory and the
current stream).

Complex SSM parameters are float32 tensors of shape (..., 2) (re, im) or
complex64 tensors.  I/O tensors are float32, float16 or bfloat16 CUDA tensors.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from . import _lib
from ._lib import check

_DT = {torch.float32: _lib.FC_F32, torch.float16: _lib.FC_F16, torch.bfloat16: _lib.FC_BF16}


def _stream():
    return ctypes_void(torch.cuda.current_stream().cuda_stream)


def ctypes_void(x):
    import ctypes
    return ctypes.c_void_p(x)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _cpx(t: torch.Tensor) -> torch.Tensor:
    if t.is_complex():
        t = torch.view_as_real(t)
    if t.dtype != torch.float32 or t.shape[-1] != 2:
        raise ValueError("complex parameters must be complex64 or float32 (..., 2)")
    return t.contiguous()


def _f32(t: torch.Tensor) -> torch.Tensor:
    if t.dtype != torch.float32:
        raise ValueError("parameters must be float32")
    return t.contiguous()


def _dtype(t: torch.Tensor) -> int:
    if t.dtype not in _DT:
        raise ValueError(f"unsupported dtype {t.dtype}")
    return _DT[t.dtype]


def _alloc_ws(nbytes: int, device) -> torch.Tensor:
    # torch's caching allocator returns >= 256-byte aligned blocks
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


def tc_timeouts() -> int:
    """Tensor-core blocks that gave up waiting on a matrix-multiply completion
    (their part of an output is unwritten); 0 in normal operation."""
    return int(_lib.load().fc_tc_timeouts())


def ssm_kernel_gen(dt, lam, Bp, Cp, L: int, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """f[h, k] = 2 Re sum_n C B A^k, A = exp(dt lambda); returns H x L float32."""
    lib = _lib.load()
    dt, lam, Bp, Cp = _f32(dt), _cpx(lam), _cpx(Bp), _cpx(Cp)
    H, N = lam.shape[0], lam.shape[1]
    if out is None:
        out = torch.empty((H, L), dtype=torch.float32, device=dt.device)
    check(lib.ssm_kernel_gen(_ptr(dt), _ptr(lam), _ptr(Bp), _ptr(Cp), H, N, L, _ptr(out), _stream()),
          "ssm_kernel_gen")
    return out


def fftconv_fwd(u: torch.Tensor, f: torch.Tensor, D: torch.Tensor,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y = causal_conv(u, f) + D u via the fused FFT kernel; u: B x H x L."""
    lib = _lib.load()
    B, H, L = u.shape
    f, D = _f32(f), _f32(D)
    if out is None:
        out = torch.empty_like(u)
    check(lib.fftconv_fwd(_ptr(u), _ptr(f), _ptr(D), _ptr(out), B, H, L, _dtype(u), _stream()), "fftconv_fwd")
    return out


def long_conv_workspace_bytes(B: int, H: int, L: int) -> int:
    return int(_lib.load().fftconv_long_workspace(B, H, L))


def fftconv_long_fwd(u: torch.Tensor, f: torch.Tensor, D: torch.Tensor, out: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y = causal_conv(u, f) + D u for L up to 65536 (arbitrary filter); u: B x H x L."""
    lib = _lib.load()
    B, H, L = u.shape
    f, D = _f32(f), _f32(D)
    if out is None:
        out = torch.empty_like(u)
    need = int(lib.fftconv_long_workspace(B, H, L))
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=u.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    check(lib.fftconv_long_fwd(_ptr(u), _ptr(f), _ptr(D), _ptr(out), B, H, L, _ptr(workspace), ws_bytes,
                               _dtype(u), _stream()), "fftconv_long_fwd")
    return out


def fftconv_bwd(dy: torch.Tensor, u: torch.Tensor, f: torch.Tensor, D: torch.Tensor, need_du: bool = True,
                need_dfilter: bool = True):
    """Gradients of y = causal_conv(u, f) + D u given dy; returns (du, df, dD)
    (None for the parts not requested)."""
    lib = _lib.load()
    B, H, L = dy.shape
    f, D = _f32(f), _f32(D)
    du = torch.empty_like(dy) if need_du else None
    df = torch.empty((H, L), dtype=torch.float32, device=dy.device) if need_dfilter else None
    dD = torch.empty((H,), dtype=torch.float32, device=dy.device) if need_dfilter else None
    check(lib.fftconv_bwd(_ptr(dy), _ptr(u), _ptr(f), _ptr(D), _ptr(du), _ptr(df), _ptr(dD), B, H, L, _dtype(dy),
                          _stream()), "fftconv_bwd")
    return du, df, dD


def ssm_decode_step(u, x, dt, lam, Bp, Cp, D, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """T tokens of the recurrent view; u: B x H x T; x: B x H x N x 2 float32
    state, updated in place.  Returns y (B x H x T)."""
    lib = _lib.load()
    B, H, Tn = u.shape
    dt, lam, Bp, Cp, D = _f32(dt), _cpx(lam), _cpx(Bp), _cpx(Cp), _f32(D)
    N = lam.shape[1]
    if x.dtype != torch.float32 or tuple(x.shape) != (B, H, N, 2) or not x.is_contiguous():
        raise ValueError("x must be a contiguous float32 B x H x N x 2 tensor")
    if out is None:
        out = torch.empty_like(u)
    check(lib.ssm_decode_step(_ptr(u), _ptr(x), _ptr(dt), _ptr(lam), _ptr(Bp), _ptr(Cp), _ptr(D), _ptr(out), B, H,
                              N, Tn, _dtype(u), _stream()), "ssm_decode_step")
    return out


def h3_decode_state(B, heads, head_dim, N, device) -> torch.Tensor:
    """Zeroed recurrent state of the H3 mixer (B x heads x hd x hd x N x 2 float32)."""
    return torch.zeros((B, heads, head_dim, head_dim, N, 2), dtype=torch.float32, device=device)


def h3_mixer_decode_step(q, k, v, kring, state, Cshift, dt, lam, Bp, Cp, D, heads: int, pos: int,
                         out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token (q, k, v: B x d_model) of the H3 mixer in recurrent form."""
    lib = _lib.load()
    B, dm = q.shape
    hd = dm // heads
    Cshift, dt, lam, Bp, Cp, D = _f32(Cshift), _f32(dt), _cpx(lam), _cpx(Bp), _cpx(Cp), _f32(D)
    N = lam.shape[1]
    S = Cshift.shape[1]
    if out is None:
        out = torch.empty_like(q)
    check(lib.h3_mixer_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(kring), _ptr(state), _ptr(Cshift), _ptr(dt),
                                   _ptr(lam), _ptr(Bp), _ptr(Cp), _ptr(D), _ptr(out), B, heads, hd, N, S, pos,
                                   _dtype(q), _stream()), "h3_mixer_decode_step")
    return out


def ssm_conv_workspace_bytes(H: int, L: int) -> int:
    return int(_lib.load().ssm_conv_workspace(H, L))


def ssm_conv_fwd(u, dt, lam, Bp, Cp, D, workspace: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Filter generation + fused FFT convolution in one call."""
    lib = _lib.load()
    B, H, L = u.shape
    dt, lam, Bp, Cp, D = _f32(dt), _cpx(lam), _cpx(Bp), _cpx(Cp), _f32(D)
    N = lam.shape[1]
    need = int(lib.ssm_conv_workspace(H, L))
    if workspace is None:
        workspace = _alloc_ws(need, u.device)
    if out is None:
        out = torch.empty_like(u)
    check(lib.ssm_conv_fwd(_ptr(u), _ptr(dt), _ptr(lam), _ptr(Bp), _ptr(Cp), _ptr(D), _ptr(out), B, H, L, N,
                           _ptr(workspace), workspace.numel() * workspace.element_size(), _dtype(u), _stream()),
          "ssm_conv_fwd")
    return out


def ssm_conv_fwd_noalloc(u, dt, lam, Bp, Cp, D, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """ssm_conv_fwd without a workspace: the filter goes to a fixed scratch
    array inside the library (H * L <= ssm_conv_noalloc_max_filter_floats())."""
    lib = _lib.load()
    B, H, L = u.shape
    dt, lam, Bp, Cp, D = _f32(dt), _cpx(lam), _cpx(Bp), _cpx(Cp), _f32(D)
    N = lam.shape[1]
    if out is None:
        out = torch.empty_like(u)
    st = lib.ssm_conv_fwd_noalloc(_ptr(u), _ptr(dt), _ptr(lam), _ptr(Bp), _ptr(Cp), _ptr(D), _ptr(out), B, H, L, N,
                                  _dtype(u), _stream())
    if st != _lib.FC_OK:
        raise _lib.FlashConvError(st, "ssm_conv_fwd_noalloc", lib.ssm_conv_noalloc_last_error().decode())
    return out


def statepass_workspace_bytes(B, H, L, N, chunk) -> int:
    return int(_lib.load().fftconv_statepass_workspace(B, H, L, N, chunk))


def fftconv_statepass(u, dt, lam, Bp, Cp, D, chunk: int, state_in: Optional[torch.Tensor] = None,
                      return_state: bool = False, workspace: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None):
    """Chunked state passing; returns y (and the final state B x H x N x 2 if
    return_state)."""
    lib = _lib.load()
    B, H, L = u.shape
    dt, lam, Bp, Cp, D = _f32(dt), _cpx(lam), _cpx(Bp), _cpx(Cp), _f32(D)
    N = lam.shape[1]
    need = int(lib.fftconv_statepass_workspace(B, H, L, N, chunk))
    if workspace is None:
        workspace = _alloc_ws(need, u.device)
    if out is None:
        out = torch.empty_like(u)
    sin = _cpx(state_in) if state_in is not None else None
    sout = torch.empty((B, H, N, 2), dtype=torch.float32, device=u.device) if return_state else None
    check(lib.fftconv_statepass(_ptr(u), _ptr(dt), _ptr(lam), _ptr(Bp), _ptr(Cp), _ptr(D), _ptr(out), B, H, L,
                                N, chunk, _ptr(sin), _ptr(sout), _ptr(workspace),
                                workspace.numel() * workspace.element_size(), _dtype(u), _stream()),
          "fftconv_statepass")
    return (out, sout) if return_state else out


def fftconv_statepass_bwd(dy, dt, lam, Bp, Cp, D, chunk: int, dstate_out: Optional[torch.Tensor] = None,
                          need_dstate_in: bool = False, workspace: Optional[torch.Tensor] = None,
                          out: Optional[torch.Tensor] = None):
    """Gradients of fftconv_statepass: du (and dstate_in, B x H x N x 2, if
    need_dstate_in) given dy and optionally dstate_out."""
    lib = _lib.load()
    B, H, L = dy.shape
    dt, lam, Bp, Cp, D = _f32(dt), _cpx(lam), _cpx(Bp), _cpx(Cp), _f32(D)
    N = lam.shape[1]
    need = int(lib.fftconv_statepass_bwd_workspace(B, H, L, N, chunk, _dtype(dy)))
    if workspace is None:
        workspace = _alloc_ws(need, dy.device)
    if out is None:
        out = torch.empty_like(dy)
    gin = _cpx(dstate_out) if dstate_out is not None else None
    gsin = torch.empty((B, H, N, 2), dtype=torch.float32, device=dy.device) if need_dstate_in else None
    check(lib.fftconv_statepass_bwd(_ptr(dy), _ptr(dt), _ptr(lam), _ptr(Bp), _ptr(Cp), _ptr(D), _ptr(out), B, H, L,
                                    N, chunk, _ptr(gin), _ptr(gsin), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), _dtype(dy), _stream()),
          "fftconv_statepass_bwd")
    return (out, gsin) if need_dstate_in else out


def h3_mixer_workspace_bytes(B, L, heads, head_dim, N) -> int:
    return int(_lib.load().h3_mixer_workspace(B, L, heads, head_dim, N))


def h3_mixer_fwd(q, k, v, Cshift, dt, lam, Bp, Cp, D, heads: int, workspace: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """H3 mixer core O = Q (.) SSM_diag(SSM_shift(K) (.) V) per head; q, k, v:
    B x L x (heads*head_dim)."""
    lib = _lib.load()
    B, L, dm = q.shape
    hd = dm // heads
    Cshift, dt, lam, Bp, Cp, D = _f32(Cshift), _f32(dt), _cpx(lam), _cpx(Bp), _cpx(Cp), _f32(D)
    N = lam.shape[1]
    S = Cshift.shape[1]
    need = int(lib.h3_mixer_workspace(B, L, heads, hd, N))
    if workspace is None:
        workspace = _alloc_ws(need, q.device)
    if out is None:
        out = torch.empty_like(q)
    check(lib.h3_mixer_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(Cshift), _ptr(dt), _ptr(lam), _ptr(Bp), _ptr(Cp),
                           _ptr(D), _ptr(out), B, L, heads, hd, N, S, _ptr(workspace),
                           workspace.numel() * workspace.element_size(), _dtype(q), _stream()),
          "h3_mixer_fwd")
    return out


# ------------------------------------------------------------------ selective SSM
# Sequences are B x H x L with contiguous time and any other strides (the halves
# of a projection need no copy); parameters are contiguous float32.  A call runs
# on its tensors' device, on that device's current stream.
def _device(first: torch.Tensor, *others) -> torch.device:
    """The one CUDA device that all tensors (None: absent) are on."""
    dev = first.device
    if dev.type != "cuda":
        raise ValueError("expected a CUDA tensor")
    for t in others:
        if t is not None and t.device != dev:
            raise ValueError(f"tensors on different devices: {dev} and {t.device}")
    return dev


# What torch.cuda.current_device() and current_stream() ask, without their checks; a torch built
# without CUDA has neither, and no tensor that gets past _device().
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _call(dev: torch.device, name: str, *args) -> None:
    """Calls the library on the device's current stream, with the device current."""
    if dev.index != _current_device():
        with torch.cuda.device(dev):
            return _call(dev, name, *args)
    status = getattr(_lib.load(), name)(*args, _raw_stream(dev.index))
    if status:
        check(status, name)


class _On:
    """Makes a device current where it is not."""

    def __init__(self, dev: torch.device):
        self.guard = None if dev.index == _current_device() else torch.cuda.device(dev)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _check(t: Optional[torch.Tensor], name: str, shape: tuple, dtype: torch.dtype) -> Optional[torch.Tensor]:
    if t is not None and not (t.dtype is dtype and t.shape == shape):
        if t.dtype is not dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _dense(t: Optional[torch.Tensor], name: str, shape: tuple, dtype: torch.dtype):
    """A contiguous tensor of this shape and type, or None."""
    if t is None or (t.dtype is dtype and t.shape == shape and t.is_contiguous()):
        return t
    _check(t, name, shape, dtype)
    raise ValueError(f"{name} must be contiguous")


def _seq(t: Optional[torch.Tensor], name: str, shape: tuple, dtype: torch.dtype):
    """A sequence of this shape and type with contiguous time, or None."""
    if t is None or (t.dtype is dtype and t.shape == shape and (t.stride(-1) == 1 or shape[-1] == 1)):
        return t
    _check(t, name, shape, dtype)
    raise ValueError(f"{name} must be contiguous along its last axis")


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


@functools.lru_cache(maxsize=256)
def _strides(*values):
    """The host array of these strides (only read by the library)."""
    return (ctypes.c_longlong * len(values))(*values)


def _need(t: Optional[torch.Tensor], nbytes: int, device) -> torch.Tensor:
    """The caller's workspace, or a new one."""
    if t is None:
        return _alloc_ws(nbytes, device)
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"the workspace must be contiguous and on {device}")
    return t


def _slots(slots: Optional[torch.Tensor], B: int):
    return _dense(slots, "slots", (B,), torch.int32)


def _lengths(lengths: Optional[torch.Tensor], B: int):
    return _dense(lengths, "lengths", (B,), torch.int32)


def _sizes(t: torch.Tensor, name: str, dims: str):
    if t.dim() != dims.count(" x ") + 1:
        raise ValueError(f"{name} must be {dims}, got shape {tuple(t.shape)}")
    if t.dtype not in _DT:
        raise ValueError(f"unsupported dtype {t.dtype}")
    return t.shape


def short_conv_fwd(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None, silu: bool = True,
                   state_in: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                   return_state: bool = False, out: Optional[torch.Tensor] = None):
    """Short causal convolution by channels: y[t] = silu(bias + sum_j w[j] x[t-j]);
    x: B x H x L, w: H x K (tap 0 = the current token).  state_in: the K-1 inputs
    before x, B x H x (K-1), oldest first.  Returns y (and the last K-1 inputs if
    return_state)."""
    B, H, L = _sizes(x, "x", "B x H x L")
    K = w.shape[-1]
    _seq(x, "x", (B, H, L), x.dtype)
    _dense(w, "w", (H, K), torch.float32)
    _dense(bias, "bias", (H,), torch.float32)
    _dense(state_in, "state_in", (B, H, K - 1), x.dtype)
    _lengths(lengths, B)
    _dense(out, "out", (B, H, L), x.dtype)
    dev = _device(x, w, bias, state_in, lengths, out)
    if out is None:
        out = x.new_empty((B, H, L))
    state = x.new_empty((B, H, K - 1)) if return_state else None
    _call(dev, "short_conv_fwd", _addr(x), _addr(w), _addr(bias), _addr(out), B, H, L, K, bool(silu), _addr(lengths),
          _strides(x.stride(0), x.stride(1)), _addr(state_in), _addr(state), _DT[x.dtype])
    return (out, state) if return_state else out


def short_conv_bwd_workspace_bytes(B: int, H: int, L: int, K: int) -> int:
    return int(_lib.load().short_conv_bwd_workspace(B, H, L, K))


def short_conv_bwd(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None,
                   silu: bool = True, state_in: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                   dstate_out: Optional[torch.Tensor] = None, need_dstate_in: bool = False,
                   workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None):
    """Gradients of short_conv_fwd given dy (and dstate_out): (dx, dw, dbias), and
    dstate_in if need_dstate_in (dbias: None without a bias)."""
    B, H, L = _sizes(x, "x", "B x H x L")
    K = w.shape[-1]
    io = x.dtype
    _seq(x, "x", (B, H, L), io)
    _seq(dy, "dy", (B, H, L), io)
    _dense(w, "w", (H, K), torch.float32)
    _dense(bias, "bias", (H,), torch.float32)
    _dense(state_in, "state_in", (B, H, K - 1), io)
    _dense(dstate_out, "dstate_out", (B, H, K - 1), io)
    _lengths(lengths, B)
    _dense(out, "out", (B, H, L), io)
    dev = _device(x, dy, w, bias, state_in, dstate_out, lengths, out)
    lib = _lib.load()
    workspace = _need(workspace, int(lib.short_conv_bwd_workspace(B, H, L, K)), dev)
    if out is None:
        out = x.new_empty((B, H, L))
    dw = torch.empty((H, K), dtype=torch.float32, device=dev)
    dbias = torch.empty((H,), dtype=torch.float32, device=dev) if bias is not None else None
    dstate = x.new_empty((B, H, K - 1)) if need_dstate_in else None
    _call(dev, "short_conv_bwd", _addr(dy), _addr(x), _addr(w), _addr(bias), _addr(out), _addr(dw), _addr(dbias), B, H,
          L, K, bool(silu), _addr(lengths), _strides(dy.stride(0), dy.stride(1), x.stride(0), x.stride(1)),
          _addr(state_in), _addr(dstate_out), _addr(dstate), _addr(workspace),
          workspace.numel() * workspace.element_size(), _DT[io])
    return (out, dw, dbias, dstate) if need_dstate_in else (out, dw, dbias)


def short_conv_step(x: torch.Tensor, state: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None,
                    silu: bool = True, slots: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token (x: B x H) of short_conv_fwd; state: S x H x (K-1), the last K-1
    inputs, updated in place.  slots: the rows' places in the state (int32; one
    outside [0, S), or one that an earlier row holds, marks a padded row: y = 0)."""
    B, H = _sizes(x, "x", "B x H")
    K, S = w.shape[-1], state.shape[0]
    _seq(x, "x", (B, H), x.dtype)
    _dense(w, "w", (H, K), torch.float32)
    _dense(bias, "bias", (H,), torch.float32)
    _dense(state, "state", (S, H, K - 1), x.dtype)
    _slots(slots, B)
    _dense(out, "out", (B, H), x.dtype)
    dev = _device(x, w, bias, state, slots, out)
    if out is None:
        out = x.new_empty((B, H))
    _call(dev, "short_conv_step", _addr(x), _addr(state), _addr(w), _addr(bias), _addr(out), B, H, K, bool(silu),
          _addr(slots), S, x.stride(0), _DT[x.dtype])
    return out


def _scan_inputs(u, delta, A, Bt, Ct, D, dt_bias, z, tail):
    """Shapes and types that the scan's calls share; tail: (L,), or () for one token."""
    B, H = u.shape[:2]
    if A.dim() != 2 or Bt.dim() != 3 + len(tail):
        raise ValueError("A must be H x N, Bt and Ct B x G x N (x L)")
    N, G, io = A.shape[1], Bt.shape[1], u.dtype
    # a token's rows are read element by element, with any stride
    seq = _seq if tail else _check
    for t, name in ((u, "u"), (delta, "delta"), (z, "z")):
        seq(t, name, (B, H, *tail), io)
    for t, name in ((Bt, "Bt"), (Ct, "Ct")):
        seq(t, name, (B, G, N, *tail), io)
    _dense(A, "A", (H, N), torch.float32)
    _dense(D, "D", (H,), torch.float32)
    _dense(dt_bias, "dt_bias", (H,), torch.float32)
    zs = z if z is not None else u
    strides = (*u.stride()[:2], *delta.stride()[:2], *zs.stride()[:2], *Bt.stride()[:3], *Ct.stride()[:3])
    return B, H, N, G, strides


def selective_scan_fwd(u: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, Bt: torch.Tensor, Ct: torch.Tensor,
                       D: Optional[torch.Tensor] = None, dt_bias: Optional[torch.Tensor] = None,
                       z: Optional[torch.Tensor] = None, softplus: bool = True,
                       state_in: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                       return_state: bool = False, return_ckpt: bool = False,
                       workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None):
    """Selective scan: dt = softplus(delta + dt_bias), x <- exp(dt A) x + dt B u,
    y = (C x + D u) silu(z); u, delta, z: B x H x L, A: H x N, Bt, Ct: B x G x N x L.
    Returns y, then the final state (B x H x N float32) if return_state, then what
    selective_scan_bwd needs if return_ckpt."""
    _sizes(u, "u", "B x H x L")
    L = u.shape[2]
    B, H, N, G, strides = _scan_inputs(u, delta, A, Bt, Ct, D, dt_bias, z, (L,))
    _dense(state_in, "state_in", (B, H, N), torch.float32)
    _lengths(lengths, B)
    _dense(out, "out", (B, H, L), u.dtype)
    dev = _device(u, delta, A, Bt, Ct, D, dt_bias, z, state_in, lengths, out)
    lib = _lib.load()
    if out is None:
        out = u.new_empty((B, H, L))
    state = torch.empty((B, H, N), dtype=torch.float32, device=dev) if return_state else None
    ckpt = None
    if return_ckpt:
        ckpt = torch.empty(int(lib.selective_scan_ckpt_bytes(B, H, L, N)) // 4, dtype=torch.float32, device=dev)
    with _On(dev):  # its size is that of the current device
        need = int(lib.selective_scan_workspace(B, H, L, N, G))
        if need or workspace is not None:
            workspace = _need(workspace, need, dev)
    _call(dev, "selective_scan_fwd", _addr(u), _addr(delta), _addr(A), _addr(Bt), _addr(Ct), _addr(D), _addr(dt_bias),
          _addr(z), _addr(out), B, H, L, N, G, bool(softplus), _addr(lengths), _strides(*strides), _addr(state_in),
          _addr(state), _addr(ckpt), _addr(workspace),
          0 if workspace is None else workspace.numel() * workspace.element_size(), _DT[u.dtype])
    more = ((state,) if return_state else ()) + ((ckpt,) if return_ckpt else ())
    return (out, *more) if more else out


def selective_scan_workspace_bytes(B: int, H: int, L: int, N: int, G: int) -> int:
    return int(_lib.load().selective_scan_workspace(B, H, L, N, G))


def selective_scan_bwd_workspace_bytes(B: int, H: int, L: int, N: int, G: int) -> int:
    return int(_lib.load().selective_scan_bwd_workspace(B, H, L, N, G))


def selective_scan_bwd(dy: torch.Tensor, u: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, Bt: torch.Tensor,
                       Ct: torch.Tensor, ckpt: torch.Tensor, D: Optional[torch.Tensor] = None,
                       dt_bias: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                       softplus: bool = True, lengths: Optional[torch.Tensor] = None,
                       dstate_out: Optional[torch.Tensor] = None, need_dstate_in: bool = False,
                       workspace: Optional[torch.Tensor] = None):
    """Gradients of selective_scan_fwd given dy, its inputs, the ckpt that it
    returned for them, and dstate_out: (du, ddelta, dA, dB, dC, dD, ddt_bias, dz), and
    dstate_in if need_dstate_in (dD, ddt_bias, dz: None where the input is)."""
    _sizes(u, "u", "B x H x L")
    L, io = u.shape[2], u.dtype
    B, H, N, G, strides = _scan_inputs(u, delta, A, Bt, Ct, D, dt_bias, z, (L,))
    _seq(dy, "dy", (B, H, L), io)
    lib = _lib.load()
    _dense(ckpt, "ckpt", (int(lib.selective_scan_ckpt_bytes(B, H, L, N)) // 4,), torch.float32)
    _dense(dstate_out, "dstate_out", (B, H, N), torch.float32)
    _lengths(lengths, B)
    dev = _device(u, dy, delta, A, Bt, Ct, ckpt, D, dt_bias, z, lengths, dstate_out)

    def new(*shape, dtype=torch.float32, when=True):
        return torch.empty(shape, dtype=dtype, device=dev) if when else None

    du, ddelta, dz = new(B, H, L, dtype=io), new(B, H, L, dtype=io), new(B, H, L, dtype=io, when=z is not None)
    dB, dC, dA = new(B, G, N, L, dtype=io), new(B, G, N, L, dtype=io), new(H, N)
    dD, dbias = new(H, when=D is not None), new(H, when=dt_bias is not None)
    dstate = new(B, H, N, when=need_dstate_in)
    with _On(dev):  # its size is that of the current device
        workspace = _need(workspace, int(lib.selective_scan_bwd_workspace(B, H, L, N, G)), dev)
    _call(dev, "selective_scan_bwd", _addr(dy), _addr(u), _addr(delta), _addr(A), _addr(Bt), _addr(Ct), _addr(D),
          _addr(dt_bias), _addr(z), _addr(ckpt), _addr(du), _addr(ddelta), _addr(dA), _addr(dB), _addr(dC), _addr(dD),
          _addr(dbias), _addr(dz), B, H, L, N, G, bool(softplus), _addr(lengths),
          _strides(dy.stride(0), dy.stride(1), *strides), _addr(dstate_out), _addr(dstate), _addr(workspace),
          workspace.numel() * workspace.element_size(), _DT[io])
    grads = (du, ddelta, dA, dB, dC, dD, dbias, dz)
    return (*grads, dstate) if need_dstate_in else grads


def selective_scan_step(u: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, Bt: torch.Tensor, Ct: torch.Tensor,
                        state: torch.Tensor, D: Optional[torch.Tensor] = None,
                        dt_bias: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                        softplus: bool = True, slots: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token of selective_scan_fwd: u, delta, z: B x H, Bt, Ct: B x G x N;
    state: S x H x N float32, updated in place.  slots: as short_conv_step."""
    _sizes(u, "u", "B x H")
    B, H, N, G, strides = _scan_inputs(u, delta, A, Bt, Ct, D, dt_bias, z, ())
    S = state.shape[0]
    _dense(state, "state", (S, H, N), torch.float32)
    _slots(slots, B)
    _dense(out, "out", (B, H), u.dtype)
    dev = _device(u, delta, A, Bt, Ct, D, dt_bias, z, state, slots, out)
    if out is None:
        out = u.new_empty((B, H))
    _call(dev, "selective_scan_step", _addr(u), _addr(delta), _addr(A), _addr(Bt), _addr(Ct), _addr(D), _addr(dt_bias),
          _addr(z), _addr(state), _addr(out), B, H, N, G, bool(softplus), _addr(slots), S, _strides(*strides),
          _DT[u.dtype])
    return out


def _norm_inputs(x, groups, weight, bias, gate, channel_major):
    _sizes(x, "x", "B x C x L" if channel_major else "B x L x C")
    B, L, C = (x.shape[0], x.shape[2], x.shape[1]) if channel_major else x.shape
    if groups < 1 or C % groups:
        raise ValueError(f"{C} channels are not a multiple of {groups} groups")
    _dense(x, "x", x.shape, x.dtype)
    _dense(gate, "gate", x.shape, x.dtype)
    _dense(weight, "weight", (C,), torch.float32)
    _dense(bias, "bias", (C,), torch.float32)
    return B, L, C


def group_norm_act_fwd(x: torch.Tensor, groups: int, weight: Optional[torch.Tensor] = None,
                       bias: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, eps: float = 1e-5,
                       channel_major: bool = False, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Group norm of every token on its own, with SiLU: y = silu(n), or n silu(gate),
    n = (x - mean) / sqrt(var + eps) weight + bias over a group's channels.  x, gate:
    B x L x C, or B x C x L with channel_major; y: B x L x C.  There is no `lengths`:
    padding is normalised too (zeros give silu(bias))."""
    B, L, C = _norm_inputs(x, groups, weight, bias, gate, channel_major)
    _dense(out, "out", (B, L, C), x.dtype)
    dev = _device(x, weight, bias, gate, out)
    if out is None:
        out = x.new_empty((B, L, C))
    _call(dev, "group_norm_act_fwd", _addr(x), _addr(weight), _addr(bias), _addr(gate), _addr(out), B, L, C, groups,
          eps, bool(channel_major), _DT[x.dtype])
    return out


def group_norm_act_bwd_workspace_bytes(B: int, L: int, C: int, groups: int, channel_major: bool = False) -> int:
    return int(_lib.load().group_norm_act_bwd_workspace(B, L, C, groups, bool(channel_major)))


def group_norm_act_bwd(dy: torch.Tensor, x: torch.Tensor, groups: int, weight: Optional[torch.Tensor] = None,
                       bias: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, eps: float = 1e-5,
                       channel_major: bool = False, workspace: Optional[torch.Tensor] = None):
    """Gradients of group_norm_act_fwd given dy (B x L x C): (dx, dweight, dbias,
    dgate), dx and dgate in x's layout (dweight, dbias, dgate: None where the input is).
    Tokens behind a padded row's end count in dweight and dbias unless their dy is zero."""
    B, L, C = _norm_inputs(x, groups, weight, bias, gate, channel_major)
    _dense(dy, "dy", (B, L, C), x.dtype)
    dev = _device(x, dy, weight, bias, gate)
    lib = _lib.load()
    dx = torch.empty_like(x)
    dgate = torch.empty_like(gate) if gate is not None else None
    dw = torch.empty((C,), dtype=torch.float32, device=dev) if weight is not None else None
    db = torch.empty((C,), dtype=torch.float32, device=dev) if bias is not None else None
    with _On(dev):  # its size is that of the current device
        workspace = _need(workspace, int(lib.group_norm_act_bwd_workspace(B, L, C, groups, bool(channel_major))), dev)
    _call(dev, "group_norm_act_bwd", _addr(dy), _addr(x), _addr(weight), _addr(bias), _addr(gate), _addr(dx),
          _addr(dw), _addr(db), _addr(dgate), B, L, C, groups, eps, bool(channel_major), _addr(workspace),
          workspace.numel() * workspace.element_size(), _DT[x.dtype])
    return dx, dw, db, dgate
