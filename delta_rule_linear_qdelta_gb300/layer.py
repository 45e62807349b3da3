"""The operators of the layer around a token mixer: the short causal convolution before it,
the selective state space scan (a mixer with a diagonal state) and the group norm with a
gate after it.  A thin binding of the C entry points of the same names (include/qdelta.h
has the formulas); every tensor is contiguous and on one CUDA device.

Shared arguments: activations are bfloat16 or float32, one dtype per call; parameters,
their gradients and the scan's state are float32.  lens [B] int32 (or None): tokens from
lens[b] on are padding, whose inputs are not used and whose outputs and gradients are 0.  Every
call also takes stream= (a torch stream of the tensors' device, or a handle, 0 being the default
stream), on which all of it is then done.  A workspace is any contiguous tensor of enough bytes.
"""
from __future__ import annotations

import functools

import torch

from . import _check, _dtype_code, _need, _same_device, load_library

F32, I32 = torch.float32, torch.int32


def _arg(t, name, dtype, shape, dev, optional=False):
    """The address of an argument that is what it has to be; an error that says what is wrong
    otherwise.  One token's call spends most of its time on the host, so the usual case is a
    single test."""
    if t is None:
        if optional:
            return None
    elif t.dtype is dtype and t.shape == shape and t.get_device() == dev.index and t.is_contiguous():
        return t.data_ptr()
    _need(t, name, dtype, shape)
    _same_device(dev, t)


def _new(t, name, dtype, shape, dev):
    """The caller's output after a check, or a fresh one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _arg(t, name, dtype, shape, dev)
    return t


def _sizes(*sizes):
    """Refuses what the C entry points' 32-bit sizes cannot hold: it would arrive there cut off."""
    if max(sizes) > 0x7fffffff:
        raise ValueError(f"a size of {max(sizes)} does not fit in 32 bits")


def _adr(t):
    return None if t is None else t.data_ptr()


def _scratch(nbytes, workspace, dev):
    """Address and size of the caller's workspace, or of a fresh one of nbytes, and its owner."""
    if workspace is None:
        if nbytes == 0:
            return None, 0, None
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _same_device(dev, workspace)
    if not workspace.is_contiguous():                   # its bytes are not where its element count says
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _run(name, dev, *args):
    """Calls the entry point `name` with `dev` current and the current stream as its last argument."""
    fn = getattr(load_library(), name)
    if torch._C._cuda_getDevice() == dev.index:
        _check(fn(*args, torch._C._cuda_getCurrentRawStream(dev.index)), name)
    else:
        with torch.cuda.device(dev):
            _check(fn(*args, torch._C._cuda_getCurrentRawStream(dev.index)), name)


def _on_stream(call):
    """Adds the argument `stream` (a torch stream or a handle; None: the current one).  The whole call
    is made on it, so outputs and scratch belong to it: PyTorch does not give scratch that a kernel
    there still uses to another stream."""
    @functools.wraps(call)
    def on(*args, stream=None, **kw):
        dev = None if stream is None else next((t.device for t in (*args, *kw.values()) if isinstance(t, torch.Tensor)), None)
        if dev is None or dev.type != "cuda":           # (no tensor on a GPU: refused by the call)
            return call(*args, **kw)
        if not isinstance(stream, torch.cuda.Stream):
            # (an ExternalStream of handle 0 would be a new stream, not the default one)
            stream = torch.cuda.ExternalStream(int(stream), device=dev) if int(stream) else torch.cuda.default_stream(dev)
        elif stream.device != dev:
            raise ValueError(f"stream of {stream.device}, expected one of {dev}, where the tensors are")
        with torch.cuda.stream(stream):
            return call(*args, **kw)
    return on


@_on_stream
def short_conv_fwd(x, w, bias=None, S0=None, *, lens=None, silu=True, y=None, S_final=None, return_final=True):
    """Depthwise causal convolution over tokens with an optional SiLU.  x [B,T,D]; w [D,W]
    (W = 2, 3 or 4), bias [D] or None; S0 [B,W-1,D] in x's dtype: the inputs just before
    the call, or None (= 0).  Returns (y, S_final), S_final the last W - 1 inputs."""
    B, T, D = x.shape
    W, dt, dev = w.shape[-1], x.dtype, x.device
    _sizes(B, T, D, W)
    args = (_arg(x, "x", dt, (B, T, D), dev), _arg(w, "w", F32, (D, W), dev), _arg(bias, "bias", F32, (D,), dev, True),
            _arg(S0, "S0", dt, (B, W - 1, D), dev, True), _arg(lens, "lens", I32, (B,), dev, True))
    code = _dtype_code(x)
    y = _new(y, "y", dt, (B, T, D), dev)
    if S_final is not None or return_final:
        S_final = _new(S_final, "S_final", dt, (B, W - 1, D), dev)
    _run("short_conv_fwd", dev, *args, y.data_ptr(), _adr(S_final), B, T, D, W, int(silu), code)
    return y, S_final


@_on_stream
def short_conv_step(S, x, w, bias=None, *, silu=True, y=None):
    """One token of the convolution: x [N,D]; S [N,W-1,D] in x's dtype, the last W - 1
    inputs, updated in place.  Returns y [N,D]."""
    N, D = x.shape
    W, dt, dev = w.shape[-1], x.dtype, x.device
    _sizes(N, D, W)
    args = (_arg(S, "S", dt, (N, W - 1, D), dev), _arg(x, "x", dt, (N, D), dev), _arg(w, "w", F32, (D, W), dev),
            _arg(bias, "bias", F32, (D,), dev, True))
    code = _dtype_code(x)
    y = torch.empty_like(x) if y is None else _new(y, "y", dt, (N, D), dev)
    _run("short_conv_step", dev, *args, y.data_ptr(), N, D, W, int(silu), code)
    return y


def short_conv_bwd_workspace_bytes(B, T, D, W, dtype) -> int:
    _sizes(B, T, D, W)
    return load_library().short_conv_bwd_workspace_bytes(B, T, D, W, dtype)


@_on_stream
def short_conv_bwd(x, w, bias, S0, dy, dS_final=None, *, lens=None, silu=True, want_dS0=True, workspace=None):
    """Backward of short_conv_fwd: gradients of sum(dy * y) + sum(dS_final * S_final).
    Returns a dict dx, dw, dbias (None without a bias), dS0 (None unless want_dS0)."""
    B, T, D = x.shape
    W, dt, dev = w.shape[-1], x.dtype, x.device
    _sizes(B, T, D, W)
    args = (_arg(x, "x", dt, (B, T, D), dev), _arg(w, "w", F32, (D, W), dev), _arg(bias, "bias", F32, (D,), dev, True),
            _arg(S0, "S0", dt, (B, W - 1, D), dev, True), _arg(lens, "lens", I32, (B,), dev, True),
            _arg(dy, "dy", dt, (B, T, D), dev), _arg(dS_final, "dS_final", dt, (B, W - 1, D), dev, True))
    code = _dtype_code(x)
    g = {"dx": torch.empty_like(x), "dw": torch.empty_like(w),
         "dbias": None if bias is None else torch.empty_like(bias),
         "dS0": torch.empty((B, W - 1, D), dtype=dt, device=dev) if want_dS0 else None}
    ws, wsb, hold = _scratch(short_conv_bwd_workspace_bytes(B, T, D, W, code), workspace, dev)
    _run("short_conv_bwd", dev, *args, *map(_adr, g.values()), B, T, D, W, int(silu), code, ws, wsb)
    return g


def _ssm_inputs(x, delta, A, B, C, D, delta_bias):
    """Checks what every form of the scan takes; tokens are x's leading dimensions."""
    tok, ch, dt, dev = tuple(x.shape[:-1]), x.shape[-1], x.dtype, x.device
    N, G = A.shape[-1], B.shape[-2]
    _sizes(*x.shape, G, N)
    args = (_arg(x, "x", dt, (*tok, ch), dev), _arg(delta, "delta", dt, (*tok, ch), dev), _arg(A, "A", F32, (ch, N), dev),
            _arg(B, "B", dt, (*tok, G, N), dev), _arg(C, "C", dt, (*tok, G, N), dev),
            _arg(D, "D", F32, (ch,), dev, True), _arg(delta_bias, "delta_bias", F32, (ch,), dev, True))
    return args, ch, G, N, _dtype_code(x), dev


def ssm_workspace_bytes(B, T, D, G, N, dtype) -> int:
    _sizes(B, T, D, G, N)
    return load_library().ssm_workspace_bytes(B, T, D, G, N, dtype)


@_on_stream
def ssm_fwd(x, delta, A, B, C, D=None, delta_bias=None, S0=None, *, lens=None, softplus=True, y=None, S_final=None,
            return_final=True, workspace=None):
    """Selective state space scan.  x, delta [B,T,D]; A [D,N] (negative: the decay rates); B, C
    [B,T,G,N], shared by the D/G channels of a group; skip weight D [D] and delta_bias [D] or
    None; S0 [B,D,N] or None.  The step size is softplus(delta + delta_bias), or the sum itself
    with softplus=False.  Returns (y, S_final)."""
    nb, T, _ = x.shape
    args, ch, G, N, code, dev = _ssm_inputs(x, delta, A, B, C, D, delta_bias)
    args += (_arg(S0, "S0", F32, (nb, ch, N), dev, True), _arg(lens, "lens", I32, (nb,), dev, True))
    y = _new(y, "y", x.dtype, (nb, T, ch), dev)
    if S_final is not None or return_final:
        S_final = _new(S_final, "S_final", F32, (nb, ch, N), dev)
    ws, wsb, hold = _scratch(ssm_workspace_bytes(nb, T, ch, G, N, code), workspace, dev)
    _run("ssm_fwd", dev, *args, y.data_ptr(), _adr(S_final), nb, T, ch, G, N, int(softplus), code, ws, wsb)
    return y, S_final


@_on_stream
def ssm_step(S, x, delta, A, B, C, D=None, delta_bias=None, *, softplus=True, y=None):
    """One token of the scan: x, delta [N,D]; B, C [N,G,states]; S [N,D,states] float32 updated in
    place; the rest as in ssm_fwd.  Returns y [N,D]."""
    nb, _ = x.shape
    args, ch, G, N, code, dev = _ssm_inputs(x, delta, A, B, C, D, delta_bias)
    S = _arg(S, "S", F32, (nb, ch, N), dev)
    y = _new(y, "y", x.dtype, (nb, ch), dev)
    _run("ssm_step", dev, S, *args, y.data_ptr(), nb, ch, G, N, int(softplus), code)
    return y


def ssm_bwd_workspace_bytes(B, T, D, G, N, dtype) -> int:
    _sizes(B, T, D, G, N)
    return load_library().ssm_bwd_workspace_bytes(B, T, D, G, N, dtype)


@_on_stream
def ssm_bwd(x, delta, A, B, C, D, delta_bias, S0, dy, dS_final=None, *, lens=None, softplus=True, want_dS0=True,
            workspace=None):
    """Backward of ssm_fwd: gradients of sum(dy * y) + sum(dS_final * S_final).  Returns a dict
    dx, ddelta, dA, dB, dC, dD and ddelta_bias (None without the parameter), dS0 (None unless
    want_dS0)."""
    nb, T, _ = x.shape
    args, ch, G, N, code, dev = _ssm_inputs(x, delta, A, B, C, D, delta_bias)
    args += (_arg(S0, "S0", F32, (nb, ch, N), dev, True), _arg(lens, "lens", I32, (nb,), dev, True),
             _arg(dy, "dy", x.dtype, (nb, T, ch), dev), _arg(dS_final, "dS_final", F32, (nb, ch, N), dev, True))
    g = {"dx": torch.empty_like(x), "ddelta": torch.empty_like(x), "dA": torch.empty_like(A),
         "dB": torch.empty_like(B), "dC": torch.empty_like(C), "dD": None if D is None else torch.empty_like(D),
         "ddelta_bias": None if delta_bias is None else torch.empty_like(delta_bias),
         "dS0": torch.empty((nb, ch, N), dtype=F32, device=dev) if want_dS0 else None}
    ws, wsb, hold = _scratch(ssm_bwd_workspace_bytes(nb, T, ch, G, N, code), workspace, dev)
    _run("ssm_bwd", dev, *args, *map(_adr, g.values()), nb, T, ch, G, N, int(softplus), code, ws, wsb)
    return g


def _norm_inputs(x, w, b, z):
    if x.dim() < 2:
        raise ValueError(f"x has shape {tuple(x.shape)}, expected [..., H, d]")
    dev, (H, d), M = x.device, x.shape[-2:], 1
    for n in x.shape[:-2]:
        M *= n
    _sizes(M, H, d)
    args = (_arg(x, "x", x.dtype, x.shape, dev), _arg(w, "w", F32, (H, d), dev, True),
            _arg(b, "b", F32, (H, d), dev, True), _arg(z, "z", x.dtype, x.shape, dev, True))
    return args, M, H, d, _dtype_code(x), dev


@_on_stream
def group_norm_fwd(x, w=None, b=None, z=None, *, eps=1e-5, center=True, silu=True, y=None):
    """Group norm of each token's channels: x [..., H, d], H groups of d channels; w, b [H,d] or
    None (1, 0).  center=False: the root mean square in place of the mean and variance.  With a
    gate z (x's shape) y = n SiLU(z), else y = SiLU(n); silu=False: the identity in its place."""
    args, M, H, d, code, dev = _norm_inputs(x, w, b, z)
    y = _new(y, "y", x.dtype, x.shape, dev)
    _run("group_norm_fwd", dev, *args, y.data_ptr(), M, H, d, eps, int(center), int(silu), code)
    return y


def group_norm_bwd_workspace_bytes(M, H, d, dtype) -> int:
    _sizes(M, H, d)
    return load_library().group_norm_bwd_workspace_bytes(M, H, d, dtype)


@_on_stream
def group_norm_bwd(x, w, b, z, dy, *, eps=1e-5, center=True, silu=True, workspace=None):
    """Backward of group_norm_fwd: gradients of sum(dy * y).  Returns a dict dx, dz, dw, db (None
    without the input)."""
    args, M, H, d, code, dev = _norm_inputs(x, w, b, z)
    dy = _arg(dy, "dy", x.dtype, x.shape, dev)
    g = {"dx": torch.empty_like(x), "dz": None if z is None else torch.empty_like(z),
         "dw": None if w is None else torch.empty_like(w), "db": None if b is None else torch.empty_like(b)}
    need = 0 if w is None and b is None else group_norm_bwd_workspace_bytes(M, H, d, code)
    ws, wsb, hold = _scratch(need, workspace, dev)
    _run("group_norm_bwd", dev, *args, dy, *map(_adr, g.values()), M, H, d, eps, int(center), int(silu), code,
         ws, wsb)
    return g
