"""The operators of the layer around a token mixer: the short causal convolution before it,
the selective state space scan (a mixer with a diagonal state) and the group norm with a
gate after it.  A thin binding of the C entry points of the same names (include/qdelta.h
has the formulas); every tensor is contiguous and on one CUDA device.

Shared arguments: activations are bfloat16 or float32, one dtype per call; parameters,
their gradients and the scan's state are float32.  lens [B] int32 (or None): tokens from
lens[b] on are padding, whose inputs are not used and whose outputs and gradients are 0.
"""
from __future__ import annotations

import torch

from . import (_call, _check, _dtype_code, _need, _ptr, _same_device, _stream, _workspace, load_library)

F32, I32 = torch.float32, torch.int32


def _new(t, shape, dtype, device, name):
    """The caller's output after a check, or a fresh one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _need(t, name, dtype, shape)
    return t


def short_conv_fwd(x, w, bias=None, S0=None, *, lens=None, silu=True, y=None, S_final=None, return_final=True,
                   stream=None):
    """Depthwise causal convolution over tokens with an optional SiLU.  x [B,T,D]; w [D,W]
    (W = 2, 3 or 4), bias [D] or None; S0 [B,W-1,D] in x's dtype: the inputs just before
    the call, or None (= 0).  Returns (y, S_final), S_final the last W - 1 inputs."""
    B, T, D = x.shape
    W, dt, dev = w.shape[-1], x.dtype, x.device
    _need(x, "x", dt, (B, T, D))
    _need(w, "w", F32, (D, W))
    _need(bias, "bias", F32, (D,), optional=True)
    _need(S0, "S0", dt, (B, W - 1, D), optional=True)
    _need(lens, "lens", I32, (B,), optional=True)
    code = _dtype_code(x)
    y = _new(y, (B, T, D), dt, dev, "y")
    if S_final is not None or return_final:
        S_final = _new(S_final, (B, W - 1, D), dt, dev, "S_final")
    _same_device(dev, w, bias, S0, lens, y, S_final)
    _check(_call(dev, load_library().short_conv_fwd, _ptr(x), _ptr(w), _ptr(bias), _ptr(S0), _ptr(lens), _ptr(y),
                 _ptr(S_final), B, T, D, W, int(silu), code, _stream(stream, dev)), "short_conv_fwd")
    return y, S_final


def short_conv_step(S, x, w, bias=None, *, silu=True, y=None, stream=None):
    """One token of the convolution: x [N,D]; S [N,W-1,D] in x's dtype, the last W - 1
    inputs, updated in place.  Returns y [N,D]."""
    N, D = x.shape
    W, dt, dev = w.shape[-1], x.dtype, x.device
    _need(x, "x", dt, (N, D))
    _need(S, "S", dt, (N, W - 1, D))
    _need(w, "w", F32, (D, W))
    _need(bias, "bias", F32, (D,), optional=True)
    code = _dtype_code(x)
    y = _new(y, (N, D), dt, dev, "y")
    _same_device(dev, S, w, bias, y)
    _check(_call(dev, load_library().short_conv_step, _ptr(S), _ptr(x), _ptr(w), _ptr(bias), _ptr(y), N, D, W,
                 int(silu), code, _stream(stream, dev)), "short_conv_step")
    return y


def short_conv_bwd_workspace_bytes(B, T, D, W, dtype) -> int:
    return load_library().short_conv_bwd_workspace_bytes(B, T, D, W, dtype)


def short_conv_bwd(x, w, bias, S0, dy, dS_final=None, *, lens=None, silu=True, want_dS0=True, workspace=None,
                   stream=None):
    """Backward of short_conv_fwd: gradients of sum(dy * y) + sum(dS_final * S_final).
    Returns a dict dx, dw, dbias (None without a bias), dS0 (None unless want_dS0)."""
    B, T, D = x.shape
    W, dt, dev = w.shape[-1], x.dtype, x.device
    _need(x, "x", dt, (B, T, D))
    _need(w, "w", F32, (D, W))
    _need(bias, "bias", F32, (D,), optional=True)
    _need(S0, "S0", dt, (B, W - 1, D), optional=True)
    _need(lens, "lens", I32, (B,), optional=True)
    _need(dy, "dy", dt, (B, T, D))
    _need(dS_final, "dS_final", dt, (B, W - 1, D), optional=True)
    code = _dtype_code(x)
    g = {"dx": torch.empty_like(x), "dw": torch.empty_like(w),
         "dbias": None if bias is None else torch.empty_like(bias),
         "dS0": torch.empty((B, W - 1, D), dtype=dt, device=dev) if want_dS0 else None}
    workspace, wsb = _workspace(short_conv_bwd_workspace_bytes(B, T, D, W, code), workspace, dev)
    _same_device(dev, w, bias, S0, lens, dy, dS_final, workspace)
    _check(_call(dev, load_library().short_conv_bwd, _ptr(x), _ptr(w), _ptr(bias), _ptr(S0), _ptr(lens), _ptr(dy),
                 _ptr(dS_final), _ptr(g["dx"]), _ptr(g["dw"]), _ptr(g["dbias"]), _ptr(g["dS0"]), B, T, D, W,
                 int(silu), code, _ptr(workspace), wsb, _stream(stream, dev)), "short_conv_bwd")
    return g


def _ssm_inputs(x, delta, A, B, C, D, delta_bias):
    """Checks what every form of the scan takes; tokens are x's leading dimensions."""
    tok, ch, dt = tuple(x.shape[:-1]), x.shape[-1], x.dtype
    N, G = A.shape[-1], B.shape[-2]
    _need(x, "x", dt, (*tok, ch))
    _need(delta, "delta", dt, (*tok, ch))
    _need(A, "A", F32, (ch, N))
    _need(B, "B", dt, (*tok, G, N))
    _need(C, "C", dt, (*tok, G, N))
    _need(D, "D", F32, (ch,), optional=True)
    _need(delta_bias, "delta_bias", F32, (ch,), optional=True)
    return ch, G, N, _dtype_code(x)


def ssm_workspace_bytes(B, T, D, G, N, dtype) -> int:
    return load_library().ssm_workspace_bytes(B, T, D, G, N, dtype)


def ssm_fwd(x, delta, A, B, C, D=None, delta_bias=None, S0=None, *, lens=None, softplus=True, y=None, S_final=None,
            return_final=True, workspace=None, stream=None):
    """Selective state space scan.  x, delta [B,T,D]; A [D,N] (negative: the decay rates); B, C
    [B,T,G,N], shared by the D/G channels of a group; skip weight D [D] and delta_bias [D] or
    None; S0 [B,D,N] or None.  The step size is softplus(delta + delta_bias), or the sum itself
    with softplus=False.  Returns (y, S_final)."""
    nb, T, _ = x.shape
    ch, G, N, code = _ssm_inputs(x, delta, A, B, C, D, delta_bias)
    dev = x.device
    _need(S0, "S0", F32, (nb, ch, N), optional=True)
    _need(lens, "lens", I32, (nb,), optional=True)
    y = _new(y, (nb, T, ch), x.dtype, dev, "y")
    if S_final is not None or return_final:
        S_final = _new(S_final, (nb, ch, N), F32, dev, "S_final")
    workspace, wsb = _workspace(ssm_workspace_bytes(nb, T, ch, G, N, code), workspace, dev)
    _same_device(dev, delta, A, B, C, D, delta_bias, S0, lens, y, S_final, workspace)
    _check(_call(dev, load_library().ssm_fwd, _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                 _ptr(delta_bias), _ptr(S0), _ptr(lens), _ptr(y), _ptr(S_final), nb, T, ch, G, N, int(softplus), code,
                 _ptr(workspace), wsb, _stream(stream, dev)), "ssm_fwd")
    return y, S_final


def ssm_step(S, x, delta, A, B, C, D=None, delta_bias=None, *, softplus=True, y=None, stream=None):
    """One token of the scan: x, delta [N,D]; B, C [N,G,states]; S [N,D,states] float32 updated in
    place; the rest as in ssm_fwd.  Returns y [N,D]."""
    nb = x.shape[0]
    if x.dim() != 2:
        raise ValueError(f"x has shape {tuple(x.shape)}, expected [N, D]")
    ch, G, N, code = _ssm_inputs(x, delta, A, B, C, D, delta_bias)
    dev = x.device
    _need(S, "S", F32, (nb, ch, N))
    y = _new(y, (nb, ch), x.dtype, dev, "y")
    _same_device(dev, S, delta, A, B, C, D, delta_bias, y)
    _check(_call(dev, load_library().ssm_step, _ptr(S), _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                 _ptr(delta_bias), _ptr(y), nb, ch, G, N, int(softplus), code, _stream(stream, dev)), "ssm_step")
    return y


def ssm_bwd_workspace_bytes(B, T, D, G, N, dtype) -> int:
    return load_library().ssm_bwd_workspace_bytes(B, T, D, G, N, dtype)


def ssm_bwd(x, delta, A, B, C, D, delta_bias, S0, dy, dS_final=None, *, lens=None, softplus=True, want_dS0=True,
            workspace=None, stream=None):
    """Backward of ssm_fwd: gradients of sum(dy * y) + sum(dS_final * S_final).  Returns a dict
    dx, ddelta, dA, dB, dC, dD and ddelta_bias (None without the parameter), dS0 (None unless
    want_dS0)."""
    nb, T, _ = x.shape
    ch, G, N, code = _ssm_inputs(x, delta, A, B, C, D, delta_bias)
    dev = x.device
    _need(S0, "S0", F32, (nb, ch, N), optional=True)
    _need(lens, "lens", I32, (nb,), optional=True)
    _need(dy, "dy", x.dtype, (nb, T, ch))
    _need(dS_final, "dS_final", F32, (nb, ch, N), optional=True)
    g = {"dx": torch.empty_like(x), "ddelta": torch.empty_like(x), "dA": torch.empty_like(A),
         "dB": torch.empty_like(B), "dC": torch.empty_like(C), "dD": None if D is None else torch.empty_like(D),
         "ddelta_bias": None if delta_bias is None else torch.empty_like(delta_bias),
         "dS0": torch.empty((nb, ch, N), dtype=F32, device=dev) if want_dS0 else None}
    workspace, wsb = _workspace(ssm_bwd_workspace_bytes(nb, T, ch, G, N, code), workspace, dev)
    _same_device(dev, delta, A, B, C, D, delta_bias, S0, lens, dy, dS_final, workspace)
    _check(_call(dev, load_library().ssm_bwd, _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                 _ptr(delta_bias), _ptr(S0), _ptr(lens), _ptr(dy), _ptr(dS_final), _ptr(g["dx"]), _ptr(g["ddelta"]),
                 _ptr(g["dA"]), _ptr(g["dB"]), _ptr(g["dC"]), _ptr(g["dD"]), _ptr(g["ddelta_bias"]), _ptr(g["dS0"]),
                 nb, T, ch, G, N, int(softplus), code, _ptr(workspace), wsb, _stream(stream, dev)), "ssm_bwd")
    return g


def _norm_inputs(x, w, b, z):
    if x.dim() < 2:
        raise ValueError(f"x has shape {tuple(x.shape)}, expected [..., H, d]")
    H, d = x.shape[-2:]
    M = 1
    for n in x.shape[:-2]:
        M *= n
    _need(x, "x", x.dtype, x.shape)
    _need(w, "w", F32, (H, d), optional=True)
    _need(b, "b", F32, (H, d), optional=True)
    _need(z, "z", x.dtype, x.shape, optional=True)
    return M, H, d, _dtype_code(x)


def group_norm_fwd(x, w=None, b=None, z=None, *, eps=1e-5, center=True, silu=True, y=None, stream=None):
    """Group norm of each token's channels: x [..., H, d], H groups of d channels; w, b [H,d] or
    None (1, 0).  center=False: the root mean square in place of the mean and variance.  With a
    gate z (x's shape) y = n SiLU(z), else y = SiLU(n); silu=False: the identity in its place."""
    M, H, d, code = _norm_inputs(x, w, b, z)
    dev = x.device
    y = _new(y, tuple(x.shape), x.dtype, dev, "y")
    _same_device(dev, w, b, z, y)
    _check(_call(dev, load_library().group_norm_fwd, _ptr(x), _ptr(w), _ptr(b), _ptr(z), _ptr(y), M, H, d, eps,
                 int(center), int(silu), code, _stream(stream, dev)), "group_norm_fwd")
    return y


def group_norm_bwd_workspace_bytes(M, H, d, dtype) -> int:
    return load_library().group_norm_bwd_workspace_bytes(M, H, d, dtype)


def group_norm_bwd(x, w, b, z, dy, *, eps=1e-5, center=True, silu=True, workspace=None, stream=None):
    """Backward of group_norm_fwd: gradients of sum(dy * y).  Returns a dict dx, dz, dw, db (None
    without the input)."""
    M, H, d, code = _norm_inputs(x, w, b, z)
    dev = x.device
    _need(dy, "dy", x.dtype, x.shape)
    g = {"dx": torch.empty_like(x), "dz": None if z is None else torch.empty_like(z),
         "dw": None if w is None else torch.empty_like(w), "db": None if b is None else torch.empty_like(b)}
    workspace, wsb = _workspace(group_norm_bwd_workspace_bytes(M, H, d, code) if w is not None or b is not None else 0,
                                workspace, dev)
    _same_device(dev, w, b, z, dy, workspace)
    _check(_call(dev, load_library().group_norm_bwd, _ptr(x), _ptr(w), _ptr(b), _ptr(z), _ptr(dy), _ptr(g["dx"]),
                 _ptr(g["dz"]), _ptr(g["dw"]), _ptr(g["db"]), M, H, d, eps, int(center), int(silu), code,
                 _ptr(workspace), wsb, _stream(stream, dev)), "group_norm_bwd")
    return g
