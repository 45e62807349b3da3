"""The mixers of a hybrid stack beside the Delta rule: linear attention with a decay for each head, and
softmax attention over a sliding window with a few first tokens that stay visible (sinks).  A thin binding
of the C entry points of the same names (include/qdelta.h has the formulas); every tensor is contiguous
and on one CUDA device.

Shared arguments: tokens are bfloat16 or float32, one dtype per call; states are float32; head dims are
multiples of 8 up to 128.  lens [B] int32 (or None): tokens from lens[b] on are padding, whose inputs are
not used and whose outputs and gradients are 0.  Every call also takes stream= (a torch stream of the
tensors' device, or a handle, 0 being the default stream), on which all of it is then done.  A workspace
is any contiguous tensor of enough bytes.
"""
from __future__ import annotations

import functools
import math

import torch

from . import _dtype_code, load_library
from .layer import F32, I32, _adr, _arg, _new, _on_stream, _run, _scratch, _sizes

# One token's call spends most of its time on the host: scratch sizes, which the sizes alone give, are asked for
# once, and new tensors are made like one at hand (1.5 us where torch.empty with a device takes 3.7).
@functools.lru_cache(maxsize=1024)
def _bytes(name, *sizes):
    return getattr(load_library(), name)(*sizes)


def _work(name, sizes, workspace, like):
    """Address, size and owner of the workspace of the entry point `name`: the caller's or a fresh one."""
    nbytes = _bytes(name + "_workspace_bytes", *sizes)
    if workspace is None and nbytes:
        workspace = like.new_empty(nbytes // like.element_size() + 1)
        return workspace.data_ptr(), nbytes, workspace
    return _scratch(nbytes, workspace, like.device)


def _like(t, name, src):
    """The caller's output after a check, or a fresh one, of src's shape and type."""
    return torch.empty_like(src) if t is None else _new(t, name, src.dtype, src.shape, src.device)


def _decay_arg(g, dt, tok, H, dev):
    """Address of the log decays, and whether there is one for each token."""
    if g is None:
        return None, 0
    if g.dim() == 1:
        return _arg(g, "g", F32, (H,), dev), 0
    return _arg(g, "g", dt, (*tok, H), dev), 1


def _lin_inputs(q, k, v, g, lead):
    """Checks what every form of linear attention takes; tokens are q's leading dimensions, named in `lead`."""
    if q.dim() != len(lead) + 2 or v.dim() != q.dim():
        raise ValueError(f"q, v have shapes {tuple(q.shape)}, {tuple(v.shape)}, expected [{', '.join(lead)}, H, d]")
    tok, (H, dk), dv, dt, dev = tuple(q.shape[:-2]), q.shape[-2:], v.shape[-1], q.dtype, q.device
    _sizes(*q.shape, dv)
    gp, per_token = _decay_arg(g, dt, tok, H, dev)
    args = (_arg(q, "q", dt, (*tok, H, dk), dev), _arg(k, "k", dt, (*tok, H, dk), dev),
            _arg(v, "v", dt, (*tok, H, dv), dev), gp)
    return args, H, dk, dv, per_token, _dtype_code(q), dev


def lin_attn_workspace_bytes(B, T, H, dk, dv, dtype) -> int:
    _sizes(B, T, H, dk, dv)
    return _bytes("lin_attn_workspace_bytes", B, T, H, dk, dv, dtype)


@_on_stream
def lin_attn_fwd(q, k, v, g=None, S0=None, *, lens=None, o=None, S_final=None, return_final=True, workspace=None):
    """Linear attention: S_t = exp(g_t) S_{t-1} + v_t k_t^T, o_t = S_t q_t.  q, k [B,T,H,dk]; v [B,T,H,dv];
    log decays g [B,T,H] in q's dtype (one for each token and head), [H] float32 (one for each head) or None
    (no decay), at most 0, -inf dropping the state; S0 [B,H,dv,dk] or None.  Returns (o, S_final)."""
    args, H, dk, dv, per_token, code, dev = _lin_inputs(q, k, v, g, "BT")
    B, T = q.shape[:2]
    args += (_arg(S0, "S0", F32, (B, H, dv, dk), dev, True), _arg(lens, "lens", I32, (B,), dev, True))
    o = _like(o, "o", v)
    if S_final is not None or return_final:
        S_final = _new(S_final, "S_final", F32, (B, H, dv, dk), dev)
    ws, wsb, hold = _work("lin_attn", (B, T, H, dk, dv, code), workspace, q)
    _run("lin_attn_fwd", dev, *args, o.data_ptr(), _adr(S_final), B, T, H, dk, dv, per_token, code, ws, wsb)
    return o, S_final


@_on_stream
def lin_attn_step(S, q, k, v, g=None, *, o=None):
    """One token of linear attention: q, k [N,H,dk]; v [N,H,dv]; g [N,H] in q's dtype, [H] float32 or None;
    S [N,H,dv,dk] float32 updated in place.  Returns o [N,H,dv]."""
    args, H, dk, dv, per_token, code, dev = _lin_inputs(q, k, v, g, "N")
    N = q.shape[0]
    S = _arg(S, "S", F32, (N, H, dv, dk), dev)
    o = _like(o, "o", v)
    _run("lin_attn_step", dev, S, *args, o.data_ptr(), N, H, dk, dv, per_token, code)
    return o


def lin_attn_bwd_workspace_bytes(B, T, H, dk, dv, dtype) -> int:
    _sizes(B, T, H, dk, dv)
    return _bytes("lin_attn_bwd_workspace_bytes", B, T, H, dk, dv, dtype)


@_on_stream
def lin_attn_bwd(q, k, v, g, S0, dO, dS_final=None, *, lens=None, want_dS0=True, workspace=None):
    """Backward of lin_attn_fwd: gradients of sum(dO * o) + sum(dS_final * S_final).  Returns a dict dq, dk, dv,
    dg (None unless g has a decay for each token), dS0 (None unless want_dS0)."""
    args, H, dk, dv, per_token, code, dev = _lin_inputs(q, k, v, g, "BT")
    B, T = q.shape[:2]
    args += (_arg(S0, "S0", F32, (B, H, dv, dk), dev, True), _arg(lens, "lens", I32, (B,), dev, True),
             _arg(dO, "dO", q.dtype, (B, T, H, dv), dev), _arg(dS_final, "dS_final", F32, (B, H, dv, dk), dev, True))
    r = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v),
         "dg": torch.empty_like(g) if per_token else None,
         "dS0": torch.empty((B, H, dv, dk), dtype=F32, device=dev) if want_dS0 else None}
    ws, wsb, hold = _work("lin_attn_bwd", (B, T, H, dk, dv, code), workspace, q)
    _run("lin_attn_bwd", dev, *args, *map(_adr, r.values()), B, T, H, dk, dv, per_token, code, ws, wsb)
    return r


def _win_inputs(q, k, v, lens, window, sinks, scale):
    """Checks the prompt's tensors; the keys before the call are those that k has more than q."""
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError(f"q, k have shapes {tuple(q.shape)}, {tuple(k.shape)}, expected [B, T, H, d] and [B, keys, Hkv, d]")
    (B, T, H, d), (_, Tk, Hkv, _), dt, dev = q.shape, k.shape, q.dtype, q.device
    if Tk < T:
        raise ValueError(f"k has {Tk} tokens, expected the {T} of q and those before them")
    window = max(1, Tk) if window is None else window
    _sizes(B, Tk, H, d, window, sinks, window + sinks)
    args = (_arg(q, "q", dt, (B, T, H, d), dev), _arg(k, "k", dt, (B, Tk, Hkv, d), dev), _arg(v, "v", dt, (B, Tk, Hkv, d), dev))
    sizes = (B, T, Tk - T, H, Hkv, d, window, sinks)
    return args, _arg(lens, "lens", I32, (B,), dev, True), sizes, _scale(scale, d), _dtype_code(q), dev


def _scale(scale, d):
    return 1.0 / math.sqrt(d) if scale is None else scale


@_on_stream
def win_attn_fwd(q, k, v, *, window=None, sinks=0, scale=None, lens=None, o=None, lse=None, return_lse=True):
    """Softmax attention over a sliding window with sinks.  q [B,T,H,d]; k, v [B,past+T,Hkv,d]: `past` keys from
    before the call, then the call's; Hkv divides H.  The query of token t, at position past + t, sees the last
    `window` keys up to its own (None: all) and the first `sinks`.  scale: 1/sqrt(d) unless given.  Returns
    (o, lse), lse [B,T,H] float32."""
    args, lens, sizes, scale, code, dev = _win_inputs(q, k, v, lens, window, sinks, scale)
    o = _like(o, "o", q)
    if lse is not None or return_lse:
        lse = _new(lse, "lse", F32, q.shape[:3], dev)
    _run("win_attn_fwd", dev, *args, lens, o.data_ptr(), _adr(lse), *sizes, scale, code)
    return o, lse


def win_attn_bwd_workspace_bytes(B, T, past, H, Hkv, d, window, sinks, dtype) -> int:
    _sizes(B, T, past, H, Hkv, d, window, sinks)
    return _bytes("win_attn_bwd_workspace_bytes", B, T, past, H, Hkv, d, window, sinks, dtype)


@_on_stream
def win_attn_bwd(q, k, v, o, lse, dO, *, window=None, sinks=0, scale=None, lens=None, workspace=None):
    """Backward of win_attn_fwd, whose o and lse it takes: gradients of sum(dO * o).  Returns a dict dq, dk, dv."""
    args, lens, sizes, scale, code, dev = _win_inputs(q, k, v, lens, window, sinks, scale)
    args += (_arg(o, "o", q.dtype, q.shape, dev), _arg(lse, "lse", F32, q.shape[:3], dev),
             _arg(dO, "dO", q.dtype, q.shape, dev), lens)
    r = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v)}
    ws, wsb, hold = _work("win_attn_bwd", (*sizes, code), workspace, q)
    _run("win_attn_bwd", dev, *args, *map(_adr, r.values()), *sizes, scale, code, ws, wsb)
    return r


def win_attn_step_workspace_bytes(N, H, Hkv, d, window, sinks, dtype) -> int:
    _sizes(N, H, Hkv, d, window, sinks)
    return _bytes("win_attn_step_workspace_bytes", N, H, Hkv, d, window, sinks, dtype)


def _cache(K, V, N, dt, window, sinks, d, dev):
    """Checks a cache [N, sinks + window, Hkv, d]."""
    if K.dim() != 4:
        raise ValueError(f"K has shape {tuple(K.shape)}, expected [{N}, {sinks} + {window}, Hkv, {d}]")
    shape = (N, window + sinks, K.shape[2], d)
    _sizes(*shape)
    return _arg(K, "K", dt, shape, dev), _arg(V, "V", dt, shape, dev)


@_on_stream
def win_attn_step(K, V, pos, q, k, v, *, window, sinks=0, scale=None, o=None, workspace=None):
    """One token of windowed attention against a cache.  K, V [N,sinks+window,Hkv,d], updated in place; pos [N]
    int32: the number of tokens before this one (negative: the sequence is idle); q [N,H,d]; k, v [N,Hkv,d].
    Returns o [N,H,d].  pos is not advanced: several layers share it."""
    if q.dim() != 3:
        raise ValueError(f"q has shape {tuple(q.shape)}, expected [N, H, d]")
    (N, H, d), Hkv, dt, dev = q.shape, K.shape[2] if K.dim() == 4 else 0, q.dtype, q.device
    kv = _cache(K, V, N, dt, window, sinks, d, dev)
    args = (*kv, _arg(pos, "pos", I32, (N,), dev), _arg(q, "q", dt, (N, H, d), dev), _arg(k, "k", dt, (N, Hkv, d), dev),
            _arg(v, "v", dt, (N, Hkv, d), dev))
    code = _dtype_code(q)
    o = _like(o, "o", q)
    ws, wsb, hold = _work("win_attn_step", (N, H, Hkv, d, window, sinks, code), workspace, q)
    _run("win_attn_step", dev, *args, o.data_ptr(), N, H, Hkv, d, window, sinks, _scale(scale, d), code, ws, wsb)
    return o


@_on_stream
def win_attn_fill(K, V, k, v, *, window, sinks=0, lens=None, past=0):
    """Fills a cache K, V [B,sinks+window,Hkv,d] from a prompt's k, v [B,past+T,Hkv,d], whose first key is token 0;
    lens counts the T.  Slots of no token are left as they are.  The next token's pos is past + lens[b]."""
    if k.dim() != 4 or not 0 <= past <= k.shape[1]:
        raise ValueError(f"k has shape {tuple(k.shape)}, expected [B, keys, Hkv, d] with at least past={past} keys")
    (B, Tk, Hkv, d), dt, dev = k.shape, k.dtype, k.device
    kv = _cache(K, V, B, dt, window, sinks, d, dev)
    _sizes(Tk)
    _arg(K, "K", dt, (B, window + sinks, Hkv, d), dev)
    _run("win_attn_fill", dev, *kv, _arg(k, "k", dt, k.shape, dev), _arg(v, "v", dt, k.shape, dev),
         _arg(lens, "lens", I32, (B,), dev, True), B, Tk - past, past, Hkv, d, window, sinks, _dtype_code(k))
