"""The layer operators' definitions in 64 bits, token by token, and their gradients by the
formulas (not by autograd): short convolution, selective scan, group norm.  CPU tensors."""
import torch

F64 = torch.float64


def _d(t):
    return None if t is None else t.detach().cpu().to(F64)


def silu(x):
    return x / (1 + torch.exp(-x))


def silu_grad(x):
    s = 1 / (1 + torch.exp(-x))
    return s + x * s * (1 - s)


def lengths(lens, B, T):
    return [T] * B if lens is None else [min(max(int(v), 0), T) for v in lens]


# ------------------------------------------------------------------ short convolution

def _taps(x, S0, b, n, W):
    """The W - 1 kept inputs of sequence b followed by its n tokens."""
    head = torch.zeros(W - 1, x.shape[-1], dtype=F64) if S0 is None else S0[b]
    return torch.cat([head, x[b, :n]])


def conv_fwd(x, w, bias=None, S0=None, lens=None, act=True):
    x, w, bias, S0 = _d(x), _d(w), _d(bias), _d(S0)
    B, T, D = x.shape
    W = w.shape[1]
    y, S = torch.zeros(B, T, D, dtype=F64), torch.zeros(B, W - 1, D, dtype=F64)
    for b, n in enumerate(lengths(lens, B, T)):
        row = _taps(x, S0, b, n, W)
        for t in range(n):
            p = (row[t:t + W] * w.T).sum(0) + (0 if bias is None else bias)
            y[b, t] = silu(p) if act else p
        S[b] = row[n:]
    return y, S


def conv_bwd(x, w, bias, S0, dy, dS_final=None, lens=None, act=True):
    x, w, bias, S0, dy, dS = _d(x), _d(w), _d(bias), _d(S0), _d(dy), _d(dS_final)
    B, T, D = x.shape
    W = w.shape[1]
    g = {"dx": torch.zeros(B, T, D, dtype=F64), "dw": torch.zeros_like(w), "dbias": torch.zeros(D, dtype=F64),
         "dS0": torch.zeros(B, W - 1, D, dtype=F64)}
    for b, n in enumerate(lengths(lens, B, T)):
        row = _taps(x, S0, b, n, W)
        drow = torch.zeros_like(row)
        for t in range(n):
            p = (row[t:t + W] * w.T).sum(0) + (0 if bias is None else bias)
            dp = dy[b, t] * (silu_grad(p) if act else 1)
            drow[t:t + W] += dp * w.T
            g["dw"] += (dp * row[t:t + W]).T
            g["dbias"] += dp
        if dS is not None:
            drow[n:] += dS[b]
        g["dS0"][b] = drow[:W - 1]
        g["dx"][b, :n] = drow[W - 1:]
    if bias is None:
        g["dbias"] = None
    return g


# ------------------------------------------------------------------ selective scan

def _step_size(delta, bias, softplus):
    raw = delta if bias is None else delta + bias
    return raw, torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw


def _spread(t, D):
    return t.repeat_interleave(D // t.shape[-2], dim=-2)


def _states(x, delta, A, B, bias, S0, softplus, b, n):
    """raw, u, decays and the states 0 .. n (h[0] the one before the first token) of sequence b."""
    D, N = A.shape
    raw, u = _step_size(delta[b, :n], bias, softplus)
    a = torch.exp(u[..., None] * A)
    h = torch.zeros(n + 1, D, N, dtype=F64)
    if S0 is not None:
        h[0] = S0[b]
    Bc = _spread(B[b, :n], D)
    for t in range(n):
        h[t + 1] = a[t] * h[t] + (u[t] * x[b, t])[:, None] * Bc[t]
    return raw, u, a, h, Bc


def ssm_fwd(x, delta, A, B, C, D=None, delta_bias=None, S0=None, lens=None, softplus=True):
    x, delta, A, B, C, D, delta_bias, S0 = (_d(v) for v in (x, delta, A, B, C, D, delta_bias, S0))
    nb, T, ch = x.shape
    y, S = torch.zeros(nb, T, ch, dtype=F64), torch.zeros(nb, ch, A.shape[1], dtype=F64)
    for b, n in enumerate(lengths(lens, nb, T)):
        h = _states(x, delta, A, B, delta_bias, S0, softplus, b, n)[3]
        y[b, :n] = (h[1:] * _spread(C[b, :n], ch)).sum(-1) + (0 if D is None else D * x[b, :n])
        S[b] = h[n]
    return y, S


def ssm_bwd(x, delta, A, B, C, D, delta_bias, S0, dy, dS_final=None, lens=None, softplus=True):
    x, delta, A, B, C, D, delta_bias, S0, dy, dS = (_d(v) for v in (x, delta, A, B, C, D, delta_bias, S0, dy, dS_final))
    nb, T, ch = x.shape
    N, G = A.shape[1], B.shape[-2]
    z = lambda *s: torch.zeros(*s, dtype=F64)
    g = {"dx": z(nb, T, ch), "ddelta": z(nb, T, ch), "dA": z(ch, N), "dB": z(nb, T, G, N), "dC": z(nb, T, G, N),
         "dD": z(ch), "ddelta_bias": z(ch), "dS0": z(nb, ch, N)}
    for b, n in enumerate(lengths(lens, nb, T)):
        raw, u, a, h, Bc = _states(x, delta, A, B, delta_bias, S0, softplus, b, n)
        Cc = _spread(C[b, :n], ch)
        dh = z(ch, N) if dS is None else dS[b].clone()
        for t in reversed(range(n)):
            dh = dh + Cc[t] * dy[b, t][:, None]
            g["dC"][b, t] = (h[t + 1] * dy[b, t][:, None]).reshape(G, ch // G, N).sum(1)
            g["dB"][b, t] = (dh * (u[t] * x[b, t])[:, None]).reshape(G, ch // G, N).sum(1)
            through = (dh * Bc[t]).sum(-1)
            r = dh * a[t] * h[t]
            du = (r * A).sum(-1) + x[b, t] * through
            dd = du / (1 + torch.exp(-raw[t])) if softplus else du
            g["dx"][b, t] = u[t] * through + (0 if D is None else D * dy[b, t])
            g["ddelta"][b, t] = dd
            g["ddelta_bias"] += dd
            g["dA"] += r * u[t][:, None]
            g["dD"] += dy[b, t] * x[b, t]
            dh = dh * a[t]
        g["dS0"][b] = dh
    if D is None:
        g["dD"] = None
    if delta_bias is None:
        g["ddelta_bias"] = None
    return g


# ------------------------------------------------------------------ group norm

def _normed(x, w, b, eps, center):
    m = x.mean(-1, keepdim=True) if center else 0.0
    rstd = 1 / torch.sqrt(((x - m) ** 2).mean(-1, keepdim=True) + eps)
    xh = (x - m) * rstd
    return xh, rstd, xh * (1 if w is None else w) + (0 if b is None else b)


def norm_fwd(x, w=None, b=None, z=None, eps=1e-5, center=True, act=True):
    x, w, b, z = _d(x), _d(w), _d(b), _d(z)
    n = _normed(x, w, b, eps, center)[2]
    t = n if z is None else z
    a = silu(t) if act else t
    return a if z is None else n * a


def norm_bwd(x, w, b, z, dy, eps=1e-5, center=True, act=True):
    x, w, b, z, dy = _d(x), _d(w), _d(b), _d(z), _d(dy)
    xh, rstd, n = _normed(x, w, b, eps, center)
    dz = None
    if z is None:
        dn = dy * silu_grad(n) if act else dy
    else:
        dn = dy * (silu(z) if act else z)
        dz = dy * n * (silu_grad(z) if act else 1)
    q = dn * (1 if w is None else w)
    dx = q - xh * (q * xh).mean(-1, keepdim=True)
    if center:
        dx = dx - q.mean(-1, keepdim=True)
    over = tuple(range(x.dim() - 2))
    return {"dx": dx * rstd, "dz": dz, "dw": None if w is None else (dn * xh).sum(over),
            "db": None if b is None else dn.sum(over)}
