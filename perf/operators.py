"""The state-space layer's operators as measured work: the short causal convolution, the selective
scan (both for prompts, for training and for single tokens) and the gated group norm.

`run` computes a case in its plain form (elementary torch operations in 32 bits) or, where `own` is
true, through the package's entry points.  A case's `op` says which operator and direction it is.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------- the cases

def _conv(name, op, B, T, D, W=4, dtype="bf16", bias=True, silu=True, s0=False, ragged=False):
    return {"name": name, "op": op, "B": B, "T": T, "D": D, "W": W, "dtype": dtype, "bias": bias, "silu": silu,
            "s0": s0, "ragged": ragged}


def _ssm(name, op, B, T, D, N=16, G=1, dtype="bf16", skip=True, bias=True, softplus=True, s0=False, ragged=False):
    return {"name": name, "op": op, "B": B, "T": T, "D": D, "N": N, "G": G, "dtype": dtype, "skip": skip,
            "bias": bias, "softplus": softplus, "s0": s0, "ragged": ragged}


def _norm(name, op, M, H, d, dtype="bf16", center=True, affine=True, gate=True, silu=True):
    return {"name": name, "op": op, "M": M, "H": H, "d": d, "dtype": dtype, "center": center, "affine": affine,
            "gate": gate, "silu": silu}


def listed():
    return [
        # the 1.3B-model layer of the benchmark (B=8, T=2048, 16 heads x 128): prompts through the convolution
        _conv("conv_prompt", "conv_fwd", 8, 2048, 2048),
        # a training step's backward of the same layer
        _conv("conv_train", "conv_bwd", 8, 2048, 2048),
        # prompts of different lengths padded to one, continued from kept inputs, at an odd width in fp32
        _conv("conv_ragged", "conv_fwd", 5, 333, 1029, W=3, dtype="f32", s0=True, ragged=True),
        # one token for each of the decode workload's 512 sequences
        _conv("conv_decode", "conv_step", 512, 1, 2048),
        # the same layer's scan over the prompts
        _ssm("ssm_prompt", "ssm_fwd", 8, 2048, 2048),
        # the long-context workload: one sequence of 32K tokens, continued from a state
        _ssm("ssm_long", "ssm_fwd", 1, 32768, 2048, s0=True),
        # a training step's backward at the 8-head shape (B=4, T=4096, 8 heads x 128)
        _ssm("ssm_train", "ssm_bwd", 4, 4096, 1024),
        # a small ragged fp32 training batch at odd sizes, two B/C groups, a sequence carried over
        _ssm("ssm_train_ragged", "ssm_bwd", 3, 517, 770, N=24, G=2, dtype="f32", s0=True, ragged=True),
        # one token for each of 512 sequences
        _ssm("ssm_decode", "ssm_step", 512, 1, 2048),
        # one token of one sequence: what a call costs at least
        _ssm("ssm_decode_one", "ssm_step", 1, 1, 2048),
        # the layer's output norm over 16 heads x 128 with its gate
        _norm("norm_prompt", "norm_fwd", 8 * 2048, 16, 128),
        # and its backward in a training step
        _norm("norm_train", "norm_bwd", 8 * 2048, 16, 128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A channel count: a whole number of 16-byte rows two times in three, any number otherwise."""
    D = _log_int(rng, lo, hi)
    return D if rng.random() < 0.34 else max(8, D // 8 * 8)


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_bwd", "conv_step", "ssm_fwd", "ssm_bwd", "ssm_step", "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    flag = lambda p: rng.random() < p
    most = 1 << (25 if dtype == "bf16" else 24)         # token-channels of one call
    if op.startswith("norm"):
        d = rng.choice([64, 128, 128, 256, _log_int(rng, 8, 4096)])
        H = _log_int(rng, 1, max(1, min(64, 4096 // d)))
        M = _log_int(rng, 1, max(1, most // (H * d)))
        return {k: v for k, v in _norm("", op, M, H, d, dtype, flag(0.5), flag(0.8), flag(0.7), flag(0.8)).items()
                if k != "name"}
    if op.endswith("step"):
        D, B, T = _width(rng, 64, 4096), _log_int(rng, 1, 512), 1
    else:
        D, T = _width(rng, 16, 4096), _log_int(rng, 1, 32768)
        B = _log_int(rng, 1, max(1, min(16, most // (T * D))))
    if op.startswith("conv"):
        if op != "conv_step":
            T = max(1, min(T, most // (B * D)))
        c = _conv("", op, B, T, D, rng.choice([2, 3, 4, 4]), dtype, flag(0.7), flag(0.8), flag(0.5), flag(0.3))
    else:
        N = rng.choice([16, 16, 16, 32, 64, _log_int(rng, 1, 128)])
        if op != "ssm_step":
            T = max(1, min(T, most // (B * D), (1 << (29 if op == "ssm_fwd" else 28)) // (B * D * N)))
        else:
            B = max(1, min(B, (1 << 24) // (D * N)))
        G = rng.choice([g for g in (1, 1, 1, 2, 4) if D % g == 0])
        c = _ssm("", op, B, T, D, N, G, dtype, flag(0.8), flag(0.8), flag(0.8), flag(0.5), flag(0.3))
    if op.endswith("step"):
        c["s0"] = c["ragged"] = False
    del c["name"]
    return c


# --------------------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev).manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    randn = lambda *s: torch.randn(*s, generator=g, device=dev)
    rand = lambda *s: torch.rand(*s, generator=g, device=dev)
    op, s = case["op"], {"case": case}
    if op.startswith("norm"):
        M, H, d = case["M"], case["H"], case["d"]
        s["x"] = (randn(M, H, d) * torch.exp(0.5 * randn(H, 1)) + 0.2 * randn(M, H, 1)).to(dt)
        s["w"] = 1 + 0.1 * randn(H, d) if case["affine"] else None
        s["b"] = 0.1 * randn(H, d) if case["affine"] else None
        s["z"] = randn(M, H, d).to(dt) if case["gate"] else None
        s["dy"] = randn(M, H, d).to(dt) if op == "norm_bwd" else None
        return s
    B, T, D = case["B"], case["T"], case["D"]
    # padded lengths: one sequence keeps the whole length, the others any, one of them possibly nothing
    s["lens"] = None
    if case["ragged"]:
        n = torch.randint(0, T + 1, (B,), generator=g, device=dev, dtype=torch.int32)
        n[0] = T
        if B > 2:
            n[B - 1] = 0
        s["lens"] = n
    if op.startswith("conv"):
        W = case["W"]
        s["w"] = (rand(D, W) * 2 - 1) / math.sqrt(W)
        s["bias"] = (rand(D) - 0.5) if case["bias"] else None
        if op == "conv_step":
            s["S"] = randn(B, W - 1, D).to(dt)
            s["x"] = randn(B, D).to(dt)
            return s
        s["x"] = randn(B, T, D).to(dt)
        s["S0"] = randn(B, W - 1, D).to(dt) if case["s0"] else None
        if op == "conv_bwd":
            s["dy"] = randn(B, T, D).to(dt)
            s["dS_final"] = randn(B, W - 1, D).to(dt) if case["s0"] else None
        return s
    N, G = case["N"], case["G"]
    # the layer's initialisation: A = -1 .. -N with a spread from training, step sizes log-uniform in [1e-3, 0.1]
    s["A"] = -torch.arange(1, N + 1, device=dev).float() * torch.exp(0.1 * randn(D, N))
    step = torch.exp(rand(D) * (math.log(0.1) - math.log(1e-3)) + math.log(1e-3))
    s["D"] = 1 + 0.1 * randn(D) if case["skip"] else None
    inv = torch.log(torch.expm1(step))
    s["delta_bias"] = (inv if case["softplus"] else step) if case["bias"] else None
    one = op == "ssm_step"
    tok = (B,) if one else (B, T)
    raw = 0.5 * randn(*tok, D)
    if not case["softplus"]:
        raw = 0.01 * raw.abs()
    elif not case["bias"]:
        raw = raw - 3.5
    s["delta"] = raw.to(dt)
    pre = randn(*tok, D)
    s["x"] = (pre * torch.sigmoid(pre)).to(dt)          # what the convolution's SiLU leaves
    s["B"], s["C"] = randn(*tok, G, N).to(dt), randn(*tok, G, N).to(dt)
    if one:
        s["S"] = 0.3 * randn(B, D, N)
        return s
    s["S0"] = 0.3 * randn(B, D, N) if case["s0"] else None
    if op == "ssm_bwd":
        s["dy"] = randn(B, T, D).to(dt)
        s["dS_final"] = 0.3 * randn(B, D, N) if case["s0"] else None
    return s


# --------------------------------------------------------------------------- the plain forms

def _f(t):
    return None if t is None else t.float()


def _valid(s):
    """[B,T,1] truth values: the tokens that are no padding, or None where all are real."""
    if s["lens"] is None:
        return None
    return (torch.arange(s["case"]["T"], device=s["lens"].device) < s["lens"][:, None])[..., None]


def _keep(valid, t):
    return t if valid is None else torch.where(valid, t, torch.zeros((), dtype=t.dtype, device=t.device))


def _silu_grad(x):
    sg = torch.sigmoid(x)
    return sg * (1 + x * (1 - sg))


def _conv_padded(s):
    """The kept inputs and the call's in one row of T + W - 1, in 32 bits, and where the last W - 1 stand."""
    case, x = s["case"], _keep(_valid(s), s["x"].float())
    B, T, W = case["B"], case["T"], case["W"]
    head = torch.zeros(B, W - 1, case["D"], device=x.device) if s["S0"] is None else s["S0"].float()
    n = torch.full((B,), T, device=x.device) if s["lens"] is None else s["lens"].long()
    at = n[:, None] + torch.arange(W - 1, device=x.device)
    return torch.cat([head, x], 1), at[..., None].expand(B, W - 1, case["D"])


def _conv_pre(s, xp):
    T, W, w = s["case"]["T"], s["case"]["W"], s["w"]
    pre = sum(xp[:, j:j + T] * w[:, j] for j in range(W))
    return pre if s["bias"] is None else pre + s["bias"]


def _plain_conv_fwd(s):
    dt, silu = s["x"].dtype, s["case"]["silu"]
    xp, at = _conv_padded(s)
    pre = _conv_pre(s, xp)
    y = pre * torch.sigmoid(pre) if silu else pre
    return {"y": _keep(_valid(s), y).to(dt), "S_final": xp.gather(1, at).to(dt)}


def _plain_conv_bwd(s):
    case, dt, w = s["case"], s["x"].dtype, s["w"]
    T, W = case["T"], case["W"]
    xp, at = _conv_padded(s)
    dpre = _keep(_valid(s), s["dy"].float())
    if case["silu"]:
        dpre = dpre * _silu_grad(_conv_pre(s, xp))
    dw = torch.stack([(dpre * xp[:, j:j + T]).sum((0, 1)) for j in range(W)], 1)
    dxp = sum(torch.nn.functional.pad(dpre * w[:, j], (0, 0, j, W - 1 - j)) for j in range(W))
    if s["dS_final"] is not None:
        dxp = dxp.scatter_add(1, at, s["dS_final"].float())
    return {"dx": dxp[:, W - 1:].to(dt), "dw": dw, "dbias": None if s["bias"] is None else dpre.sum((0, 1)),
            "dS0": dxp[:, :W - 1].to(dt)}


def _plain_conv_step(s):
    x, S, case = s["x"], s["S"], s["case"]
    xp = torch.cat([S, x[:, None]], 1)
    pre = (xp.float() * s["w"].t()).sum(1)
    pre = pre if s["bias"] is None else pre + s["bias"]
    S.copy_(xp[:, 1:])
    return {"y": (pre * torch.sigmoid(pre) if case["silu"] else pre).to(x.dtype), "S": S}


def _recur(a, b):
    """h_t = a_t h_{t-1} + b_t along axis 1 from h = 0, by doubling: log2(T) passes over the arrays."""
    h, a, s = b.clone(), a.clone(), 1
    while s < a.shape[1]:
        h[:, s:] += a[:, s:] * h[:, :-s].clone()
        a[:, s:] *= a[:, :-s].clone()
        s *= 2
    return h


def _per_channel(t, D):
    """[..., G, N] per group -> [..., D, N] per channel."""
    return t.float().repeat_interleave(D // t.shape[-2], dim=-2)


def _step_size(s):
    raw = s["delta"].float()
    raw = raw if s["delta_bias"] is None else raw + s["delta_bias"]
    return raw, torch.nn.functional.softplus(raw) if s["case"]["softplus"] else raw


def _ssm_states(s):
    """The decays, the states after each token and what the backward reuses, in 32 bits."""
    valid, D = _valid(s), s["case"]["D"]
    raw, u = _step_size(s)
    u, x = _keep(valid, u), _keep(valid, s["x"].float())
    deep = None if valid is None else valid[..., None]
    Bc, Cc = _keep(deep, _per_channel(s["B"], D)), _keep(deep, _per_channel(s["C"], D))
    a = torch.exp(u[..., None] * s["A"])
    b = (u * x)[..., None] * Bc
    if s["S0"] is not None:
        b[:, 0] += a[:, 0] * s["S0"]
    return raw, u, x, Bc, Cc, a, _recur(a, b)


def _plain_ssm_fwd(s):
    raw, u, x, Bc, Cc, a, h = _ssm_states(s)
    y = (h * Cc).sum(-1)
    y = y if s["D"] is None else y + s["D"] * x
    return {"y": _keep(_valid(s), y).to(s["x"].dtype), "S_final": h[:, -1].clone()}


def _plain_ssm_bwd(s):
    case, dt, A, valid = s["case"], s["x"].dtype, s["A"], _valid(s)
    D, N, G = case["D"], case["N"], case["G"]
    raw, u, x, Bc, Cc, a, h = _ssm_states(s)
    g = _keep(valid, s["dy"].float())
    q = Cc * g[..., None]
    if s["dS_final"] is not None:
        q[:, -1] += s["dS_final"]
    after = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)      # the decay between t and t + 1
    dh = _recur(after.flip(1), q.flip(1)).flip(1)
    first = torch.zeros_like(h[:, 0]) if s["S0"] is None else s["S0"]
    r = dh * a * torch.cat([first[:, None], h[:, :-1]], 1)           # the gradient of u A
    through = (dh * Bc).sum(-1)
    du = (r * A).sum(-1) + x * through
    ddelta = _keep(valid, du * torch.sigmoid(raw) if case["softplus"] else du)
    dx = u * through if s["D"] is None else u * through + s["D"] * g
    groups = lambda t: t.unflatten(2, (G, D // G)).sum(3).to(dt)
    return {"dx": dx.to(dt), "ddelta": ddelta.to(dt), "dA": (r * u[..., None]).sum((0, 1)),
            "dB": groups(dh * (u * x)[..., None]), "dC": groups(h * g[..., None]),
            "dD": None if s["D"] is None else (g * x).sum((0, 1)),
            "ddelta_bias": None if s["delta_bias"] is None else ddelta.sum((0, 1)), "dS0": a[:, 0] * dh[:, 0]}


def _plain_ssm_step(s):
    S, x, D = s["S"], s["x"].float(), s["case"]["D"]
    _, u = _step_size(s)
    S.copy_(S * torch.exp(u[..., None] * s["A"]) + (u * x)[..., None] * _per_channel(s["B"], D))
    y = (S * _per_channel(s["C"], D)).sum(-1)
    return {"y": (y if s["D"] is None else y + s["D"] * x).to(s["x"].dtype), "S": S}


EPS = 1e-5


def _normed(s):
    x, center = s["x"].float(), s["case"]["center"]
    mean = x.mean(-1, keepdim=True) if center else 0.0
    rstd = torch.rsqrt((x - mean).square().mean(-1, keepdim=True) + EPS)
    xh = (x - mean) * rstd
    n = xh if s["w"] is None else xh * s["w"] + s["b"]
    return xh, rstd, n


def _plain_norm_fwd(s):
    _, _, n = _normed(s)
    t = n if s["z"] is None else s["z"].float()
    act = t * torch.sigmoid(t) if s["case"]["silu"] else t
    return {"y": (act if s["z"] is None else n * act).to(s["x"].dtype)}


def _plain_norm_bwd(s):
    case, dt = s["case"], s["x"].dtype
    xh, rstd, n = _normed(s)
    dn, z, dz = s["dy"].float(), _f(s["z"]), None
    if z is not None:
        dz = (dn * n * (_silu_grad(z) if case["silu"] else 1.0)).to(dt)
        dn = dn * (z * torch.sigmoid(z) if case["silu"] else z)
    elif case["silu"]:
        dn = dn * _silu_grad(n)
    dxh = dn if s["w"] is None else dn * s["w"]
    dx = dxh - xh * (dxh * xh).mean(-1, keepdim=True)
    if case["center"]:
        dx = dx - dxh.mean(-1, keepdim=True)
    return {"dx": (dx * rstd).to(dt), "dz": dz, "dw": None if s["w"] is None else (dn * xh).sum(0),
            "db": None if s["w"] is None else dn.sum(0)}


# --------------------------------------------------------------------------- the framework's operators

def _own_run(s):
    import delta_rule_linear_qdelta_gb300 as qd
    case, op = s["case"], s["case"]["op"]
    if op == "conv_fwd":
        y, S = qd.short_conv_fwd(s["x"], s["w"], s["bias"], s["S0"], lens=s["lens"], silu=case["silu"])
        return {"y": y, "S_final": S}
    if op == "conv_bwd":
        return qd.short_conv_bwd(s["x"], s["w"], s["bias"], s["S0"], s["dy"], s["dS_final"], lens=s["lens"],
                                 silu=case["silu"])
    if op == "conv_step":
        return {"y": qd.short_conv_step(s["S"], s["x"], s["w"], s["bias"], silu=case["silu"]), "S": s["S"]}
    if op == "ssm_fwd":
        y, S = qd.ssm_fwd(s["x"], s["delta"], s["A"], s["B"], s["C"], s["D"], s["delta_bias"], s["S0"],
                          lens=s["lens"], softplus=case["softplus"])
        return {"y": y, "S_final": S}
    if op == "ssm_bwd":
        return qd.ssm_bwd(s["x"], s["delta"], s["A"], s["B"], s["C"], s["D"], s["delta_bias"], s["S0"], s["dy"],
                          s["dS_final"], lens=s["lens"], softplus=case["softplus"])
    if op == "ssm_step":
        return {"y": qd.ssm_step(s["S"], s["x"], s["delta"], s["A"], s["B"], s["C"], s["D"], s["delta_bias"],
                                 softplus=case["softplus"]), "S": s["S"]}
    kw = {"eps": EPS, "center": case["center"], "silu": case["silu"]}
    if op == "norm_fwd":
        return {"y": qd.group_norm_fwd(s["x"], s["w"], s["b"], s["z"], **kw)}
    return qd.group_norm_bwd(s["x"], s["w"], s["b"], s["z"], s["dy"], **kw)


_PLAIN = {"conv_fwd": _plain_conv_fwd, "conv_bwd": _plain_conv_bwd, "conv_step": _plain_conv_step,
          "ssm_fwd": _plain_ssm_fwd, "ssm_bwd": _plain_ssm_bwd, "ssm_step": _plain_ssm_step,
          "norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd}


def run(state):
    return _own_run(state) if own else _PLAIN[state["case"]["op"]](state)


# --------------------------------------------------------------------------- the least work

def work(case):
    """Each input read once and each output written once; an exponential counts as one operation."""
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op.startswith("norm"):
        n, c = case["M"] * case["H"] * case["d"], case["H"] * case["d"]
        arrays = (2 + case["gate"]) if op == "norm_fwd" else (3 + 2 * case["gate"])
        params = 2 * c * case["affine"] * (1 if op == "norm_fwd" else 2)
        return {"bytes": n * e * arrays + 4 * params, "flops": n * (14 if op == "norm_fwd" else 30)}
    B, T, D = case["B"], case["T"], case["D"]
    n = B * T * D
    if op.startswith("conv"):
        W = case["W"]
        params, kept = 4 * D * (W + case["bias"]), B * (W - 1) * D * e
        if op == "conv_fwd":
            return {"bytes": 2 * n * e + params + kept * (1 + case["s0"]), "flops": n * (2 * W + 4)}
        if op == "conv_bwd":
            return {"bytes": 3 * n * e + 2 * params + kept * (1 + 2 * case["s0"]), "flops": n * (6 * W + 10)}
        return {"bytes": 2 * n * e + params + 2 * kept, "flops": n * (2 * W + 4)}
    N, G = case["N"], case["G"]
    params, groups, state = 4 * D * (N + case["skip"] + case["bias"]), 2 * B * T * G * N * e, 4 * B * D * N
    if op == "ssm_fwd":
        return {"bytes": 3 * n * e + params + groups + state * (1 + case["s0"]), "flops": n * (7 * N + 8)}
    if op == "ssm_bwd":
        return {"bytes": 5 * n * e + 2 * params + 2 * groups + state * (1 + 2 * case["s0"]), "flops": n * (18 * N + 16)}
    return {"bytes": 3 * n * e + params + groups + 2 * state, "flops": n * (7 * N + 8)}


# --------------------------------------------------------------------------- the definitions in 64 bits

def _exact_conv(s):
    """Token by token over the kept inputs and the call's, differentiated by autograd for the backward."""
    case, op = s["case"], s["case"]["op"]
    W, B, T, D = case["W"], case["B"], case["T"], case["D"]
    w = s["w"].double().requires_grad_()
    bias = None if s["bias"] is None else s["bias"].double().requires_grad_()
    x = (s["x"][:, None] if op == "conv_step" else s["x"]).double().requires_grad_()
    S0 = s["S"] if op == "conv_step" else s["S0"]
    S0 = (torch.zeros(B, W - 1, D, device=x.device) if S0 is None else S0).double().requires_grad_()
    n = [T] * B if s["lens"] is None else [int(v) for v in s["lens"].tolist()]
    ys, ends = [], []
    for b in range(B) if max(n) != min(n) or T == 0 else [slice(None)]:
        xb, sb, nb = (x, S0, n[0]) if isinstance(b, slice) else (x[b:b + 1], S0[b:b + 1], n[b])
        row = torch.cat([sb, xb[:, :nb]], 1)
        y = torch.nn.functional.conv1d(row.transpose(1, 2), w[:, None], bias, groups=D).transpose(1, 2) if nb else xb[:, :0]
        y = y / (1 + torch.exp(-y)) if case["silu"] else y
        ys.append(torch.nn.functional.pad(y, (0, 0, 0, T - nb)))
        ends.append(row[:, nb:])
    y, end = torch.cat(ys), torch.cat(ends)
    if op == "conv_step":
        return {"y": y[:, 0].detach(), "S": end.detach()}
    if op == "conv_fwd":
        return {"y": y.detach(), "S_final": end.detach()}
    L = (y * s["dy"].double()).sum()
    L = L if s["dS_final"] is None else L + (end * s["dS_final"].double()).sum()
    want = [x, w, S0] + ([] if bias is None else [bias])
    got = torch.autograd.grad(L, want, allow_unused=True)
    got = [torch.zeros_like(v) if t is None else t for v, t in zip(want, got)]
    return {"dx": got[0], "dw": got[1], "dbias": None if bias is None else got[3], "dS0": got[2]}


def _exact_ssm(s):
    """The recurrence token by token; the backward is autograd's through it."""
    case, op = s["case"], s["case"]["op"]
    back, D, G = op == "ssm_bwd", case["D"], case["G"]
    d = {}
    for k in ("x", "delta", "A", "B", "C", "D", "delta_bias"):
        v = s[k] if op != "ssm_step" or k in ("A", "D", "delta_bias") or s[k] is None else s[k][:, None]
        d[k] = None if v is None else v.double().requires_grad_(back)
    h = s["S"] if op == "ssm_step" else s["S0"]
    h = torch.zeros(case["B"], D, case["N"], device=s["A"].device) if h is None else h
    h0 = h = h.double().requires_grad_(back)
    T = d["x"].shape[1]
    with torch.set_grad_enabled(back):
        u = d["delta"] if d["delta_bias"] is None else d["delta"] + d["delta_bias"]
        u = torch.logaddexp(u, torch.zeros_like(u)) if case["softplus"] else u
        real = None if s["lens"] is None else torch.arange(T, device=u.device) < s["lens"][:, None]
        if real is not None:
            u = u * real[..., None]                     # a step of no length leaves the state as it is
        ys = []
        cols = [t.unbind(1) for t in (u, d["x"], d["B"], d["C"])]
        for ut, xt, Bt, Ct in zip(*cols):
            Bt, Ct = (t[:, :, None].expand(-1, G, D // G, -1).reshape(-1, D, case["N"]) for t in (Bt, Ct))
            h = torch.exp(ut[..., None] * d["A"]) * h + (ut * xt)[..., None] * Bt
            ys.append(torch.einsum("bdn,bdn->bd", h, Ct))
        y = torch.stack(ys, 1)
        y = y if d["D"] is None else y + d["D"] * d["x"]
        y = y if real is None else y * real[..., None]
    if op == "ssm_step":
        return {"y": y[:, 0], "S": h}
    if not back:
        return {"y": y, "S_final": h}
    L = (y * s["dy"].double()).sum()
    L = L if s["dS_final"] is None else L + (h * s["dS_final"].double()).sum()
    names = [k for k in d if d[k] is not None]
    got = dict(zip(["S0"] + names, torch.autograd.grad(L, [h0] + [d[k] for k in names])))
    return {"d" + k: got.get(k) for k in ("x", "delta", "A", "B", "C", "D", "delta_bias", "S0")}


def _exact_norm(s):
    case, back = s["case"], s["case"]["op"] == "norm_bwd"
    v = {k: None if s[k] is None else s[k].double().requires_grad_(back) for k in ("x", "w", "b", "z")}
    with torch.set_grad_enabled(back):
        x = v["x"]
        x = x - x.sum(-1, keepdim=True) / case["d"] if case["center"] else x
        n = x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["d"] + EPS)
        n = n if v["w"] is None else v["w"] * n + v["b"]
        t = n if v["z"] is None else v["z"]
        t = t / (1 + torch.exp(-t)) if case["silu"] else t
        y = t if v["z"] is None else n * t
    if not back:
        return {"y": y}
    names = [k for k in v if v[k] is not None]
    got = dict(zip(names, torch.autograd.grad(y, [v[k] for k in names], s["dy"].double())))
    return {"d" + k: got.get(k) for k in ("x", "z", "w", "b")}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    return _exact_norm(s) if op.startswith("norm") else _exact_conv(s) if op.startswith("conv") else _exact_ssm(s)
