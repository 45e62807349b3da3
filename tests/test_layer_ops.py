"""The layer operators (short convolution, selective scan, group norm) against their
definitions in 64 bits (tests/layer_reference.py).

Tolerances, set before any run:
  fp32 outputs (and every parameter gradient, state and state gradient): relative L2 <= 1e-5,
    the library's fp32 tolerance: roundings of 2^-24 and hardware exponentials of 2^-22 per
    token, over states that forget within some hundred tokens.
  bf16 outputs: computed in fp32 and rounded once, so each is within half a bf16 ulp of the
    exact value, 2^-8 |ref| (8 significant bits), plus the fp32 error, 1e-5 of the largest |ref|.
"""
import ctypes

import pytest
import torch

import layer_reference as ref

F32, BF16 = torch.float32, torch.bfloat16
NAN = float("nan")


@pytest.fixture(scope="module")
def qd():
    import delta_rule_linear_qdelta_gb300 as m
    from delta_rule_linear_qdelta_gb300 import build
    build.build()
    m.load_library()
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


def close(got, want, what):
    if want is None:
        assert got is None, what
        return
    assert got.shape == want.shape, (what, got.shape, want.shape)
    if want.numel() == 0:
        return
    g = got.detach().cpu().double()
    assert torch.isfinite(g).all(), f"{what}: not finite"
    err = (g - want).abs()
    if got.dtype == BF16:
        over = (err - 2.0 ** -8 * want.abs() - 1e-5 * want.abs().max()).max()
        assert over <= 0, f"{what}: {over:.3e} beyond half an ulp"
    else:
        rel = err.norm() / want.norm().clamp_min(1e-30)
        assert rel <= 1e-5 or err.max() == 0, f"{what}: relative L2 {rel:.3e}"


def close_all(got, want):
    assert set(got) == set(want)
    for k in want:
        close(got[k], want[k], k)


def cu(d):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in d.items()}


def lens_of(how, B, T, g):
    if not how:
        return None
    n = torch.randint(0, T + 1, (B,), generator=g, dtype=torch.int32)
    n[0] = T
    n[B - 1] = 0
    if B > 2:
        n[1] = min(T, 1)
    return n


def poison(t, lens):
    """The padded tokens of t as NaN."""
    if lens is not None:
        for b, n in enumerate(lens.tolist()):
            t[b, max(n, 0):] = NAN
    return t


# ------------------------------------------------------------------ inputs

def conv_inputs(B, T, D, W, dt, seed, bias=True, s0=True, lens=False):
    g = gen(seed)
    n = lens_of(lens, B, T, g)
    r = lambda *s: torch.randn(*s, generator=g)
    return {"x": poison(r(B, T, D).to(dt), n), "w": 0.5 * r(D, W), "bias": 0.5 * r(D) if bias else None,
            "S0": r(B, W - 1, D).to(dt) if s0 else None, "lens": n, "dy": poison(r(B, T, D).to(dt), n),
            "dS_final": r(B, W - 1, D).to(dt) if s0 else None}


def ssm_inputs(B, T, D, N, G, dt, seed, skip=True, bias=True, s0=True, lens=False, softplus=True):
    g = gen(seed)
    n = lens_of(lens, B, T, g)
    r = lambda *s: torch.randn(*s, generator=g)
    step = torch.exp(torch.rand(D, generator=g) * 4.6 - 6.9)                 # 1e-3 .. 0.1
    raw = 0.5 * r(B, T, D) if softplus else 0.02 * r(B, T, D).abs()
    if softplus and not bias:
        raw = raw - 3
    return {"x": poison(r(B, T, D).to(dt), n), "delta": poison(raw.to(dt), n),
            "A": -(1 + torch.arange(N).float()) * torch.exp(0.1 * r(D, N)), "B": poison(r(B, T, G, N).to(dt), n),
            "C": poison(r(B, T, G, N).to(dt), n), "D": 1 + 0.1 * r(D) if skip else None,
            "delta_bias": (torch.log(torch.expm1(step)) if softplus else step) if bias else None,
            "S0": 0.3 * r(B, D, N) if s0 else None, "lens": n, "dy": poison(r(B, T, D).to(dt), n),
            "dS_final": 0.3 * r(B, D, N) if s0 else None}


def norm_inputs(M, H, d, dt, seed, affine=True, gate=True):
    g = gen(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    return {"x": (2 * r(M, H, d) + r(M, H, 1)).to(dt), "w": 1 + 0.2 * r(H, d) if affine else None,
            "b": 0.2 * r(H, d) if affine else None, "z": r(M, H, d).to(dt) if gate else None,
            "dy": r(M, H, d).to(dt)}


SSM_IN = ("x", "delta", "A", "B", "C", "D", "delta_bias", "S0")


# ------------------------------------------------------------------ the definitions themselves

def _differences(f, inputs, grads, seed):
    """Central differences of f (four points, so the error is of the step's fourth power) along
    random directions of every input, against its gradient."""
    g = gen(seed)
    for k, v in inputs.items():
        if grads.get("d" + k) is None or v is None:
            continue
        way = torch.randn(v.shape, generator=g, dtype=torch.float64)
        h = 3e-5
        at = lambda s: f({**inputs, k: v + s * h * way})
        num = (8 * (at(1) - at(-1)) - (at(2) - at(-2))) / (12 * h)
        got = (grads["d" + k].double().cpu() * way).sum()
        yield k, num, got


def _conv_loss(d, dy, dS, lens, act):
    y, S = ref.conv_fwd(d["x"], d["w"], d["bias"], d["S0"], lens, act)
    return (y * dy).sum() + (S * dS).sum()


def _ssm_loss(d, dy, dS, lens, softplus):
    y, S = ref.ssm_fwd(*(d[k] for k in SSM_IN), lens, softplus)
    return (y * dy).sum() + (S * dS).sum()


def _f64(d, names):
    return {k: None if d[k] is None else torch.nan_to_num(d[k].double()) for k in names}


@pytest.mark.parametrize("act", [True, False])
def test_conv_gradient_formula_against_differences(act):
    d = conv_inputs(2, 7, 3, 4, F32, 1, lens=True)
    v, dy, dS = _f64(d, ("x", "w", "bias", "S0")), torch.nan_to_num(d["dy"].double()), d["dS_final"].double()
    g = ref.conv_bwd(v["x"], v["w"], v["bias"], v["S0"], dy, dS, d["lens"], act)
    for k, num, got in _differences(lambda e: _conv_loss(e, dy, dS, d["lens"], act), v, g, 2):
        assert abs(num - got) <= 1e-8 * max(1, abs(num)), k


@pytest.mark.parametrize("softplus", [True, False])
def test_ssm_gradient_formula_against_differences(softplus):
    d = ssm_inputs(2, 9, 4, 5, 2, F32, 3, lens=True, softplus=softplus)
    v, dy, dS = _f64(d, SSM_IN), torch.nan_to_num(d["dy"].double()), d["dS_final"].double()
    g = ref.ssm_bwd(*(v[k] for k in SSM_IN), dy, dS, d["lens"], softplus)
    for k, num, got in _differences(lambda e: _ssm_loss(e, dy, dS, d["lens"], softplus), v, g, 4):
        assert abs(num - got) <= 1e-8 * max(1, abs(num)), k


@pytest.mark.parametrize("gate,center,act", [(True, True, True), (False, True, True), (True, False, False),
                                             (False, False, True)])
def test_norm_gradient_formula_against_differences(gate, center, act):
    d = norm_inputs(3, 2, 7, F32, 5, gate=gate)
    v, dy = _f64(d, ("x", "w", "b", "z")), d["dy"].double()
    g = ref.norm_bwd(*(v[k] for k in ("x", "w", "b", "z")), dy, 1e-5, center, act)
    f = lambda e: (ref.norm_fwd(e["x"], e["w"], e["b"], e["z"], 1e-5, center, act) * dy).sum()
    for k, num, got in _differences(f, v, g, 6):
        assert abs(num - got) <= 1e-7 * max(1, abs(num)), k


# ------------------------------------------------------------------ refusals (no GPU needed)

def _lib_call(qd, fn, **over):
    """A valid call's arguments with some replaced; pointers are never followed on the host."""
    p = ctypes.c_void_p(256)
    base = {
        "short_conv_fwd": dict(x=p, w=p, bias=None, S0=None, lens=None, y=p, S_final=None, B=1, T=8, D=16, W=4, silu=1,
                               dtype=1, stream=None),
        "short_conv_step": dict(S=p, x=p, w=p, bias=None, y=p, N=1, D=16, W=4, silu=1, dtype=1, stream=None),
        "short_conv_bwd": dict(x=p, w=p, bias=None, S0=None, lens=None, dy=p, dS_final=None, dx=p, dw=p, dbias=None,
                               dS0=None, B=1, T=8, D=16, W=4, silu=1, dtype=1, workspace=p, nbytes=1 << 30, stream=None),
        "ssm_fwd": dict(x=p, delta=p, A=p, Bm=p, Cm=p, D_=None, bias=None, S0=None, lens=None, y=p, S_final=None, B=1, T=8,
                        D=16, G=1, N=16, softplus=1, dtype=1, workspace=None, nbytes=0, stream=None),
        "ssm_step": dict(S=p, x=p, delta=p, A=p, Bm=p, Cm=p, D_=None, bias=None, y=p, B=1, D=16, G=1, N=16, softplus=1,
                         dtype=1, stream=None),
        "ssm_bwd": dict(x=p, delta=p, A=p, Bm=p, Cm=p, D_=None, bias=None, S0=None, lens=None, dy=p, dS_final=None, dx=p,
                        ddelta=p, dA=p, dB=p, dC=p, dD=None, dbias=None, dS0=None, B=1, T=8, D=16, G=1, N=16, softplus=1,
                        dtype=1, workspace=p, nbytes=1 << 30, stream=None),
        "group_norm_fwd": dict(x=p, w=None, b=None, z=None, y=p, M=2, H=2, d=16, eps=1e-5, center=1, silu=1, dtype=1,
                               stream=None),
        "group_norm_bwd": dict(x=p, w=p, b=None, z=p, dy=p, dx=p, dz=p, dw=p, db=None, M=2, H=2, d=16, eps=1e-5, center=1,
                               silu=1, dtype=1, workspace=p, nbytes=1 << 30, stream=None),
    }[fn]
    return getattr(qd.load_library(), fn)(*{**base, **over}.values())


OFF = ctypes.c_void_p(258)
REFUSED = [
    ("short_conv_fwd", dict(x=None), 1, "x is NULL"), ("short_conv_fwd", dict(y=OFF), 1, "aligned"),
    ("short_conv_fwd", dict(W=5), 2, "taps"), ("short_conv_fwd", dict(W=1), 2, "taps"),
    ("short_conv_fwd", dict(T=-1), 1, "negative"), ("short_conv_fwd", dict(dtype=7), 2, "dtype"),
    ("short_conv_fwd", dict(B=1 << 20, T=1 << 20), 1, "overflow"), ("short_conv_fwd", dict(lens=OFF), 1, "lens"),
    ("short_conv_step", dict(S=None), 1, "S is NULL"), ("short_conv_step", dict(N=-1), 1, "negative"),
    ("short_conv_bwd", dict(dw=None), 1, "dw is NULL"), ("short_conv_bwd", dict(nbytes=8), 5, "workspace"),
    ("short_conv_bwd", dict(workspace=None), 5, "workspace"),
    ("ssm_fwd", dict(A=None), 1, "A is NULL"), ("ssm_fwd", dict(N=0), 2, "states"), ("ssm_fwd", dict(N=129), 2, "states"),
    ("ssm_fwd", dict(G=3), 1, "groups"), ("ssm_fwd", dict(G=0), 1, "groups"), ("ssm_fwd", dict(S0=OFF), 1, "S0"),
    ("short_conv_bwd", dict(B=2000000000, T=1, D=33), 1, "overflow"),
    ("ssm_fwd", dict(B=1 << 20, T=1, D=1 << 16, G=1 << 16, N=1), 1, "overflow"),
    ("ssm_step", dict(B=1 << 20, D=1 << 14, N=128), 1, "overflow"), ("group_norm_fwd", dict(M=1 << 30, d=128), 1, "overflow"),
    ("ssm_fwd", dict(T=65536), 5, "workspace"), ("ssm_fwd", dict(dtype=2), 2, "dtype"),
    ("ssm_step", dict(Cm=None), 1, "C is NULL"), ("ssm_step", dict(D=-4), 1, "negative"),
    ("ssm_bwd", dict(dB=None), 1, "dB is NULL"), ("ssm_bwd", dict(nbytes=64), 5, "workspace"),
    ("ssm_bwd", dict(dS0=OFF), 1, "dS0"), ("ssm_bwd", dict(N=200), 2, "states"),
    ("group_norm_fwd", dict(eps=0.0), 1, "eps"), ("group_norm_fwd", dict(eps=NAN), 1, "eps"),
    ("group_norm_fwd", dict(d=8193), 2, "8192"), ("group_norm_fwd", dict(d=0), 1, "size"),
    ("group_norm_fwd", dict(z=OFF), 1, "z"), ("group_norm_bwd", dict(dz=None), 1, "dz is NULL"),
    ("group_norm_bwd", dict(nbytes=0), 5, "workspace"), ("group_norm_bwd", dict(M=-1), 1, "size"),
]


@pytest.mark.parametrize("fn,over,code,words", REFUSED)
def test_bad_arguments_are_refused(qd, fn, over, code, words):
    assert _lib_call(qd, fn, **over) == code
    msg = qd.qd_last_error()
    assert fn in msg and words in msg, msg


def test_empty_batches_need_no_device(qd):
    none = dict(x=None, w=None, y=None)
    assert _lib_call(qd, "short_conv_fwd", **none, B=0) == qd.QD_OK
    assert _lib_call(qd, "short_conv_step", **none, S=None, N=0) == qd.QD_OK
    assert _lib_call(qd, "ssm_fwd", x=None, delta=None, A=None, Bm=None, Cm=None, y=None, B=0) == qd.QD_OK
    assert _lib_call(qd, "group_norm_fwd", x=None, y=None, M=0) == qd.QD_OK


def test_binding_refuses_what_it_cannot_run(qd):
    x, w = torch.zeros(1, 4, 8), torch.zeros(8, 4)
    with pytest.raises(ValueError, match="CUDA"):
        qd.short_conv_fwd(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        qd.short_conv_step(torch.zeros(4, 3, 8), x[0], w)
    with pytest.raises(ValueError, match="CUDA"):
        qd.short_conv_bwd(x, w, None, None, x)
    A, BC = torch.zeros(8, 4), torch.zeros(1, 4, 1, 4)
    with pytest.raises(ValueError, match="CUDA"):
        qd.ssm_fwd(x, x, A, BC, BC)
    with pytest.raises(ValueError, match="CUDA"):
        qd.ssm_step(torch.zeros(4, 8, 4), x[0], x[0], A, BC[0], BC[0])
    with pytest.raises(ValueError, match="CUDA"):
        qd.ssm_bwd(x, x, A, BC, BC, None, None, None, x)
    with pytest.raises(ValueError, match="CUDA"):
        qd.group_norm_fwd(x)
    with pytest.raises(ValueError, match="CUDA"):
        qd.group_norm_bwd(x, None, None, None, x)


@pytest.mark.gpu
def test_binding_checks_shapes_types_and_layout(qd):
    x, w = torch.zeros(2, 4, 8, device="cuda"), torch.zeros(8, 4, device="cuda")
    with pytest.raises(TypeError, match="w has dtype"):
        qd.short_conv_fwd(x, w.half())
    with pytest.raises(TypeError, match="unsupported dtype"):
        qd.short_conv_fwd(x.half(), w)
    with pytest.raises(ValueError, match="contiguous"):
        qd.short_conv_fwd(x.transpose(0, 1).contiguous().transpose(0, 1), w)
    with pytest.raises(TypeError, match="lens"):
        qd.short_conv_fwd(x, w, lens=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="S0 has shape"):
        qd.short_conv_fwd(x, w, S0=torch.zeros(2, 4, 8, device="cuda"))
    A, BC = torch.zeros(8, 4, device="cuda"), torch.zeros(2, 4, 1, 4, device="cuda")
    with pytest.raises(ValueError, match="C has shape"):
        qd.ssm_fwd(x, x, A, BC, BC[:, :, :, :3].contiguous())
    with pytest.raises(ValueError, match="y must be a CUDA tensor"):
        qd.group_norm_fwd(x, y=torch.zeros_like(x, device="cpu"))
    with pytest.raises(qd.QDError):
        qd.ssm_fwd(x, x, A, BC.expand(2, 4, 3, 4).contiguous(), BC.expand(2, 4, 3, 4).contiguous())


# ------------------------------------------------------------------ short convolution on the GPU

CONV = [  # B, T, D, W, dtype, silu, bias, s0, lens
    (1, 1, 8, 4, BF16, True, True, True, False), (2, 2, 8, 4, F32, True, True, True, False),
    (3, 17, 40, 4, BF16, True, True, True, True), (3, 33, 64, 3, F32, False, True, False, True),
    (4, 100, 33, 4, BF16, True, False, True, True), (2, 65, 7, 2, F32, True, True, True, True),
    (2, 257, 1028, 4, BF16, True, True, False, False), (1, 1000, 24, 2, BF16, False, False, False, False),
    (5, 3, 12, 3, BF16, True, True, True, True), (2, 130, 513, 4, F32, True, True, True, True),
    (2, 64, 260, 3, BF16, True, True, True, False), (1, 4100, 16, 4, F32, True, True, True, False),
    (2, 75, 130, 4, BF16, True, True, True, True), (2, 40, 50, 2, F32, True, True, True, True),
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,D,W,dt,act,bias,s0,lens", CONV)
def test_conv_forward_and_backward(qd, B, T, D, W, dt, act, bias, s0, lens):
    d = conv_inputs(B, T, D, W, dt, 10 + T, bias, s0, lens)
    c = cu(d)
    y, S = qd.short_conv_fwd(c["x"], c["w"], c["bias"], c["S0"], lens=c["lens"], silu=act)
    y_ref, S_ref = ref.conv_fwd(d["x"], d["w"], d["bias"], d["S0"], d["lens"], act)
    close(y, y_ref, "y")
    assert torch.equal(S.cpu().double(), S_ref)
    g = qd.short_conv_bwd(c["x"], c["w"], c["bias"], c["S0"], c["dy"], c["dS_final"], lens=c["lens"], silu=act)
    close_all(g, ref.conv_bwd(d["x"], d["w"], d["bias"], d["S0"], d["dy"], d["dS_final"], d["lens"], act))


@pytest.mark.gpu
@pytest.mark.parametrize("N,D,W,dt", [(1, 8, 4, BF16), (5, 33, 3, F32), (64, 2048, 4, BF16), (7, 12, 2, BF16)])
def test_conv_tokens_one_by_one_are_the_sequence(qd, N, D, W, dt):
    d = conv_inputs(N, 6, D, W, dt, 40 + D)
    c = cu(d)
    y, S_end = qd.short_conv_fwd(c["x"], c["w"], c["bias"], c["S0"])
    S = c["S0"].clone()
    for t in range(6):
        yt = qd.short_conv_step(S, c["x"][:, t].contiguous(), c["w"], c["bias"])
        close(yt, ref.conv_fwd(d["x"], d["w"], d["bias"], d["S0"])[0][:, t], f"token {t}")
    assert torch.equal(S, S_end)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 2, 5, 40])
def test_conv_state_may_be_carried_in_place(qd, T):
    d = conv_inputs(3, T, 48, 4, BF16, 60)
    c = cu(d)
    want = qd.short_conv_fwd(c["x"], c["w"], c["bias"], c["S0"])
    S = c["S0"].clone()
    y, S2 = qd.short_conv_fwd(c["x"], c["w"], c["bias"], S, S_final=S)
    assert S2 is S and torch.equal(y, want[0]) and torch.equal(S, want[1])


# ------------------------------------------------------------------ selective scan on the GPU

SSM = [  # B, T, D, N, G, dtype, skip, bias, s0, lens, softplus
    (1, 1, 8, 16, 1, BF16, True, True, True, False, True), (2, 31, 64, 16, 1, F32, True, True, True, True, True),
    (2, 33, 72, 16, 2, BF16, True, True, True, True, True), (3, 70, 33, 16, 1, F32, False, False, False, True, True),
    (1, 130, 40, 1, 1, F32, True, True, True, False, True), (2, 50, 130, 3, 2, BF16, True, False, True, True, True),
    (1, 64, 136, 8, 1, BF16, True, True, False, False, False), (2, 47, 24, 24, 3, F32, True, True, True, True, True),
    (1, 95, 65, 32, 1, BF16, False, True, True, False, True), (2, 40, 40, 64, 1, F32, True, True, True, True, False),
    (1, 66, 36, 50, 2, BF16, True, True, True, False, True), (2, 34, 20, 128, 1, F32, True, True, True, True, True),
    (1, 48, 16, 100, 4, BF16, True, True, False, False, True), (3, 16, 9, 17, 9, F32, True, True, True, True, True),
    (1, 1500, 16, 16, 1, F32, True, True, True, False, True), (2, 1111, 24, 32, 1, BF16, True, True, True, True, True),
    (1, 700, 8, 128, 1, F32, True, True, True, False, True), (2, 901, 7, 5, 1, F32, True, True, True, True, True),
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,D,N,G,dt,skip,bias,s0,lens,softplus", SSM)
def test_ssm_forward_and_backward(qd, B, T, D, N, G, dt, skip, bias, s0, lens, softplus):
    d = ssm_inputs(B, T, D, N, G, dt, 100 + T, skip, bias, s0, lens, softplus)
    c = cu(d)
    y, S = qd.ssm_fwd(*(c[k] for k in SSM_IN), lens=c["lens"], softplus=softplus)
    y_ref, S_ref = ref.ssm_fwd(*(d[k] for k in SSM_IN), d["lens"], softplus)
    close(y, y_ref, "y")
    close(S, S_ref, "S_final")
    g = qd.ssm_bwd(*(c[k] for k in SSM_IN), c["dy"], c["dS_final"], lens=c["lens"], softplus=softplus)
    close_all(g, ref.ssm_bwd(*(d[k] for k in SSM_IN), d["dy"], d["dS_final"], d["lens"], softplus))


@pytest.mark.gpu
def test_the_long_shapes_are_cut_into_segments(qd):
    """The shapes above meet both forms of the scan."""
    assert qd.ssm_workspace_bytes(1, 1500, 16, 1, 16, qd.QD_F32) > 0
    assert qd.ssm_workspace_bytes(2, 33, 72, 2, 16, qd.QD_BF16) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("N", [4, 16, 30, 64, 128, 5])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_ssm_tokens_one_by_one_are_the_sequence(qd, N, dt):
    d = ssm_inputs(3, 4, 70, N, 2, dt, 200 + N)
    c = cu(d)
    y_ref, S_ref = ref.ssm_fwd(*(d[k] for k in SSM_IN))
    S = c["S0"].clone()
    for t in range(4):
        tok = [c[k][:, t].contiguous() for k in ("x", "delta", "B", "C")]
        yt = qd.ssm_step(S, tok[0], tok[1], c["A"], tok[2], tok[3], c["D"], c["delta_bias"])
        close(yt, y_ref[:, t], f"token {t}")
    close(S, S_ref, "S")


@pytest.mark.gpu
@pytest.mark.parametrize("T", [40, 1500])
def test_ssm_state_may_be_carried_in_place_and_a_sequence_cut(qd, T):
    d = ssm_inputs(1, T, 24, 16, 1, F32, 300)
    c = cu(d)
    y, S = qd.ssm_fwd(*(c[k] for k in SSM_IN))
    Si = c["S0"].clone()
    y2, _ = qd.ssm_fwd(*(c[k] for k in SSM_IN[:-1]), Si, S_final=Si)
    assert torch.equal(y, y2) and torch.equal(S, Si)
    cut, Sc, ys = T // 3, c["S0"].clone(), []
    for part in (slice(0, cut), slice(cut, T)):
        tok = {k: c[k][:, part].contiguous() for k in ("x", "delta", "B", "C")}
        yp, _ = qd.ssm_fwd(tok["x"], tok["delta"], c["A"], tok["B"], tok["C"], c["D"], c["delta_bias"], Sc, S_final=Sc)
        ys.append(yp)
    y_ref, S_ref = ref.ssm_fwd(*(d[k] for k in SSM_IN))
    close(torch.cat(ys, 1), y_ref, "y in two calls")
    close(Sc, S_ref, "S in two calls")


@pytest.mark.gpu
def test_ssm_steps_of_no_length_and_very_long_ones(qd):
    """u = 0 leaves the state as it is; a huge u forgets it without a NaN."""
    d = ssm_inputs(1, 12, 16, 16, 1, F32, 310, bias=False, softplus=False)
    d["delta"][:, 3:6] = 0.0
    d["delta"][:, 8] = 500.0
    c = cu(d)
    y, S = qd.ssm_fwd(*(c[k] for k in SSM_IN), softplus=False)
    y_ref, S_ref = ref.ssm_fwd(*(d[k] for k in SSM_IN), softplus=False)
    close(y, y_ref, "y")
    close(S, S_ref, "S")
    d["delta_bias"] = torch.linspace(-110, 110, 16)                  # softplus from underflow to the identity
    c = cu(d)
    y, S = qd.ssm_fwd(*(c[k] for k in SSM_IN))
    y_ref, S_ref = ref.ssm_fwd(*(d[k] for k in SSM_IN))
    close(y, y_ref, "y")
    close(S, S_ref, "S")
    close_all(qd.ssm_bwd(*(c[k] for k in SSM_IN), c["dy"], c["dS_final"]),
              ref.ssm_bwd(*(d[k] for k in SSM_IN), d["dy"], d["dS_final"]))


@pytest.mark.gpu
def test_ssm_gradient_against_differences_of_the_definition(qd):
    d = ssm_inputs(2, 40, 24, 16, 2, F32, 320)
    c = cu(d)
    g = qd.ssm_bwd(*(c[k] for k in SSM_IN), c["dy"], c["dS_final"])
    v = _f64(d, SSM_IN)
    dy, dS = d["dy"].double(), d["dS_final"].double()
    for k, num, got in _differences(lambda e: _ssm_loss(e, dy, dS, None, True), v, g, 7):
        assert abs(num - got) <= 1e-4 * max(1, abs(num)), k


# ------------------------------------------------------------------ group norm on the GPU

NORM = [  # M, H, d, dtype, affine, gate, center, silu
    (1, 1, 1, F32, True, True, True, True), (3, 2, 3, BF16, True, False, True, True), (5, 6, 8, BF16, True, True, True, True),
    (33, 3, 20, F32, True, True, False, True), (64, 16, 64, BF16, True, True, True, True),
    (100, 16, 128, BF16, True, True, True, True), (100, 6, 128, F32, False, True, False, True),
    (17, 1, 200, BF16, True, False, True, False), (9, 5, 256, BF16, True, True, True, False), (21, 40, 16, F32, True, True, True, True),
    (7, 2, 1000, F32, True, False, False, True), (6, 1, 1001, BF16, True, True, True, True), (5, 1, 2048, BF16, True, True, False, True),
    (4, 2, 4096, F32, True, True, True, True), (3, 1, 5000, BF16, True, True, True, True), (2, 1, 8192, F32, True, False, True, True),
    (2, 1, 8191, BF16, False, True, True, True), (2500, 2, 100, F32, True, True, True, True), (40, 3, 33, BF16, True, True, True, True),
    (30, 4, 100, BF16, True, True, True, True), (11, 2, 250, F32, True, True, True, True), (3, 2, 1500, BF16, True, False, True, True),
    (2, 1, 8190, F32, True, True, False, True), (4, 1, 3002, BF16, True, True, True, True),
]


@pytest.mark.gpu
@pytest.mark.parametrize("M,H,d,dt,affine,gate,center,act", NORM)
def test_norm_forward_and_backward(qd, M, H, d, dt, affine, gate, center, act):
    v = norm_inputs(M, H, d, dt, 400 + d, affine, gate)
    c = cu(v)
    a, ca = [v[k] for k in ("x", "w", "b", "z")], [c[k] for k in ("x", "w", "b", "z")]
    # one channel a group: centring leaves 0 / sqrt(eps), so everything is exactly b
    close(qd.group_norm_fwd(*ca, center=center, silu=act), ref.norm_fwd(*a, 1e-5, center, act), "y")
    close_all(qd.group_norm_bwd(*ca, c["dy"], center=center, silu=act), ref.norm_bwd(*a, v["dy"], 1e-5, center, act))


@pytest.mark.gpu
def test_norm_of_constant_and_far_off_groups(qd):
    """A group of one value everywhere has no variance; one far from zero keeps its own."""
    x = torch.randn(6, 4, 64, generator=gen(9))
    x[0] = 3.0
    x[1] = 0.0
    x[2] += 4096.0
    y = qd.group_norm_fwd(x.cuda(), silu=False)
    close(y[3:], ref.norm_fwd(x, act=False)[3:], "ordinary")
    assert (y[1] == 0).all() and y[0].abs().max() <= 1e-3
    # the input's own rounding at 4096 is part of the input: what is left is the mean's, 2^-24 4096 against 1
    assert (y[2].cpu().double() - ref.norm_fwd(x, act=False)[2]).abs().max() <= 1e-3


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 7, 15, 50, 125])
@pytest.mark.parametrize("B", [1, 5])
def test_ssm_step_with_states_no_multiple_of_four(qd, N, B):
    """States are moved one by one then; a group of sequences and the last channels are not full."""
    d = ssm_inputs(B, 1, 77, N, 1, F32, 300 + N)
    c = cu(d)
    y_ref, S_ref = ref.ssm_fwd(*(d[k] for k in SSM_IN))
    S = c["S0"].clone()
    tok = [c[k][:, 0].contiguous() for k in ("x", "delta", "B", "C")]
    y = qd.ssm_step(S, tok[0], tok[1], c["A"], tok[2], tok[3], c["D"], c["delta_bias"])
    close(y, y_ref[:, 0], "y")
    close(S, S_ref, "S")


@pytest.mark.gpu
def test_norm_takes_any_leading_shape(qd):
    v = norm_inputs(12, 4, 32, BF16, 3)
    c = cu(v)
    flat = qd.group_norm_fwd(c["x"], c["w"], c["b"], c["z"])
    y = qd.group_norm_fwd(c["x"].view(2, 6, 4, 32), c["w"], c["b"], c["z"].view(2, 6, 4, 32))
    assert torch.equal(y.view(12, 4, 32), flat)


# ------------------------------------------------------------------ every operator

def _all_calls(qd):
    """name -> (call, outputs) of each operator on small inputs in device memory."""
    cv, ss, nm = cu(conv_inputs(2, 50, 40, 4, BF16, 1, lens=True)), cu(ssm_inputs(2, 600, 24, 16, 1, BF16, 2, lens=True)), \
        cu(norm_inputs(70, 4, 128, BF16, 3))
    ssm, nrm = [ss[k] for k in SSM_IN], [nm[k] for k in ("x", "w", "b", "z")]
    one = [ss[k][:, 0].contiguous() for k in ("x", "delta", "B", "C")]

    def conv_step():
        S = cv["S0"].clone()
        return qd.short_conv_step(S, cv["x"][:, 0].contiguous(), cv["w"], cv["bias"]), S

    def ssm_step():
        S = ss["S0"].clone()
        return qd.ssm_step(S, one[0], one[1], ss["A"], one[2], one[3], ss["D"], ss["delta_bias"]), S

    return {
        "short_conv_fwd": lambda: qd.short_conv_fwd(cv["x"], cv["w"], cv["bias"], cv["S0"], lens=cv["lens"]),
        "short_conv_bwd": lambda: qd.short_conv_bwd(cv["x"], cv["w"], cv["bias"], cv["S0"], cv["dy"], cv["dS_final"],
                                                    lens=cv["lens"]).values(),
        "short_conv_step": conv_step,
        "ssm_fwd": lambda: qd.ssm_fwd(*ssm, lens=ss["lens"]),
        "ssm_bwd": lambda: qd.ssm_bwd(*ssm, ss["dy"], ss["dS_final"], lens=ss["lens"]).values(),
        "ssm_step": ssm_step,
        "group_norm_fwd": lambda: [qd.group_norm_fwd(*nrm)],
        "group_norm_bwd": lambda: qd.group_norm_bwd(*nrm, nm["dy"]).values(),
    }


NAMES = ["short_conv_fwd", "short_conv_bwd", "short_conv_step", "ssm_fwd", "ssm_bwd", "ssm_step", "group_norm_fwd",
         "group_norm_bwd"]


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_results_do_not_change_and_other_streams_work(qd, name):
    call = _all_calls(qd)[name]
    first = [t.clone() for t in call()]
    assert qd.last_launch_count() >= 1
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = list(call())
    side.synchronize()
    for a, b in zip(first, again):
        assert torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float())), name


@pytest.mark.gpu
def test_the_stream_argument(qd):
    """A call on a given stream, as an object or a handle, allocates there and runs there: what it
    leaves behind may be reused at once by another call on that stream."""
    d = cu(ssm_inputs(1, 1500, 16, 16, 1, F32, 2))
    want = qd.ssm_bwd(*(d[k] for k in SSM_IN), d["dy"], d["dS_final"])
    y = qd.ssm_fwd(*(d[k] for k in SSM_IN))[0]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        for _ in range(3):
            got = qd.ssm_bwd(*(d[k] for k in SSM_IN), d["dy"], d["dS_final"], stream=stream)
            y2 = qd.ssm_fwd(*(d[k] for k in SSM_IN), stream=stream)[0]
        side.synchronize()
        assert torch.equal(y, y2)
        for k in want:
            assert torch.equal(want[k], got[k]), k


@pytest.mark.gpu
def test_sequences_of_no_tokens(qd):
    d = cu(conv_inputs(2, 0, 16, 4, BF16, 1))
    y, S = qd.short_conv_fwd(d["x"], d["w"], d["bias"], d["S0"])
    assert y.shape == (2, 0, 16) and torch.equal(S, d["S0"])
    g = qd.short_conv_bwd(d["x"], d["w"], d["bias"], d["S0"], d["dy"], d["dS_final"])
    assert torch.equal(g["dS0"], d["dS_final"]) and not g["dw"].any() and not g["dbias"].any()
    d = cu(ssm_inputs(2, 0, 16, 16, 1, F32, 1))
    y, S = qd.ssm_fwd(*(d[k] for k in SSM_IN))
    assert y.shape == (2, 0, 16) and torch.equal(S, d["S0"])
    g = qd.ssm_bwd(*(d[k] for k in SSM_IN), d["dy"], d["dS_final"])
    assert torch.equal(g["dS0"], d["dS_final"])
    assert not any(g[k].any() for k in ("dA", "dD", "ddelta_bias"))
    # and no sequences at all: parameter gradients are zero
    x, w = torch.zeros(0, 5, 8, device="cuda"), torch.ones(8, 4, device="cuda")
    assert not qd.short_conv_bwd(x, w, None, None, x)["dw"].any()
    A, BC = -torch.ones(8, 4, device="cuda"), torch.zeros(0, 5, 1, 4, device="cuda")
    assert not qd.ssm_bwd(x, x, A, BC, BC, None, None, None, x)["dA"].any()
    n = torch.zeros(0, 2, 8, device="cuda")
    assert not qd.group_norm_bwd(n, torch.ones(2, 8, device="cuda"), None, None, n)["dw"].any()


# ------------------------------------------------------------------ offsets beyond 32 bits

@pytest.mark.gpu
def test_arrays_of_more_than_two_to_the_31_elements(qd):
    """The tail of a very long sequence is that of a short one that starts from its state."""
    T, D, N, tail = (1 << 20) + 37, 2056, 16, 45
    assert T * D > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x = torch.empty(1, T, D, dtype=BF16, device="cuda").normal_(generator=g)
    w, bias = 0.5 * r(D, 4), 0.1 * r(D)
    cut = lambda t: t[:, T - tail:].contiguous()
    half = lambda a, b: (a.float() - b.float()).abs().max() <= 2.0 ** -7 * b.float().abs().max()   # one bf16 ulp

    y, S = qd.short_conv_fwd(x, w, bias)
    before = x[:, T - tail - 3:T - tail].contiguous()
    y2, S2 = qd.short_conv_fwd(cut(x), w, bias, before)
    assert torch.equal(cut(y), y2) and torch.equal(S, S2)
    gx = qd.short_conv_bwd(x, w, bias, None, y)["dx"]
    g2 = qd.short_conv_bwd(cut(x), w, bias, before, cut(y))["dx"]
    assert torch.equal(cut(gx), g2)
    del gx

    n = qd.group_norm_fwd(x.view(T, 8, 257))
    assert torch.equal(n[T - tail:], qd.group_norm_fwd(x.view(T, 8, 257)[T - tail:].contiguous()))
    gn = qd.group_norm_bwd(x.view(T, 8, 257), None, None, None, n)["dx"]
    want = qd.group_norm_bwd(x.view(T, 8, 257)[T - tail:].contiguous(), None, None, None, n[T - tail:].contiguous())["dx"]
    assert torch.equal(gn[T - tail:], want)
    del n, gn

    delta = y
    A, skip, db = -(1 + torch.arange(N, device="cuda").float()).repeat(D, 1), torch.ones(D, device="cuda"), -3 + r(D)
    B, C = r(1, T, 1, N).to(BF16), r(1, T, 1, N).to(BF16)
    args = lambda f, S0=None: (f(x), f(delta), A, f(B), f(C), skip, db, S0)
    ys, Ss = qd.ssm_fwd(*args(lambda t: t))
    _, mid = qd.ssm_fwd(*args(lambda t: t[:, :T - tail].contiguous()))
    y3, S3 = qd.ssm_fwd(*args(cut, mid))
    assert half(cut(ys), y3)
    assert (Ss - S3).norm() <= 1e-5 * S3.norm()
    gs = qd.ssm_bwd(*args(lambda t: t), x)
    g3 = qd.ssm_bwd(*args(cut, mid), cut(x))
    for k in ("dx", "ddelta", "dB", "dC"):
        assert half(cut(gs[k]), g3[k]), k
