"""The layer operators at the edges of what they take: arguments that must be refused before a kernel
sees them, streams given in every form, values that are not finite, states that grow."""
import ctypes

import pytest
import torch

import layer_reference as ref

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def qd():
    import delta_rule_linear_qdelta_gb300 as m
    from delta_rule_linear_qdelta_gb300 import build
    build.build()
    m.load_library()
    return m


@pytest.fixture(scope="module")
def layer(qd):
    from delta_rule_linear_qdelta_gb300 import layer as m
    return m


# ------------------------------------------------------------------ workspaces

def test_a_workspace_has_the_memory_that_its_size_says(layer):
    """An expanded tensor has many elements and one byte behind them; a strided one has gaps that are not its own."""
    cpu = torch.device("cpu")
    base = torch.empty(4096, dtype=torch.uint8)
    for bad in (base[:1].expand(4096), base[::2], base.view(64, 64).t()):
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            layer._scratch(1024, bad, cpu)
    assert layer._scratch(1024, base, cpu)[:2] == (base.data_ptr(), 4096)
    assert layer._scratch(1024, base.view(torch.float32), cpu)[:2] == (base.data_ptr(), 4096)


# ------------------------------------------------------------------ sizes near 2^31

MOST = 2 ** 31 - 2 ** 17


@pytest.mark.parametrize("fn,over", [
    ("short_conv_fwd", dict(T=MOST + 1, D=1)), ("short_conv_fwd", dict(T=1, D=MOST + 1)),
    ("short_conv_step", dict(D=MOST + 1)), ("short_conv_bwd", dict(T=MOST + 1, D=1)),
    ("short_conv_bwd", dict(T=1, D=MOST + 1)), ("ssm_fwd", dict(T=MOST + 1, D=1, N=1)), ("ssm_fwd", dict(T=1, D=MOST + 1, N=1)),
    ("ssm_step", dict(D=MOST + 1, N=1)), ("ssm_bwd", dict(T=MOST + 1, D=1, N=1)),
    ("group_norm_fwd", dict(M=1, H=MOST + 1, d=1)), ("group_norm_bwd", dict(M=1, H=MOST + 1, d=1))])
def test_sizes_whose_index_arithmetic_would_wrap_are_refused(qd, fn, over):
    """The kernels add up to a CTA's tokens or channels to a size in 32 bits."""
    from test_layer_ops import _lib_call
    assert _lib_call(qd, fn, **over) == 1
    assert fn in qd.qd_last_error() and "overflow" in qd.qd_last_error()


def test_workspaces_of_refused_sizes_are_none(qd):
    for T, D in ((MOST + 1, 1), (1, MOST + 1)):
        assert qd.short_conv_bwd_workspace_bytes(1, T, D, 4, qd.QD_F32) == 0
        assert qd.ssm_workspace_bytes(1, T, D, 1, 1, qd.QD_F32) == 0
        assert qd.ssm_bwd_workspace_bytes(1, T, D, 1, 1, qd.QD_F32) == 0
    assert qd.group_norm_bwd_workspace_bytes(1, MOST + 1, 1, qd.QD_F32) == 0
    assert qd.short_conv_bwd_workspace_bytes(1, MOST, 1, 4, qd.QD_F32) > 0


def test_the_plan_of_very_long_sequences(qd):
    """19 segments of 32 channels with 128 states each: the start and the ends of 18, and their sums of u; in the backward
    a checkpoint per 8 tokens (states and u), ends, sums and R of all 19, dB and dC per token and group, one row of
    parameter gradients a segment; every array rounded to 64 floats."""
    S, D, N, T = 19, 32, 128, MOST
    assert qd.ssm_workspace_bytes(1, T, D, D, N, qd.QD_F32) == 4 * (S * D * N + (S - 1) * D)
    up = lambda n: (n + 63) // 64 * 64
    chunks = T // 8
    want = up(chunks * D * N) + up(chunks * D) + 2 * up(S * D * N) + up(S * D) + up(T * D * 2 * N) + up(S * D * (N + 2))
    assert qd.ssm_bwd_workspace_bytes(1, T, D, D, N, qd.QD_F32) == 4 * want


def test_sizes_beyond_32_bits_are_refused_by_the_binding(qd):
    """The C entry points take 32-bit sizes: 2^32 rows would reach them as none."""
    big = 2 ** 32
    x = torch.zeros(1).expand(1, big, 1)
    w, A, bc = torch.zeros(1, 4), torch.zeros(1, 1), torch.zeros(1).expand(1, big, 1, 1)
    tok = torch.zeros(1).expand(big, 1)
    calls = [lambda: qd.short_conv_fwd(x, w), lambda: qd.short_conv_bwd(x, w, None, None, x),
             lambda: qd.short_conv_step(torch.zeros(1).expand(big, 3, 1), tok, w), lambda: qd.ssm_fwd(x, x, A, bc, bc),
             lambda: qd.ssm_bwd(x, x, A, bc, bc, None, None, None, x),
             lambda: qd.ssm_step(torch.zeros(1).expand(big, 1, 1), tok, tok, A, bc[0], bc[0]),
             lambda: qd.group_norm_fwd(x.unsqueeze(-1)), lambda: qd.group_norm_bwd(x.unsqueeze(-1), None, None, None, x),
             lambda: qd.group_norm_fwd(x.view(1, 2 ** 16, 2 ** 16, 1, 1)),
             lambda: qd.short_conv_bwd_workspace_bytes(1, big, 1, 4, qd.QD_F32),
             lambda: qd.ssm_workspace_bytes(1, big, 1, 1, 1, qd.QD_F32),
             lambda: qd.ssm_bwd_workspace_bytes(1, big, 1, 1, 1, qd.QD_F32),
             lambda: qd.group_norm_bwd_workspace_bytes(big, 1, 1, qd.QD_F32)]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError, match="32 bits"):
            call()
            pytest.fail(f"call {i} was taken")


# ------------------------------------------------------------------ streams

class OnGpu(torch.Tensor):
    """A tensor that says it is on the first GPU, for what the binding decides before any CUDA call."""
    device = property(lambda self: torch.device("cuda", 0))


def on_gpu():
    return torch.zeros(1).as_subclass(OnGpu)


@pytest.mark.gpu
def test_handle_zero_is_the_default_stream(layer):
    x, seen = torch.zeros(1, device="cuda"), layer._on_stream(lambda t: torch.cuda.current_stream().cuda_stream)
    assert torch.cuda.default_stream().cuda_stream == 0
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert seen(x) == side.cuda_stream
        assert seen(x, stream=0) == 0
        assert seen(x, stream=torch.cuda.default_stream()) == 0
    assert seen(x, stream=side.cuda_stream) == side.cuda_stream


def test_handle_zero_needs_no_new_stream(layer, monkeypatch):
    import contextlib
    used = []
    monkeypatch.setattr(torch.cuda, "default_stream", lambda dev: ("default", dev))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device: ("external", h, device))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: used.append(s) or contextlib.nullcontext())
    call = layer._on_stream(lambda t: None)
    call(on_gpu(), stream=0)
    call(on_gpu(), stream=64)
    assert used == [("default", torch.device("cuda", 0)), ("external", 64, torch.device("cuda", 0))]


def test_a_handle_with_arguments_by_name(qd, layer, monkeypatch):
    import contextlib
    used = []
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device: (h, device))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: used.append(s) or contextlib.nullcontext())
    layer._on_stream(lambda *, x=None, eps=0.0: None)(eps=1.0, x=on_gpu(), stream=64)
    assert used == [(64, torch.device("cuda", 0))]
    monkeypatch.undo()
    x, w = torch.zeros(1, 4, 8), torch.zeros(8, 4)
    with pytest.raises(ValueError, match="CUDA"):                    # the call's own refusals
        qd.short_conv_fwd(x=x, w=w, stream=64)
    with pytest.raises(TypeError, match="required"):
        qd.short_conv_fwd(stream=64)


@pytest.mark.gpu
def test_a_handle_with_arguments_by_name_on_the_gpu(qd):
    x, w = torch.randn(2, 9, 16, device="cuda"), torch.randn(16, 4, device="cuda")
    want = qd.short_conv_fwd(x, w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = qd.short_conv_fwd(x=x, w=w, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_a_stream_of_another_device_is_refused(layer, monkeypatch):
    """The call would run on the tensors' device, on a stream that nobody named."""
    class Stream:
        def __init__(self, index):
            self.device = torch.device("cuda", index)

    import contextlib
    ran = []
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    call = layer._on_stream(lambda t: ran.append(t))
    with pytest.raises(ValueError, match="stream of cuda:1"):
        call(on_gpu(), stream=Stream(1))
    assert not ran
    call(on_gpu(), stream=Stream(0))
    assert len(ran) == 1


# ------------------------------------------------------------------ values that are not finite

@pytest.mark.gpu
@pytest.mark.parametrize("D,dt", [(16, F32), (33, BF16), (40, BF16)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_kept_inputs_of_a_sequence_without_tokens_give_no_weight_gradient(qd, D, dt, bad):
    """No token of it meets them, whatever they hold.  Likewise the last inputs of a sequence and its padding."""
    g = torch.Generator().manual_seed(7)
    r = lambda *s: torch.randn(*s, generator=g)
    x, dy, w, bias, S0 = r(3, 9, D).to(dt), r(3, 9, D).to(dt), r(D, 4), r(D), r(3, 3, D).to(dt)
    lens = torch.tensor([9, 0, 4], dtype=torch.int32)
    S0[1] = bad
    args = (x, w, bias, S0, dy, None)
    S0_fine = S0.clone()
    S0_fine[1] = 0.0                                     # the definition, where those rows are used by nothing
    want = ref.conv_bwd(x, w, bias, S0_fine, dy, None, lens)
    got = qd.short_conv_bwd(*(t if t is None else t.cuda() for t in args), lens=lens.cuda())
    for k in ("dw", "dbias", "dx", "dS0"):
        e = (got[k].cpu().double() - want[k]).abs()
        # fp32: a sum of 13 terms, 2^-24 and the hardware exponential's 2^-22 each; bf16: half an ulp more
        assert (e <= 1e-5 * want[k].abs().max() + (2.0 ** -8 * want[k].abs() if got[k].dtype is BF16 else 0)).all(), k


@pytest.mark.gpu
def test_an_infinite_last_input_meets_no_padding(qd):
    """Without an activation dw is dy x: infinite where the token is, and in no other tap."""
    x, dy, w = torch.ones(1, 8, 8, device="cuda"), torch.ones(1, 8, 8, device="cuda"), torch.ones(8, 4, device="cuda")
    x[0, 4] = float("inf")
    g = qd.short_conv_bwd(x, w, None, None, dy, lens=torch.tensor([5], dtype=torch.int32, device="cuda"), silu=False)
    assert torch.equal(g["dw"], torch.tensor([2.0, 3.0, 4.0, float("inf")], device="cuda").expand(8, 4))


@pytest.mark.gpu
@pytest.mark.parametrize("d,dt", [(128, BF16), (64, F32), (20, F32), (1000, BF16), (4096, F32), (33, BF16), (1, F32)])
@pytest.mark.parametrize("center", [True, False])
def test_a_group_whose_squares_overflow_is_normalised_to_nothing(qd, d, dt, center):
    """Its reciprocal root is 0 (1 / sqrt(inf)), so y = act(b), and nothing flows to x and w; other groups are as ever."""
    g = torch.Generator().manual_seed(11)
    r = lambda *s: torch.randn(*s, generator=g)
    x, w, b, dy = r(5, 2, d).to(dt), 1 + 0.1 * r(2, d), r(2, d), r(5, 2, d).to(dt)
    sign = torch.where(torch.arange(d) % 2 == 0, 1.0, -1.0)
    big = (3e19 * sign).to(dt)                           # its square is above the largest number of 32 bits, its sum is not
    x[1, 0] = big
    c = [t.cuda() for t in (x, w, b)]
    y = qd.group_norm_fwd(*c, center=center, silu=False)
    grads = qd.group_norm_bwd(*c, None, dy.cuda(), center=center, silu=False)
    if d == 1 and center:
        return                                           # one channel: nothing is left of it after centring
    assert torch.equal(y[1, 0], c[2][0].to(dt)) and (grads["dx"][1, 0] == 0).all()
    for t in (y, *(grads[k] for k in ("dx", "dw", "db"))):
        assert torch.isfinite(t).all()
    x[1, 0] = 0                                          # the same xh = 0 for that group
    c = [t.cuda() for t in (x, w, b)]
    y0 = qd.group_norm_fwd(*c, center=center, silu=False)
    g0 = qd.group_norm_bwd(*c, None, dy.cuda(), center=center, silu=False)
    assert torch.equal(y, y0) and torch.equal(grads["dw"], g0["dw"]) and torch.equal(grads["db"], g0["db"])


# ------------------------------------------------------------------ states that grow

GROW = [(16, 16), (7, 5), (16, 64)]                      # D, N: one CTA along the channels, so 1500 tokens are cut into segments


def growing(D, N, seed):
    """A > 0 and step sizes as they come; everything else 0."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    z = torch.zeros(1, 1500, D)
    return g, {"x": z.clone(), "delta": z.clone(), "A": 6 + 0.1 * r(D, N), "B": r(1, 1500, 1, N), "C": r(1, 1500, 1, N),
               "D": None, "delta_bias": None, "S0": None, "dy": z.clone(), "dS_final": None}


SSM_IN = ("x", "delta", "A", "B", "C", "D", "delta_bias", "S0")


def scan_both(qd, d, tol, softplus=False):
    assert qd.ssm_workspace_bytes(1, 1500, d["x"].shape[-1], 1, d["A"].shape[-1], qd.QD_F32) > 0
    c = {k: None if v is None else v.cuda() for k, v in d.items()}
    y, S = qd.ssm_fwd(*(c[k] for k in SSM_IN), softplus=softplus)
    g = qd.ssm_bwd(*(c[k] for k in SSM_IN), c["dy"], c["dS_final"], softplus=softplus)
    y_ref, S_ref = ref.ssm_fwd(*(d[k] for k in SSM_IN), softplus=softplus)
    want = {"y": y_ref, "S_final": S_ref, **ref.ssm_bwd(*(d[k] for k in SSM_IN), d["dy"], d["dS_final"], softplus=softplus)}
    for k, v in {"y": y, "S_final": S, **g}.items():
        if want[k] is None:
            assert v is None, k
            continue
        assert torch.isfinite(v).all(), k
        err = (v.cpu().double() - want[k]).norm()
        assert err <= tol * want[k].norm(), (k, float(err), float(want[k].norm()))


@pytest.mark.gpu
@pytest.mark.parametrize("D,N", GROW)
@pytest.mark.parametrize("how", ["rates", "rates and softplus", "steps back"])
def test_a_state_of_zero_stays_zero_while_decays_overflow(qd, D, N, how):
    """Between the tokens that send gradients and those that have inputs, exp(A u) would multiply up to e^1900, by
    positive rates or by negative step sizes."""
    g, d = growing(D, N, 20)
    softplus, u = how == "rates and softplus", torch.full((1500,), 0.01)
    u[100:1400] = 0.25
    if how == "steps back":
        u[100:1400] *= -1
        d["A"] *= -1
    d["delta"][:] = (torch.log(torch.expm1(u.double())).float() if softplus else u)[None, :, None]
    d["x"][:, 1400:] = torch.randn(1, 100, D, generator=g)
    d["dy"][:, :100] = torch.randn(1, 100, D, generator=g)
    # fp32 tolerance of the scan: the tokens with inputs or gradients make 100 steps of at most e^0.07
    scan_both(qd, d, 1e-5, softplus)


@pytest.mark.gpu
@pytest.mark.parametrize("D,N", GROW)
@pytest.mark.parametrize("way", [1, -1])
def test_a_tiny_state_grows_over_a_segment_by_more_than_fp32_holds(qd, D, N, way):
    """1e-30 e^96 is an ordinary number.  Tolerance: the exponent, 139 as a power of two, has a relative error of 2^-24 from
    A log2(e) and, taken at once in two halves or in 64 steps, 8e-6 from its roundings: 1.2e-5 in all, and the
    products of a state and a gradient have it twice and the sums' 1e-5."""
    g, d = growing(D, N, 21)
    d["delta"][:, 80:144] = 0.25 * way
    d["A"] *= way
    d["S0"], d["dS_final"] = (1e-30 * torch.randn(1, D, N, generator=g) for _ in range(2))
    scan_both(qd, d, 5e-5)


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_step_size_that_is_no_number_is_not_hidden(qd, bad):
    g, d = growing(16, 16, 22)
    d["delta"][:, :] = 0.01
    d["delta"][0, 300, 3] = bad
    d["S0"] = torch.ones(1, 16, 16)
    c = {k: None if v is None else v.cuda() for k, v in d.items()}
    y, S = qd.ssm_fwd(*(c[k] for k in SSM_IN), softplus=False)
    assert not torch.isfinite(S[0, 3]).any() and not torch.isfinite(y[0, 300:, 3]).any()
    # the other channels are finite where their definition is within fp32 (S0 e^90 is not everywhere)
    fine = ref.ssm_fwd(*(d[k] for k in SSM_IN), softplus=False)[1][0].abs() <= torch.finfo(F32).max
    other = torch.arange(16) != 3
    assert torch.equal(torch.isfinite(S[0].cpu())[other], fine[other]) and torch.isfinite(y[0, :300]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("D,N,dt,lens", [(16, 16, F32, None), (21, 5, F32, 30011), (24, 16, BF16, None)])
def test_hundreds_of_segments(qd, D, N, dt, lens):
    """Few channels over very many tokens, within the tolerances of the other scan tests: fp32 relative L2 1e-5, bf16
    half an ulp and 1e-5 of the largest."""
    from test_layer_ops import close, close_all, ssm_inputs
    T = 32768
    d = ssm_inputs(1, T, D, N, 1, dt, 500 + D)
    assert qd.ssm_workspace_bytes(1, T, D, 1, N, qd.QD_F32) >= 4 * 400 * D * N
    if lens:
        d["lens"] = torch.tensor([lens], dtype=torch.int32)
        for k in ("x", "delta", "B", "C", "dy"):
            d[k][:, lens:] = float("nan")
    c = {k: None if v is None else v.cuda() for k, v in d.items()}
    y, S = qd.ssm_fwd(*(c[k] for k in SSM_IN), lens=c["lens"])
    y_ref, S_ref = ref.ssm_fwd(*(d[k] for k in SSM_IN), d["lens"])
    close(y, y_ref, "y")
    close(S, S_ref, "S_final")
    g = qd.ssm_bwd(*(c[k] for k in SSM_IN), c["dy"], c["dS_final"], lens=c["lens"])
    close_all(g, ref.ssm_bwd(*(d[k] for k in SSM_IN), d["dy"], d["dS_final"], d["lens"]))
