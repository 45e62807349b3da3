"""The mixers beside the Delta rule (linear attention with decays, windowed attention with sinks) against
their definitions in 64 bits (tests/mixer_reference.py).

Tolerances, set before any run.  A result is a sum of products whose factors are held in fp32 or rounded to
bf16; A is the same sum over absolute values, so a factor off by a relative e moves the result by at
most e A.
  fp32 calls and fp32 outputs (states and their gradients, lse): relative L2 <= 1e-5, the library's fp32
    tolerance; an element by at most 1e-5 (A + the largest |ref|).
  bf16 outputs, by 2^-8 (half a step of bf16, relative) for each rounding that a term meets:
    o of linear attention: a pair's weight and the output, or the decayed query, the entering state and
      the output: 3
    its gradients dq, dk, dv: the same, and for dv the state's gradient: 3.  dg: a pair's gradient or
      both states, and the output: 3
    o of windowed attention: the probability and the output: 2
    its gradients: the probability's gradient, the o that enters it, and the output: 3
  each time plus 1e-5 (A + the largest |ref|) for what is done in fp32.
"""
import ctypes
import math

import pytest
import torch

import mixer_reference as ref

F32, BF16, F64 = torch.float32, torch.bfloat16, torch.float64
NAN, INF = float("nan"), float("inf")
HALF = 2.0 ** -8


@pytest.fixture(scope="module")
def qd():
    import delta_rule_linear_qdelta_gb300 as m
    from delta_rule_linear_qdelta_gb300 import build
    build.build()
    m.load_library()
    return m


def close(got, want, mag, what, roundings=3, extra=0.0):
    assert got.shape == want.shape, (what, got.shape, want.shape)
    if want.numel() == 0:
        return
    g = got.detach().cpu().double()
    assert torch.isfinite(g).all(), f"{what}: not finite"
    err = (g - want).abs()
    small = 1e-5 * (mag + want.abs().max()) + extra
    if got.dtype == BF16:
        over = (err - roundings * HALF * mag - small).max()
        assert over <= 0, f"{what}: {over:.3e} beyond {roundings} roundings"
    else:
        assert (err - small).max() <= 0, f"{what}: {(err - small).max():.3e} beyond fp32"
        # relative to the terms where all of them cancel (a query that sees one key alone: dP = D, each a sum of
        # d products with its own roundings)
        size = want.norm() if want.norm() > 1e-6 * mag.norm() else mag.norm()
        rel = (err - extra).clamp_min(0).norm() / size.clamp_min(1e-30)
        assert rel <= 1e-5 or err.max() == 0, f"{what}: relative L2 {rel:.3e}"


def decay_noise(d, mag):
    """What fp32 may leave of the terms that cancel in dg.  dg_t is the sum over the tokens from t to its
    chunk's end of q . dq - k . dk, in which the pairs of two such tokens cancel: each q_i . dq_i is a sum of up
    to 128 products with a dq that is itself one of up to 256, so 2^9 roundings of 2^-24 and random signs, 2^-19.5
    of the term, are left of each (chunks of 64 or 128 tokens: here all of an aligned 128)."""
    t = (d["q"].abs() * mag["dq"]).sum(-1) + (d["k"].abs() * mag["dk"]).sum(-1)
    T = t.shape[1]
    t = torch.nn.functional.pad(t, (0, 0, 0, -T % 128)).unflatten(1, (-1, 128))
    return 2.0 ** -19.5 * t.sum(2, keepdim=True).expand_as(t).flatten(1, 2)[:, :T]


def cu(d):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in d.items()}


def wide(d):
    """The inputs in 64 bits, what padding holds replaced by 0."""
    out = {}
    for x, t in d.items():
        out[x] = torch.nan_to_num(t.double(), nan=0.0, neginf=-INF) if isinstance(t, torch.Tensor) and t.is_floating_point() else t
    return out


def mags(d):
    return {x: t.abs() if isinstance(t, torch.Tensor) and t.is_floating_point() and x != "g" else t for x, t in d.items()}


def lens_of(how, B, T, g):
    if not how:
        return None
    n = torch.randint(0, T + 1, (B,), generator=g, dtype=torch.int32)
    n[0] = T + 7                                        # clamped
    n[B - 1] = 0
    if B > 2:
        n[1] = min(T, 1)
    return n


def poison(t, lens, past=0):
    """The padded tokens of t as NaN."""
    if lens is not None:
        for b, n in enumerate(lens.tolist()):
            t[b, past + max(n, 0):] = NAN
    return t


# ------------------------------------------------------------------ linear attention: inputs and shapes

def lin_inputs(B, T, H, dk, dv, dt, seed, decay="token", s0=True, lens=False):
    """decay: token, strong (down to e^-20 a token), drop (some tokens drop the state), head, none."""
    g = torch.Generator().manual_seed(seed)
    n = lens_of(lens, B, T, g)
    r = lambda *s: torch.randn(*s, generator=g)
    unit = lambda t: t / t.norm(dim=-1, keepdim=True).clamp_min(1e-6)
    ld = None
    if decay == "head":
        ld = -torch.exp(-6 * torch.rand(H, generator=g) - 1)
    elif decay != "none":
        ld = -torch.nn.functional.softplus(0.5 * r(B, T, H) - 4)
        if decay == "strong":
            ld = torch.where(torch.rand(B, T, H, generator=g) < 0.3, -20 * torch.rand(B, T, H, generator=g), ld)
        if decay == "drop":
            ld = torch.where(torch.rand(B, T, H, generator=g) < 0.05, torch.full((), -INF), ld)
            ld[:, ::64] = torch.where(torch.rand(B, (T + 63) // 64, H, generator=g) < 0.5, torch.full((), -88.0), ld[:, ::64])
        ld = poison(ld.to(dt), n)
    return {"q": poison(unit(r(B, T, H, dk)).to(dt), n), "k": poison(unit(r(B, T, H, dk)).to(dt), n),
            "v": poison(r(B, T, H, dv).to(dt), n), "g": ld, "S0": 0.3 * r(B, H, dv, dk) if s0 else None, "lens": n,
            "dO": poison(r(B, T, H, dv).to(dt), n), "dS_final": 0.3 * r(B, H, dv, dk) if s0 else None}


def dropped(d):
    """The decays with -inf in the place of those below the smallest normal number, as the kernels take them."""
    if d["g"] is not None:
        d["g"] = torch.where(d["g"] < -87, torch.full((), -INF, dtype=F64), d["g"])
    return d


LIN = [  # B, T, H, dk, dv, decay, s0, lens
    (1, 1, 1, 8, 8, "token", False, False),
    (2, 1, 3, 128, 128, "token", True, False),
    (1, 2, 2, 16, 40, "none", True, False),
    (2, 63, 2, 64, 64, "token", False, False),
    (1, 64, 3, 128, 128, "token", True, False),
    (2, 65, 1, 32, 128, "drop", True, False),
    (1, 127, 2, 72, 104, "token", True, False),
    (2, 128, 2, 128, 64, "head", True, False),
    (1, 129, 2, 128, 128, "token", True, False),
    (4, 150, 2, 64, 128, "token", True, True),
    (4, 200, 3, 128, 128, "drop", True, True),
    (2, 300, 2, 128, 128, "strong", True, False),
    (3, 270, 1, 40, 24, "strong", False, True),
    (3, 260, 2, 128, 128, "none", False, True),
    (2, 513, 1, 64, 64, "drop", True, False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("B,T,H,dk,dv,decay,s0,lens", LIN)
def test_linear_attention(qd, B, T, H, dk, dv, decay, s0, lens, dt):
    d = lin_inputs(B, T, H, dk, dv, dt, 100 * T + dk, decay, s0, lens)
    w = dropped(wide(d))
    args = ("q", "k", "v", "g", "S0", "lens")
    o, S = qd.lin_attn_fwd(*(cu(d)[x] for x in args[:5]), lens=cu(d)["lens"])
    want, mag = (ref.lin_fwd(*(e[x] for x in args)) for e in (w, mags(w)))
    close(o, want[0], mag[0], "o")
    close(S, want[1], mag[1], "S_final")
    if lens:
        for b, n in enumerate(ref.lens_list(d["lens"], B, T)):
            assert (o[b, n:] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("B,T,H,dk,dv,decay,s0,lens", LIN)
def test_linear_attention_gradients(qd, B, T, H, dk, dv, decay, s0, lens, dt):
    d = lin_inputs(B, T, H, dk, dv, dt, 100 * T + dv, decay, s0, lens)
    w = dropped(wide(d))
    c = cu(d)
    got = qd.lin_attn_bwd(c["q"], c["k"], c["v"], c["g"], c["S0"], c["dO"], c["dS_final"], lens=c["lens"])
    want, mag = (ref.lin_bwd(e, d["lens"]) for e in (w, mags(w)))
    if decay in ("head", "none"):
        assert got.pop("dg") is None
        want.pop("dg", None)
    assert set(got) == set(want)
    for x in want:
        close(got[x], want[x], mag[x], x, extra=decay_noise(w, mag) if x == "dg" else 0.0)
    if "dg" in got:
        assert (got["dg"].cpu()[torch.nan_to_num(d["g"].float()) < -87] == 0).all()


@pytest.mark.gpu
def test_linear_attention_gradients_against_differences(qd):
    d = lin_inputs(2, 140, 2, 64, 40, F32, 5, "token")
    c, w = cu(d), wide(d)
    got = qd.lin_attn_bwd(c["q"], c["k"], c["v"], c["g"], c["S0"], c["dO"], c["dS_final"])
    g = torch.Generator().manual_seed(6)

    def loss(e):
        o, S = ref.lin_fwd(e["q"], e["k"], e["v"], e["g"], e["S0"])
        return float((o * w["dO"]).sum() + (S * w["dS_final"]).sum())

    for x in ("q", "k", "v", "g", "S0"):
        way = torch.randn(w[x].shape, generator=g, dtype=F64)
        if x == "g":
            way *= 0.01
        h = 1e-4
        num = (loss({**w, x: w[x] + h * way}) - loss({**w, x: w[x] - h * way})) / (2 * h)
        have = float((got["d" + x].cpu().double() * way).sum())
        # 1e-5 of the gradient's norm in any direction, and the differences' own error (h^2 and 2^-52 / h)
        size = float(got["d" + x].cpu().double().norm() * way.norm())
        assert abs(num - have) <= 1e-5 * size + 1e-6 * (1 + abs(num)), x


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("N,H,dk,dv,decay", [(1, 1, 8, 8, "token"), (3, 5, 128, 128, "token"), (2, 2, 40, 72, "head"),
                                             (5, 3, 64, 16, "none"), (4, 2, 128, 24, "drop"), (700, 2, 16, 128, "token")])
def test_linear_attention_step(qd, N, H, dk, dv, decay, dt):
    d = lin_inputs(N, 1, H, dk, dv, dt, N + dk, "token" if decay == "drop" else decay)
    if decay == "drop":
        d["g"][::2] = -INF
        d["S0"][::2] = NAN                                  # dropped, whatever it holds
    w = wide(d)
    c = cu(d)
    S = c["S0"].clone()
    g = c["g"] if c["g"] is None or c["g"].dim() == 1 else c["g"][:, 0].contiguous()
    o = qd.lin_attn_step(S, *(c[x][:, 0].contiguous() for x in "qkv"), g)
    want, mag = (ref.lin_fwd(*(e[x] for x in ("q", "k", "v", "g", "S0"))) for e in (w, mags(w)))
    close(o, want[0][:, 0], mag[0][:, 0], "o", 1)           # all in fp32 but the output
    close(S, want[1], mag[1], "S")


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16])
def test_a_prompt_in_pieces_and_tokens_is_the_whole(qd, dt):
    """Pieces carry the state in place; the last tokens go one at a time."""
    B, T, H, dk, dv = 2, 211, 3, 128, 64
    d = lin_inputs(B, T, H, dk, dv, dt, 9, "token", True, False)
    c, w = cu(d), wide(d)
    S, outs, at = c["S0"].clone(), [], 0
    for n in (1, 130, 64, 9):
        part = [c[x][:, at:at + n].contiguous() for x in ("q", "k", "v", "g")]
        o, _ = qd.lin_attn_fwd(*part, S, S_final=S)
        outs.append(o)
        at += n
    for t in range(at, T):
        outs.append(qd.lin_attn_step(S, *(c[x][:, t].contiguous() for x in ("q", "k", "v", "g")))[:, None])
    want, mag = (ref.lin_fwd(*(e[x] for x in ("q", "k", "v", "g", "S0"))) for e in (w, mags(w)))
    close(torch.cat(outs, 1), want[0], mag[0], "o")
    close(S, want[1], mag[1], "S")


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("B,T,H,lens", [(1, 8192, 2, None), (3, 2000, 5, [2000, 130, 0]), (2, 897, 38, [1, 897]), (1, 40000, 1, [200])])
def test_a_state_carried_in_place_through_long_sequences(qd, B, T, H, lens, dt):
    """S_final over S0 where a sequence is cut into segments, some of them of padding alone: as in a buffer of its own."""
    d = lin_inputs(B, T, H, 64, 128, dt, T + H, "token", True)
    c = cu(d)
    n = None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda()
    o, S = qd.lin_attn_fwd(c["q"], c["k"], c["v"], c["g"], c["S0"], lens=n)
    for _ in range(3):
        carried = c["S0"].clone()
        again, end = qd.lin_attn_fwd(c["q"], c["k"], c["v"], c["g"], carried, lens=n, S_final=carried)
        assert end is carried and torch.equal(carried, S) and torch.equal(again, o)
    if lens is not None and 0 in lens:
        assert torch.equal(S[lens.index(0)], c["S0"][lens.index(0)])


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("a_token", [0.1, 0.31, 0.45, 0.49, 0.6])
@pytest.mark.parametrize("power", [-56, -30, 30, 56])
def test_linear_attention_of_small_and_large_values(qd, power, a_token, dt):
    """Queries, and a loss, scaled by a power of two: outputs and gradients are linear in them, whatever the decays of a
    chunk sum to.  All results are far inside the range of both types."""
    d = lin_inputs(1, 200, 2, 64, 64, dt, 17, "token", True)
    d["g"] = torch.full((1, 200, 2), -a_token).to(dt)
    f = 2.0 ** power
    fwd = {**d, "q": (d["q"].float() * f).to(dt)}
    c, w = cu(fwd), wide(fwd)
    o, S = qd.lin_attn_fwd(c["q"], c["k"], c["v"], c["g"], c["S0"])
    want, mag = (ref.lin_fwd(*(e[x] for x in ("q", "k", "v", "g", "S0"))) for e in (w, mags(w)))
    close(o, want[0], mag[0], "o")
    close(S, want[1], mag[1], "S_final")
    bwd = {**d, "dO": (d["dO"].float() * f).to(dt), "dS_final": d["dS_final"] * f}
    c, w = cu(bwd), wide(bwd)
    got = qd.lin_attn_bwd(c["q"], c["k"], c["v"], c["g"], c["S0"], c["dO"], c["dS_final"])
    want, mag = (ref.lin_bwd(e) for e in (w, mags(w)))
    for x in want:
        close(got[x], want[x], mag[x], x, extra=decay_noise(w, mag) if x == "dg" else 0.0)


def chunked(q, k, v, g, S0, C=128):
    """Linear attention in 64 bits by chunks, for long sequences on the GPU: [T,d] q, k, v, [T] g, one head."""
    S, o = S0.clone(), []
    for t in range(0, q.shape[0], C):
        qc, kc, vc, P = q[t:t + C], k[t:t + C], v[t:t + C], torch.cumsum(g[t:t + C], 0)
        M = torch.exp(P[:, None] - P).tril()
        o.append(((qc @ kc.t()) * M) @ vc + torch.exp(P)[:, None] * (qc @ S.t()))
        S = torch.exp(P[-1]) * S + (torch.exp(P[-1] - P)[:, None] * vc).t() @ kc
    return torch.cat(o), S


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("T,n", [(8192, None), (5001, 4133)])
def test_long_sequences_of_few_heads(qd, T, n, dt):
    """So few streams that a sequence has to be cut, with decays that remember thousands of tokens."""
    B, H, d = 1, 2, 128
    x = lin_inputs(B, T, H, d, d, dt, T, "none", True)
    x["g"] = (-torch.rand(B, T, H, generator=torch.Generator().manual_seed(3)) * 2e-3).to(dt)
    c = cu(x)
    lens = None if n is None else torch.tensor([n], dtype=torch.int32).cuda()
    o, S = qd.lin_attn_fwd(c["q"], c["k"], c["v"], c["g"], c["S0"], lens=lens)
    got = qd.lin_attn_bwd(c["q"], c["k"], c["v"], c["g"], c["S0"], c["dO"], c["dS_final"], lens=lens)
    m = T if n is None else n
    assert (o[:, m:] == 0).all()
    for h in range(H):
        leaf = [c[y][0, :m, h].double().requires_grad_() for y in ("q", "k", "v", "g")] + [c["S0"][0, h].double().requires_grad_()]
        wo, wS = chunked(*leaf)
        grads = torch.autograd.grad((wo * c["dO"][0, :m, h].double()).sum() + (wS * c["dS_final"][0, h].double()).sum(), leaf)
        # random signs: the error of a sum of roundings is of one rounding's relative size (root mean square
        # 2^-8 / sqrt 3 at most), here of up to four that are independent; sums of 2^-24 for fp32
        tol = 5e-3 if dt == BF16 else 1e-5
        for name, a, b, t in [("o", o[0, :m, h], wo, tol), ("S", S[0, h], wS, 1e-5)] + [
                ("d" + y, got["d" + y][0, :m, h], z, tol) for y, z in zip(("q", "k", "v", "g"), grads)] + [
                ("dS0", got["dS0"][0, h], grads[4], 1e-5)]:
            rel = float((a.double() - b.detach()).norm() / b.detach().norm())
            assert rel <= t, (name, rel)


def chunked_batch(q, k, v, g, S0, C=128):
    """The same in 64 bits for a batch of heads, q, k, v [N,T,d], g [N,T] or None, S0 [N,dv,dk]; decays below -87 drop the
    state.  Exponents of pairs that do not see each other never enter an exponential."""
    N, T, _ = q.shape
    g = torch.zeros(N, T, dtype=q.dtype, device=q.device) if g is None else g
    drop = g < -87
    g = torch.where(drop, torch.zeros_like(g), g)
    if S0 is None:
        S0 = torch.zeros(N, v.shape[-1], q.shape[-1], dtype=q.dtype, device=q.device)
    zero, S, o = torch.zeros((), dtype=q.dtype, device=q.device), S0, []
    weight = lambda x, see: torch.where(see, torch.exp(torch.where(see, x, zero)), zero)
    for t in range(0, T, C):
        qc, kc, vc, P, piece = q[:, t:t + C], k[:, t:t + C], v[:, t:t + C], torch.cumsum(g[:, t:t + C], 1), drop[:, t:t + C].cumsum(1)
        n = P.shape[1]
        see = torch.ones(n, n, dtype=torch.bool, device=q.device).tril() & (piece[:, :, None] == piece[:, None])
        M = weight(P[:, :, None] - P[:, None], see)
        o.append(((qc @ kc.mT) * M) @ vc + weight(P, piece == 0)[..., None] * (qc @ S.mT))
        S = weight(P[:, -1], piece[:, -1] == 0)[:, None, None] * S + (weight(P[:, -1:] - P, piece == piece[:, -1:])[..., None] * vc).mT @ kc
    return torch.cat(o, 1), S


def chunked_bwd(d, lens):
    """Gradients in 64 bits as ref.lin_bwd's, sequence by sequence, on the GPU; padded tokens' are 0."""
    B, T, H, _ = d["q"].shape
    names = [x for x in ("q", "k", "v", "g", "S0") if d[x] is not None]
    out = {"d" + x: torch.zeros(d[x].shape, dtype=F64) for x in names}
    for b, n in enumerate(ref.lens_list(lens, B, T)):
        if n == 0:
            out["dS0"][b] = d["dS_final"][b]
            continue
        heads = lambda x: d[x][b] if x == "S0" else d[x][b, :n].transpose(0, 1)
        leaf = {x: heads(x).cuda().contiguous().requires_grad_() for x in names}
        o, S = chunked_batch(*(leaf.get(x) for x in ("q", "k", "v", "g", "S0")))
        loss = (o * heads("dO").cuda()).sum() + (S * d["dS_final"][b].cuda()).sum()
        for x, t in zip(names, torch.autograd.grad(loss, list(leaf.values()))):
            if x == "S0":
                out["dS0"][b] = t.cpu()
            else:
                out["d" + x][b, :n] = t.transpose(0, 1).cpu()
    return out


def test_the_chunked_definition_is_the_definition():
    d = dropped(wide(lin_inputs(2, 140, 2, 16, 8, F32, 31, "drop")))
    o, S = ref.lin_fwd(*(d[x] for x in ("q", "k", "v", "g", "S0")))
    for b in range(2):
        got = chunked_batch(*(d[x][b].transpose(0, 1) for x in ("q", "k", "v", "g")), d["S0"][b])
        assert torch.allclose(got[0].transpose(0, 1), o[b], rtol=1e-12, atol=1e-12)
        assert torch.allclose(got[1], S[b], rtol=1e-12, atol=1e-12)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (128, 40), (24, 128)])
@pytest.mark.parametrize("decays", ["mixed", "none"])
def test_linear_attention_gradients_of_many_chunks(qd, decays, dk, dv, dt):
    """More chunks than the GPU has SMs twice over, so that each CTA takes several in turn: whole, cut by padding and all
    padding ones, chunks whose decays are weak, strong and drop the state side by side.  The same bits every time."""
    B, T, H = 4, 1200, 16
    x = lin_inputs(B, T, H, dk, dv, dt, dk + dv, "none")
    g = torch.Generator().manual_seed(5)
    n = torch.tensor([1300, 1, 700, 1100], dtype=torch.int32)
    assert H * sum(-(-min(m, T) // 128) for m in n.tolist()) > 2 * 152
    for y in ("q", "k", "v", "dO"):
        poison(x[y], n)
    x["lens"] = n
    if decays == "mixed":
        ld = -torch.nn.functional.softplus(0.5 * torch.randn(B, T, H, generator=g) - 4)
        kind = torch.randint(0, 4, (B, -(-T // 128), H), generator=g).repeat_interleave(128, 1)[:, :T]   # a chunk's: weak, weak, strong, drops
        ld = torch.where((kind == 2) & (torch.rand(B, T, H, generator=g) < 0.3), -20 * torch.rand(B, T, H, generator=g), ld)
        ld = torch.where((kind == 3) & (torch.rand(B, T, H, generator=g) < 0.05), torch.full((), -INF), ld)
        x["g"] = poison(ld.to(dt), n)
    w, c = dropped(wide(x)), cu(x)
    run = lambda: qd.lin_attn_bwd(c["q"], c["k"], c["v"], c["g"], c["S0"], c["dO"], c["dS_final"], lens=c["lens"])
    got = run()
    want, mag = (chunked_bwd(e, n) for e in (w, mags(w)))
    if decays == "none":
        assert got.pop("dg") is None
    assert set(got) == set(want)
    for y in want:
        close(got[y], want[y], mag[y], y, extra=decay_noise(w, mag) if y == "dg" else 0.0)
        # random signs: the relative error is of one rounding's size, of up to four that are independent (root mean square
        # 2^-8 / sqrt 3 at most)
        if got[y].dtype == BF16:
            rel = float((got[y].cpu().double() - want[y]).norm() / want[y].norm())
            assert rel <= 5e-3, (y, rel)
    for _ in range(5):
        again = run()
        assert all(torch.equal(again[y], got[y]) for y in want)


# ------------------------------------------------------------------ windowed attention

def win_inputs(B, T, past, H, Hkv, d, dt, seed, lens=False):
    g = torch.Generator().manual_seed(seed)
    n = lens_of(lens, B, T, g)
    r = lambda *s: torch.randn(*s, generator=g)
    return {"q": poison(r(B, T, H, d).to(dt), n), "k": poison(r(B, past + T, Hkv, d).to(dt), n, past),
            "v": poison(r(B, past + T, Hkv, d).to(dt), n, past), "lens": n, "dO": poison(r(B, T, H, d).to(dt), n)}


WIN = [  # B, T, past, H, Hkv, d, window, sinks, lens
    (1, 1, 0, 1, 1, 8, 1, 0, False),
    (2, 1, 40, 4, 2, 128, 16, 3, False),
    (1, 64, 0, 2, 2, 64, 1, 0, False),
    (1, 65, 0, 2, 1, 64, 2, 1, False),
    (2, 127, 0, 4, 2, 128, 1000, 0, False),
    (1, 128, 0, 2, 2, 128, 128, 0, False),
    (1, 129, 0, 3, 1, 128, 129, 4, False),
    (2, 200, 0, 6, 2, 72, 50, 5, False),
    (1, 300, 100, 4, 1, 128, 64, 4, False),
    (4, 190, 33, 6, 3, 64, 70, 2, True),
    (3, 260, 0, 2, 2, 128, 40, 130, True),
    (1, 513, 0, 8, 4, 128, 200, 4, False),
    (1, 520, 7, 2, 1, 40, 130, 260, False),
    (2, 384, 0, 5, 1, 128, 1 << 30, 0, False),
    (1, 300, 0, 2, 2, 32, 3, (1 << 30) - 3, False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("B,T,past,H,Hkv,d,window,sinks,lens", WIN)
def test_windowed_attention(qd, B, T, past, H, Hkv, d, window, sinks, lens, dt):
    x = win_inputs(B, T, past, H, Hkv, d, dt, 10 * T + d, lens)
    c, w, scale = cu(x), wide(x), 0.7 / math.sqrt(d)
    o, lse = qd.win_attn_fwd(c["q"], c["k"], c["v"], window=window, sinks=sinks, scale=scale, lens=c["lens"])
    want, z = ref.win_fwd(w["q"], w["k"], w["v"], window, sinks, scale, x["lens"])
    mag, _ = ref.win_fwd(w["q"], w["k"], w["v"].abs(), window, sinks, scale, x["lens"])
    close(o, want, mag, "o", 2)
    close(lse, z, z.abs() + 1, "lse")
    if window == 1 and sinks == 0:                          # a query sees itself alone
        assert torch.equal(o, c["v"][:, past:].repeat_interleave(H // Hkv, 2))
    got = qd.win_attn_bwd(c["q"], c["k"], c["v"], o, lse, c["dO"], window=window, sinks=sinks, scale=scale, lens=c["lens"])
    want, mag = ref.win_bwd(w["q"], w["k"], w["v"], w["dO"], window, sinks, scale, x["lens"])
    assert set(got) == set(want)
    for y in want:
        close(got[y], want[y], mag[y], y)
    if lens:
        for b, n in enumerate(ref.lens_list(x["lens"], B, T)):
            assert (o[b, n:] == 0).all() and (lse[b, n:] == 0).all() and (got["dq"][b, n:] == 0).all()
            assert (got["dk"][b, past + n:] == 0).all() and (got["dv"][b, past + n:] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("B,T,past,H,Hkv,d,window,sinks,lens", [
    (1, 700, 0, 8, 1, 128, 1 << 30, 0, False),
    (1, 1500, 5, 16, 1, 64, 130, 3, False),
    (3, 400, 33, 8, 1, 72, 300, 2, True),
    (2, 129, 200, 16, 1, 40, 150, 140, True),
])
def test_many_heads_on_few_key_heads(qd, B, T, past, H, Hkv, d, window, sinks, lens, dt):
    """So few key tiles that what is summed over heads and queries is cut."""
    test_windowed_attention(qd, B, T, past, H, Hkv, d, window, sinks, lens, dt)


@pytest.mark.gpu
def test_windowed_attention_gradients_against_differences(qd):
    B, T, past, H, Hkv, d, window, sinks = 2, 90, 5, 4, 2, 40, 30, 3
    x = win_inputs(B, T, past, H, Hkv, d, F32, 8)
    c, w, scale = cu(x), wide(x), 1 / math.sqrt(d)
    kw = {"window": window, "sinks": sinks}
    o, lse = qd.win_attn_fwd(c["q"], c["k"], c["v"], **kw)
    got = qd.win_attn_bwd(c["q"], c["k"], c["v"], o, lse, c["dO"], **kw)
    g = torch.Generator().manual_seed(6)
    loss = lambda e: float((ref.win_fwd(e["q"], e["k"], e["v"], window, sinks, scale)[0] * w["dO"]).sum())
    for y in "qkv":
        way = torch.randn(w[y].shape, generator=g, dtype=F64)
        h = 1e-4
        num = (8 * (loss({**w, y: w[y] + h * way}) - loss({**w, y: w[y] - h * way}))
               - (loss({**w, y: w[y] + 2 * h * way}) - loss({**w, y: w[y] - 2 * h * way}))) / (12 * h)
        have = float((got["d" + y].cpu().double() * way).sum())
        size = float(got["d" + y].cpu().double().norm() * way.norm())
        assert abs(num - have) <= 1e-5 * size + 1e-7 * (1 + abs(num)), y


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("scale,far", [(1.0, 60.0), (20.0, 3.0), (0.0, 1.0), (-0.2, 1.0)])
def test_scores_of_any_size(qd, scale, far, dt):
    """Scores of thousands, all equal ones and a negative scale: the softmax's maximum is taken off first."""
    x = win_inputs(1, 150, 0, 2, 1, 64, dt, 3)
    x["q"] = (far * x["q"].float()).to(dt)
    c, w = cu(x), wide(x)
    o, lse = qd.win_attn_fwd(c["q"], c["k"], c["v"], window=50, sinks=2, scale=scale)
    want, z = ref.win_fwd(w["q"], w["k"], w["v"], 50, 2, scale)
    # a score of size s is a sum of fp32 products, off by up to 2^-24 sqrt(d) s, as is its exponent's: it moves
    # each probability by that
    s = float((scale * w["q"].abs()).abs().max() * w["k"].abs().max() * 8)
    off = 2.0 ** -24 * 8 * 8 * s
    mag, _ = ref.win_fwd(w["q"], w["k"], w["v"].abs(), 50, 2, scale)
    err = (o.cpu().double() - want).abs()
    assert (err <= (2 * HALF if dt == BF16 else 0) * mag + (2 * off + 1e-5) * (mag + want.abs().max())).all()
    assert ((lse.cpu().double() - z).abs() <= off + 1e-5 * (1 + z.abs())).all()


def bwd_terms(q, k, v, dO, window, sinks, scale):
    """For dq, dk, dv of one sequence [T,H,d]: the sum over the terms of what a relative error of each probability can move
    (D among it: the sum of all of the row's), in units of that error."""
    r = q.shape[1] // k.shape[1]
    kr, vr = (t.repeat_interleave(r, 1).abs() for t in (k, v))
    P, _ = ref.win_probs(q, k, window, sinks, scale)
    dP = torch.einsum("thd,shd->hts", dO.abs(), vr)
    dS = P * (dP + (P * dP).sum(-1, keepdim=True))
    fold = lambda t: t.unflatten(1, (-1, r)).sum(2)
    return {"dq": abs(scale) * torch.einsum("hts,shd->thd", dS, kr), "dk": fold(abs(scale) * torch.einsum("hts,thd->shd", dS, q.abs())),
            "dv": fold(torch.einsum("hts,thd->shd", P, dO.abs()))}


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("scale,far", [(1.0, 60.0), (20.0, 3.0), (0.0, 1.0), (-0.2, 1.0)])
@pytest.mark.parametrize("T,H,window,sinks", [(150, 2, 50, 2), (700, 2, 50, 5), (400, 8, 1 << 30, 0)])
def test_gradients_with_scores_of_any_size(qd, T, H, window, sinks, scale, far, dt):
    """As above for the backward: one walk a key tile, sinks in slices, walks in pieces."""
    d = 64
    x = win_inputs(1, T, 0, H, 1, d, dt, 3)
    x["q"] = (far * x["q"].float()).to(dt)
    c, w, kw = cu(x), wide(x), {"window": window, "sinks": sinks, "scale": scale}
    if T > 150:                                         # parts beside the rows' D
        assert qd.win_attn_bwd_workspace_bytes(1, T, 0, H, 1, d, window, sinks, qd.QD_BF16 if dt == BF16 else qd.QD_F32) > 4 * T * H + 256
    o, lse = qd.win_attn_fwd(c["q"], c["k"], c["v"], **kw)
    got = qd.win_attn_bwd(c["q"], c["k"], c["v"], o, lse, c["dO"], **kw)
    want, mag = ref.win_bwd(w["q"], w["k"], w["v"], w["dO"], window, sinks, scale)
    terms = bwd_terms(*(w[y][0] for y in ("q", "k", "v", "dO")), window, sinks, scale)
    # a score is a sum of 64 products, whose 64 roundings of 2^-24 of the sum of their sizes have random signs; a
    # probability's exponent has its own, the one in lse, and lse's own rounding and product, each no larger
    size = abs(scale) * torch.einsum("thd,sd->hts", w["q"][0].abs(), w["k"][0, :, 0].abs()).max()
    off = 3 * 8 * 2.0 ** -24 * float(size)
    for y in want:
        g, m = got[y].cpu().double(), mag[y].abs()
        assert torch.isfinite(g).all(), y
        # roundings to bf16 as everywhere here: the probability's gradient, the o that enters it, the output
        over = (g - want[y]).abs() - (3 * HALF if dt == BF16 else 0) * m - (off + 1e-5) * terms[y][None] - 1e-5 * (m + want[y].abs().max())
        assert over.max() <= 0, (y, float(over.max()))
        if scale == 0 and y != "dv":
            assert (g == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [False, True])
def test_keys_beyond_what_stays_in_l2(qd, lens):
    """A batch whose windows' keys are more than 64 MB takes its query blocks in another order than its sequences alone do:
    the same bits."""
    B, T, past, H, d, window, sinks = 16, 640, 33, 16, 128, 600, 4
    g = torch.Generator("cuda").manual_seed(7)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=BF16)
    q, k, v, dO = r(B, T, H, d), r(B, past + T, H, d), r(B, past + T, H, d), r(B, T, H, d)
    assert 4 * B * H * d * window > 64e6 > 4 * H * d * window
    n = torch.randint(0, T + 1, (B,), dtype=torch.int32, device="cuda", generator=g) if lens else None
    kw = {"window": window, "sinks": sinks}
    o, lse = qd.win_attn_fwd(q, k, v, lens=n, **kw)
    got = qd.win_attn_bwd(q, k, v, o, lse, dO, lens=n, **kw)
    for b in range(B):
        one, m = (lambda t: t[b:b + 1]), None if n is None else n[b:b + 1]
        o1, lse1 = qd.win_attn_fwd(one(q), one(k), one(v), lens=m if m is None else m.clone(), **kw)
        assert torch.equal(o1, one(o)) and torch.equal(lse1, one(lse))
        r1 = qd.win_attn_bwd(one(q), one(k), one(v), o1, lse1, one(dO), lens=m if m is None else m.clone(), **kw)
        assert torch.equal(r1["dq"], one(got["dq"]))
        for y in ("dk", "dv"):                          # (walks may be cut otherwise: sums in fp32, rounded once)
            a, z = one(got[y]).float(), r1[y].float()
            assert (a - z).abs().max() <= 2 * HALF * z.abs().max()
            assert (a - z).norm() <= 1e-3 * z.norm()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("N,H,Hkv,d,window,sinks", [(1, 1, 1, 8, 1, 0), (3, 4, 2, 128, 33, 4), (2, 16, 1, 64, 200, 1),
                                                    (5, 6, 6, 72, 5, 0), (2, 20, 1, 128, 130, 3), (1, 4, 2, 128, 3000, 4),
                                                    (40, 8, 2, 128, 70, 2)])
def test_windowed_attention_step(qd, N, H, Hkv, d, window, sinks, dt):
    """Every stage of a cache: its first token, not yet full, just full, wrapped, far on, idle.  Slots not in
    use hold NaN."""
    slots = window + sinks
    g = torch.Generator().manual_seed(d + window)
    stages = [0, slots // 2, slots - 1, slots, slots + 1, slots + 3 * window - 1, 2000000000, -1]
    for first in range(0, len(stages), N) if N < len(stages) else [0]:
        pos = torch.tensor([stages[(first + i) % len(stages)] for i in range(N)], dtype=torch.int32)
        r = lambda *s: torch.randn(*s, generator=g).to(dt)
        K, V, q, k, v = r(N, slots, Hkv, d), r(N, slots, Hkv, d), r(N, H, d), r(N, Hkv, d), r(N, Hkv, d)
        for b, p in enumerate(pos.tolist()):
            K[b, max(p, 0):] = NAN                          # (a full cache: nothing)
            V[b, max(p, 0):] = NAN
        Kc, Vc = K.cuda(), V.cuda()
        o = qd.win_attn_step(Kc, Vc, pos.cuda(), q.cuda(), k.cuda(), v.cuda(), window=window, sinks=sinks)
        for b, p in enumerate(pos.tolist()):
            if p < 0:
                assert (o[b] == 0).all()
                held = 0
            else:
                at = p if p < slots else sinks + (p - sinks) % window
                K[b, at], V[b, at] = k[b], v[b]
                held = min(p + 1, slots)
                one = [t.double() for t in (q[b][None, None], K[b, :held][None], V[b, :held][None])]
                want = ref.win_fwd(*one, slots, 0, 1 / math.sqrt(d))[0][0, 0]
                mag = ref.win_fwd(one[0], one[1], one[2].abs(), slots, 0, 1 / math.sqrt(d))[0][0, 0]
                close(o[b], want, mag, f"o at {p}", 2)
        same = lambda a, b: torch.equal(torch.nan_to_num(a.float(), nan=99.0), torch.nan_to_num(b.cpu().float(), nan=99.0))
        assert same(K, Kc) and same(V, Vc)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("window,sinks,past", [(20, 3, 0), (1, 0, 0), (64, 0, 9), (500, 5, 0), (7, 40, 50)])
def test_a_cache_from_a_prompt_goes_on_as_the_prompt_would(qd, window, sinks, past, dt):
    """Prompts of different lengths, padded; the caches filled from them; then tokens, each at its own position."""
    B, T, more, H, Hkv, d = 4, 100, 12, 4, 2, 64
    g = torch.Generator().manual_seed(window)
    lens = torch.tensor([100, 37, 0, 2], dtype=torch.int32)
    r = lambda *s: torch.randn(*s, generator=g).to(dt)
    q, k, v = r(B, T + more, H, d), r(B, past + T + more, Hkv, d), r(B, past + T + more, Hkv, d)
    pad = lambda t: poison(t[:, :past + T].clone(), lens, past).cuda()
    kw = {"window": window, "sinks": sinks}
    qp = poison(q[:, :T].clone(), lens).cuda()
    o, _ = qd.win_attn_fwd(qp, pad(k), pad(v), lens=lens.cuda(), **kw)
    K = torch.full((B, window + sinks, Hkv, d), 7.0, dtype=dt).cuda()
    V = K.clone()
    qd.win_attn_fill(K, V, pad(k), pad(v), lens=lens.cuda(), past=past, **kw)
    for b, n in enumerate(lens.tolist()):
        assert (K[b, past + n:] == 7).all() and (V[b, past + n:] == 7).all()
    pos = (lens + past).cuda()
    steps = []
    for t in range(more):
        at = [int(n) + t for n in lens]
        pick = lambda x, off: torch.stack([x[b, off + a] for b, a in enumerate(at)]).cuda()
        steps.append(qd.win_attn_step(K, V, pos, pick(q, 0), pick(k, past), pick(v, past), **kw))
        pos += 1
    for b, n in enumerate(lens.tolist()):
        one = [t[b:b + 1, :m].double() for t, m in ((q, n + more), (k, past + n + more), (v, past + n + more))]
        want, _ = ref.win_fwd(*one, window, sinks, 1 / math.sqrt(d))
        mag, _ = ref.win_fwd(one[0], one[1], one[2].abs(), window, sinks, 1 / math.sqrt(d))
        close(torch.cat([o[b, :n], torch.stack([s[b] for s in steps])]), want[0], mag[0], "o", 2)


@pytest.mark.gpu
@pytest.mark.parametrize("heads,window,sinks,T", [(1 << 24, 1, 0, 2), ((1 << 24) + 8, 1, 0, 1), (16, 1 << 20, 40, (1 << 20) + 100)])
def test_a_cache_whose_rows_or_whole_pass_32_bits(qd, heads, window, sinks, T):
    """A token's keys of 2^31 elements and more, and a cache of so many."""
    d, slots = 128, window + sinks
    K, V = (torch.zeros(1, slots, heads, d, dtype=BF16, device="cuda") for _ in range(2))
    k, v = (torch.randn(1, T, heads, d, dtype=BF16, device="cuda", generator=torch.Generator("cuda").manual_seed(i)) for i in range(2))
    qd.win_attn_fill(K, V, k, v, window=window, sinks=sinks)
    for cache, new in ((K, k), (V, v)):
        for p in range(T) if T < 4 else (0, sinks - 1, T - slots + sinks, T - 100, T - 1):
            at = p if p < slots else sinks + (p - sinks) % window
            if p < sinks or p >= T - window:
                assert torch.equal(cache[0, at], new[0, p]), p
    if T > 4:                                           # every slot behind the sinks: the ring, turned
        turned = torch.roll(k[0, T - window:], (T - sinks) % window, 0)
        assert torch.equal(K[0, sinks:], turned)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16])
def test_a_prompt_in_pieces(qd, dt):
    """A piece's kept keys are the sinks' and the last window - 1."""
    T, H, Hkv, d, window, sinks = 301, 2, 1, 64, 45, 6
    x = win_inputs(1, T, 0, H, Hkv, d, dt, 77)
    c, w = cu(x), wide(x)
    outs, at = [], 0
    for n in (60, 1, 130, 110):
        first = max(sinks, at - (window - 1))
        cut = lambda t: torch.cat([t[:, :min(sinks, at)], t[:, first:at], t[:, at:at + n]], 1).contiguous()
        outs.append(qd.win_attn_fwd(c["q"][:, at:at + n].contiguous(), cut(c["k"]), cut(c["v"]), window=window, sinks=sinks)[0])
        at += n
    want, _ = ref.win_fwd(w["q"], w["k"], w["v"], window, sinks, 1 / math.sqrt(d))
    mag, _ = ref.win_fwd(w["q"], w["k"], w["v"].abs(), window, sinks, 1 / math.sqrt(d))
    close(torch.cat(outs, 1), want, mag, "o", 2)


@pytest.mark.gpu
@pytest.mark.parametrize("dt,tol", [(F32, 1e-5), (BF16, 5e-3)])
def test_sinks_of_a_long_sequence(qd, dt, tol):
    """The sinks' gradients are sums over every query; a window a small part of the sequence.  (bf16: errors of
    random signs, of one rounding's relative size, from up to four independent roundings.)"""
    B, T, H, Hkv, d, window, sinks = 1, 3000, 4, 2, 128, 300, 5
    x = win_inputs(B, T, 0, H, Hkv, d, dt, 4)
    x["dO"] = (x["dO"].float() + 0.5).to(dt)                # so that the sums do not average out
    c = cu(x)
    kw = {"window": window, "sinks": sinks}
    o, lse = qd.win_attn_fwd(c["q"], c["k"], c["v"], **kw)
    got = qd.win_attn_bwd(c["q"], c["k"], c["v"], o, lse, c["dO"], **kw)
    leaf = [c[y][0].double().requires_grad_() for y in "qkv"]
    mask = ref.seen(T, 0, window, sinks).cuda()
    s = torch.einsum("thd,shd->hts", leaf[0], leaf[1].repeat_interleave(2, 1)) / math.sqrt(d)
    P = torch.softmax(s.masked_fill(~mask, -math.inf), -1)
    want = torch.einsum("hts,shd->thd", P, leaf[2].repeat_interleave(2, 1))
    grads = torch.autograd.grad((want * c["dO"][0].double()).sum(), leaf)
    rel = lambda a, b: float((a.double() - b.detach()).norm() / b.detach().norm())
    assert rel(o[0], want) <= tol
    for y, b in zip("qkv", grads):
        assert rel(got["d" + y][0], b) <= tol, y
        if y != "q":
            assert rel(got["d" + y][0, :sinks], b[:sinks]) <= tol, y


# ------------------------------------------------------------------ arrays beyond 2^31 elements

def _first_and_last(small, n):
    """[2, ...] as the first and the last of n, zeros between."""
    big = torch.zeros(n, *small.shape[1:], dtype=small.dtype, device="cuda")
    big[0], big[-1] = small[0], small[1]
    return big


def _same_at_the_ends(big, small):
    assert torch.equal(big[0], small[0]) and torch.equal(big[-1], small[1])


@pytest.mark.gpu
@pytest.mark.parametrize("dt,H,d", [(BF16, 16, 128), (F32, 128, 16)])
def test_linear_attention_of_arrays_beyond_32_bits(qd, dt, H, d):
    """Sequences that are not cut: the first and the last of a batch as in a batch of two, nothing in the others."""
    B, T = 2049, 512
    assert B * T * H * d > 1 << 31
    c = cu(lin_inputs(2, T, H, d, d, dt, 1, "token"))
    x = {y: _first_and_last(c[y], B) for y in ("q", "k", "v", "g", "S0", "dO", "dS_final")}
    o, S = qd.lin_attn_fwd(x["q"], x["k"], x["v"], x["g"], x["S0"])
    want = qd.lin_attn_fwd(c["q"], c["k"], c["v"], c["g"], c["S0"])
    _same_at_the_ends(o, want[0])
    _same_at_the_ends(S, want[1])
    assert not o[1:-1].any() and not S[1:-1].any()
    del o, S
    got = qd.lin_attn_bwd(x["q"], x["k"], x["v"], x["g"], x["S0"], x["dO"], x["dS_final"])
    want = qd.lin_attn_bwd(c["q"], c["k"], c["v"], c["g"], c["S0"], c["dO"], c["dS_final"])
    for y in want:
        _same_at_the_ends(got[y], want[y])
        assert not got[y][1:-1].any()


@pytest.mark.gpu
@pytest.mark.parametrize("dt,H,d,sinks", [(BF16, 16, 128, 3), (F32, 128, 16, 0)])
def test_windowed_attention_of_arrays_beyond_32_bits(qd, dt, H, d, sinks):
    B, T, kw = 2049, 512, {"window": 100, "sinks": sinks}
    c = cu(win_inputs(2, T, 0, H, H, d, dt, 1))
    x = {y: _first_and_last(c[y], B) for y in ("q", "k", "v", "dO")}
    o, lse = qd.win_attn_fwd(x["q"], x["k"], x["v"], **kw)
    o2, lse2 = qd.win_attn_fwd(c["q"], c["k"], c["v"], **kw)
    _same_at_the_ends(o, o2)
    _same_at_the_ends(lse, lse2)
    assert not o[1:-1].any()
    got = qd.win_attn_bwd(x["q"], x["k"], x["v"], o, lse, x["dO"], **kw)
    want = qd.win_attn_bwd(c["q"], c["k"], c["v"], o2, lse2, c["dO"], **kw)
    for y in want:
        _same_at_the_ends(got[y], want[y])
        assert not got[y][1:-1].any()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16])
def test_steps_of_states_and_caches_beyond_32_bits(qd, dt):
    N, H, d = 8193, 16, 128
    c = cu(lin_inputs(2, 1, H, d, d, dt, 1, "token"))
    x = {y: _first_and_last(c[y] if y == "S0" else c[y][:, 0].contiguous(), N) for y in ("q", "k", "v", "g", "S0")}
    assert x["S0"].numel() > 1 << 31
    o = qd.lin_attn_step(x["S0"], x["q"], x["k"], x["v"], x["g"])
    S = c["S0"].clone()
    _same_at_the_ends(o, qd.lin_attn_step(S, *(c[y][:, 0].contiguous() for y in ("q", "k", "v", "g"))))
    _same_at_the_ends(x["S0"], S)
    del x, o
    N, H, Hkv, window, sinks = 4, 8, 4, 1 << 20, 3
    g = torch.Generator("cuda").manual_seed(9)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=dt)
    K, V = (torch.zeros(N, window + sinks, Hkv, d, dtype=dt, device="cuda") for _ in range(2))
    assert K.numel() > 1 << 31
    K[-1], V[-1] = r(window + sinks, Hkv, d), r(window + sinks, Hkv, d)
    q, k, v = r(N, H, d), r(N, Hkv, d), r(N, Hkv, d)
    p = 5 * window + 77
    o = qd.win_attn_step(K, V, torch.full((N,), p, dtype=torch.int32, device="cuda"), q, k, v, window=window, sinks=sinks)
    at = sinks + (p - sinks) % window
    assert torch.equal(K[-1, at], k[-1]) and torch.equal(V[-1, at], v[-1]) and torch.equal(K[0, at], k[0])
    # relative L2 over a million keys: errors of random signs, of one rounding's size each (the probability's, the output's)
    for h in range(H):
        s = (K[-1, :, h // 2].double() @ q[-1, h].double()) / math.sqrt(d)
        want = torch.softmax(s, 0) @ V[-1, :, h // 2].double()
        rel = float((o[-1, h].double() - want).norm() / want.norm())
        assert rel <= (5e-3 if dt == BF16 else 1e-5), (h, rel)


# ------------------------------------------------------------------ how they are called

def _calls(qd):
    """Every entry point on small inputs of both types: a function of the inputs that returns its outputs."""
    def lin(dt):
        d = cu(lin_inputs(2, 150, 2, 128, 64, dt, 1, "token"))
        yield d, lambda d: list(qd.lin_attn_fwd(d["q"], d["k"], d["v"], d["g"], d["S0"]))
        yield d, lambda d: list(qd.lin_attn_bwd(d["q"], d["k"], d["v"], d["g"], d["S0"], d["dO"], d["dS_final"]).values())
        one = {x: (t if x == "S0" or t is None else t[:, 0].contiguous()) for x, t in d.items() if x != "lens"}
        yield one, lambda d: (lambda S: [qd.lin_attn_step(S, d["q"], d["k"], d["v"], d["g"]), S])(d["S0"].clone())
        long = cu(lin_inputs(1, 3000, 1, 64, 64, dt, 1, "token"))
        yield long, lambda d: list(qd.lin_attn_fwd(d["q"], d["k"], d["v"], d["g"], d["S0"]))
        yield long, lambda d: list(qd.lin_attn_bwd(d["q"], d["k"], d["v"], d["g"], d["S0"], d["dO"], d["dS_final"]).values())

    def win(dt):
        d = cu(win_inputs(2, 400, 0, 4, 2, 128, dt, 2))
        kw = {"window": 60, "sinks": 3}
        yield d, lambda d: list(qd.win_attn_fwd(d["q"], d["k"], d["v"], **kw))
        o, lse = qd.win_attn_fwd(d["q"], d["k"], d["v"], **kw)
        yield {**d, "o": o, "lse": lse}, lambda d: list(qd.win_attn_bwd(d["q"], d["k"], d["v"], d["o"], d["lse"], d["dO"], **kw).values())
        e = cu({"K": torch.randn(2, 2003, 2, 128).to(dt), "V": torch.randn(2, 2003, 2, 128).to(dt),
                "pos": torch.tensor([5000, 900], dtype=torch.int32), "q": torch.randn(2, 4, 128).to(dt),
                "k": torch.randn(2, 2, 128).to(dt), "v": torch.randn(2, 2, 128).to(dt)})

        def step(e):
            K, V = e["K"].clone(), e["V"].clone()
            return [qd.win_attn_step(K, V, e["pos"], e["q"], e["k"], e["v"], window=2000, sinks=3), K, V]
        yield e, step

        def fill(d):
            K = torch.zeros(2, 63, 2, 128, dtype=dt, device="cuda")
            V = torch.zeros_like(K)
            qd.win_attn_fill(K, V, d["k"], d["v"], window=60, sinks=3)
            return [K, V]
        yield d, fill

    for dt in (F32, BF16):
        yield from lin(dt)
        yield from win(dt)


@pytest.mark.gpu
def test_the_same_inputs_give_the_same_bits_on_any_stream(qd):
    for d, call in _calls(qd):
        first = call(d)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            again = call(d)
        third = call(d)
        torch.cuda.synchronize()
        for a, b, c in zip(first, again, third):
            assert (a is None and b is None) or (torch.equal(a, b) and torch.equal(a, c))


@pytest.mark.gpu
def test_calls_on_two_streams_at_once(qd):
    """Every call on one stream while the others run on another: the same bits as alone."""
    calls = list(_calls(qd))
    alone = [call(d) for d, call in calls]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for i in range(len(calls)):                     # (the second stream takes them from the other end)
            for s, at, out in zip(streams, (i, len(calls) - 1 - i), got):
                with torch.cuda.stream(s):
                    out.append((at, calls[at][1](calls[at][0])))
    torch.cuda.synchronize()
    for at, out in got[0] + got[1]:
        for a, b in zip(out, alone[at]):
            assert (a is None and b is None) or torch.equal(a, b)
    assert qd.qd_device_status() == 0


@pytest.mark.gpu
def test_captured_and_replayed(qd):
    """A call captured into a graph and replayed on new inputs gives what a direct call gives."""
    for d, call in _calls(qd):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            call(d)
            with torch.cuda.graph(graph, stream=side):
                out = call(d)
        torch.cuda.current_stream().wait_stream(side)
        for x in ("q", "dO"):
            if d.get(x) is not None:
                d[x].mul_(0.5)
        graph.replay()
        want = call(d)
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert (a is None and b is None) or torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16])
def test_a_workspace_may_hold_anything_and_be_shared(qd, dt):
    """Two graphs of each call with one workspace between them, which held NaN before: as with workspaces of their own."""
    d = cu(lin_inputs(2, 700, 2, 128, 64, dt, 1, "token"))
    e = cu(win_inputs(2, 400, 0, 4, 2, 128, dt, 2))
    kw = {"window": 60, "sinks": 3}
    o, lse = qd.win_attn_fwd(e["q"], e["k"], e["v"], **kw)
    K, V = torch.randn(2, 2003, 2, 128).to(dt).cuda(), torch.randn(2, 2003, 2, 128).to(dt).cuda()
    pos = torch.tensor([5000, 900], dtype=torch.int32).cuda()
    one = lambda t: t[:, 5].contiguous()
    calls = [
        lambda ws: qd.lin_attn_fwd(d["q"], d["k"], d["v"], d["g"], d["S0"], workspace=ws),
        lambda ws: qd.lin_attn_bwd(d["q"], d["k"], d["v"], d["g"], d["S0"], d["dO"], d["dS_final"], workspace=ws).values(),
        lambda ws: qd.win_attn_bwd(e["q"], e["k"], e["v"], o, lse, e["dO"], **kw, workspace=ws).values(),
        lambda ws: [qd.win_attn_step(K, V, pos, one(e["q"]), one(e["k"]), one(e["v"]), window=2000, sinks=3, workspace=ws)],
    ]
    ws = torch.full((1 << 24,), NAN, device="cuda")
    want = [list(call(None)) for call in calls]
    graphs, outs = [], []
    for call in calls + calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(list(call(ws)))
        graphs.append(graph)
    for _ in range(2):
        ws.fill_(NAN)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for got, w in zip(outs, want + want):
            for a, b in zip(got, w):
                assert torch.equal(a, b)


@pytest.mark.gpu
def test_nothing_to_do(qd):
    """No tokens, no sequences: states carried over, gradients of what is not seen 0."""
    S0 = torch.randn(2, 3, 16, 8, device="cuda")
    z = lambda *s, dt=BF16: torch.zeros(*s, dtype=dt, device="cuda")
    o, S = qd.lin_attn_fwd(z(2, 0, 3, 8), z(2, 0, 3, 8), z(2, 0, 3, 16), None, S0)
    assert o.shape == (2, 0, 3, 16) and torch.equal(S, S0)
    r = qd.lin_attn_bwd(z(2, 0, 3, 8), z(2, 0, 3, 8), z(2, 0, 3, 16), None, S0, z(2, 0, 3, 16), S0)
    assert torch.equal(r["dS0"], S0)
    o, S = qd.lin_attn_fwd(z(0, 5, 3, 8), z(0, 5, 3, 8), z(0, 5, 3, 16))
    assert o.shape == (0, 5, 3, 16) and S.shape == (0, 3, 16, 8)
    o, lse = qd.win_attn_fwd(z(2, 0, 4, 8), z(2, 5, 2, 8), z(2, 5, 2, 8), window=3)
    assert o.shape == (2, 0, 4, 8) and lse.shape == (2, 0, 4)
    r = qd.win_attn_bwd(z(2, 0, 4, 8), z(2, 5, 2, 8), z(2, 5, 2, 8), o, lse, o, window=3)
    assert r["dk"].shape == (2, 5, 2, 8) and (r["dk"] == 0).all() and (r["dv"] == 0).all()
    assert qd.win_attn_step(z(0, 4, 2, 8), z(0, 4, 2, 8), z(0, dt=torch.int32), z(0, 4, 8), z(0, 2, 8), z(0, 2, 8),
                            window=4).shape == (0, 4, 8)


# ------------------------------------------------------------------ refusals (on the CPU)

P256 = ctypes.c_void_p(256)


def _c_calls(qd, lib):
    """name -> call(pointer overrides by place, sizes overrides by name) with valid arguments otherwise."""
    p, bf = P256, qd.QD_BF16

    def make(fn, npointers, names, sizes, tail):
        def call(at=None, ptr=None, ws=True, **over):
            ps = [p] * npointers
            if at is not None:
                ps[at] = ptr
            vals = {**sizes, **over}
            t = list(tail)
            if t and t[0] == "ws":
                t = [p, 1 << 40, None] if ws else [None, 0, None]
            return getattr(lib, fn)(*ps, *(vals[n] for n in names), *t)
        return call
    lin = {"B": 1, "T": 8, "H": 2, "dk": 64, "dv": 64, "tok": 1, "dt": bf}
    win = {"B": 1, "T": 8, "past": 0, "H": 4, "Hkv": 2, "d": 64, "window": 4, "sinks": 1, "scale": 0.1, "dt": bf}
    step = {x: v for x, v in win.items() if x not in ("T", "past")}
    fill = {x: v for x, v in win.items() if x not in ("H", "scale")}
    return {
        "lin_attn_fwd": make("lin_attn_fwd", 8, list(lin), lin, ["ws"]),
        "lin_attn_step": make("lin_attn_step", 6, ["B", "H", "dk", "dv", "tok", "dt"], lin, [None]),
        "lin_attn_bwd": make("lin_attn_bwd", 13, list(lin), lin, ["ws"]),
        "win_attn_fwd": make("win_attn_fwd", 6, list(win), win, [None]),
        "win_attn_bwd": make("win_attn_bwd", 10, list(win), win, ["ws"]),
        "win_attn_step": make("win_attn_step", 7, list(step), step, ["ws"]),
        "win_attn_fill": make("win_attn_fill", 5, list(fill), fill, [None]),
    }


OPTIONAL = {"lin_attn_fwd": (3, 4, 5, 7), "lin_attn_step": (4,), "lin_attn_bwd": (3, 4, 5, 7, 11, 12), "win_attn_fwd": (3, 5),
            "win_attn_bwd": (6,), "win_attn_step": (), "win_attn_fill": (4,)}
POINTERS = {"lin_attn_fwd": 8, "lin_attn_step": 6, "lin_attn_bwd": 13, "win_attn_fwd": 6, "win_attn_bwd": 10, "win_attn_step": 7,
            "win_attn_fill": 5}


@pytest.mark.parametrize("fn", sorted(POINTERS))
def test_pointers_are_checked(qd, fn):
    call = _c_calls(qd, qd.load_library())[fn]
    for i in range(POINTERS[fn]):
        assert call(i, ctypes.c_void_p(264)) == qd.QD_ERR_ARG and "aligned" in qd.qd_last_error()
        if i not in OPTIONAL[fn]:
            assert call(i, None) == qd.QD_ERR_ARG and "NULL" in qd.qd_last_error() and fn in qd.qd_last_error()


@pytest.mark.parametrize("fn,over,status", [
    *[(f, {"B": -1}, 1) for f in sorted(POINTERS)],
    *[(f, {"dt": 5}, 2) for f in sorted(POINTERS)],
    *[(f, {"dk": x}, 2) for f in ("lin_attn_fwd", "lin_attn_step", "lin_attn_bwd") for x in (0, 12, 136)],
    *[(f, {"dv": x}, 2) for f in ("lin_attn_fwd", "lin_attn_step", "lin_attn_bwd") for x in (4, 65, 256)],
    *[(f, {"d": x}, 2) for f in ("win_attn_fwd", "win_attn_bwd", "win_attn_step", "win_attn_fill") for x in (0, 20, 136)],
    *[(f, {"window": 0}, 1) for f in ("win_attn_fwd", "win_attn_bwd", "win_attn_step", "win_attn_fill")],
    *[(f, {"sinks": -1}, 1) for f in ("win_attn_fwd", "win_attn_bwd", "win_attn_step", "win_attn_fill")],
    *[(f, {"Hkv": 3}, 1) for f in ("win_attn_fwd", "win_attn_bwd", "win_attn_step")],
    *[(f, {"past": -1}, 1) for f in ("win_attn_fwd", "win_attn_bwd", "win_attn_fill")],
    *[(f, {"T": 2 ** 31 - 1}, 1) for f in ("lin_attn_fwd", "lin_attn_bwd", "win_attn_fwd", "win_attn_bwd", "win_attn_fill")],
    ("win_attn_fwd", {"T": 2 ** 30, "past": 2 ** 30}, 1),
    ("win_attn_step", {"window": 2 ** 31 - 1, "sinks": 2 ** 31 - 1}, 1),
    ("win_attn_fill", {"window": 2 ** 30, "sinks": 2 ** 30, "Hkv": 64}, 1),
    ("lin_attn_fwd", {"B": 2 ** 20, "H": 2 ** 20}, 1),
    ("lin_attn_step", {"B": 2 ** 20, "H": 2 ** 12}, 1),
])
def test_sizes_are_checked(qd, fn, over, status):
    assert _c_calls(qd, qd.load_library())[fn](**over) == status
    assert fn in qd.qd_last_error()


@pytest.mark.parametrize("fn", ["lin_attn_fwd", "lin_attn_bwd", "win_attn_bwd", "win_attn_step"])
def test_a_missing_workspace_is_refused(qd, fn):
    lib = qd.load_library()
    need = {"lin_attn_fwd": lambda: lib.lin_attn_workspace_bytes(1, 30000, 2, 64, 64, qd.QD_F32),
            "lin_attn_bwd": lambda: lib.lin_attn_bwd_workspace_bytes(1, 30000, 2, 64, 64, qd.QD_F32),
            "win_attn_bwd": lambda: lib.win_attn_bwd_workspace_bytes(1, 30000, 0, 4, 2, 64, 4, 1, qd.QD_F32),
            "win_attn_step": lambda: lib.win_attn_step_workspace_bytes(1, 4, 2, 64, 30000, 1, qd.QD_F32)}[fn]()
    call = _c_calls(qd, lib)[fn]
    over = {"window": 30000} if fn == "win_attn_step" else {"T": 30000}
    if need:
        assert call(ws=False, dt=qd.QD_F32, **over) == qd.QD_ERR_WORKSPACE
        assert f"{need} bytes" in qd.qd_last_error()


def test_a_gradient_of_decays_that_have_none_is_refused(qd):
    lib = qd.load_library()
    call = _c_calls(qd, lib)["lin_attn_bwd"]
    assert call(tok=0) == qd.QD_ERR_ARG and "dg" in qd.qd_last_error()
    assert call(3, None) == qd.QD_ERR_ARG and "dg" in qd.qd_last_error()


def test_empty_calls_need_no_pointers(qd):
    lib, n, bf = qd.load_library(), None, 1
    assert lib.lin_attn_fwd(*[n] * 8, 0, 8, 2, 64, 64, 1, bf, n, 0, n) == 0
    assert lib.lin_attn_step(*[n] * 6, 0, 2, 64, 64, 1, bf, n) == 0
    assert lib.lin_attn_bwd(*[n] * 13, 0, 8, 2, 64, 64, 0, bf, n, 0, n) == 0
    assert lib.win_attn_fwd(*[n] * 6, 0, 8, 0, 4, 2, 64, 4, 1, 0.1, bf, n) == 0
    assert lib.win_attn_bwd(*[n] * 10, 0, 8, 0, 4, 2, 64, 4, 1, 0.1, bf, n, 0, n) == 0
    assert lib.win_attn_step(*[n] * 7, 0, 4, 2, 64, 4, 1, 0.1, bf, n, 0, n) == 0
    assert lib.win_attn_fill(*[n] * 5, 0, 8, 0, 2, 64, 4, 1, bf, n) == 0


def test_workspaces_of_refused_sizes_are_none(qd):
    lib, bf = qd.load_library(), 1
    assert lib.lin_attn_workspace_bytes(-1, 8, 2, 64, 64, bf) == 0 and lib.lin_attn_workspace_bytes(1, 8, 2, 65, 64, bf) == 0
    assert lib.lin_attn_bwd_workspace_bytes(1, 2 ** 31 - 1, 2, 64, 64, bf) == 0
    assert lib.win_attn_bwd_workspace_bytes(1, 8, 0, 4, 3, 64, 4, 1, bf) == 0
    assert lib.win_attn_step_workspace_bytes(1, 4, 2, 64, 0, 1, bf) == 0


def test_the_binding_refuses(qd):
    """Wrong shapes, types and host tensors, before any launch."""
    x = lambda *s, dt=BF16: torch.zeros(*s, dtype=dt)
    q, v, S = x(2, 8, 3, 64), x(2, 8, 3, 64), x(2, 3, 64, 64, dt=F32)
    cache = x(2, 10, 3, 64)
    calls = [lambda **k: qd.lin_attn_fwd(k.get("q", q), q, v, k.get("g"), S), lambda **k: qd.lin_attn_bwd(k.get("q", q), q, v, k.get("g"), S, v),
             lambda **k: qd.lin_attn_step(S, k.get("q", q)[:, 0], q[:, 0], v[:, 0], None),
             lambda **k: qd.win_attn_fwd(k.get("q", q), q, v, window=4), lambda **k: qd.win_attn_bwd(k.get("q", q), q, v, q, x(2, 8, 3, dt=F32), q),
             lambda **k: qd.win_attn_step(cache, cache, x(2, dt=torch.int32), k.get("q", q)[:, 0], q[:, 0], v[:, 0], window=8, sinks=2),
             lambda **k: qd.win_attn_fill(cache, cache, k.get("q", q), v, window=8, sinks=2)]
    for call in calls:
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError):
        qd.win_attn_step(cache, cache, x(2, dt=torch.int32), q[:, 0], q[:, 0], v[:, 0], window=9, sinks=2)
    with pytest.raises(ValueError):
        qd.win_attn_fwd(q, q[:, :5], v[:, :5], window=4)
    with pytest.raises(ValueError):
        qd.win_attn_fill(cache, cache, q, v, window=8, sinks=2, past=9)
    with pytest.raises(ValueError):
        qd.win_attn_fwd(q[0], q[0], v[0], window=4)


@pytest.mark.parametrize("form,lead,wrong", [
    ("fwd", "B, T", (100,)), ("fwd", "B, T", (2, 3, 5)), ("fwd", "B, T", ()),
    ("bwd", "B, T", (100,)), ("bwd", "B, T", (2, 3, 5)),
    ("step", "N", (2, 5)), ("step", "N", ()),
])
def test_linear_attention_refuses_other_ranks(qd, form, lead, wrong):
    """One sequence without its batch dimension, several leading dimensions: sizes taken from them would be others'."""
    q, S = torch.zeros(*wrong, 8, 64, dtype=BF16), torch.zeros(2, 8, 64, 64)
    call = {"fwd": lambda: qd.lin_attn_fwd(q, q, q), "bwd": lambda: qd.lin_attn_bwd(q, q, q, None, None, q),
            "step": lambda: qd.lin_attn_step(S, q, q, q)}[form]
    with pytest.raises(ValueError, match=rf"expected \[{lead}, H, d\]"):
        call()


@pytest.mark.gpu
def test_the_binding_refuses_on_the_gpu(qd):
    x = lambda *s, dt=BF16: torch.zeros(*s, dtype=dt, device="cuda")
    q, S = x(2, 8, 3, 64), x(2, 3, 64, 64, dt=F32)
    for bad in (lambda: qd.lin_attn_fwd(q, q, q.float()), lambda: qd.lin_attn_fwd(q, q, q, x(3)),           # types
                lambda: qd.lin_attn_fwd(q, q, q, x(2, 8, 3, dt=F32)), lambda: qd.lin_attn_fwd(q, q, q, None, S.half()),
                lambda: qd.win_attn_step(x(2, 4, 3, 64), x(2, 4, 3, 64), x(2, dt=torch.int64), q[:, 0].contiguous(),
                                         q[:, 0].contiguous(), q[:, 0].contiguous(), window=4)):
        with pytest.raises((TypeError, ValueError)):
            bad()
    for bad in (lambda: qd.lin_attn_fwd(q.transpose(1, 2), q, q), lambda: qd.win_attn_fwd(q[:, ::2], q, q, window=3),  # strides
                lambda: qd.lin_attn_fwd(q, q[:, :4].contiguous(), q), lambda: qd.win_attn_fwd(q, q, q[:, :, :2].contiguous()),
                lambda: qd.lin_attn_fwd(q, q, q, None, S[:1].contiguous())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ValueError, match="32 bits"):
        qd.win_attn_fwd(q, q, q, window=2 ** 31 - 1, sinks=2)
    with pytest.raises(qd.QDError):
        qd.lin_attn_fwd(x(1, 4, 2, 20), x(1, 4, 2, 20), x(1, 4, 2, 20))
