"""The example layer: the operators as a model uses them together (prompt, one token at a
time, gradients), against the same layer from their 64-bit definitions."""
import os
import sys

import pytest
import torch

import layer_reference as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

WIDTH, HEADS, DIM, N, RANK = 24, 3, 16, 16, 4


@pytest.fixture(scope="module")
def layer():
    from delta_rule_linear_qdelta_gb300 import build
    build.build()
    import state_space_layer as m
    return m.StateSpaceLayer(WIDTH, HEADS, DIM, N, rank=RANK, dtype=torch.float32)


def reference(p, h, lens=None):
    """The layer in 64 bits on the CPU, from the operators' definitions."""
    D = HEADS * DIM
    xz = h @ p["W_in"]
    x, _ = ref.conv_fwd(xz[..., :D], p["conv_w"], p["conv_b"], None, lens)
    dbc = x @ p["W_x"]
    dt, B, C = dbc.split([RANK, N, N], dim=-1)
    y, _ = ref.ssm_fwd(x, dt @ p["W_dt"], p["A"], B.unsqueeze(-2), C.unsqueeze(-2), p["skip"], p["delta_bias"], None, lens)
    rows = lambda t: t.view(*t.shape[:-1], HEADS, DIM)
    return ref.norm_fwd(rows(y), p["norm_w"], p["norm_b"], rows(xz[..., D:])).reshape(y.shape) @ p["W_out"]


def rel(a, b):
    return float((a.double().cpu() - b).norm() / b.norm())


def test_prompt_then_tokens_is_the_whole_sequence(layer):
    """Sequences of different lengths, padded; then each goes on from its own last token."""
    g = torch.Generator().manual_seed(3)
    lens, more = [20, 7, 0, 13], 5
    h = torch.randn(4, 20 + more, WIDTH, generator=g)
    padded = torch.full((4, 20, WIDTH), float("nan"))
    for b, n in enumerate(lens):
        padded[b, :n] = h[b, :n]
    _, state = layer.prompt(padded.cuda(), lens=torch.tensor(lens, dtype=torch.int32).cuda())
    p64 = {k: v.double().cpu() for k, v in layer.p.items()}
    whole = reference(p64, h.double())
    for t in range(more):
        tok = torch.stack([h[b, n + t] for b, n in enumerate(lens)])
        out = layer.step(tok.cuda(), state)
        want = torch.stack([whole[b, n + t] for b, n in enumerate(lens)])
        # fp32 throughout: the operators' 1e-5 through five products of up to 48 terms
        assert rel(out, want) <= 1e-4, t


def test_gradients_against_differences_of_the_definitions(layer):
    g = torch.Generator().manual_seed(4)
    h, wt = torch.randn(2, 12, WIDTH, generator=g), torch.randn(2, 12, WIDTH, generator=g)
    out, grads, dh = layer.grads(h.cuda(), lambda o: wt.cuda())
    p64 = {k: v.double().cpu() for k, v in layer.p.items()}
    assert rel(out, reference(p64, h.double())) <= 1e-4
    loss = lambda p, h: (reference(p, h) * wt.double()).sum()
    eps = 3e-5
    for k in list(p64) + ["h"]:
        base = h.double() if k == "h" else p64[k]
        way = torch.randn(base.shape, generator=g, dtype=torch.float64)
        at = lambda s: loss(p64, base + s * eps * way) if k == "h" else loss(p64 | {k: base + s * eps * way}, h.double())
        num = (8 * (at(1) - at(-1)) - (at(2) - at(-2))) / (12 * eps)
        got = (dh if k == "h" else grads[k]).double().cpu()
        # fp32 gradients: 1e-4 of the sum of the terms' magnitudes
        assert abs((got * way).sum() - num) <= 1e-4 * (got * way).abs().sum(), k
