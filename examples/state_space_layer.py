"""A state space layer from this package's operators, as it is trained and served.

    x, z    = split(h W_in)
    x       = SiLU(causal convolution of x)                    short_conv_*
    dt,B,C  = split(x W_x),  delta = dt W_dt
    y       = selective scan of x with delta, B, C             ssm_*
    out     = (group norm of y, gated by z) W_out              group_norm_*

`prompt` runs whole (possibly padded) sequences and returns the state after each, `step` one
token per sequence from that state, `grads` the gradients of a scalar loss.  The projections
are plain matrix products.

    python examples/state_space_layer.py        # on a GPU: prompt, decode, a few training steps
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import delta_rule_linear_qdelta_gb300 as qd  # noqa: E402


class StateSpaceLayer:
    """width: the model's; heads x head_dim = D channels; states N per channel, rank of delta."""

    def __init__(self, width, heads, head_dim, states=16, taps=4, rank=16, dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator().manual_seed(seed)
        self.heads, self.head_dim, self.N, self.W, self.rank = heads, head_dim, states, taps, rank
        D = self.D = heads * head_dim
        r = lambda *s: torch.randn(*s, generator=g)
        step = torch.exp(torch.rand(D, generator=g) * (math.log(0.1) - math.log(1e-3)) + math.log(1e-3))
        f32 = {"conv_w": r(D, taps) / math.sqrt(taps), "conv_b": torch.zeros(D),
               "A": -torch.arange(1, states + 1).float().repeat(D, 1), "skip": torch.ones(D),
               "delta_bias": torch.log(torch.expm1(step)), "norm_w": torch.ones(heads, head_dim),
               "norm_b": torch.zeros(heads, head_dim)}
        mats = {"W_in": r(width, 2 * D) / math.sqrt(width), "W_x": r(D, rank + 2 * states) / math.sqrt(D),
                "W_dt": r(rank, D) / math.sqrt(rank), "W_out": r(D, width) / math.sqrt(D)}
        self.p = {k: v.to(device) for k, v in f32.items()} | {k: v.to(device, dtype) for k, v in mats.items()}

    # ------------------------------------------------------------------ shared pieces
    def _split_in(self, h):
        xz = h @ self.p["W_in"]
        return xz[..., :self.D].contiguous(), xz[..., self.D:].contiguous()

    def _split_x(self, x):
        """delta and the scan's B, C (one group) from the convolved channels."""
        dbc = x @ self.p["W_x"]
        dt, B, C = dbc.split([self.rank, self.N, self.N], dim=-1)
        return dt, dt @ self.p["W_dt"], B.unsqueeze(-2).contiguous(), C.unsqueeze(-2).contiguous()

    def _rows(self, t):
        return t.view(*t.shape[:-1], self.heads, self.head_dim)

    # ------------------------------------------------------------------ serving
    def prompt(self, h, state=None, lens=None):
        """h [B,T,width] -> (out [B,T,width], state).  lens [B] int32: real tokens of each sequence."""
        out, state, _ = self._forward(h, state, lens)
        return out, state

    def _forward(self, h, state, lens):
        p = self.p
        S_conv, S_ssm = state if state is not None else (None, None)
        x_in, z = self._split_in(h)
        x, S_conv1 = qd.short_conv_fwd(x_in, p["conv_w"], p["conv_b"], S_conv, lens=lens)
        dt, delta, B, C = self._split_x(x)
        y, S_ssm1 = qd.ssm_fwd(x, delta, p["A"], B, C, p["skip"], p["delta_bias"], S_ssm, lens=lens)
        n = qd.group_norm_fwd(self._rows(y), p["norm_w"], p["norm_b"], self._rows(z))
        out = n.view(y.shape) @ p["W_out"]
        return out, (S_conv1, S_ssm1), (h, x_in, z, x, dt, delta, B, C, y, n, S_conv, S_ssm, lens)

    def step(self, h, state):
        """One token per sequence: h [B,width] -> out [B,width]; the state is updated in place."""
        p, (S_conv, S_ssm) = self.p, state
        x_in, z = self._split_in(h)
        x = qd.short_conv_step(S_conv, x_in, p["conv_w"], p["conv_b"])
        _, delta, B, C = self._split_x(x)
        y = qd.ssm_step(S_ssm, x, delta, p["A"], B, C, p["skip"], p["delta_bias"])
        return qd.group_norm_fwd(self._rows(y), p["norm_w"], p["norm_b"], self._rows(z)).view(y.shape) @ p["W_out"]

    # ------------------------------------------------------------------ training
    def grads(self, h, dout_of, state=None, lens=None):
        """Runs the layer and returns (out, {parameter: gradient}, dh) for the loss whose gradient with
        respect to out is dout_of(out)."""
        p = self.p
        out, _, saved = self._forward(h, state, lens)
        h, x_in, z, x, dt, delta, B, C, y, n, S_conv, S_ssm, lens = saved
        dout = dout_of(out)
        flat = lambda t: t.reshape(-1, t.shape[-1])
        g = {"W_out": flat(n.view(y.shape)).t() @ flat(dout)}
        gn = qd.group_norm_bwd(self._rows(y), p["norm_w"], p["norm_b"], self._rows(z),
                               self._rows((dout @ p["W_out"].t()).contiguous()))
        g["norm_w"], g["norm_b"] = gn["dw"], gn["db"]
        gs = qd.ssm_bwd(x, delta, p["A"], B, C, p["skip"], p["delta_bias"], S_ssm, gn["dx"].view(y.shape), lens=lens)
        g["A"], g["skip"], g["delta_bias"] = gs["dA"], gs["dD"], gs["ddelta_bias"]
        g["W_dt"] = flat(dt).t() @ flat(gs["ddelta"])
        ddbc = torch.cat([gs["ddelta"] @ p["W_dt"].t(), gs["dB"].squeeze(-2), gs["dC"].squeeze(-2)], -1)
        g["W_x"] = flat(x).t() @ flat(ddbc)
        gc = qd.short_conv_bwd(x_in, p["conv_w"], p["conv_b"], S_conv, gs["dx"] + ddbc @ p["W_x"].t(), lens=lens)
        g["conv_w"], g["conv_b"] = gc["dw"], gc["dbias"]
        dxz = torch.cat([gc["dx"], gn["dz"].view(z.shape)], -1)
        g["W_in"] = flat(h).t() @ flat(dxz)
        return out, g, dxz @ p["W_in"].t()


def main():
    layer = StateSpaceLayer(width=1024, heads=6, head_dim=128)
    gen = torch.Generator(device="cuda").manual_seed(1)
    h = torch.randn(4, 256, 1024, generator=gen, device="cuda").bfloat16()
    lens = torch.tensor([256, 200, 31, 0], dtype=torch.int32, device="cuda")
    out, state = layer.prompt(h, lens=lens)
    for _ in range(8):                                  # continues every sequence after its own last token
        out = layer.step(torch.randn(4, 1024, generator=gen, device="cuda").bfloat16(), state)
    print("decoded", tuple(out.shape), "finite", bool(torch.isfinite(out).all()))
    target = torch.randn(4, 256, 1024, generator=gen, device="cuda").bfloat16()
    for it in range(5):
        out, g, _ = layer.grads(h, lambda o: ((o - target) / o.numel()).to(o.dtype))
        print("step", it, "loss", float((out.float() - target.float()).square().mean() / 2))
        for k, v in g.items():                          # steps of one size for every parameter
            v = v.float()
            layer.p[k] -= (1e-3 * v / v.square().mean().sqrt().clamp_min(1e-30)).to(layer.p[k].dtype)


if __name__ == "__main__":
    main()
