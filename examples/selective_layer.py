"""A selective state-space layer on libgdn: short convolution, selective scan, gated group norm.

    python examples/selective_layer.py            # needs an MI355X and the built library

Runs a prompt through the layer, continues it token by token from the states the prompt left (the
convolution's line and the scan's state, both updated in place), checks that the tokens agree with
one pass over everything, and trains the layer's parameters for a few steps, the gradients coming
from the library's backward calls.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_chunked_02_amd as gdn  # noqa: E402


class SelectiveLayer:
    """x -> u = silu(conv(x W_in)), gate = x W_gate -> (dt, B, C) = u W_dbc -> scan -> norm(y) silu(gate)
    -> W_out, in bf16 with fp32 parameters of the recurrence."""

    def __init__(self, model=256, inner=512, dstate=16, groups=8, width=4, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        n = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
        self.inner, self.dstate, self.groups, self.width = inner, dstate, groups, width
        self.w_in = (n(model, 2 * inner) * model ** -0.5).bfloat16()
        self.w_dbc = (n(inner, inner + 2 * dstate) * inner ** -0.5).bfloat16()
        self.w_out = (n(inner, model) * inner ** -0.5).bfloat16()
        self.conv_w, self.conv_b = n(inner, width) * width ** -0.5, torch.zeros(inner, device=device)
        self.A = -torch.arange(1, dstate + 1, device=device).float().repeat(inner, 1)
        self.D = torch.ones(inner, device=device)
        first = torch.exp(torch.rand(inner, generator=g, device=device) * 4.6 - 6.9)  # 0.001 .. 0.1
        self.dt_bias = first + torch.log(-torch.expm1(-first))
        self.norm_w, self.norm_b = torch.ones(inner, device=device), torch.zeros(inner, device=device)

    def new_states(self, batch):
        dev = self.w_in.device
        return (torch.zeros(batch, self.width - 1, self.inner, dtype=torch.bfloat16, device=dev),
                torch.zeros(batch, self.inner, self.dstate, device=dev))

    def _split(self, u):
        dbc = u @ self.w_dbc
        i, s = self.inner, self.dstate
        B = dbc[..., i:i + s].unflatten(-1, (1, s))  # slices: read in place
        return dbc[..., :i], B, dbc[..., i + s:].unflatten(-1, (1, s))

    def _norm(self, y, gate):
        flat = y.reshape(-1, self.inner)
        out, mean, rstd = gdn.group_norm(flat, self.groups, self.norm_w, self.norm_b,
                                         activation="silu", gate=gate.reshape(-1, self.inner))
        return out.view(y.shape), mean, rstd

    def prompt(self, x, states):
        """y for x [B, T, model]; the states are carried in and out, in place."""
        line, state = states
        xz = x @ self.w_in
        u = gdn.causal_conv1d(xz[..., :self.inner].contiguous(), self.conv_w, self.conv_b,
                              conv_state=line, activation="silu")
        dt, B, C = self._split(u)
        y, ht = gdn.selective_scan(u, dt, self.A, B, C, D=self.D, dt_bias=self.dt_bias,
                                   dt_softplus=True, initial_state=state)
        state.copy_(ht)
        return self._norm(y, xz[..., self.inner:])[0] @ self.w_out

    def token(self, x, states):
        """y for one token x [B, model]."""
        line, state = states
        xz = x @ self.w_in
        u = gdn.causal_conv1d(xz[:, None, :self.inner].contiguous(), self.conv_w, self.conv_b,
                              conv_state=line, activation="silu")[:, 0]
        dt, B, C = self._split(u)
        y = gdn.selective_state_update(state, u, dt, self.A, B, C, D=self.D, dt_bias=self.dt_bias,
                                       dt_softplus=True)
        return self._norm(y, xz[:, self.inner:])[0] @ self.w_out

    def step(self, x, target, rate=0.02):
        """One step of gradient descent on the layer's own parameters (the projections stay);
        returns the loss."""
        xz = x @ self.w_in
        xi, gate = xz[..., :self.inner].contiguous(), xz[..., self.inner:]
        u = gdn.causal_conv1d(xi, self.conv_w, self.conv_b, activation="silu")
        dt, B, C = self._split(u)
        common = dict(D=self.D, dt_bias=self.dt_bias, dt_softplus=True)
        y, _ = gdn.selective_scan(u, dt, self.A, B, C, output_final_state=False, **common)
        v, mean, rstd = self._norm(y, gate)
        out = v @ self.w_out
        diff = out.float() - target.float()
        loss = diff.square().mean()

        dv = ((2.0 / diff.numel()) * diff).bfloat16() @ self.w_out.T
        flat = lambda t: t.reshape(-1, self.inner)  # noqa: E731
        dy, dnw, dnb, _ = gdn.group_norm_bwd(flat(dv), flat(y), self.groups, mean, rstd,
                                             self.norm_w, self.norm_b, activation="silu",
                                             gate=flat(gate))
        du, ddt, dA, dB, dC, dD, _, dbias, _ = gdn.selective_scan_bwd(
            u, dt, self.A, B, C, dy.view(u.shape), **common)
        # the scan's inputs dt, B and C came from u as well
        du = du + torch.cat([ddt, dB.flatten(2), dC.flatten(2)], -1) @ self.w_dbc.T
        _, dcw, dcb, _ = gdn.causal_conv1d_bwd(xi, self.conv_w, du, bias=self.conv_b,
                                               activation="silu")
        for p, g in ((self.norm_w, dnw), (self.norm_b, dnb), (self.D, dD), (self.dt_bias, dbias),
                     (self.conv_w, dcw), (self.conv_b, dcb)):
            p -= rate / (g.norm() + 1e-12) * p.norm().clamp_min(1.0) * g
        self.A *= torch.exp(-rate * torch.sign(dA * self.A) * 0.1)  # stays negative
        return float(loss)


def main():
    layer = SelectiveLayer()
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(2, 300, 256, generator=g, device="cuda").bfloat16()

    whole = layer.prompt(x, layer.new_states(2))
    states = layer.new_states(2)
    parts = [layer.prompt(x[:, :260], states)]
    parts += [layer.token(x[:, t], states)[:, None] for t in range(260, 300)]
    parts = torch.cat(parts, 1)
    err = float((parts.float() - whole.float()).norm() / whole.float().norm())
    print("prompt of 260 and 40 tokens against one prompt of 300: relative difference %.2e" % err)

    target = SelectiveLayer(seed=7).prompt(x, layer.new_states(2)) * 0.5
    losses = [layer.step(x, target) for _ in range(20)]
    print("loss over 20 steps: %.4f -> %.4f" % (losses[0], losses[-1]))
    return err, losses


if __name__ == "__main__":
    main()
