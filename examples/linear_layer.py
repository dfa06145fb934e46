"""A linear attention block on libgdn: norm, linear attention with a decay for each token and head, a
gated group norm, and the norms after the block.

    python examples/linear_layer.py            # needs an MI355X and the built library

Runs a prompt through the block, continues it token by token from the state the prompt left (a line of
a pool, updated in place), checks that the tokens agree with one pass over everything, and takes a few
steps on the block's parameters, the gradients coming from the library's backward calls.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_chunked_02_amd as gdn  # noqa: E402


class LinearLayer:
    """y = norm(x) -> q, k, v, gate = y W_in, g = logsigmoid(y W_g + 4) -> attention -> norm(o)
    silu(gate) -> h = . W_out -> x' = x + norm(h), and norm(x'), which the next block takes.  The
    residual stream x is fp32, the block's own tensors are of ``dtype``."""

    names = ("pre", "post", "scale", "following", "norm_w", "norm_b", "w_in", "w_g", "w_out")

    def __init__(self, model=256, heads=4, shared=2, dk=64, dv=64, dtype=torch.bfloat16,
                 device="cuda", seed=0):
        r = torch.Generator(device=device).manual_seed(seed)
        n = lambda *s: torch.randn(*s, generator=r, device=device)  # noqa: E731
        self.heads, self.shared, self.dk, self.dv = heads, shared, dk, dv
        inner = heads * dv
        self.w_in = (n(model, 2 * shared * dk + 2 * inner) * model ** -0.5).to(dtype)
        self.w_g = (n(model, heads) * model ** -0.5).to(dtype)
        self.w_out = (n(inner, model) * inner ** -0.5).to(dtype)
        self.pre, self.post, self.following = (1 + 0.1 * n(model) for _ in range(3))
        self.scale = 0.5 + 0.1 * n(model)
        self.norm_w, self.norm_b = 1 + 0.1 * n(inner), 0.1 * n(inner)

    def pool(self, lines):
        return torch.zeros(lines, self.heads, self.dk, self.dv, device=self.w_in.device)

    def _project(self, y):
        """q, k, v and the gate as slices of one projection, read in place, and the log-decays."""
        p = y @ self.w_in
        a, b = self.shared * self.dk, self.heads * self.dv
        q, k = (p[..., i * a:(i + 1) * a].unflatten(-1, (self.shared, self.dk)) for i in (0, 1))
        v = p[..., 2 * a:2 * a + b].unflatten(-1, (self.heads, self.dv))
        z = (y @ self.w_g).float() + 4.0
        return q, k, v, p[..., 2 * a + b:], z, torch.nn.functional.logsigmoid(z)

    def _gated(self, o, gate):
        rows = o.numel() // (self.heads * self.dv)
        return gdn.group_norm(o.reshape(rows, -1), self.heads, self.norm_w, self.norm_b,
                              activation="silu", gate=gate.reshape(rows, -1))

    def _after(self, x, h, inplace=False):
        return gdn.block_norm(x, h, weight=self.following, post_norm=True, post_weight=self.post,
                              scale=self.scale, inplace=inplace)

    def prompt(self, x, state, cu_seqlens=None):
        """(x', the next block's input) for x [B, T, model]; ``state`` [sequences, ...] is carried in
        and out, in place."""
        y = gdn.block_norm(x, weight=self.pre, dtype=self.w_in.dtype)[1]
        q, k, v, gate, _, g = self._project(y)
        o, ht = gdn.linear_attention(q, k, v, g, initial_state=state, cu_seqlens=cu_seqlens)
        state.copy_(ht)
        n = self._gated(o, gate)[0]
        return self._after(x, (n @ self.w_out).view(x.shape[:-1] + (-1,)))[:2]

    def token(self, x, pool, lines):
        """The same for one token x [B, model] of the sequences at ``lines`` of the pool."""
        y = gdn.block_norm(x, weight=self.pre, dtype=self.w_in.dtype)[1]
        q, k, v, gate, _, g = self._project(y)
        o = gdn.linear_state_update(pool, q, k, v, g, cache_indices=lines)
        return self._after(x, self._gated(o, gate)[0] @ self.w_out)[:2]

    def gradients(self, x, dxo, dy, cu_seqlens=None):
        """One pass there and back, given the gradients of x' and of the next block's input: the
        gradients of x and, in the order of ``names``, of the parameters."""
        dtype = self.w_in.dtype
        _, y, _, rstd = gdn.block_norm(x, weight=self.pre, dtype=dtype)
        q, k, v, gate, z, g = self._project(y)
        o, _ = gdn.linear_attention(q, k, v, g, output_final_state=False, cu_seqlens=cu_seqlens)
        n, mean, nrstd = self._gated(o, gate)
        h = (n @ self.w_out).view(y.shape)
        _, _, prstd, frstd = self._after(x, h)

        dx, dh, _, dfollowing, dpost, dscale = gdn.block_norm_bwd(
            dy, dxo, x, h, prstd, frstd, weight=self.following, post_norm=True,
            post_weight=self.post, scale=self.scale)
        flat = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
        dn = flat(dh) @ self.w_out.T
        dwo = n.T @ flat(dh)
        do, dnw, dnb, dgate = gdn.group_norm_bwd(dn, o.view(n.shape), self.heads, mean, nrstd,
                                                 self.norm_w, self.norm_b, activation="silu",
                                                 gate=flat(gate))
        dq, dk, dv, dg, _ = gdn.linear_attention_bwd(q, k, v, g, do.view(o.shape),
                                                     cu_seqlens=cu_seqlens)
        dz = (dg * torch.sigmoid(-z)).to(dtype)
        dp = torch.cat([dq.flatten(2), dk.flatten(2), dv.flatten(2),
                        dgate.view(y.shape[:-1] + (-1,))], -1)
        dyin = dp @ self.w_in.T + dz @ self.w_g.T
        dx, _, _, dpre, _, _ = gdn.block_norm_bwd(dyin, dx, x, rstd=rstd, weight=self.pre)
        return (dx, dpre, dpost, dscale, dfollowing, dnw, dnb, flat(y).T @ flat(dp),
                flat(y).T @ flat(dz), dwo)

    def step(self, x, target, rate=0.02):
        """One step of gradient descent on the distance of x' from a target; returns the loss."""
        diff = self.prompt(x, self.pool(x.shape[0]))[0] - target
        grads = self.gradients(x, (2.0 / diff.numel()) * diff,
                               torch.zeros_like(x, dtype=self.w_in.dtype))
        for name, d in zip(self.names, grads[1:]):
            w = getattr(self, name)
            w -= (rate / (d.float().norm() + 1e-12) * w.float().norm() * d.float()).to(w.dtype)
        return float(diff.square().mean())


def main():
    layer = LinearLayer()
    r = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(2, 300, 256, generator=r, device="cuda")

    whole = layer.prompt(x, layer.pool(2))[0]
    pool = layer.pool(5)
    lines = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    state = layer.pool(2)
    parts = [layer.prompt(x[:, :260], state)[0]]
    pool[lines.long()] = state
    parts += [layer.token(x[:, t], pool, lines)[0][:, None] for t in range(260, 300)]
    parts = torch.cat(parts, 1)
    err = float((parts - whole).norm() / (whole - x).norm())
    print("prompt of 260 and 40 tokens against one prompt of 300: relative difference %.2e" % err)

    target = x + 0.5 * (LinearLayer(seed=7).prompt(x, layer.pool(2))[0] - x)
    losses = [layer.step(x, target) for _ in range(20)]
    print("loss over 20 steps: %.4f -> %.4f" % (losses[0], losses[-1]))
    return err, losses


if __name__ == "__main__":
    main()
