"""A gated-delta-rule block trained and served with DeltaRule and BlockNorm.

    q, k, v, z, a, b = n W_in                    one projection, used in place as slices
    q, k   = unit length per head                (BlockNorm with the constant weight Dk^-1/2)
    g      = -rate softplus(a),  beta = sigma(b)
    o      = gated delta rule (q, k, v, g, beta)
    y      = (RMSNorm(o; w_head) * silu(z)) W_out      per value head
    x', n' = x + scale * RMSNorm(y; w_post),  RMSNorm(x'; w_next)

``n`` is the normed residual stream that the block before leaves.  Run as a
program it trains the block for a few steps, then prefills a prompt and decodes.
"""
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bwd_persistent_cta_gb300 as R  # noqa: E402


class GatedDeltaBlock:
    """Weights of one block, and its operators for ``batch`` sequences of ``seq_len`` tokens (batch first)."""

    def __init__(self, batch, seq_len, width, heads_k, heads_v, dim, dtype="bf16", weights=None, seed=0):
        self.B, self.T, self.width, self.Hk, self.Hv, self.D, self.dtype = batch, seq_len, width, heads_k, heads_v, dim, dtype
        rows, td = batch * seq_len, torch.bfloat16 if dtype == "bf16" else torch.float32
        self.cuts = [2 * heads_k * dim, heads_v * dim, heads_v * dim, heads_v, heads_v]        # qk, v, z, a, b
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
        self.w = weights or {
            "in": (rnd(width, sum(self.cuts)) / width ** 0.5).to(td),
            "out": (rnd(heads_v * dim, width) / (heads_v * dim) ** 0.5).to(td),
            "head": torch.ones(dim, device="cuda", dtype=td), "post": torch.ones(width, device="cuda", dtype=td),
            "scale": torch.full((width,), 0.5, device="cuda", dtype=td), "next": torch.ones(width, device="cuda", dtype=td)}
        self.rate = torch.logspace(-3, -0.5, heads_v, device="cuda")
        self.unit = torch.full((dim,), dim ** -0.5, device="cuda", dtype=td)
        self.qk_norm = R.BlockNorm(rows, dim, groups=2 * heads_k, dtype=dtype, eps=1e-12)
        self.delta = R.DeltaRule(batch, seq_len, heads_k, heads_v, dim, dim, dtype=dtype, batch_first=True)
        self.head = R.BlockNorm(rows, dim, groups=heads_v, dtype=dtype, gate="silu")
        self.boundary = R.BlockNorm(rows, width, dtype=dtype, residual=True, norm_out=True)

    def _mix_inputs(self, n):
        """The projection and what the recurrence takes of it."""
        B, T, Hk, Hv, D = self.B, self.T, self.Hk, self.Hv, self.D
        p = n.reshape(B * T, self.width) @ self.w["in"]
        qk, v, z, a, b = p.split(self.cuts, 1)
        qkn, _ = self.qk_norm.forward(qk, w_in=self.unit)
        q, k = (t.unflatten(1, (Hk, D)).unflatten(0, (B, T)) for t in qkn.split(Hk * D, 1))
        g = (-self.rate * F.softplus(a.float())).to(p.dtype).view(B, T, Hv)
        beta = torch.sigmoid(b.float()).to(p.dtype).view(B, T, Hv)
        return (q, k, v.unflatten(1, (Hv, D)).unflatten(0, (B, T)), g, beta), z, (qk, a, b)

    def _finish(self, x, o, z):
        o = o.reshape(self.B * self.T, -1)
        h, _ = self.head.forward(o, z=z, w_in=self.w["head"])
        y = h @ self.w["out"]
        x1, n1 = self.boundary.forward(y, x=x.reshape(self.B * self.T, -1), w_in=self.w["post"], scale=self.w["scale"],
                                       w_out=self.w["next"])
        return x1.view(x.shape), n1.view(x.shape), (o, h, y)

    def forward(self, x, n, state=None, train=False):
        """(x', n', state after the last token) for x, n [batch, seq_len, width]."""
        ins, z, raw = self._mix_inputs(n)
        o, sT = self.delta.forward(*ins, s0=state, train=train)
        x1, n1, mid = self._finish(x, o, z)
        if train:
            self.saved = (x, n, ins, z, raw, mid)
        return x1, n1, sT

    def decode(self, x, n, pool, slots):
        """(x', n') for seq_len new tokens a sequence; its state in ``pool`` at ``slots`` is updated in place."""
        ins, z, _ = self._mix_inputs(n)
        o = self.delta.step(*ins, pool, slots=slots)
        x1, n1, _ = self._finish(x, o, z)
        return x1, n1

    def backward(self, dx1, dn1):
        """(dx, dn, gradients of the weights) after a training forward."""
        x, n, ins, z, (qk, a, b), (o, h, y) = self.saved
        rows, w, Hk, D = self.B * self.T, self.w, self.Hk, self.D
        flat = lambda t: None if t is None else t.reshape(rows, -1)  # noqa: E731
        d = self.boundary.backward(flat(dx1), flat(dn1), y, x=flat(x), w_in=w["post"], scale=w["scale"], w_out=w["next"])
        dw = {"post": d["dw_in"], "scale": d["dscale"], "next": d["dw_out"], "out": h.T @ d["dy"]}
        dx = d["dx"]
        dh = self.head.backward(d["dy"] @ w["out"].T, None, o, z=z, w_in=w["head"])
        dw["head"] = dh["dw_in"]
        dq, dk, dv, dg, dbeta, _ = self.delta.backward(dh["dy"].view(ins[2].shape), *ins)
        dqk = self.qk_norm.backward(torch.cat([dq.reshape(rows, Hk * D), dk.reshape(rows, Hk * D)], 1), None, qk,
                                    w_in=self.unit)["dy"]
        da = -self.rate * torch.sigmoid(a.float()) * flat(dg).float()
        s = torch.sigmoid(b.float())
        db = s * (1 - s) * flat(dbeta).float()
        dp = torch.cat([dqk, flat(dv), dh["dz"], da.to(dv.dtype), db.to(dv.dtype)], 1)
        dw["in"] = flat(n).T @ dp
        return dx.view(x.shape), (dp @ w["in"].T).view(n.shape), dw


def main():
    B, T, width = 4, 512, 1024
    block = GatedDeltaBlock(B, T, width, 4, 8, 128)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(B, T, width, device="cuda", generator=gen).to(torch.bfloat16)
    n = (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)
    want = torch.roll(n, 1, 1)                              # a delay line: yesterday's token
    for step in range(40):
        x1, n1, _ = block.forward(x, n, train=True)
        err = n1.float() - want.float()
        _, _, dw = block.backward(None, (2 * err / err.numel()).to(torch.bfloat16))
        for name, w in block.w.items():                     # steps of 1 % of each weight's length
            d = dw[name].float()
            w.copy_((w.float() - 0.01 * w.float().norm() * d / d.norm().clamp_min(1e-30)).to(w.dtype))
        if step % 10 == 0 or step == 39:
            print(f"step {step}: mean squared error {err.square().mean().item():.4f}")
    # serving: prefill into a pool of states, then one token at a time
    x1, n1, sT = block.forward(x, n)
    pool = torch.zeros(16, 8, 128, 128, device="cuda")
    slots = torch.tensor([5, 2, 11, 7], dtype=torch.int32, device="cuda")
    pool[slots.long()] = sT
    one = GatedDeltaBlock(B, 1, width, 4, 8, 128, weights=block.w)
    for t in range(8):
        y1, m1 = one.decode(x[:, t:t + 1].contiguous(), n[:, t:t + 1].contiguous(), pool, slots)
    one.delta.sync()
    print("decoded", t + 1, "tokens; output", tuple(m1.shape))


if __name__ == "__main__":
    main()
