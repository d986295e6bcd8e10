"""A selective-scan block trained and served with CausalConv, SelectiveScan, BlockNorm and GradClip.

    x, z        = n W_in                          one projection, used in place as slices
    u           = CausalConv(x)                   depthwise, silu
    r, B, C     = u W_x                           low rank of the steps, and the scan's B and C
    dt          = r W_dt
    o           = SelectiveScan(u, dt, A, B, C; z, D, dt_bias)
    y           = o W_out
    x', n'      = x + scale * RMSNorm(y; w_post),  RMSNorm(x'; w_next)

``n`` is the normed residual stream that the block before leaves.  Run as a
program it trains the block for a few steps, with the gradients clipped by their
norm together, then prefills a prompt and decodes.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bwd_persistent_cta_gb300 as R  # noqa: E402


class SelectiveScanBlock:
    """Weights of one block, and its operators for ``batch`` sequences of ``seq_len`` tokens (batch first).  The scan's
    own weights (A, D, dt_bias) are fp32."""

    def __init__(self, batch, seq_len, width, channels, states, rank, taps=4, dtype="bf16", weights=None, seed=0):
        self.B, self.T, self.width, self.D, self.N, self.rank = batch, seq_len, width, channels, states, rank
        rows, td = batch * seq_len, torch.bfloat16 if dtype == "bf16" else torch.float32
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
        step = torch.logspace(-3, -1, channels, device="cuda")
        self.w = weights or {
            "in": (rnd(width, 2 * channels) / width ** 0.5).to(td),
            "conv": (rnd(channels, taps) / taps ** 0.5).to(td), "conv_bias": torch.zeros(channels, device="cuda", dtype=td),
            "x": (rnd(channels, rank + 2 * states) / channels ** 0.5).to(td),
            "dt": (rnd(rank, channels) / rank ** 0.5).to(td),
            "dt_bias": step + torch.log(-torch.expm1(-step)),
            "A": -torch.arange(1.0, states + 1, device="cuda").repeat(channels, 1),
            "D": torch.ones(channels, device="cuda"),
            "out": (rnd(channels, width) / channels ** 0.5).to(td),
            "post": torch.ones(width, device="cuda", dtype=td),
            "scale": torch.full((width,), 0.5, device="cuda", dtype=td), "next": torch.ones(width, device="cuda", dtype=td)}
        self.conv = R.CausalConv(batch, seq_len, channels, taps, dtype=dtype, batch_first=True)
        self.scan = R.SelectiveScan(batch, seq_len, channels, states, dtype=dtype, batch_first=True)
        self.boundary = R.BlockNorm(rows, width, dtype=dtype, residual=True, norm_out=True)

    def _projected(self, n):
        """x and z, slices of one projection."""
        p = n.reshape(self.B * self.T, self.width) @ self.w["in"]
        return p.view(self.B, self.T, -1).split(self.D, 2)

    def _scan_inputs(self, u):
        """The scan's inputs from the convolution's output, and the projection that B and C are slices of."""
        q = u.reshape(self.B * self.T, self.D) @ self.w["x"]
        dt = (q[:, :self.rank] @ self.w["dt"]).view(u.shape)
        bc = q.view(self.B, self.T, -1)
        B, C = (bc[..., self.rank + i * self.N:self.rank + (i + 1) * self.N].unflatten(2, (1, self.N)) for i in (0, 1))
        return (u, dt, self.w["A"], B, C), q

    def _finish(self, x, o):
        y = o.reshape(self.B * self.T, self.D) @ self.w["out"]
        w = self.w
        x1, n1 = self.boundary.forward(y, x=x.reshape(self.B * self.T, -1), w_in=w["post"], scale=w["scale"], w_out=w["next"])
        return x1.view(x.shape), n1.view(x.shape), y

    def _more(self, z):
        return dict(z=z, D=self.w["D"], dt_bias=self.w["dt_bias"])

    def forward(self, x, n, conv_state=None, state=None, train=False):
        """(x', n', the convolution's state, the scan's) for x, n [batch, seq_len, width]."""
        xc, z = self._projected(n)
        u, sT = self.conv.forward(xc, self.w["conv"], bias=self.w["conv_bias"], s0=conv_state)
        ins, q = self._scan_inputs(u)
        o, hT = self.scan.forward(*ins, **self._more(z), h0=state, train=train)
        x1, n1, y = self._finish(x, o)
        if train:
            self.saved = (x, n, xc, z, ins, q, o, y)
        return x1, n1, sT, hT

    def decode(self, x, n, conv_pool, pool, slots):
        """(x', n') for seq_len new tokens a sequence; its states in the pools at ``slots`` are updated in place."""
        xc, z = self._projected(n)
        u = self.conv.step(xc, self.w["conv"], conv_pool, bias=self.w["conv_bias"], slots=slots)
        ins, _ = self._scan_inputs(u)
        o = self.scan.step(*ins, pool, **self._more(z), slots=slots)
        return self._finish(x, o)[:2]

    def backward(self, dx1, dn1):
        """(dx, dn, gradients of the weights) after a training forward."""
        x, n, xc, z, ins, q, o, y = self.saved
        rows, w = self.B * self.T, self.w
        flat = lambda t: None if t is None else t.reshape(rows, -1)  # noqa: E731
        d = self.boundary.backward(flat(dx1), flat(dn1), y, x=flat(x), w_in=w["post"], scale=w["scale"], w_out=w["next"])
        dw = {"post": d["dw_in"], "scale": d["dscale"], "next": d["dw_out"], "out": flat(o).T @ d["dy"]}
        dx = d["dx"]
        s = self.scan.backward((d["dy"] @ w["out"].T).view(o.shape), *ins, **self._more(z))
        dw.update(A=s["dA"], D=s["dD"], dt_bias=s["ddt_bias"])
        ddt = flat(s["ddt"])
        dw["dt"] = q[:, :self.rank].T @ ddt
        dq = torch.cat([ddt @ w["dt"].T, flat(s["dB"]), flat(s["dC"])], 1)
        dw["x"] = flat(ins[0]).T @ dq
        du = flat(s["dx"]) + dq @ w["x"].T
        c = self.conv.backward(du.view(o.shape), xc, w["conv"], bias=w["conv_bias"])
        dw.update(conv=c["dw"], conv_bias=c["dbias"])
        dp = torch.cat([flat(c["dx"]), flat(s["dz"])], 1)
        dw["in"] = flat(n).T @ dp
        return dx.view(x.shape), (dp @ w["in"].T).view(n.shape), dw


def main():
    B, T, width = 4, 512, 512
    block = SelectiveScanBlock(B, T, width, 1024, 16, 32)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(B, T, width, device="cuda", generator=gen).to(torch.bfloat16)
    n = (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)
    want = torch.roll(n, 1, 1)                              # a delay line: yesterday's token
    names = list(block.w)
    clip = None
    for step in range(40):
        x1, n1, _, _ = block.forward(x, n, train=True)
        err = n1.float() - want.float()
        _, _, dw = block.backward(None, (2 * err / err.numel()).to(torch.bfloat16))
        grads = [dw[m].contiguous() for m in names]
        if clip is None:
            clip = R.GradClip([g.numel() for g in grads], ["bf16" if g.dtype == torch.bfloat16 else "f32" for g in grads])
        norm = clip.clip(grads, 1e-3)
        for m, g in zip(names, grads):
            block.w[m].copy_((block.w[m].float() - 100.0 * g.float()).to(block.w[m].dtype))
        if step % 10 == 0 or step == 39:
            print(f"step {step}: mean squared error {err.square().mean().item():.4f}, gradient norm {norm.item():.2e}")
    # serving: prefill into pools of states, then one token at a time
    _, _, sT, hT = block.forward(x, n)
    slots = torch.tensor([5, 2, 11, 7], dtype=torch.int32, device="cuda")
    conv_pool, pool = torch.zeros(16, 3, 1024, device="cuda", dtype=torch.bfloat16), torch.zeros(16, 1024, 16, device="cuda")
    conv_pool[slots.long()], pool[slots.long()] = sT, hT
    one = SelectiveScanBlock(B, 1, width, 1024, 16, 32, weights=block.w)
    for t in range(8):
        y1, m1 = one.decode(x[:, t:t + 1].contiguous(), n[:, t:t + 1].contiguous(), conv_pool, pool, slots)
    torch.cuda.synchronize()
    print("decoded", t + 1, "tokens; output", tuple(m1.shape))


if __name__ == "__main__":
    main()
