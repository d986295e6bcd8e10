"""The selective scan's decays, steps and gates beside 64 bits where roundings add up or
grow: memories of many thousand tokens, and steps and gates far from zero."""
import math

import pytest

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24               # half a step of fp32


def _reference(t, dy, dhT):
    """Channel d reads group d // 8: y, hT, dh0, dA in 64 bits on the GPU (no gate, D or softplus)."""
    import torch
    x, dt, A, Bm, Cm, h = (t[n].double() for n in ("x", "dt", "A", "B", "C", "h0"))
    T, B, D = x.shape
    chan = lambda v: v.repeat_interleave(D // v.shape[1], 1)  # noqa: E731
    kept, y = [], torch.empty_like(x)
    for i in range(T):
        kept.append(h)
        h = torch.exp(dt[i][..., None] * A) * h + (dt[i] * x[i])[..., None] * chan(Bm[i])
        y[i] = (chan(Cm[i]) * h).sum(-1)
    hT, g, dA = h, dhT.double(), torch.zeros_like(A)
    for i in reversed(range(T)):
        g = torch.exp(dt[i][..., None] * A) * (g + dy[i].double()[..., None] * chan(Cm[i]))
        dA += (g * kept.pop() * dt[i][..., None]).sum(0)
    return y, hT, g, dA


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_memories(dtype):
    """|delta A| from 1e-5 to 1e-3 over 8192 tokens, whose steps vary, in one piece (8 channels a group fill the SMs).

    An exponential in fp32 that is off by b on average moves what is remembered over T tokens by T b; its own rounding
    and the state's are walks.  fp32 storage: b = 3e-9, a walk of sqrt(T) * (4e-8 + 2^-25): 3.1e-5; dA has two such
    states in it.  bf16 storage: b = 1.1e-8 (what its decays' approximation is off by, for decays this near to one),
    and outputs rounded to bf16."""
    import torch
    import bwd_persistent_cta_gb300 as R
    T, B, G, N = 8192, 1, 800, 8
    D = 8 * G
    walk = math.sqrt(T) * (4e-8 + EPS / 2)
    tol = T * (3e-9 if dtype == "f32" else 1.1e-8) + walk
    td = torch.float32 if dtype == "f32" else torch.bfloat16
    gen = torch.Generator(device="cuda").manual_seed(41)
    rnd = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    t = {"x": (0.1 * rnd(T, B, D)).to(td), "dt": (0.01 * torch.exp(0.5 * rnd(T, B, D))).to(td), "B": rnd(T, B, G, N).to(td),
         "C": rnd(T, B, G, N).to(td), "h0": 1 + 0.3 * rnd(B, D, N),
         "A": -torch.logspace(-3, -1, N, device="cuda") * torch.exp(0.1 * rnd(D, N))}
    dy, dhT = (0.01 * rnd(T, B, D)).to(td), 1 + 0.3 * rnd(B, D, N)
    op = R.SelectiveScan(B, T, D, N, groups=G, dtype=dtype, softplus=False)
    args = [t[n] for n in ("x", "dt", "A", "B", "C")]
    before = op.launches()
    y, hT = op.forward(*args, h0=t["h0"])
    assert op.launches() == before + 1                     # one piece
    d = op.backward(dy, *args, dhT=dhT)
    wy, wh, wdh, wdA = _reference(t, dy, dhT)
    out = 0.0 if dtype == "f32" else 1.5 * 2.0 ** -9
    for name, got, want, bound in (("y", y, wy, tol + out), ("hT", hT, wh, tol), ("dh0", d["dh0"], wdh, tol),
                                   ("dA", d["dA"], wdA, 2 * tol)):
        e = (got.double() - want).norm().item() / want.norm().item()
        assert e <= bound, f"{name}: {e:.2e} > {bound:.1e}"
    for n in range(N):
        e = (hT[..., n].double() - wh[..., n]).norm().item() / wh[..., n].norm().item()
        assert e <= tol, f"state {n}: {e:.2e} > {tol:.1e}"


@pytest.mark.parametrize("T", [1, 4096])
def test_long_memories_of_a_step(T):
    """Serving: 4096 tokens in one call or one by one."""
    import torch
    import bwd_persistent_cta_gb300 as R
    total, B, D, N = 4096, 1, 16, 8
    gen = torch.Generator(device="cuda").manual_seed(42)
    rnd = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    t = {"x": 0.1 * rnd(total, B, D), "dt": 0.01 * torch.exp(0.5 * rnd(total, B, D)), "B": rnd(total, B, 1, N),
         "C": rnd(total, B, 1, N), "h0": 1 + 0.3 * rnd(B, D, N), "A": -torch.logspace(-3, -1, N, device="cuda").repeat(D, 1)}
    op = R.SelectiveScan(B, T, D, N, dtype="f32", softplus=False)
    st = t["h0"].clone()
    for i in range(0, total, T):
        x, dt, Bm, Cm = (t[n][i:i + T] for n in ("x", "dt", "B", "C"))
        op.step(x, dt, t["A"], Bm, Cm, st)
    h = t["h0"].double()
    for i in range(total):
        dt = t["dt"][i].double()
        h = torch.exp(dt[..., None] * t["A"].double()) * h + (dt * t["x"][i].double())[..., None] * t["B"][i].double()
    tol = total * 3e-9 + math.sqrt(total) * (4e-8 + EPS / 2)
    e = (st.double() - h).norm().item() / h.norm().item()
    assert e <= tol, f"{e:.2e} > {tol:.1e}"


def _values():
    import torch
    v = torch.cat([torch.linspace(-80, 80, 8001), torch.logspace(-6, 1, 500), -torch.logspace(-6, 1, 500)])
    return torch.cat([v, v.new_zeros(-v.numel() % 8)])


def _allowed(v):
    return (11.2 + 1.3 * v.abs()) * EPS


@pytest.mark.parametrize("how", ["forward", "step"])
def test_steps_far_from_zero(how):
    """One token from a state of zero with B = C = x = 1 returns the step 8 times.  softplus, relative: the exponent
    |v| log2(e) is a product rounded to half a step and a constant rounded by 0.32 * 2^-24 |v|, which the exponential
    scales by log(2): 1.3 |v| * 2^-24 at most; its own approximation and the reciprocal's 2^-22.7 and 2^-23, two sums,
    two products and the polynomial (0.13) one each: (5 + 2 + 4.13) * 2^-24."""
    import torch
    import bwd_persistent_cta_gb300 as R
    v = _values()
    D, N = v.numel(), 8
    op = R.SelectiveScan(1, 1, D, N, dtype="f32")
    one = torch.ones(1, 1, D, device="cuda")
    bc, A = torch.ones(1, 1, 1, N, device="cuda"), -torch.ones(D, N, device="cuda")
    args = (one, v.cuda().view(1, 1, D), A, bc, bc)
    if how == "forward":
        y, _ = op.forward(*args, train=False)
    else:
        y = op.step(*args, torch.zeros(1, D, N, device="cuda"))
    w = v.double()
    want = 8 * (w.clamp(min=0) + torch.log1p(torch.exp(-w.abs())))
    err = ((y.view(-1).cpu().double() - want) / want).abs() / _allowed(w)
    assert err.max().item() <= 1, (err.max().item(), v[err.argmax()].item())


@pytest.mark.parametrize("how", ["forward", "step", "ddt"])
def test_gates_far_from_zero(how):
    """silu of the gate, and the sigmoid in the step's gradient, to what the exponent's rounding leaves of them (as above,
    with a sum, a reciprocal and two products behind it)."""
    import torch
    import bwd_persistent_cta_gb300 as R
    v = _values()
    D, N = v.numel(), 8
    one, row = torch.ones(1, 1, D, device="cuda"), v.cuda().view(1, 1, D)
    bc, A = torch.ones(1, 1, 1, N, device="cuda"), torch.zeros(D, N, device="cuda")
    w = v.double()
    s = torch.exp(w.clamp(max=0)) / (1 + torch.exp(-w.abs()))
    if how == "ddt":
        # with dy = 1, x = 1 and A = 0: ddt = sum_n C B sigma(dt) = 8 sigma(dt)
        op = R.SelectiveScan(1, 1, D, N, dtype="f32")
        args = (one, row, A, bc, bc)
        op.forward(*args)
        got, want = op.backward(one, *args)["ddt"], 8 * s
    else:
        # without softplus a step of one: y = 8 silu(z)
        op = R.SelectiveScan(1, 1, D, N, dtype="f32", softplus=False)
        args = (one, one, A, bc, bc)
        got = op.forward(*args, z=row, train=False)[0] if how == "forward" else op.step(
            *args, torch.zeros(1, D, N, device="cuda"), z=row)
        want = 8 * w * s
    keep = want != 0
    err = ((got.view(-1).cpu().double() - want)[keep] / want[keep]).abs() / _allowed(w)[keep]
    assert err.max().item() <= 1, (err.max().item(), v[keep][err.argmax()].item())
