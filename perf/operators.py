"""Timed cases of the gated delta rule and of the block norm.

Each case runs one operator once.  Where ``own`` is false the operator is
computed in its plain form: elementary torch operations in 32 bits on the
inputs as they come, rounded once at the end.  Where it is true the case makes
the calls a user makes of ``bwd_persistent_cta_gb300``.  ``exact`` computes the
same outputs in 64 bits from the operator's definition, token by token.

Gated delta rule, per sequence and value head, with the state S [Dv, Dk], the
decay a_t = exp(g_t) and the key head shared by Hv / Hk value heads:

    e_t = v_t - a_t S_{t-1} k_t
    S_t = a_t S_{t-1} + beta_t e_t k_t^T
    o_t = scale S_t q_t                      scale = Dk^-1/2

Block norm, per row (and per group of ``cols`` columns):

    b = RMSNorm(y; w_in) * act(z),  x' = x + scale * b,  n = RMSNorm(x'; w_out)
"""
import math

import torch

own = False

CHUNK = 64
EPS = 1e-6


# --- the cases ---------------------------------------------------------------
def _prefill(B, T, Hk, Hv, Dk, Dv, dtype="bf16", ragged=False, bfirst=True):
    return dict(op="prefill", B=B, T=T, Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, dtype=dtype, ragged=ragged, bfirst=bfirst)


def _train(B, T, Hk, Hv, Dk, Dv, dtype="bf16", ragged=False, bfirst=True, state=False):
    return dict(op="train", B=B, T=T, Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, dtype=dtype, ragged=ragged, bfirst=bfirst,
                state=state)


def _step(B, T, Hk, Hv, Dk, Dv, dtype="bf16", ragged=False):
    return dict(op="step", B=B, T=T, Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, dtype=dtype, ragged=ragged)


def _norm(rows, groups, cols, dtype="bf16", train=True, gate="silu", block=True):
    return dict(op="norm", rows=rows, groups=groups, cols=cols, dtype=dtype, train=train, gate=gate, block=block)


def listed():
    return [
        # one short turn of a conversation added to a state kept from before
        dict(_prefill(1, 77, 4, 8, 64, 64), name="prefill_turn"),
        # a batch of prompts of unequal lengths, two value heads on a key head
        dict(_prefill(8, 1000, 8, 16, 128, 128, ragged=True), name="prefill_batch"),
        # one long document
        dict(_prefill(1, 16384, 16, 32, 128, 128), name="prefill_long"),
        # truncated backpropagation over a short ragged segment: a state comes in and its gradient goes out
        dict(_train(3, 190, 4, 4, 64, 64, ragged=True, bfirst=False, state=True), name="train_segment"),
        # an ordinary training batch
        dict(_train(8, 2048, 16, 16, 128, 128), name="train_batch"),
        # a run in 32 bits, unequal key and value widths
        dict(_train(2, 513, 2, 4, 64, 128, dtype="f32"), name="train_f32"),
        # one new token of one sequence: latency
        dict(_step(1, 1, 8, 16, 128, 128), name="step_one"),
        # one new token for each of a full serving batch
        dict(_step(256, 1, 16, 32, 128, 128), name="step_batch"),
        # up to four tokens accepted from a draft, a different number for each sequence
        dict(_step(48, 4, 8, 16, 128, 128, ragged=True), name="step_draft"),
        # the block boundary while decoding
        dict(_norm(16, 1, 2048, train=False), name="norm_decode"),
        # the gated norm of each value head's output, forward and backward
        dict(_norm(16384, 16, 128, block=False), name="norm_heads"),
        # the block boundary of a training step, forward and backward
        dict(_norm(16384, 1, 2048), name="norm_block"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: sizes over the logarithm of their range, odd ones among them."""
    op = rng.choice(("prefill", "prefill", "train", "train", "step", "norm"))
    if op == "norm":
        block = rng.random() < 0.5
        dtype = rng.choice(("bf16", "bf16", "f32"))
        train = rng.random() < 0.7
        cols = 8 * _log(rng, 8, 1024) if block else rng.choice((64, 128, 256))
        groups = 1 if block else rng.choice((4, 8, 16, 32))
        rows = _log(rng, 1, max(1, min(65536, (1 << 25) // (cols * groups))))
        return _norm(rows, groups, cols, dtype, train, rng.choice(("silu", "sigmoid")), block)
    Dk, Dv = rng.choice(((64, 64), (128, 128), (128, 128), (64, 128), (128, 64)))
    Hk = rng.choice((1, 2, 3, 4, 8, 16))
    Hv = Hk * rng.choice((1, 1, 2, 4) if Hk <= 8 else (1, 2))
    ragged = rng.random() < 0.5
    if op == "step":
        return _step(_log(rng, 1, 256), rng.choice((1, 1, 2, 3, 5)), Hk, min(Hv, 32), Dk, Dv, "bf16", ragged)
    bfirst = rng.random() < 0.6
    if op == "prefill":
        T = _log(rng, 1, 16384)
        B = _log(rng, 1, max(1, min(64, 262144 // (T * Hv))))
        return _prefill(B, T, Hk, Hv, Dk, Dv, "bf16", ragged, bfirst)
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    T = _log(rng, 1, 4096 if dtype == "bf16" else 1024)
    B = _log(rng, 1, max(1, min(32, (131072 if dtype == "bf16" else 8192) // (T * Hv))))
    return _train(B, T, Hk, Hv, Dk, Dv, dtype, ragged, bfirst, rng.random() < 0.5)


def _lengths(c):
    """Valid tokens of each sequence of a ragged case: from all of T down to none of it in a draft, to half elsewhere."""
    B, T = c["B"], c["T"]
    if c["op"] == "step":
        return [(b * 7 + 1) % (T + 1) for b in range(B)]
    return [T - (b * (T // 2)) // max(1, B - 1) for b in range(B)]


def _tokens(c):
    return sum(_lengths(c)) if c["ragged"] else c["B"] * c["T"]


def work(c):
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "norm":
        n = c["rows"] * c["groups"] * c["cols"]
        # forward: y, z (and x) in, x' (and n) out; backward: those inputs and the upstream gradients in, as many
        # gradients as inputs out.  Weights and their gradients are one row each.
        fwd, bwd = (5, 8) if c["block"] else (3, 5)
        return {"bytes": n * e * (fwd + (bwd if c["train"] else 0)), "flops": n * ((14 if c["block"] else 10) * (3 if c["train"] else 1))}
    tok, Hk, Hv, Dk, Dv = _tokens(c), c["Hk"], c["Hv"], c["Dk"], c["Dv"]
    io = tok * e * (2 * Hk * Dk + 2 * Hv * Dv + 2 * Hv)          # q, k, v, g, beta, o
    state = 4 * c["B"] * Hv * Dk * Dv
    if c["op"] == "step":
        # only sequences with a token touch their state
        live = sum(1 for n in _lengths(c) if n) if c["ragged"] else c["B"]
        state = 2 * 4 * live * Hv * Dk * Dv
        return {"bytes": io + state, "flops": 6 * tok * Hv * Dk * Dv}
    if c["op"] == "prefill":
        return {"bytes": io + 2 * state, "flops": 6 * tok * Hv * Dk * Dv}
    # the forward, then the backward: q, k, v, g, beta and do in, their five gradients out
    back = tok * e * (4 * Hk * Dk + 3 * Hv * Dv + 4 * Hv)
    return {"bytes": io + back + (4 * state if c["state"] else 0), "flops": 18 * tok * Hv * Dk * Dv}


# --- inputs ------------------------------------------------------------------
def _dt(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _delta_inputs(c, gen):
    """q, k, v as slices of one packed projection, g and beta of another, in the case's order of batch and time."""
    B, T, Hk, Hv, Dk, Dv = (c[n] for n in ("B", "T", "Hk", "Hv", "Dk", "Dv"))
    lead = (B, T) if c.get("bfirst", True) else (T, B)
    rnd = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    unit = lambda x: x / x.square().sum(-1, keepdim=True).add(1e-6).sqrt()  # noqa: E731
    act = lambda x: x * torch.sigmoid(x)  # noqa: E731
    packed = torch.empty(*lead, 2 * Hk * Dk + Hv * Dv, device="cuda", dtype=_dt(c))
    q, k, v = (t.unflatten(-1, (-1, d)) for t, d in zip(packed.split([Hk * Dk, Hk * Dk, Hv * Dv], -1), (Dk, Dk, Dv)))
    q.copy_(unit(act(rnd(*lead, Hk, Dk))))
    k.copy_(unit(act(rnd(*lead, Hk, Dk))))
    v.copy_(rnd(*lead, Hv, Dv))
    gates = torch.empty(*lead, 2 * Hv, device="cuda", dtype=_dt(c))
    g, beta = gates.split([Hv, Hv], -1)
    # memories of about three to a thousand tokens, one rate for each head
    rate = torch.exp(torch.empty(Hv, device="cuda").uniform_(math.log(1e-3), math.log(0.3), generator=gen))
    g.copy_(-rate * torch.log1p(torch.exp(0.5 + rnd(*lead, Hv))))
    beta.copy_(torch.sigmoid(rnd(*lead, Hv)))
    return q, k, v, g, beta


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rnd = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    s = {"case": c}
    if own:
        import bwd_persistent_cta_gb300 as R
    if c["op"] == "norm":
        rows, width, dt = c["rows"], c["groups"] * c["cols"], _dt(c)
        s["y"] = (rnd(rows, width) * torch.exp(rnd(rows, 1))).to(dt)
        s["z"] = rnd(rows, 2 * width).to(dt)[:, width:]          # the gate's half of a projection
        s["w_in"] = (1 + 0.1 * rnd(c["cols"])).to(dt)
        block = c["block"]
        s["x"] = (4 * rnd(rows, width)).to(dt) if block else None
        s["scale"] = (0.5 + 0.1 * rnd(c["cols"])).to(dt) if block else None
        s["w_out"] = (1 + 0.1 * rnd(c["cols"])).to(dt) if block else None
        s["dx_out"] = rnd(rows, width).to(dt) if c["train"] else None
        s["dn_out"] = rnd(rows, width).to(dt) if c["train"] and block else None
        if own:
            s["op"] = R.BlockNorm(rows, c["cols"], groups=c["groups"], dtype=c["dtype"], norm_in=True, gate=c["gate"],
                                  residual=block, norm_out=block, eps=EPS)
        return s
    s["in"] = _delta_inputs(c, gen)
    B, T, Hv, Dk, Dv = c["B"], c["T"], c["Hv"], c["Dk"], c["Dv"]
    lens = _lengths(c) if c["ragged"] else None
    s["lens"] = torch.tensor(lens if lens else [T] * B, device="cuda")
    if c["op"] == "step":
        # a pool of states, the batch's slots anywhere in it
        pool = B + B // 4 + 1
        s["state"] = 0.3 * rnd(pool, Hv, Dv, Dk)
        s["slots"] = torch.randperm(pool, device="cuda", generator=gen)[:B].to(torch.int32)
        s["o"] = torch.empty(B, T, Hv, Dv, device="cuda", dtype=_dt(c))
    else:
        given = c["op"] == "prefill" or c["state"]
        s["s0"] = 0.3 * rnd(B, Hv, Dv, Dk) if given else None
        if c["op"] == "train":
            s["do"] = rnd(*s["in"][2].shape).to(_dt(c))
            s["dsT"] = 0.1 * rnd(B, Hv, Dv, Dk) if given else None
    if own:
        s["op"] = R.DeltaRule(B, T, c["Hk"], Hv, Dk, Dv, dtype=c["dtype"], batch_first=c.get("bfirst", True))
        if lens:
            s["op"].set_seq_lengths(lens)
    return s


# --- one pass ----------------------------------------------------------------
def run(state):
    c = state["case"]
    if c["op"] == "norm":
        return _norm_own(state) if own else _norm_plain(state)
    if c["op"] == "step":
        return _step_own(state) if own else _step_plain(state)
    return _seq_own(state) if own else _seq_plain(state)


def _seq_own(s):
    c, op = s["case"], s["op"]
    o, sT = op.forward(*s["in"], s0=s["s0"], train=c["op"] == "train")
    if c["op"] == "prefill":
        return {"o": o, "sT": sT}
    dq, dk, dv, dg, dbeta, ds0 = op.backward(s["do"], *s["in"], s0=s["s0"], dsT=s["dsT"])
    out = {"o": o, "dq": dq, "dk": dk, "dv": dv, "dg": dg, "dbeta": dbeta}
    return dict(out, sT=sT, ds0=ds0) if c["state"] else out


def _step_own(s):
    s["op"].step(*s["in"], s["state"], slots=s["slots"], o=s["o"])
    return {"o": s["o"], "state": s["state"]}


def _norm_own(s):
    op = s["op"]
    x_out, n_out = op.forward(s["y"], z=s["z"], x=s["x"], w_in=s["w_in"], scale=s["scale"], w_out=s["w_out"])
    out = {"x_out": x_out} if n_out is None else {"x_out": x_out, "n_out": n_out}
    if s["case"]["train"]:
        d = op.backward(s["dx_out"], s["dn_out"], s["y"], z=s["z"], x=s["x"], w_in=s["w_in"], scale=s["scale"],
                        w_out=s["w_out"])
        out.update({n: t for n, t in d.items() if t is not None})
    return out


# --- plain forms -------------------------------------------------------------
def _chunked(s):
    """The inputs in 32 bits as [B, Hv, N, 64, D] (gates without D), zero beyond each sequence's length."""
    c = s["case"]
    T, pad = c["T"], -c["T"] % CHUNK
    live = torch.arange(T, device="cuda")[None, :] < s["lens"][:, None]

    def one(x, group):
        x = x.float() if c.get("bfirst", True) else x.float().transpose(0, 1)
        x = torch.where(live.reshape(live.shape + (1,) * (x.dim() - 2)), x, 0.0)
        x = torch.cat([x, x.new_zeros(x.shape[0], pad, *x.shape[2:])], 1) if pad else x
        x = x.transpose(1, 2).unflatten(2, (-1, CHUNK))
        return x.repeat_interleave(group, 1) if group > 1 else x

    n = c["Hv"] // c["Hk"]
    q, k, v, g, beta = s["in"]
    return live, one, [one(q, n), one(k, n), one(v, 1), one(g, 1), one(beta, 1)]


def _inverse(A):
    """(I + A)^-1 for strictly lower triangular A [..., 64, 64]: the inverses of blocks of 1, 2, 4, ... joined in pairs,
    [[X, 0], [-Y L X, Y]]."""
    X = torch.ones(*A.shape[:-2], CHUNK, 1, 1, device=A.device)
    for b in (1, 2, 4, 8, 16, 32):
        m = CHUNK // (2 * b)
        L = A.unflatten(-1, (m, 2, b)).unflatten(-4, (m, 2, b))       # [..., m, 2, b, m, 2, b]
        L = torch.diagonal(L[..., :, 1, :, :, 0, :], dim1=-4, dim2=-2).movedim(-1, -3)
        X = X.unflatten(-3, (m, 2))
        top, low = X[..., 0, :, :], X[..., 1, :, :]
        X = torch.cat([torch.cat([top, torch.zeros_like(top)], -1), torch.cat([-(low @ L @ top), low], -1)], -2)
    return X.squeeze(-3)


def _seq_plain(s):
    c = s["case"]
    B, T, Hk, Hv, Dk, Dv = (c[n] for n in ("B", "T", "Hk", "Hv", "Dk", "Dv"))
    live, one, (q, k, v, g, beta) = _chunked(s)
    scale = Dk ** -0.5
    G = g.cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, device="cuda", dtype=torch.bool).tril()
    D = torch.exp(torch.where(low, G[..., :, None] - G[..., None, :], -math.inf))
    eG, eE, eC = torch.exp(G)[..., None], torch.exp(G[..., -1:] - G)[..., None], torch.exp(G[..., -1])
    A = (D * (k @ k.mT)).tril(-1)
    P = scale * D * (q @ k.mT)
    X = _inverse(A * beta[..., None, :])                          # e = X (v - exp(G) k S)
    W, V = X @ (eG * k), X @ v
    S = torch.zeros(B, Hv, Dk, Dv, device="cuda") if s["s0"] is None else s["s0"].mT
    b1 = beta[..., None]
    kE = eE * k
    before, e = [], []
    for n in range(k.shape[2]):
        before.append(S)
        e.append(V[:, :, n] - W[:, :, n] @ S)
        S = eC[:, :, n, None, None] * S + kE[:, :, n].mT @ (b1[:, :, n] * e[n])
    S0, e = torch.stack(before, 2), torch.stack(e, 2)
    u = b1 * e
    o = scale * eG * (q @ S0) + P @ u

    def back(x, heads=None, dtype=None):
        """[B, Hv, N, 64, ...] to the caller's order, the value heads of a key head summed."""
        x = x.flatten(2, 3)[:, :, :T]
        if heads and heads != Hv:
            x = x.unflatten(1, (heads, Hv // heads)).sum(2)
        x = x.transpose(1, 2)
        x = torch.where(live.reshape(live.shape + (1,) * (x.dim() - 2)), x, 0.0)
        x = x if c["bfirst"] else x.transpose(0, 1)
        return x.to(dtype or _dt(c)).contiguous()

    if c["op"] == "prefill":
        return {"o": back(o), "sT": S.mT.contiguous()}

    do = one(s["do"], 1)
    Y = _inverse(beta[..., :, None] * A).mT                       # y = Y du
    y0, Yk = Y @ (P.mT @ do), Y @ kE
    SQ = (scale * eG * q).mT @ do
    kX = (eG * b1 * k).mT
    dS = torch.zeros(B, Hv, Dk, Dv, device="cuda") if s["dsT"] is None else s["dsT"].mT
    after, y = [None] * k.shape[2], [None] * k.shape[2]
    for n in reversed(range(k.shape[2])):
        after[n] = dS
        y[n] = y0[:, :, n] + Yk[:, :, n] @ dS
        dS = eC[:, :, n, None, None] * dS + SQ[:, :, n] - kX[:, :, n] @ y[n]
    dS1, y = torch.stack(after, 2), torch.stack(y, 2)
    de = b1 * y
    dP = (do @ u.mT) * P                                          # times P: what reaches the decays
    dA = -(de @ u.mT) * A
    dq1 = scale * eG * (do @ S0.mT)
    dk1 = -eG * (de @ S0.mT)
    dk3 = eE * (u @ dS1.mT)
    mP, mA = scale * D * (do @ u.mT), -(D * (de @ u.mT)).tril(-1)
    dq = dq1 + mP @ k
    dk = dk1 + dk3 + mP.mT @ q + mA @ k + mA.mT @ k
    dbeta = (y * e).sum(-1)
    out_of = (k * dk3).sum(-1)
    dG = (dP + dA).sum(-1) - (dP + dA).sum(-2) + (q * dq1).sum(-1) + (k * dk1).sum(-1) - out_of
    last = out_of.sum(-1) + eC * (S0 * dS1).sum((-1, -2))
    dg = dG.flip(-1).cumsum(-1).flip(-1) + last[..., None]
    out = {"o": back(o), "dq": back(dq, Hk), "dk": back(dk, Hk), "dv": back(de), "dg": back(dg), "dbeta": back(dbeta)}
    return dict(out, sT=S.mT.contiguous(), ds0=dS.mT.contiguous()) if c["state"] else out


def _step_plain(s):
    c = s["case"]
    n = c["Hv"] // c["Hk"]
    q, k, v, g, beta = (x.float() for x in s["in"])
    q, k = (x.repeat_interleave(n, 2) if n > 1 else x for x in (q, k))
    at = s["slots"].long()
    S = s["state"][at]
    for t in range(c["T"]):
        live = (t < s["lens"])[:, None, None]
        Sn = S * torch.exp(g[:, t])[..., None, None]
        e = v[:, t] - (Sn * k[:, t, :, None, :]).sum(-1)
        Sn = Sn + (beta[:, t, :, None] * e)[..., None] * k[:, t, :, None, :]
        o = c["Dk"] ** -0.5 * (Sn * q[:, t, :, None, :]).sum(-1)
        s["o"][:, t] = torch.where(live, o, 0.0).to(s["o"].dtype)
        S = torch.where(live[..., None], Sn, S)
    s["state"][at] = S
    return {"o": s["o"], "state": s["state"]}


def _act(z, gate):
    sg = torch.sigmoid(z)
    return (z * sg, sg * (1 + z * (1 - sg))) if gate == "silu" else (sg, sg * (1 - sg))


def _norm_plain(s):
    c = s["case"]
    rows, dt = c["rows"], _dt(c)
    f = lambda x: None if x is None else x.float().reshape(rows, c["groups"], c["cols"])  # noqa: E731
    w = lambda x: None if x is None else x.float()  # noqa: E731
    y, z, x, w_in, scale, w_out = f(s["y"]), f(s["z"]), f(s["x"]), w(s["w_in"]), w(s["scale"]), w(s["w_out"])
    rms = lambda t: torch.rsqrt(t.square().mean(-1, keepdim=True) + EPS)  # noqa: E731
    act, dact = _act(z, c["gate"])
    r1 = rms(y)
    a = y * r1 * w_in
    b = a * act
    x1 = x + scale * b if c["block"] else b
    flat = lambda t: t.reshape(rows, -1).to(dt)  # noqa: E731
    out = {"x_out": flat(x1)}
    if c["block"]:
        r2 = rms(x1)
        out["n_out"] = flat(x1 * r2 * w_out)
    if not c["train"]:
        return out
    dx = f(s["dx_out"])
    if c["block"]:
        dn = f(s["dn_out"])
        out["dw_out"] = (dn * x1 * r2).sum((0, 1))
        h = dn * w_out
        dx = dx + r2 * h - x1 * r2 ** 3 * (h * x1).mean(-1, keepdim=True)
        out["dx"] = flat(dx)
        out["dscale"] = (dx * b).sum((0, 1))
        dx = dx * scale
    out["dz"] = flat(dx * a * dact)
    da = dx * act
    out["dw_in"] = (da * y * r1).sum((0, 1))
    h = da * w_in
    out["dy"] = flat(r1 * h - y * r1 ** 3 * (h * y).mean(-1, keepdim=True))
    return out


# --- 64 bits, from the definitions ---------------------------------------------
def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "norm":
        return _norm_exact(s)
    if c["op"] == "step":
        return _step_exact(s)
    return _seq_exact(s)


def _dbl(x):
    return None if x is None else x.double()


def _seq_exact(s):
    c = s["case"]
    B, T, Hk, Hv, Dk, Dv = (c[n] for n in ("B", "T", "Hk", "Hv", "Dk", "Dv"))
    train, n = c["op"] == "train", c["Hv"] // c["Hk"]
    time_first = lambda x: _dbl(x.transpose(0, 1) if c["bfirst"] else x)  # noqa: E731
    q, k, v, g, beta = (time_first(x) for x in s["in"])
    do = time_first(s["do"]) if train else None
    out = {m: torch.zeros_like(x) for m, x in (("o", v), ("dq", q), ("dk", k), ("dv", v), ("dg", g), ("dbeta", beta))}
    zero = torch.zeros(B, Hv, Dv, Dk, device="cuda", dtype=torch.float64)
    sT, ds0 = zero.clone(), zero.clone()
    # as many sequences at once as their saved states have room for
    many = max(1, int(8e9 // (T * Hv * Dk * Dv * 8))) if train else B
    scale = Dk ** -0.5
    heads = lambda x: x.repeat_interleave(n, 1)  # noqa: E731
    fold = lambda x: x.unflatten(1, (Hk, n)).sum(2)  # noqa: E731
    for b in range(0, B, many):
        z = slice(b, min(B, b + many))
        S = zero[z].clone() if s["s0"] is None else s["s0"][z].double()
        kept = []
        for t in range(T):
            live = (t < s["lens"][z]).double()[:, None]
            a = torch.exp(g[t, z] * live)
            kt, bt = heads(k[t, z]), beta[t, z] * live
            Sa = a[..., None, None] * S
            e = v[t, z] - torch.einsum("bhvk,bhk->bhv", Sa, kt)
            kept.append((S, e) if train else None)
            S = Sa + (bt[..., None] * e)[..., None] * kt[:, :, None, :]
            out["o"][t, z] = live[..., None] * scale * torch.einsum("bhvk,bhk->bhv", S, heads(q[t, z]))
        sT[z] = S
        if not train:
            continue
        dS = zero[z].clone() if s["dsT"] is None else s["dsT"][z].double()
        after = S
        for t in reversed(range(T)):
            live = (t < s["lens"][z]).double()[:, None]
            a = torch.exp(g[t, z] * live)
            kt, qt, bt, (S, e) = heads(k[t, z]), heads(q[t, z]), beta[t, z] * live, kept.pop()
            dot = scale * live[..., None] * do[t, z]
            out["dq"][t, z] = fold(torch.einsum("bhvk,bhv->bhk", after, dot))
            dS = dS + dot[..., None] * qt[:, :, None, :]
            du = torch.einsum("bhvk,bhk->bhv", dS, kt)
            de = bt[..., None] * du
            Sa = a[..., None, None] * S
            dk = torch.einsum("bhvk,bhv->bhk", dS, bt[..., None] * e) - torch.einsum("bhvk,bhv->bhk", Sa, de)
            out["dk"][t, z] = fold(dk)
            out["dv"][t, z] = de
            out["dbeta"][t, z] = live * (du * e).sum(-1)
            dS = dS - de[..., None] * kt[:, :, None, :]
            out["dg"][t, z] = live * (dS * Sa).sum((-1, -2))
            dS = a[..., None, None] * dS
            after = S
        ds0[z] = dS
    order = lambda x: x.transpose(0, 1).contiguous() if c["bfirst"] else x  # noqa: E731
    if not train:
        return {"o": order(out["o"]), "sT": sT}
    out = {m: order(x) for m, x in out.items()}
    return dict(out, sT=sT, ds0=ds0) if c["state"] else out


def _step_exact(s):
    c = s["case"]
    n = c["Hv"] // c["Hk"]
    q, k, v, g, beta = (_dbl(x) for x in s["in"])
    o = torch.zeros(v.shape, device="cuda", dtype=torch.float64)
    pool = s["state"].double()
    at = s["slots"].long()
    S = pool[at]
    for t in range(c["T"]):
        live = (t < s["lens"]).double()[:, None]
        kt, qt = (x[:, t].repeat_interleave(n, 1) for x in (k, q))
        S = torch.exp(g[:, t] * live)[..., None, None] * S
        u = (beta[:, t] * live)[..., None] * (v[:, t] - torch.einsum("bhvk,bhk->bhv", S, kt))
        S = S + u[..., None] * kt[:, :, None, :]
        o[:, t] = live[..., None] * c["Dk"] ** -0.5 * torch.einsum("bhvk,bhk->bhv", S, qt)
    pool[at] = S
    return {"o": o, "state": pool}


def _norm_exact(s):
    """The forward in 64 bits; the gradients as those of the sum of outputs times upstream gradients, by the quotient rule."""
    c = s["case"]
    rows, groups, cols = c["rows"], c["groups"], c["cols"]
    f = lambda x: None if x is None else x.double().reshape(rows * groups, cols)  # noqa: E731
    y, z, x = f(s["y"]), f(s["z"]), f(s["x"])
    w_in, scale, w_out = _dbl(s["w_in"]), _dbl(s["scale"]), _dbl(s["w_out"])
    n1 = ((y * y).sum(1, keepdim=True) / cols + EPS).sqrt()
    sg = 1 / (1 + torch.exp(-z))
    act = z * sg if c["gate"] == "silu" else sg
    b = y / n1 * w_in * act
    x1 = b if x is None else x + scale * b
    flat = lambda t: t.reshape(rows, groups * cols)  # noqa: E731
    out = {"x_out": flat(x1)}
    n2 = ((x1 * x1).sum(1, keepdim=True) / cols + EPS).sqrt()
    if x is not None:
        out["n_out"] = flat(x1 / n2 * w_out)
    if not c["train"]:
        return out
    norm_back = lambda h, t, m: (h - t * ((h * t).sum(1, keepdim=True) / (cols * m * m))) / m  # noqa: E731
    d = f(s["dx_out"])
    if x is not None:
        dn = f(s["dn_out"])
        out["dw_out"] = (dn * x1 / n2).sum(0)
        d = d + norm_back(dn * w_out, x1, n2)
        out["dx"], out["dscale"] = flat(d), (d * b).sum(0)
        d = d * scale
    dact = sg + z * sg * (1 - sg) if c["gate"] == "silu" else sg * (1 - sg)
    out["dz"] = flat(d * y / n1 * w_in * dact)
    out["dw_in"] = (d * act * y / n1).sum(0)
    out["dy"] = flat(norm_back(d * act * w_in, y, n1))
    return out
