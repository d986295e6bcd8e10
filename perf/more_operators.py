"""Timed cases of the selective scan, of the causal convolution before it and of
gradient clipping.

Each case runs one operator once.  Where ``own`` is false the operator is
computed in its plain form: elementary torch operations in 32 bits (64 for the
sums of a whole model's squares), rounded once at the end.  Where it is true the
case makes the calls a user makes of ``bwd_persistent_cta_gb300``.  ``exact``
computes the same outputs in 64 bits from the operator's definition, token by
token.

Selective scan, per sequence and channel d, with N states a channel, d's group
of B and C, and delta_t = softplus(dt_t + dt_bias):

    h_t[n] = exp(delta_t A[n]) h_{t-1}[n] + delta_t x_t B_t[n]
    y_t    = (sum_n C_t[n] h_t[n] + D x_t) * silu(z_t)

Causal convolution, per sequence and channel, W taps, x before the sequence from
the state of the last W - 1 inputs:

    y_t = silu(bias + sum_k w[k] x_{t-W+1+k})

Clipping, over a list of gradient tensors:

    norm = sqrt(sum of all squares),  out = g * min(1, max_norm / (norm + 1e-6))
"""
import math

import torch

own = False

CLIP_EPS = 1e-6


# --- the cases ---------------------------------------------------------------
def _scan(op, B, T, D, N=16, G=1, dtype="bf16", ragged=False, bfirst=True, state=False):
    return dict(op=op, B=B, T=T, D=D, N=N, G=G, dtype=dtype, ragged=ragged, bfirst=bfirst, state=state)


def _conv(op, B, T, D, W=4, dtype="bf16", ragged=False, bfirst=True, state=False):
    return dict(op=op, B=B, T=T, D=D, W=W, dtype=dtype, ragged=ragged, bfirst=bfirst, state=state)


def _clip(blocks, width, dtype="bf16", flat=False, inplace=False, size=1.0):
    return dict(op="clip", blocks=blocks, width=width, dtype=dtype, flat=flat, inplace=inplace, size=size)


def listed():
    return [
        # one short turn of a conversation, added to the state kept from before
        dict(_scan("scan_prefill", 1, 77, 1024, state=True), name="scan_turn"),
        # a batch of prompts of unequal lengths
        dict(_scan("scan_prefill", 8, 1000, 2048, ragged=True), name="scan_batch"),
        # one long document
        dict(_scan("scan_prefill", 1, 16384, 4096), name="scan_long"),
        # an ordinary training batch
        dict(_scan("scan_train", 8, 2048, 2048), name="scan_train"),
        # a run in 32 bits: two groups, truncated segments of unequal lengths, a state in and its gradient out
        dict(_scan("scan_train", 3, 513, 528, G=2, dtype="f32", ragged=True, bfirst=False, state=True), name="scan_train_f32"),
        # one new token of one sequence: latency
        dict(_scan("scan_step", 1, 1, 2048, state=True), name="scan_step_one"),
        # one new token for each of a full serving batch
        dict(_scan("scan_step", 256, 1, 4096, state=True), name="scan_step_batch"),
        # the convolution of that batch of prompts
        dict(_conv("conv_prefill", 8, 1000, 2048, ragged=True, state=True), name="conv_batch"),
        # the convolution of a training batch, forward and backward
        dict(_conv("conv_train", 8, 2048, 4096), name="conv_train"),
        # the convolution of a serving batch's new tokens
        dict(_conv("conv_step", 256, 1, 4096, state=True), name="conv_step_batch"),
        # a small model's gradients, many of them small, as slices of one buffer
        dict(_clip(12, 64, dtype="f32", flat=True), name="clip_small"),
        # a large model's gradients, matrices and vectors
        dict(_clip(24, 2048), name="clip_large"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: sizes over the logarithm of their range, odd ones among them."""
    op = rng.choice(("scan_prefill", "scan_prefill", "scan_train", "scan_train", "scan_step", "conv_prefill", "conv_train",
                     "conv_step", "clip"))
    if op == "clip":
        width = _log(rng, 8, 4096)
        return _clip(min(32, _log(rng, 1, max(1, min(48, (1 << 25) // (width * width))))), width,
                     rng.choice(("bf16", "f32", "mixed")), rng.random() < 0.3, rng.random() < 0.5, rng.choice((1.0, 1.0, 1e-3, 0.01)))
    D = 8 * _log(rng, 1, 512)
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    ragged, bfirst, state = rng.random() < 0.5, rng.random() < 0.6, rng.random() < 0.5
    if op.startswith("conv"):
        W = rng.choice((2, 3, 4, 4, 4))
        if op == "conv_step":
            return _conv(op, _log(rng, 1, 256), rng.choice((1, 1, 2, 3, 5)), D, W, dtype, ragged, True, True)
        T = _log(rng, 1, 16384)
        return _conv(op, _log(rng, 1, max(1, min(64, (1 << 25) // (T * D)))), T, D, W, dtype, ragged, bfirst, state)
    N = rng.choice((16, 16, 16, 8, 32, 64))
    G = rng.choice((1, 1, 2, 4)) if D % 32 == 0 else 1
    if op == "scan_step":
        return _scan(op, _log(rng, 1, 256), rng.choice((1, 1, 2, 3, 5)), D, N, G, dtype, ragged, True, True)
    T = _log(rng, 1, 16384 if op == "scan_prefill" else 4096)
    B = _log(rng, 1, max(1, min(64, (1 << (28 if op == "scan_prefill" else 27)) // (T * D * N))))
    return _scan(op, B, T, D, N, G, dtype, ragged, bfirst, state)


def _lengths(c):
    """Valid tokens of each sequence of a ragged case: from all of T down to none of it in a step, to half elsewhere."""
    B, T = c["B"], c["T"]
    if c["op"].endswith("step"):
        return [(b * 7 + 1) % (T + 1) for b in range(B)]
    return [T - (b * (T // 2)) // max(1, B - 1) for b in range(B)]


def _sizes(c):
    """Elements of each gradient of a clipping case: three matrices and four vectors a block."""
    w = c["width"]
    return [2 * w * w, 2 * w * w, w * w, w, 2 * w, 7, w + 1] * c["blocks"]


def work(c):
    if c["op"] == "clip":
        s = _sizes(c)
        e = [_bytes(c, i) for i in range(len(s))]
        return {"bytes": 2 * sum(n * b for n, b in zip(s, e)), "flops": 3 * sum(s)}
    e = 2 if c["dtype"] == "bf16" else 4
    lens = _lengths(c) if c["ragged"] else [c["T"]] * c["B"]
    tok, live, D = sum(lens), sum(1 for n in lens if n), c["D"]
    train = c["op"].endswith("train")
    if c["op"].startswith("conv"):
        W = c["W"]
        state = e * D * (W - 1) * (live if c["op"] == "conv_step" else c["B"])
        # x in, y out; in training x and the gradient of y in again, the gradient of x out
        io = tok * D * e * (5 if train else 2) + D * (W + 1) * (e + (4 if train else 0))
        moves = 4 if train and c["state"] else 2 if c["state"] or not train else 0
        return {"bytes": io + moves * state, "flops": tok * D * ((2 * W + 4) * (3 if train else 1))}
    N, G = c["N"], c["G"]
    # x, dt, z, B and C in, y out
    io = tok * e * (4 * D + 2 * G * N) + 4 * D * (N + 2)
    state = 4 * D * N * (live if c["op"] == "scan_step" else c["B"])
    if train:
        # those inputs and the gradient of y in again, and the gradients of the inputs out
        io += tok * e * (7 * D + 4 * G * N) + 4 * 2 * D * (N + 2)
        return {"bytes": io + (4 * state if c["state"] else 0), "flops": tok * D * (21 * N + 40)}
    return {"bytes": io + state * (2 if c["state"] else 1), "flops": tok * D * (7 * N + 12)}


# --- inputs ------------------------------------------------------------------
def _dt(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _bytes(c, i):
    """Of an element of gradient i: vectors of a mixed model are held in 32 bits."""
    return 4 if c["dtype"] == "f32" or (c["dtype"] == "mixed" and i % 7 >= 3) else 2


def _silu(x):
    return x * torch.sigmoid(x)


def _prepare_clip(c, rnd):
    sizes = _sizes(c)
    types = [torch.float32 if _bytes(c, i) == 4 else torch.bfloat16 for i in range(len(sizes))]
    # gradients of one model: of sizes a few powers of ten apart, and together about ``size`` times sqrt(1000) long
    spread = [10.0 ** (i % 4 - 2) for i in range(len(sizes))]
    norm = math.sqrt(sum(n * s * s for n, s in zip(sizes, spread)))
    many = [c["size"] * 30 / norm * s for s in spread]
    # in one buffer of each type, end to end or each on a boundary of its own
    grain = 1 if c["flat"] else 64
    place, used = [], dict.fromkeys(types, 0)
    for n, t in zip(sizes, types):
        place.append((t, used[t], n))
        used[t] += (n + grain - 1) // grain * grain
    whole = {t: torch.zeros(n, device="cuda", dtype=t) for t, n in used.items()}
    grads = [whole[t][at:at + n] for t, at, n in place]
    for g, m in zip(grads, many):
        g.copy_(m * rnd(g.numel()))
    s = {"case": c, "place": place, "grads": grads, "whole": list(whole.values())}
    if not c["inplace"]:
        whole = {t: torch.zeros_like(w) for t, w in whole.items()}
        s["out"] = [whole[t][at:at + n] for t, at, n in place]
        s["whole"] = list(whole.values())
    if own:
        import bwd_persistent_cta_gb300 as R
        s["op"] = R.GradClip(sizes, ["f32" if t is torch.float32 else "bf16" for t in types])
    return s


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rnd = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    if c["op"] == "clip":
        return _prepare_clip(c, rnd)
    B, T, D, dt = c["B"], c["T"], c["D"], _dt(c)
    lead = (B, T) if c["bfirst"] else (T, B)
    lens = _lengths(c) if c["ragged"] else None
    s = {"case": c, "lens": torch.tensor(lens if lens else [T] * B, device="cuda")}
    step, train = c["op"].endswith("step"), c["op"].endswith("train")
    # a pool of states, the batch's slots anywhere in it
    pool = B + B // 4 + 1
    if step:
        s["slots"] = torch.randperm(pool, device="cuda", generator=gen)[:B].to(torch.int32)
        s["y"] = torch.empty(B, T, D, device="cuda", dtype=dt)
    # x and z: halves of one projection
    xz = rnd(*lead, 2 * D).to(dt)
    if train:
        s["dy"] = rnd(*lead, D).to(dt)
    if c["op"].startswith("conv"):
        W = c["W"]
        s["x"], _ = xz.split(D, -1)
        s["w"] = (rnd(D, W) / W ** 0.5).to(dt)
        s["bias"] = (0.1 * rnd(D)).to(dt)
        if step:
            s["state"] = rnd(pool, W - 1, D).to(dt)
        else:
            s["s0"] = rnd(B, W - 1, D).to(dt) if c["state"] else None
            s["dsT"] = rnd(B, W - 1, D).to(dt) if c["state"] and train else None
        if own:
            import bwd_persistent_cta_gb300 as R
            s["op"] = R.CausalConv(B, T, D, W, dtype=c["dtype"], act="silu", batch_first=c["bfirst"])
            if lens:
                s["op"].set_seq_lengths(lens)
        return s
    N, G = c["N"], c["G"]
    _, s["z"] = xz.split(D, -1)
    s["x"] = _silu(rnd(*lead, D)).to(dt)
    # the steps' low rank, B and C: slices of another projection
    rank = 8 * ((D + 127) // 128)
    _, b, cc = rnd(*lead, rank + 2 * G * N).to(dt).split([rank, G * N, G * N], -1)
    s["B"], s["C"] = b.unflatten(-1, (G, N)), cc.unflatten(-1, (G, N))
    s["dt"] = (0.7 * rnd(*lead, D)).to(dt)
    # steps from 0.001 to 0.1, rates from 1 to N
    step0 = torch.exp(torch.empty(D, device="cuda").uniform_(math.log(1e-3), math.log(0.1), generator=gen))
    s["dt_bias"] = step0 + torch.log(-torch.expm1(-step0))
    s["A"] = -torch.arange(1, N + 1, device="cuda") * torch.exp(0.2 * rnd(D, N))
    s["D"] = 1 + 0.1 * rnd(D)
    if step:
        s["state"] = 0.3 * rnd(pool, D, N)
    else:
        s["h0"] = 0.3 * rnd(B, D, N) if c["state"] else None
        s["dhT"] = 0.1 * rnd(B, D, N) if c["state"] and train else None
    if own:
        import bwd_persistent_cta_gb300 as R
        s["op"] = R.SelectiveScan(B, T, D, N, groups=G, dtype=c["dtype"], batch_first=c["bfirst"])
        if lens:
            s["op"].set_seq_lengths(lens)
    return s


# --- one pass ----------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if op == "clip":
        return _clip_own(state) if own else _clip_plain(state)
    if op.startswith("conv"):
        return _conv_own(state) if own else _conv_plain(state)
    return _scan_own(state) if own else _scan_plain(state)


def _scan_own(s):
    c, op = s["case"], s["op"]
    ins = (s["x"], s["dt"], s["A"], s["B"], s["C"])
    more = dict(z=s["z"], D=s["D"], dt_bias=s["dt_bias"])
    if c["op"] == "scan_step":
        op.step(*ins, s["state"], **more, slots=s["slots"], y=s["y"])
        return {"y": s["y"], "state": s["state"]}
    train = c["op"] == "scan_train"
    y, hT = op.forward(*ins, **more, h0=s["h0"], train=train)
    if not train:
        return {"y": y, "hT": hT}
    d = op.backward(s["dy"], *ins, **more, dhT=s["dhT"])
    out = {"y": y, **{n: d[n] for n in ("dx", "ddt", "dA", "dB", "dC", "dz", "dD", "ddt_bias")}}
    return dict(out, hT=hT, dh0=d["dh0"]) if c["state"] else out


def _conv_own(s):
    c, op = s["case"], s["op"]
    if c["op"] == "conv_step":
        op.step(s["x"], s["w"], s["state"], bias=s["bias"], slots=s["slots"], y=s["y"])
        return {"y": s["y"], "state": s["state"]}
    y, sT = op.forward(s["x"], s["w"], bias=s["bias"], s0=s["s0"])
    if c["op"] == "conv_prefill":
        return {"y": y, "sT": sT}
    d = op.backward(s["dy"], s["x"], s["w"], bias=s["bias"], s0=s["s0"], dsT=s["dsT"])
    out = {"y": y, **{n: d[n] for n in ("dx", "dw", "dbias")}}
    return dict(out, sT=sT, ds0=d["ds0"]) if c["state"] else out


def _clip_own(s):
    norm = s["op"].clip(s["grads"], 1.0, eps=CLIP_EPS, out=s.get("out"))
    return {"norm": norm, "out": s["whole"]}


# --- plain forms -------------------------------------------------------------
def _live(s, t):
    """Whether each token of [B, T] is valid, with ``t``'s trailing dimensions."""
    c = s["case"]
    live = torch.arange(c["T"], device="cuda")[None, :] < s["lens"][:, None]
    return live.reshape(live.shape + (1,) * (t.dim() - 2))


def _batch(s, x):
    """``x`` in 32 bits as [B, T, ...], zero beyond each sequence's length."""
    x = x if s["case"]["bfirst"] else x.transpose(0, 1)
    return torch.where(_live(s, x), x.float(), 0.0)


def _back(s, x):
    """[B, T, ...] in the caller's order and type, zero beyond each sequence's length."""
    x = torch.where(_live(s, x), x, 0.0).to(_dt(s["case"]))
    return (x if s["case"]["bfirst"] else x.transpose(0, 1)).contiguous()


def _recur(a, b, h0):
    """h_t = a_t h_{t-1} + b_t over dimension 1 of [B, T, ...]: about sqrt(T) chunks side by side, then joined."""
    B, T = a.shape[:2]
    L = max(1, math.isqrt(T))
    pad = -T % L
    if pad:
        a = torch.cat([a, a.new_ones(B, pad, *a.shape[2:])], 1)
        b = torch.cat([b, b.new_zeros(B, pad, *b.shape[2:])], 1)
    a, b = a.unflatten(1, (-1, L)).clone(), b.unflatten(1, (-1, L)).clone()
    for t in range(1, L):
        b[:, :, t] += a[:, :, t] * b[:, :, t - 1]
        a[:, :, t] *= a[:, :, t - 1]
    carry = [h0]
    for n in range(a.shape[1] - 1):
        carry.append(a[:, n, -1] * carry[-1] + b[:, n, -1])
    h = b + a * torch.stack(carry, 1)[:, :, None]
    return h.flatten(1, 2)[:, :T]


def _scan_plain(s):
    c = s["case"]
    B, T, D, N, G = (c[n] for n in ("B", "T", "D", "N", "G"))
    x, dt, z, Bm, Cm = (_batch(s, s[n]) for n in ("x", "dt", "z", "B", "C"))
    Bm, Cm = (t.repeat_interleave(D // G, 2) for t in (Bm, Cm))                # [B, T, D, N]
    v = dt + s["dt_bias"]
    delta = torch.where(_live(s, v), v.clamp(min=0) + torch.log1p(torch.exp(-v.abs())), 0.0)
    a = torch.exp(delta[..., None] * s["A"])
    step = c["op"] == "scan_step"
    h0 = s["state"][s["slots"].long()] if step else x.new_zeros(B, D, N) if s["h0"] is None else s["h0"]
    h = _recur(a, (delta * x)[..., None] * Bm, h0)
    y = (h * Cm).sum(-1) + s["D"] * x
    sz = torch.sigmoid(z)
    out = {"y": _back(s, y * z * sz)}
    if step:
        s["state"][s["slots"].long()] = h[:, -1]
        s["y"].copy_(out["y"])
        return {"y": s["y"], "state": s["state"]}
    if c["op"] == "scan_prefill":
        return dict(out, hT=h[:, -1].contiguous())
    do = _batch(s, s["dy"])
    dy = do * z * sz
    out["dz"] = _back(s, do * y * sz * (1 + z * (1 - sz)))
    after = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1).flip(1)
    end = x.new_zeros(B, D, N) if s["dhT"] is None else s["dhT"]
    g = _recur(after, (dy[..., None] * Cm).flip(1), end).flip(1)
    over = lambda t: t.unflatten(2, (G, -1)).sum(3)  # noqa: E731
    out["dC"] = _back(s, over(dy[..., None] * h))
    out["dB"] = _back(s, over(g * (delta * x)[..., None]))
    ga = g * a
    p = ga * torch.cat([h0[:, None], h[:, :-1]], 1)
    gB = (g * Bm).sum(-1)
    out["dx"] = _back(s, delta * gB + s["D"] * dy)
    ddt = (x * gB + (p * s["A"]).sum(-1)) * torch.sigmoid(v)
    ddt = torch.where(_live(s, ddt), ddt, 0.0)
    out["ddt"] = _back(s, ddt)
    out["dA"] = (p * delta[..., None]).sum((0, 1))
    out["dD"] = (dy * x).sum((0, 1))
    out["ddt_bias"] = ddt.sum((0, 1))
    return dict(out, hT=h[:, -1].contiguous(), dh0=ga[:, 0].contiguous()) if c["state"] else out


def _conv_plain(s):
    c = s["case"]
    B, T, D, W = (c[n] for n in ("B", "T", "D", "W"))
    step = c["op"] == "conv_step"
    x, w, bias = _batch(s, s["x"]), s["w"].float(), s["bias"].float()
    s0 = s["state"][s["slots"].long()] if step else x.new_zeros(B, W - 1, D) if s["s0"] is None else s["s0"]
    ext = torch.cat([s0.float(), x], 1)
    pre = bias + sum(w[:, k] * ext[:, k:k + T] for k in range(W))
    sg = torch.sigmoid(pre)
    out = {"y": _back(s, pre * sg)}
    last = s["lens"][:, None] + torch.arange(W - 1, device="cuda")             # of the extended rows
    sT = torch.gather(ext, 1, last[..., None].expand(B, W - 1, D)).to(_dt(c))
    if step:
        s["state"][s["slots"].long()] = sT
        s["y"].copy_(out["y"])
        return {"y": s["y"], "state": s["state"]}
    if c["op"] == "conv_prefill":
        return dict(out, sT=sT)
    dp = _batch(s, s["dy"]) * sg * (1 + pre * (1 - sg))
    dext = torch.zeros_like(ext)
    if s["dsT"] is not None:
        dext.scatter_add_(1, last[..., None].expand(B, W - 1, D), s["dsT"].float())
    for k in range(W):
        dext[:, k:k + T] += w[:, k] * dp
    out["dw"] = torch.stack([(dp * ext[:, k:k + T]).sum((0, 1)) for k in range(W)], 1)
    out["dbias"] = dp.sum((0, 1))
    out["dx"] = _back(s, dext[:, W - 1:])
    return dict(out, sT=sT, ds0=dext[:, :W - 1].to(_dt(c))) if c["state"] else out


def _clip_plain(s):
    # a model's squares in 64 bits: their sum has up to a few hundred million terms
    norm = torch.stack([g.double().square().sum() for g in s["grads"]]).sum().sqrt().float()
    scale = (1.0 / (norm + CLIP_EPS)).clamp(max=1.0)
    out = s.get("out", s["grads"])
    for o, g in zip(out, s["grads"]):
        o.copy_(g.float() * scale)
    return {"norm": norm.reshape(1), "out": s["whole"]}


# --- 64 bits, from the definitions ---------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        return _clip_exact(s)
    return _conv_exact(s) if case["op"].startswith("conv") else _scan_exact(s)


def _times(s, name):
    """An input in 64 bits, its tokens first."""
    t = s[name]
    return (t.transpose(0, 1) if s["case"]["bfirst"] else t).double()


def _order(s, t):
    return t.transpose(0, 1).contiguous() if s["case"]["bfirst"] else t


def _scan_exact(s):
    c = s["case"]
    B, T, D, N, G = (c[n] for n in ("B", "T", "D", "N", "G"))
    x, dt, z, Bm, Cm = (_times(s, n) for n in ("x", "dt", "z", "B", "C"))
    A, skip, bias = s["A"].double(), s["D"].double(), s["dt_bias"].double()
    train = c["op"] == "scan_train"
    zero = torch.zeros(B, D, N, device="cuda", dtype=torch.float64)
    start = s["state"][s["slots"].long()] if c["op"] == "scan_step" else s["h0"]
    h = zero.clone() if start is None else start.double()
    chan = lambda t: t[:, :, None, :].expand(B, G, D // G, N).reshape(B, D, N)  # noqa: E731
    fold = lambda t: t.reshape(B, G, D // G, N).sum(2)  # noqa: E731
    valid = [(t < s["lens"]).double()[:, None] for t in range(T)]
    soft = lambda t: torch.where(t > 0, t + torch.log1p(torch.exp(-t)), torch.log1p(torch.exp(t)))  # noqa: E731
    y, ys, kept = torch.zeros_like(x), torch.zeros_like(x), []
    for t in range(T):
        d = soft(dt[t] + bias) * valid[t]
        kept.append(h if train else None)
        h = torch.exp(d[..., None] * A) * h + (d * x[t])[..., None] * chan(Bm[t])
        y[t] = ((h * chan(Cm[t])).sum(-1) + skip * x[t]) * valid[t]
        ys[t] = y[t] * z[t] / (1 + torch.exp(-z[t]))
    if c["op"] == "scan_step":
        pool = s["state"].double()
        pool[s["slots"].long()] = h
        return {"y": _order(s, ys), "state": pool}
    if not train:
        return {"y": _order(s, ys), "hT": h}
    do, last = _times(s, "dy"), h
    out = {"y": ys, **{n: torch.zeros_like(r) for n, r in (("dx", x), ("ddt", x), ("dB", Bm), ("dC", Cm), ("dz", x))}}
    dA, dD, db = torch.zeros_like(A), torch.zeros_like(skip), torch.zeros_like(bias)
    g = zero.clone() if s["dhT"] is None else s["dhT"].double()
    for t in reversed(range(T)):
        raw = dt[t] + bias
        d, sz = soft(raw) * valid[t], 1 / (1 + torch.exp(-z[t]))
        gate = z[t] * sz
        out["dz"][t] = valid[t] * do[t] * y[t] * (sz + gate * (1 - sz))
        dy = valid[t] * do[t] * gate
        out["dC"][t] = fold(dy[..., None] * h)
        h = kept.pop()
        g = g + dy[..., None] * chan(Cm[t])
        e = torch.exp(d[..., None] * A)
        out["dB"][t] = fold(g * (d * x[t])[..., None])
        gb = (g * chan(Bm[t])).sum(-1)
        out["dx"][t] = d * gb + dy * skip
        dd = x[t] * gb + (g * e * h * A).sum(-1)
        dA += (g * e * h * d[..., None]).sum(0)
        out["ddt"][t] = valid[t] * dd / (1 + torch.exp(-raw))
        dD += (dy * x[t]).sum(0)
        db += out["ddt"][t].sum(0)
        g = e * g
    out = {n: _order(s, t) for n, t in out.items()}
    out.update(dA=dA, dD=dD, ddt_bias=db)
    out = {n: out[n] for n in ("y", "dz", "dC", "dB", "dx", "ddt", "dA", "dD", "ddt_bias")}
    return dict(out, hT=last, dh0=g) if c["state"] else out


def _conv_exact(s):
    c = s["case"]
    B, T, D, W = (c[n] for n in ("B", "T", "D", "W"))
    x, w, bias = _times(s, "x"), s["w"].double(), s["bias"].double()
    train = c["op"] == "conv_train"
    start = s["state"][s["slots"].long()] if c["op"] == "conv_step" else s["s0"]
    past = torch.zeros(B, W - 1, D, device="cuda", dtype=torch.float64) if start is None else start.double()
    y, kept = torch.zeros_like(x), []
    for t in range(T):
        row = torch.cat([past, x[t][:, None]], 1)                               # the W inputs of token t
        pre = torch.einsum("bkd,dk->bd", row, w) + bias
        live = (t < s["lens"])[:, None]
        y[t] = torch.where(live, pre / (1 + torch.exp(-pre)), 0.0)
        kept.append((row, pre) if train else None)
        past = torch.where(live[..., None], row[:, 1:], past)
    if c["op"] == "conv_step":
        pool = s["state"].double()
        pool[s["slots"].long()] = past
        return {"y": _order(s, y), "state": pool}
    if not train:
        return {"y": _order(s, y), "sT": past}
    do = _times(s, "dy")
    dx, dw, db = torch.zeros_like(x), torch.zeros_like(w), torch.zeros_like(bias)
    dpast = torch.zeros_like(past) if s["dsT"] is None else s["dsT"].double()
    for t in reversed(range(T)):
        row, pre = kept.pop()
        live = (t < s["lens"]).double()[:, None]
        sg = 1 / (1 + torch.exp(-pre))
        dp = live * do[t] * (sg + pre * sg * (1 - sg))
        dw += torch.einsum("bd,bkd->dk", dp, row)
        db += dp.sum(0)
        # a valid token's row moved on by one: the state's gradient goes back to where it came from
        drow = torch.cat([torch.zeros_like(x[0])[:, None], dpast], 1) + dp[:, None] * w.T
        dx[t] = live * drow[:, -1]
        dpast = torch.where(live[..., None] > 0, drow[:, :-1], dpast)
    out = {"y": _order(s, y), "dw": dw, "dbias": db, "dx": _order(s, dx)}
    return dict(out, sT=past, ds0=dpast) if c["state"] else out


def _clip_exact(s):
    total = torch.zeros((), device="cuda", dtype=torch.float64)
    for g in s["grads"]:
        total = total + torch.dot(g.double(), g.double())
    norm = torch.sqrt(total)
    factor = 1 / (norm + CLIP_EPS) if norm + CLIP_EPS > 1 else 1.0
    whole = {w.dtype: torch.zeros_like(w, dtype=torch.float64) for w in s["whole"]}
    for (t, at, n), g in zip(s["place"], s["grads"]):
        whole[t][at:at + n] = g.double() * factor
    return {"norm": norm[None], "out": list(whole.values())}
