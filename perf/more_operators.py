"""Measured cases of the operators of a state-space layer: the short causal
convolution (forward over a piece, forward with backward, single tokens) and
the selective state-space scan that follows it (the same three forms), both
with their state carried from piece to piece.

`own` chooses between their plain form (elementary torch operations in 32
bits) and the calls of state_passing_amd.linrec.
"""
import math

import torch

own = False

DEV = "cuda"


# ----------------------------------------------------------------- cases

def listed():
    bf, f32 = "bf16", "f32"
    return [
        # one token of 64 sequences through the convolution, states in a pool addressed by slots (generation)
        dict(op="conv", kind="token", name="conv token", B=64, T=1, C=4096, K=4, dtype=bf, act=True, ragged=True),
        # a prompt piece of four sequences that end at their own lengths
        dict(op="conv", kind="piece", name="conv piece ragged", B=4, T=4096, C=2048, K=4, dtype=bf, act=True, ragged=True),
        # training step in fp32: odd length, a channel count that is no power of two, three taps, no activation
        dict(op="conv", kind="train", name="conv train f32", B=3, T=4099, C=1000, K=3, dtype=f32, act=False, ragged=False),
        # training step on one long sequence
        dict(op="conv", kind="train", name="conv train 64k", B=1, T=65536, C=2048, K=4, dtype=bf, act=True, ragged=False),
        # one token of one sequence: the latency of a single user
        dict(op="scan", kind="token", name="scan token one user", B=1, T=1, C=2048, N=16, G=1, dtype=bf, gate=True, ragged=False),
        # one token of 128 sequences, states in a pool addressed by slots
        dict(op="scan", kind="token", name="scan token batch", B=128, T=1, C=4096, N=16, G=1, dtype=bf, gate=True, ragged=True),
        # the pieces of four prompts that end at their own lengths
        dict(op="scan", kind="piece", name="scan piece ragged", B=4, T=4096, C=2048, N=16, G=1, dtype=bf, gate=True, ragged=True),
        # a short prompt of one user in fp32, wide states, two groups of channels with their own projections
        dict(op="scan", kind="piece", name="scan piece f32", B=1, T=777, C=1000, N=64, G=2, dtype=f32, gate=False, ragged=False),
        # training step on a small ragged batch, a channel count that is no power of two
        dict(op="scan", kind="train", name="scan train ragged", B=3, T=1023, C=1000, N=16, G=1, dtype=bf, gate=True, ragged=True),
        # training step on one piece of a long sequence
        dict(op="scan", kind="train", name="scan train piece", B=1, T=16384, C=2048, N=16, G=1, dtype=bf, gate=True, ragged=False),
        # training step on a batch of sequences
        dict(op="scan", kind="train", name="scan train batch", B=8, T=2048, C=4096, N=16, G=1, dtype=bf, gate=True, ragged=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv", "scan", "scan"])
    kind = rng.choice(["token", "piece", "train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    most = 65536 * 2048 if op == "conv" else 8 * 2048 * 4096
    if op == "conv":
        C = _log(rng, 64, 4096) if rng.random() < 0.3 else 8 * _log(rng, 8, 512)
        rest = dict(K=rng.choice([2, 3, 4, 4]), act=rng.random() < 0.7)
    else:
        N, G = rng.choice([8, 16, 16, 32, 64]), rng.choice([1, 1, 2, 4])
        C = _log(rng, 64, 4096) if G == 1 and rng.random() < 0.3 else 8 * G * _log(rng, 8, 512 // G)
        rest = dict(N=N, G=G, gate=rng.random() < 0.7)
        most = most * 16 // N
    if dtype == "f32":
        most //= 2
    T = _log(rng, 1, 4) if kind == "token" else _log(rng, 2, min(32768 if op == "scan" else 65536, most // C))
    B = _log(rng, 1, max(1, min(128 if kind == "token" else 64, most // (T * C))))
    return dict(op=op, kind=kind, B=B, T=T, C=C, dtype=dtype, ragged=rng.random() < 0.5, **rest)


def work(case):
    B, T, C = case["B"], case["T"], case["C"]
    # of a ragged batch one sequence is whole, the others end on average at four fifths
    there = round(T * (1 + 0.8 * (B - 1))) if case["ragged"] and case["kind"] != "token" else B * T
    n, e = there * C, 2 if case["dtype"] == "bf16" else 4
    train = case["kind"] == "train"
    if case["op"] == "conv":
        K = case["K"]
        state, taps = 4 * B * (K - 1) * C, 4 * C * (K + 1)
        if train:
            return {"bytes": 4 * n * e + 4 * state + 2 * taps, "flops": n * (6 * K + (16 if case["act"] else 2))}
        return {"bytes": 2 * n * e + 2 * state + taps, "flops": n * (2 * K + (5 if case["act"] else 1))}
    N, gate = case["N"], case["gate"]
    state, proj, params = 4 * B * C * N, 2 * there * case["G"] * N * e, 4 * C * (N + 2)
    # a state and token: the gate's product and exponential, the product that is added, the two sums; the
    # backward's seven sums and products; a channel and token: softplus, gate and their gradients
    if train:
        return {"bytes": n * e * (7 + 3 * gate) + 4 * state + 2 * proj + 2 * params, "flops": n * (21 * N + 30)}
    return {"bytes": n * e * (3 + gate) + 2 * state + proj + params, "flops": n * (7 * N + 12)}


# ----------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    B, T, C, kind = case["B"], case["T"], case["C"], case["kind"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    pad = -(-C // 8) * 8

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device=DEV)

    def rows(scale=1.0):   # token rows that begin at 16 bytes
        return (randn(B, T, pad, dtype=dt) * scale)[..., :C]

    def slots(n):
        return torch.randperm(n, generator=g, device=DEV)[:B].to(torch.int32)

    s = dict(case)
    # the layer's two streams leave one projection side by side
    both = randn(B, T, 2 * pad, dtype=dt)
    s["x"] = both[..., :C]
    ragged = case["ragged"]
    s["n"] = s["slot"] = None
    pool = B + 3 if ragged else B
    if kind == "token":
        s["slot"] = slots(pool) if ragged else None
    elif ragged:
        n = T - (rand(B) * 0.4 * T).long()
        n[0] = T
        s["n"] = n.to(torch.int32)
    # where sequences end early the rows behind them are kept
    s["out"] = {}
    if s["n"] is not None:
        names = ["y"] if kind == "piece" else ["y", "dx"] if case["op"] == "conv" else ["y", "dx", "ddt"] + ["dz"] * case["gate"]
        s["out"] = {k: torch.zeros(B, T, pad, device=DEV, dtype=dt)[..., :C] for k in names}
    if case["op"] == "conv":
        K = case["K"]
        s["w"], s["bias"] = randn(C, K) * K ** -0.5, randn(C) * 0.1
        s["S"] = randn(pool if kind == "token" else B, K - 1, C)
        if kind == "train":
            s["dy"], s["dS"] = rows(), randn(B, K - 1, C)
        return s
    N, G = case["N"], case["G"]
    s["z"] = both[..., pad:pad + C] if case["gate"] else None
    s["dt"] = rows(0.5)
    # steps from 1/1000 to 1/10 of a unit of time, states that forget at rates of 1 to N
    first = torch.exp(math.log(1e-3) + math.log(100.0) * rand(C))
    s["dt_bias"] = first + torch.log(-torch.expm1(-first))
    s["A"] = -torch.arange(1, N + 1, device=DEV) * torch.exp(0.2 * randn(C, N))
    s["D"] = 1.0 + 0.1 * randn(C)
    proj = randn(B, T, 2, G, N, dtype=dt)
    s["Bp"], s["Cp"] = proj[:, :, 0].transpose(1, 2), proj[:, :, 1].transpose(1, 2)
    s["S"] = randn(pool if kind == "token" else B, C, N) * 0.3
    if kind == "train":
        s["dy"], s["dS"] = rows(), randn(B, C, N) * 0.1
        if s["n"] is not None:
            s["out"] |= {k: torch.zeros(B, G, T, N, device=DEV, dtype=dt) for k in ("dB", "dC")}
    return s


# ----------------------------------------------------------------- plain forms

def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1, by doubling."""
    T, step = a.shape[1], 1
    while step < T:
        b = torch.cat([b[:, :step], a[:, step:] * b[:, :-step] + b[:, step:]], 1)
        a = torch.cat([a[:, :step], a[:, step:] * a[:, :-step]], 1)
        step *= 2
    return b


def _live(s):
    """[B,T,1]: the tokens that are there."""
    T = s["T"]
    if s["n"] is None:
        return torch.ones(s["B"], T, 1, dtype=torch.bool, device=DEV)
    return (torch.arange(T, device=DEV) < s["n"][:, None])[..., None]


def _keep(s, name, new, live):
    """Rounded to the layer's type; rows that are not there as they were."""
    new = new.to(s["x"].dtype)
    return torch.where(live, new, s["out"][name]) if name in s["out"] else new


def _total(t):
    """Sum over sequences and tokens."""
    return t.sum((0, 1), dtype=torch.float64).float()


def _conv(s):
    T, K, w, live = s["T"], s["K"], s["w"], _live(s)
    slot = None if s["slot"] is None else s["slot"].long()
    S = s["S"] if slot is None else s["S"][slot]
    x = torch.cat([S, s["x"].float()], 1)                                  # [B,K-1+T,C]
    win = x.unfold(1, K, 1)                                                # [B,T,C,K]
    pre = (win * w).sum(-1) + s["bias"]
    sig = torch.sigmoid(pre)
    y = _keep(s, "y", pre * sig if s["act"] else pre, live)
    end = torch.full((s["B"],), T, device=DEV) if s["n"] is None else s["n"].long()
    last = (end[:, None] + torch.arange(K - 1, device=DEV))[..., None].expand(-1, -1, s["C"])
    new = x.gather(1, last)
    if s["kind"] == "token":
        if slot is None:
            s["S"].copy_(new)
        else:
            s["S"][slot] = new
        return [y, s["S"]]
    if s["kind"] == "piece":
        return [y, new]
    dpre = s["dy"].float() * (sig * (1.0 + pre * (1.0 - sig)) if s["act"] else 1.0)
    dpre = torch.where(live, dpre, 0.0)
    edge = torch.zeros_like(S)
    dx = (torch.cat([edge, dpre, edge], 1).unfold(1, K, 1) * w.flip(1)).sum(-1)
    dx.scatter_add_(1, last, s["dS"])
    dw = _total(dpre[..., None] * torch.where(live[..., None], win, 0.0))
    return [y, new, _keep(s, "dx", dx[:, K - 1:], live), dw, _total(dpre), dx[:, :K - 1].clone()]


def _ssm(s):
    B, T, C, N, G, live = s["B"], s["T"], s["C"], s["N"], s["G"], _live(s)
    A, D = s["A"], s["D"]
    slot = None if s["slot"] is None else s["slot"].long()
    S = s["S"] if slot is None else s["S"][slot]
    x, raw = torch.where(live, s["x"].float(), 0.0), s["dt"].float() + s["dt_bias"]
    dt = torch.where(live, raw.clamp_min(0.0) + torch.log1p(torch.exp(-raw.abs())), 0.0)
    wide = lambda t: t.float().transpose(1, 2)[:, :, :, None].expand(B, T, G, C // G, N).reshape(B, T, C, N)  # noqa: E731
    Bp, Cp = wide(s["Bp"]), wide(s["Cp"])
    a = torch.exp(dt[..., None] * A)
    b = (dt * x)[..., None] * Bp
    b[:, 0] += a[:, 0] * S
    h = _scan(a, b)
    del b
    y = (h * Cp).sum(-1) + D * x
    gate = 1.0
    if s["gate"]:
        z = torch.where(live, s["z"].float(), 0.0)
        sig = torch.sigmoid(z)
        gate = z * sig
    out = [_keep(s, "y", y * gate, live), h[:, -1].clone()]
    if s["kind"] == "token":
        if slot is None:
            s["S"].copy_(out[1])
        else:
            s["S"][slot] = out[1]
        return [out[0], s["S"]]
    if s["kind"] == "piece":
        return out
    dy = torch.where(live, s["dy"].float(), 0.0)
    if s["gate"]:
        dz = _keep(s, "dz", dy * y * sig * (1.0 + z * (1.0 - sig)), live)
    dy = dy * gate
    up = dy[..., None] * Cp
    up[:, -1] += s["dS"]
    Gr = _scan(torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1).flip(1), up.flip(1)).flip(1)
    del up
    group = lambda t: t.view(B, T, G, C // G, N).sum(3).transpose(1, 2)  # noqa: E731
    dB, dC = group(Gr * (dt * x)[..., None]), group(dy[..., None] * h)
    du = (Gr * Bp).sum(-1)
    Gr = Gr * a
    dS = Gr[:, 0].clone()
    Gr = Gr * torch.cat([S[:, None], h[:, :-1]], 1)
    ddt = ((Gr * A).sum(-1) + du * x) * torch.sigmoid(raw)
    ddt = torch.where(live, ddt, 0.0)
    dA = _total(Gr * dt[..., None])
    deep = live[:, None]
    out += [_keep(s, "dx", dy * D + du * dt, live), _keep(s, "ddt", ddt, live), dA, _keep(s, "dB", dB, deep),
            _keep(s, "dC", dC, deep), dS, _total(dy * x), _total(ddt)]
    return out + [dz] if s["gate"] else out


def run(state):
    s = state
    if own:
        return _own(s)
    return _conv(s) if s["op"] == "conv" else _ssm(s)


# ----------------------------------------------------------------- the framework's calls

def _own(s):
    from state_passing_amd import linrec
    out = s["out"]
    if s["op"] == "conv":
        act = "silu" if s["act"] else None
        if s["kind"] == "token":
            return [linrec.conv_step(s["x"], s["w"], s["bias"], s["S"], slots=s["slot"], act=act), s["S"]]
        y, new = linrec.conv_fwd(s["x"], s["w"], s["bias"], s["S"], act=act, n_new=s["n"], y=out.get("y"))
        if s["kind"] == "piece":
            return [y, new]
        dx, dw, dbias, dS = linrec.conv_bwd(s["x"], s["w"], s["bias"], s["S"], s["dy"], s["dS"], act=act, n_new=s["n"],
                                            dx=out.get("dx"))
        return [y, new, dx, dw, dbias, dS]
    layer = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"])
    if s["kind"] == "token":
        return [linrec.scan_step(s["x"], s["dt"], s["A"], s["Bp"], s["Cp"], s["S"], slots=s["slot"], **layer), s["S"]]
    train = s["kind"] == "train"
    y, new, saved = linrec.scan_fwd(s["x"], s["dt"], s["A"], s["Bp"], s["Cp"], s["S"], n_new=s["n"], y=out.get("y"),
                                    save=train, **layer)
    if not train:
        return [y, new]
    r = linrec.scan_bwd(s["x"], s["dt"], s["A"], s["Bp"], s["Cp"], saved, s["dy"], s["dS"], n_new=s["n"],
                        **{k: out[k] for k in ("dx", "ddt", "dB", "dC", "dz") if k in out}, **layer)
    got = [y, new, r.dx, r.ddt, r.dA, r.dB, r.dC, r.dh_in, r.dD, r.ddt_bias]
    return got + [r.dz] if s["gate"] else got


# ----------------------------------------------------------------- the definitions in 64 bits

def _exact_conv(s):
    """Sequence by sequence, tap by tap."""
    B, T, C, K = s["B"], s["T"], s["C"], s["K"]
    w, bias = s["w"].double(), s["bias"].double()
    f64 = dict(dtype=torch.float64, device=DEV)
    y, S = torch.zeros(B, T, C, **f64), s["S"].double()
    dx, dw, db, dS = torch.zeros(B, T, C, **f64), torch.zeros(C, K, **f64), torch.zeros(C, **f64), torch.zeros_like(S)
    tail = torch.empty_like(S)
    for b in range(B):
        n = T if s["n"] is None else int(s["n"][b])
        i = b if s["slot"] is None else int(s["slot"][b])
        x = torch.cat([S[i], s["x"][b, :n].double()])
        p = bias.expand(n, C).clone()
        for k in range(K):
            p += w[:, k] * x[k:k + n]
        q = 1.0 / (1.0 + torch.exp(-p))
        y[b, :n] = p * q if s["act"] else p
        if s["kind"] == "token":
            S[i] = x[n:]
            continue
        tail[b] = x[n:]
        if s["kind"] == "train":
            d = s["dy"][b, :n].double()
            if s["act"]:
                d = d * (q + p * q * (1.0 - q))
            full = torch.zeros_like(x)
            full[n:] += s["dS"][b].double()
            for k in range(K):
                full[k:k + n] += w[:, k] * d
                dw[:, k] += (d * x[k:k + n]).sum(0)
            db += d.sum(0)
            dS[b], dx[b, :n] = full[:K - 1], full[K - 1:]
    if s["kind"] == "token":
        return [y, S]
    return [y, tail] if s["kind"] == "piece" else [y, tail, dx, dw, db, dS]


def _exact_ssm(s):
    """Token by token."""
    B, T, C, N, G = (s[k] for k in ("B", "T", "C", "N", "G"))
    A, D = s["A"].double(), s["D"].double()
    f64 = dict(dtype=torch.float64, device=DEV)
    train = s["kind"] == "train"
    at = torch.arange(B, device=DEV) if s["slot"] is None else s["slot"].long()
    n = torch.full((B,), T, device=DEV) if s["n"] is None else s["n"].long()
    h = s["S"].double()[at]
    y = torch.zeros(B, T, C, **f64)
    hs = torch.empty(T + 1 if train else 1, B, C, N, **f64)
    hs[0] = h

    def token(t):
        there = (t < n)[:, None]
        x = torch.where(there, s["x"][:, t].double(), 0.0)
        v = s["dt"][:, t].double() + s["dt_bias"].double()
        d = torch.where(there, torch.logaddexp(v, torch.zeros_like(v)), 0.0)
        Bt, Ct = (s[k][:, :, t].double().repeat_interleave(C // G, 1) for k in ("Bp", "Cp"))
        zt = torch.where(there, s["z"][:, t].double(), 0.0) if s["gate"] else None
        return there, x, v, d, Bt, Ct, zt

    for t in range(T):
        there, x, _, d, Bt, Ct, zt = token(t)
        h = torch.exp(d[..., None] * A) * h + (d * x)[..., None] * Bt
        if train:
            hs[t + 1] = h
        o = (h * Ct).sum(-1) + D * x
        y[:, t] = torch.where(there, o if zt is None else o * zt / (1.0 + torch.exp(-zt)), 0.0)
    if s["kind"] == "token":
        S = s["S"].double()
        S[at] = h
        return [y, S]
    if not train:
        return [y, h]
    dx, ddt, dz = (torch.zeros(B, T, C, **f64) for _ in range(3))
    dBp, dCp = (torch.zeros(B, G, T, N, **f64) for _ in range(2))
    dA, dD, dbias = torch.zeros(C, N, **f64), torch.zeros(C, **f64), torch.zeros(C, **f64)
    carry = s["dS"].double()
    for t in range(T - 1, -1, -1):
        there, x, v, d, Bt, Ct, zt = token(t)
        up = torch.where(there, s["dy"][:, t].double(), 0.0)
        if zt is not None:
            q = 1.0 / (1.0 + torch.exp(-zt))
            o = (hs[t + 1] * Ct).sum(-1) + D * x
            dz[:, t] = up * o * (q + zt * q * (1.0 - q))
            up = up * zt * q
        g = carry + up[..., None] * Ct
        dCp[:, :, t] = (up[..., None] * hs[t + 1]).view(B, G, C // G, N).sum(2)
        dBp[:, :, t] = (g * (d * x)[..., None]).view(B, G, C // G, N).sum(2)
        du = (g * Bt).sum(-1)
        carry = torch.exp(d[..., None] * A) * g
        e = carry * hs[t]
        dA += (e * d[..., None]).sum(0)
        dx[:, t] = up * D + du * d
        r = torch.where(there, ((e * A).sum(-1) + du * x) / (1.0 + torch.exp(-v)), 0.0)
        ddt[:, t] = r
        dD += (up * x).sum(0)
        dbias += r.sum(0)
    out = [y, h, dx, ddt, dA, dBp, dCp, carry, dD, dbias]
    return out + [dz] if s["gate"] else out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_conv(s) if case["op"] == "conv" else _exact_ssm(s)
