"""Measured cases of the operators a hybrid recurrent / softmax model runs
around the layer: the elementwise gated recurrence (forward, and forward with
backward), the single-token step of the linear and delta-rule layers, the
append of rotated keys and values to a paged 8-bit cache, and the attention
over that cache.

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
        # one token of 64 sequences through an elementwise recurrent layer (generation)
        dict(op="diag", name="diag token", B=64, T=1, C=2048, dtype=bf, mix=True, train=False),
        # a prompt piece in fp32
        dict(op="diag", name="diag prompt f32", B=2, T=4096, C=1024, dtype=f32, mix=False, train=False),
        # training step on a ragged batch: odd length, a channel count that is no power of two
        dict(op="diag", name="diag train ragged", B=3, T=4099, C=1000, dtype=bf, mix=True, train=True),
        # training step on one long sequence
        dict(op="diag", name="diag train 64k", B=1, T=65536, C=2048, dtype=bf, mix=False, train=True),
        # one token of a small batch, linear layer with a decay per head
        dict(op="step", name="step linear small", B=4, H=16, d=128, delta=False, slots=False),
        # one token of a large batch, gated delta rule, states in a pool addressed by slots
        dict(op="step", name="step delta batch", B=96, H=32, d=128, delta=True, slots=True),
        # one token of 64 sequences appended at their own lengths
        dict(op="append", name="append token", B=64, T=1, Hq=32, Hkv=8, D=128, page=64, past=1500, rot=128,
             inter=False),
        # a piece of 4096 prompt tokens of two sequences (ragged), a quarter of each head rotated
        dict(op="append", name="append piece", B=2, T=4096, Hq=32, Hkv=8, D=128, page=64, past=4000, rot=32,
             inter=True),
        # one token of one sequence: the latency of a single user
        dict(op="attn", name="attn token one user", B=1, T=1, Hq=16, Hkv=4, D=128, page=64, past=4095, window=0),
        # one token of 32 sequences around 16K tokens
        dict(op="attn", name="attn token batch", B=32, T=1, Hq=32, Hkv=8, D=128, page=64, past=16384, window=0),
        # a few tokens (a draft to be verified), small heads, a sliding window, small pages
        dict(op="attn", name="attn draft window", B=16, T=5, Hq=16, Hkv=2, D=64, page=16, past=6001, window=2048),
        # a piece of 4096 prompt tokens behind 12K cached ones
        dict(op="attn", name="attn piece", B=1, T=4096, Hq=16, Hkv=4, D=128, page=64, past=12288, window=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["diag", "step", "append", "attn"])
    if op == "diag":
        C = 8 * _log(rng, 8, 256)
        T = 1 if rng.random() < 0.2 else _log(rng, 2, 65536)
        B = _log(rng, 1, max(1, min(64, 65536 * 2048 // (T * C))))
        return dict(op=op, B=B, T=T, C=C, dtype=rng.choice(["bf16", "f32"]) if B * T * C <= 1 << 26 else "bf16",
                    mix=rng.random() < 0.5, train=rng.random() < 0.6)
    if op == "step":
        H = rng.choice([4, 12, 16, 32])
        return dict(op=op, B=_log(rng, 1, 96), H=H, d=rng.choice([64, 128]), delta=rng.random() < 0.5,
                    slots=rng.random() < 0.5)
    Hkv = rng.choice([1, 2, 4, 8])
    D, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    if op == "append":
        T = 1 if rng.random() < 0.4 else _log(rng, 2, 4096)
        B = _log(rng, 1, max(1, min(64, 8192 // T)))
        return dict(op=op, B=B, T=T, Hq=Hkv * rng.choice([1, 2, 4]), Hkv=Hkv, D=D, page=page,
                    past=_log(rng, 1, 4096) - 1, rot=rng.choice([D, D // 2, D // 4]), inter=rng.random() < 0.5)
    g = rng.choice([1, 2, 4, 6, 8])
    T = 1 if rng.random() < 0.4 else _log(rng, 2, 4096)
    past = _log(rng, 1, 16384) - 1
    most = min(32 * 8 * 16384 // (Hkv * (past + T)), 4096 * 16 * 16384 // (T * Hkv * g * (past + T)))
    return dict(op=op, B=_log(rng, 1, max(1, min(32, most))), T=T, Hq=Hkv * g, Hkv=Hkv, D=D, page=page, past=past,
                window=rng.choice([0, 0, 256, 1000]))


def _elem(case):
    return 2 if case.get("dtype", "bf16") == "bf16" else 4


def _keys(case):
    """(query, key) pairs of one sequence with every query present, and the cached tokens that they read."""
    T, past, w = case["T"], case["past"], case["window"]
    if not w:
        return T * past + T * (T + 1) // 2, past + T
    pairs = sum(min(w, past + i + 1) for i in range(T))
    return pairs, min(past + T, w + T - 1)


def work(case):
    op = case["op"]
    if op == "diag":
        n, e = case["B"] * case["T"] * case["C"], _elem(case)
        carry = 4 * case["B"] * case["C"]
        if case["train"]:
            return {"bytes": 8 * n * e + 5 * carry, "flops": 12 * n}
        return {"bytes": 3 * n * e + 2 * carry, "flops": 3 * n}
    if op == "step":
        n, d = case["B"] * case["H"], case["d"]
        return {"bytes": n * (8 * d * d + 8 * d), "flops": n * d * d * (8 if case["delta"] else 5)}
    B, T, Hq, Hkv, D = (case[k] for k in ("B", "T", "Hq", "Hkv", "D"))
    if op == "append":
        return {"bytes": B * T * D * (4 * Hq + 6 * Hkv), "flops": B * T * 3 * (Hq + Hkv) * case["rot"]}
    pairs, read = _keys(case)
    return {"bytes": B * (2 * Hkv * D * read + 4 * T * Hq * D), "flops": 4 * B * Hq * D * pairs}


# ----------------------------------------------------------------- inputs

def _cache(case, g, pages):
    """Filled pages of unit-variance keys and values under power-of-two scales."""
    Hkv, D, P = case["Hkv"], case["D"], case["page"]

    def codes(*shape):
        return (torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16) * 100).clamp_(-448, 448).to(torch.float8_e4m3fn)

    def scales():
        return torch.exp2(torch.randint(-8, -5, (pages, Hkv), generator=g, device=DEV).float())

    return codes(pages, Hkv, P, D), codes(pages, Hkv, D, P), scales(), scales()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device=DEV)

    s = dict(case)
    if op == "diag":
        B, T, C = case["B"], case["T"], case["C"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        # log gates of channels that remember from a few to a few thousand tokens
        rate = torch.exp2(-1.0 - 10.0 * rand(C))
        s["g"] = -(rate * (0.5 + rand(B, T, C))).to(dt)
        s["x"] = randn(B, T, C, dtype=dt)
        s["h_in"] = randn(B, C)
        if case["train"]:
            s["dh"] = randn(B, T, C, dtype=dt)
            s["dh_out"] = randn(B, C)
        return s
    if op == "step":
        B, H, d = case["B"], case["H"], case["d"]
        unit = lambda x: (x / torch.linalg.vector_norm(x, dim=-1, keepdim=True)).to(torch.bfloat16)  # noqa: E731
        s["q"], s["k"] = unit(randn(B, H, 1, d)), unit(randn(B, H, 1, d))
        s["v"] = randn(B, H, 1, d, dtype=torch.bfloat16)
        pool = B + 3 if case["slots"] else B
        s["S"] = randn(pool, H, d, d) * 0.1
        s["slot"] = torch.randperm(pool, generator=g, device=DEV)[:B].to(torch.int32) if case["slots"] else None
        if case["delta"]:
            s["beta"] = torch.sigmoid(randn(B, H, 1))
            s["decay"] = 0.9 + 0.1 * torch.sigmoid(randn(B, H, 1) + 2.0)
        else:
            s["beta"] = None
            s["decay"] = 1.0 - torch.exp2(-(5.0 + 8.0 * rand(H)))
        return s
    B, T, Hq, Hkv, D, P = (case[k] for k in ("B", "T", "Hq", "Hkv", "D", "page"))
    # sequences of their own lengths; every second one ends its piece early
    past = case["past"] - (rand(B) * 0.25 * case["past"]).long()
    past[0] = case["past"]
    n = torch.full((B,), T, dtype=torch.int64, device=DEV)
    n[1::2] = (T - (rand(B) * 0.25 * T).long())[1::2]
    per = -(-(case["past"] + T) // P)
    pages = B * per + 1
    s["kc"], s["vc"], s["ks"], s["vs"] = _cache(case, g, pages)
    # page 0 belongs to nobody
    s["table"] = (1 + torch.randperm(pages - 1, generator=g, device=DEV)).view(B, per).to(torch.int32)
    s["past"], s["n"] = past.to(torch.int32), n.to(torch.int32)
    s["q"] = randn(B, Hq, T, D, dtype=torch.bfloat16)
    if op == "append":
        s["k"], s["v"] = randn(B, Hkv, T, D, dtype=torch.bfloat16), randn(B, Hkv, T, D, dtype=torch.bfloat16)
        half = case["rot"] // 2
        s["freq"] = torch.pow(10000.0, -torch.arange(half, device=DEV, dtype=torch.float64) / half)
        s["q_out"] = torch.zeros_like(s["q"])
    else:
        s["o"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(B, Hq, T, device=DEV)
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


def _diag(s):
    dt = s["x"].dtype
    g, x, h_in = s["g"].float(), s["x"].float(), s["h_in"]
    a = torch.exp(g)
    b = -torch.expm1(g) * x if s["mix"] else x.clone()
    b[:, 0] += a[:, 0] * h_in
    h = _scan(a, b)
    out = [h.to(dt), h[:, -1].clone()]
    if s["train"]:
        up = s["dh"].to(torch.float32, copy=True)   # (float() of a float32 tensor is the tensor itself)
        up[:, -1] += s["dh_out"]
        nxt = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
        G = _scan(nxt.flip(1), up.flip(1)).flip(1)
        prev = torch.cat([h_in[:, None], h[:, :-1]], 1)
        dg = a * G * (prev - x) if s["mix"] else a * G * prev
        dx = -torch.expm1(g) * G if s["mix"] else G
        out += [dg.to(dt), dx.to(dt), a[:, 0] * G[:, 0]]
    return out


def _step(s):
    q, k, v = (s[n][:, :, 0].float() for n in ("q", "k", "v"))
    S = s["S"] if s["slot"] is None else s["S"][s["slot"].long()]
    if s["beta"] is None:
        new = s["decay"][:, None, None] * S + k[..., None] * v[:, :, None]
    else:
        a, beta = s["decay"][:, :, 0, None], s["beta"]
        u = beta * (v - a * (k[..., None] * S).sum(2))
        new = a[..., None] * S + k[..., None] * u[:, :, None]
    o = (q[..., None] * new).sum(2)
    if s["slot"] is None:
        s["S"].copy_(new)
    else:
        s["S"][s["slot"].long()] = new
    return [o[:, :, None].to(torch.bfloat16), s["S"]]


def _rotate(x, pos, freq, inter):
    """x [B,H,T,D] with the first 2 * len(freq) features of each head rotated by pos [B,T] * freq."""
    half = freq.numel()
    turn = pos[:, None, :, None].double() * freq
    c, n = torch.cos(turn).float(), torch.sin(turn).float()
    r, rest = x[..., :2 * half].float(), x[..., 2 * half:].float()
    if inter:
        u, w = r[..., 0::2], r[..., 1::2]
        r = torch.stack([u * c - w * n, u * n + w * c], -1).flatten(-2)
    else:
        u, w = r[..., :half], r[..., half:]
        r = torch.cat([u * c - w * n, u * n + w * c], -1)
    return torch.cat([r, rest], -1)


def _put(cache, scale, new, page, fresh, old, has_old):
    """Codes of `new` [B,N,H,P,D] into the pages; a scale is the least power of two that holds the block."""
    amax = torch.where(fresh, new.abs(), 0.0).amax((3, 4))
    m, e = torch.frexp(amax)
    need = torch.ldexp(torch.ones_like(amax), e - 9 + (m > 0.875).int()).clamp_min(2.0 ** -100)
    was = scale[page]
    s = torch.where(has_old, torch.maximum(was, need), need)
    has = cache[page].float()
    grown = has * (was / s)[..., None, None]
    put = torch.where(fresh, new / s[..., None, None], torch.where(old, grown, has))
    cache[page] = put.clamp(-448, 448).to(cache.dtype)
    # the page nobody owns takes what blocks without a new token would write
    scale[page] = torch.where(fresh.flatten(2).any(2)[:, :, None], s, was)


def _append(s):
    B, T, P = s["B"], s["T"], s["page"]
    past, n = s["past"].long(), s["n"].long()
    pos = past[:, None] + torch.arange(T, device=DEV)
    k = _rotate(s["k"], pos, s["freq"], s["inter"])
    q = _rotate(s["q"], pos, s["freq"], s["inter"])
    live = (torch.arange(T, device=DEV) < n[:, None])[:, None, :, None]
    q_out = torch.where(live, q.to(torch.bfloat16), s["q_out"])
    N = (T + P - 2) // P + 1
    first = past // P
    at = first[:, None] * P + torch.arange(N * P, device=DEV)          # positions of the touched blocks
    fresh = (at >= past[:, None]) & (at < (past + n)[:, None])
    old = at < past[:, None]
    touched = fresh.view(B, N, P).any(-1)
    block = (first[:, None] + torch.arange(N, device=DEV)).clamp_max(s["table"].shape[1] - 1)
    page = torch.where(touched, s["table"].long().gather(1, block), 0)
    src = (at - past[:, None]).clamp(0, T - 1)[:, None, :, None].expand(-1, s["Hkv"], -1, s["D"])
    split = lambda x: x.gather(2, src).unflatten(2, (N, P)).transpose(1, 2)  # noqa: E731  [B,N,H,P,D]
    mask = lambda m: m.view(B, N, 1, P, 1)  # noqa: E731
    fresh, old = mask(fresh), mask(old) & touched[:, :, None, None, None]
    has_old = old.any(3).squeeze(-1)
    _put(s["kc"], s["ks"], split(k), page, fresh, old, has_old)
    _put(s["vc"].transpose(2, 3), s["vs"], split(s["v"].float()), page, fresh, old, has_old)
    return [s["kc"], s["vc"], s["ks"], s["vs"], q_out]


def _attn(s):
    B, T, Hq, Hkv, D = (s[k] for k in ("B", "T", "Hq", "Hkv", "D"))
    page = s["table"].long()
    K = (s["kc"][page].float() * s["ks"][page][..., None, None]).transpose(1, 2).flatten(2, 3)
    V = (s["vc"][page].float() * s["vs"][page][..., None, None]).transpose(3, 4).transpose(1, 2).flatten(2, 3)
    L, g = K.shape[2], Hq // Hkv
    row = s["past"].long()[:, None] + torch.arange(T, device=DEV)
    key = torch.arange(L, device=DEV)
    see = key <= row[..., None]
    if s["window"]:
        see &= key > row[..., None] - s["window"]
    live = torch.arange(T, device=DEV) < s["n"][:, None]
    see = see[:, None, None]                                           # [B,1,1,T,L]
    x = torch.matmul(s["q"].float().reshape(B, Hkv, g * T, D), K.transpose(2, 3).contiguous())
    x = (x.view(B, Hkv, g, T, L) / math.sqrt(D)).masked_fill_(~see, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = (torch.matmul(x.view(B, Hkv, g * T, L), V).view(B, Hkv, g, T, D) / total).reshape(B, Hq, T, D)
    lse = (top + torch.log(total)).reshape(B, Hq, T)
    return [torch.where(live[:, None, :, None], o.to(torch.bfloat16), s["o"]),
            torch.where(live[:, None], lse, s["lse"])]


def run(state):
    s = state
    if own:
        return _own(s)
    return {"diag": _diag, "step": _step, "append": _append, "attn": _attn}[s["op"]](s)


# ----------------------------------------------------------------- the framework's calls

def _own(s):
    from state_passing_amd import linrec
    if s["op"] == "diag":
        form = "mix" if s["mix"] else "plain"
        h, h_out, states = linrec.diag_fwd(s["g"], s["x"], s["h_in"], form=form)
        if not s["train"]:
            return [h, h_out]
        dg, dx, dh_in = linrec.diag_bwd(s["g"], s["x"], states, s["dh"], s["dh_out"], form=form)
        return [h, h_out, dg, dx, dh_in]
    if s["op"] == "step":
        return [linrec.step(s["q"], s["k"], s["v"], s["decay"], s["S"], beta=s["beta"], slots=s["slot"]), s["S"]]
    cache = linrec.KvCache(s["kc"], s["vc"], s["ks"], s["vs"], s["table"])
    if s["op"] == "append":
        linrec.kv_append(cache, s["k"], s["v"], s["past"], n_new=s["n"], inv_freq=s["freq"], interleaved=s["inter"],
                         q=s["q"], q_out=s["q_out"])
        return [s["kc"], s["vc"], s["ks"], s["vs"], s["q_out"]]
    linrec.kv_attn(cache, s["q"], s["past"], n_new=s["n"], window=s["window"], o=s["o"], lse=s["lse"])
    return [s["o"], s["lse"]]


# ----------------------------------------------------------------- the definitions in 64 bits

def _exact_diag(s):
    g, x, h = s["g"].double(), s["x"].double(), s["h_in"].double()
    T = g.shape[1]
    a, w = g.exp(), (-torch.expm1(g) if s["mix"] else torch.ones_like(g))
    hs = torch.empty_like(x)
    for t in range(T):
        h = torch.addcmul(w[:, t] * x[:, t], a[:, t], h)
        hs[:, t] = h
    out = [hs, h]
    if s["train"]:
        dg, dx, G = torch.empty_like(x), torch.empty_like(x), s["dh_out"].double()
        dh = s["dh"].double()
        for t in range(T - 1, -1, -1):
            G = G + dh[:, t]
            dx[:, t] = w[:, t] * G
            prev = hs[:, t - 1] if t else s["h_in"].double()
            aG = a[:, t] * G
            dg[:, t] = aG * (prev - x[:, t] if s["mix"] else prev)
            G = aG
        out += [dg, dx, G]
    return out


def _exact_step(s):
    S = s["S"].double()
    o = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    eye = torch.eye(s["d"], dtype=torch.float64, device=DEV)
    for b in range(s["B"]):
        i = b if s["slot"] is None else int(s["slot"][b])
        q, k, v = (s[n][b, :, 0].double() for n in ("q", "k", "v"))
        outer = k[:, :, None] * v[:, None, :]
        if s["beta"] is None:
            S[i] = s["decay"].double()[:, None, None] * S[i] + outer
        else:
            a, beta = s["decay"][b].double()[:, :, None], s["beta"][b].double()[:, :, None]
            erase = eye - beta * k[:, :, None] * k[:, None, :]
            S[i] = a * torch.bmm(erase, S[i]) + beta * outer
        o[b, :, 0] = torch.bmm(q[:, None, :], S[i])[:, 0]
    return [o, S]


def _exact_append(s):
    """Sequence by sequence and page by page; codes as the values before their rounding."""
    P, half = s["page"], s["freq"].numel()
    kc, vc, ks, vs = s["kc"].double(), s["vc"].double().transpose(2, 3).contiguous(), s["ks"].double(), s["vs"].double()
    q_out = s["q_out"].double()
    lead = torch.arange(half, device=DEV) * (2 if s["inter"] else 1)
    follow = lead + (1 if s["inter"] else half)
    past, n, table = s["past"].tolist(), s["n"].tolist(), s["table"].tolist()
    for b in range(s["B"]):
        pos = past[b] + torch.arange(n[b], device=DEV, dtype=torch.float64)
        unit = torch.polar(torch.ones_like(pos)[:, None].expand(-1, half).contiguous(), pos[:, None] * s["freq"])

        def turned(x):
            x = x[b, :, :n[b]].double().clone()
            z = torch.complex(x[..., lead], x[..., follow]) * unit
            x[..., lead], x[..., follow] = z.real, z.imag
            return x

        q_out[b, :, :n[b]] = turned(s["q"])
        for new, codes, scale in ((turned(s["k"]), kc, ks), (s["v"][b, :, :n[b]].double(), vc, vs)):
            t = 0
            while t < n[b]:
                p, off = table[b][(past[b] + t) // P], (past[b] + t) % P
                m = min(P - off, n[b] - t)
                part = new[:, t:t + m]
                need = torch.exp2(torch.ceil(torch.log2(part.abs().amax((1, 2)) / 448)).clamp_min(-100))
                if off:
                    need = torch.maximum(need, scale[p])
                    codes[p, :, :off] *= (scale[p] / need)[:, None, None]
                codes[p, :, off:off + m] = part / need[:, None, None]
                scale[p] = need
                t += m
    return [kc, vc.transpose(2, 3).contiguous(), ks, vs, q_out]


def _exact_attn(s):
    T, Hq, Hkv, P = s["T"], s["Hq"], s["Hkv"], s["page"]
    g = Hq // Hkv
    o, lse = s["o"].double(), s["lse"].double()
    for b in range(s["B"]):
        past, n = int(s["past"][b]), int(s["n"][b])
        lo = max(0, past - s["window"] + 1) if s["window"] else 0
        page = s["table"][b, lo // P:-(-(past + n) // P)].long()
        lo -= lo % P
        row = past + torch.arange(n, device=DEV)[:, None]
        for h in range(Hkv):
            K = (s["kc"][page, h].double() * s["ks"][page, h].double()[:, None, None]).flatten(0, 1)
            V = (s["vc"][page, h].double() * s["vs"][page, h].double()[:, None, None]).transpose(1, 2).flatten(0, 1)
            key = lo + torch.arange(K.shape[0], device=DEV)
            hide = (key > row) | ((key <= row - s["window"]) if s["window"] else (key < 0))
            x = torch.matmul(s["q"][b, h * g:(h + 1) * g, :n].double() * s["D"] ** -0.5, K.t())
            x.masked_fill_(hide, -math.inf)
            z = torch.logsumexp(x, -1)
            lse[b, h * g:(h + 1) * g, :n] = z
            o[b, h * g:(h + 1) * g, :n] = torch.matmul(torch.exp(x - z[..., None]), V)
    return [o, lse]


def exact(case, seed):
    s = prepare(case, seed)
    return {"diag": _exact_diag, "step": _exact_step, "append": _exact_append, "attn": _exact_attn}[case["op"]](s)
