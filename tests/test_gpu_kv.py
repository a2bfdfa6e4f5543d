"""GPU tests of the paged 8-bit key/value cache: the append with rotation
(linrec_kv_append) and the attention over the cache (linrec_kv_attn) against
plain implementations in 64 bits on the CPU.

Tolerances, from the roundings made:
- a stored value: half an e4m3 step, 2^-4 of the value, or half the smallest
  step, 2^-10 of the scale; what is rounded carries fp32 errors of the rotation
  (sine, cosine and three fp32 operations: 2^-21 of the pair's norm);
- the weights enter the second product as bf16 (half a step: 2^-8), so o is off
  by 2^-8 of sum_j p_j |v_j|; scores are sums of D exact products in fp32,
  off by D 2^-24 sum |q k| scale <= 2^-13 relative in p for what is drawn here,
  with 2^-21 for the exponential: 2^-12 in all; o is then rounded to bf16.
"""
import math

import pytest
import torch

from state_passing_amd import linrec

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F8 = torch.float8_e4m3fn


def filled_cache(g, B, H, D, page, max_pages, spare=2):
    """A cache whose pages hold unit-variance values, on the CPU; page ids shuffled."""
    pages = B * max_pages + spare
    codes = lambda *s: (torch.randn(*s, generator=g) * 100).clamp_(-448, 448).to(F8)  # noqa: E731
    scale = lambda: torch.exp2(torch.randint(-8, -5, (pages, H), generator=g).float())  # noqa: E731
    table = torch.randperm(pages, generator=g)[:B * max_pages].view(B, max_pages).to(torch.int32)
    return linrec.KvCache(codes(pages, H, page, D), codes(pages, H, D, page), scale(), scale(), table)


def to_dev(cache):
    return linrec.KvCache(*(t.to(DEV) for t in cache))


def dense(cache, b):
    """Keys and values [H, tokens, D] of sequence b in 64 bits, and which tokens have a page."""
    pages = cache.k.shape[0]
    ids = cache.table[b].long()
    ok = (ids >= 0) & (ids < pages)
    i = torch.where(ok, ids, 0)
    K = cache.k[i].double() * cache.k_scale[i].double()[..., None, None]
    V = (cache.v[i].double() * cache.v_scale[i].double()[..., None, None]).transpose(2, 3)
    flat = lambda x: x.transpose(0, 1).flatten(1, 2)  # noqa: E731
    return flat(K), flat(V), ok.repeat_interleave(cache.k.shape[2])


def attn_reference(cache, q, past, n, scale, window):
    """(o, sum_j p_j |v_j|, lse) in 64 bits; NaN and infinities only from what a row sees."""
    B, Hq, T, D = q.shape
    H = cache.k.shape[1]
    o, mag, lse = (torch.zeros(B, Hq, T, *s, dtype=torch.float64) for s in ((D,), (D,), ()))
    for b in range(B):
        K, V, ok = dense(cache, b)
        for i in range(n[b]):
            pos = past[b] + i
            see = torch.arange(K.shape[1])
            see = ok & (see <= pos) & ((see > pos - window) if window > 0 else True)
            idx = see.nonzero()[:, 0]
            for h in range(Hq):
                kv = h // (Hq // H)
                if not len(idx):
                    lse[b, h, i] = -math.inf
                    continue
                s = K[kv, idx] @ q[b, h, i].double() * scale
                lse[b, h, i] = torch.logsumexp(s, 0)
                p = torch.softmax(s, 0)
                o[b, h, i] = p @ V[kv, idx]
                mag[b, h, i] = p @ V[kv, idx].abs()
    return o, mag, lse


def check_attn(cache, q, past, n, *, scale=None, window=0, n_new=True, view=None, **kw):
    """Runs kv_attn on the GPU and compares every row that is there; the others keep their fill."""
    B, Hq, T, D = q.shape
    sc = D ** -0.5 if scale is None else scale
    ref, mag, ref_lse = attn_reference(cache, q, past, n, sc, window)
    dq = q.to(DEV) if view is None else view(q.to(DEV))
    o = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    o = o if view is None else view(o)
    lse = torch.full((B, Hq, T), 7.0, device=DEV)
    args = dict(n_new=torch.tensor(n, dtype=torch.int32, device=DEV) if n_new else None, scale=scale,
                window=window, o=o, lse=lse, **kw)
    gpu, past_d = to_dev(cache), torch.tensor(past, dtype=torch.int32, device=DEV)
    linrec.kv_attn(gpu, dq, past_d, **args)
    torch.cuda.synchronize()
    got, got_lse = o.double().cpu(), lse.double().cpu()
    for b in range(B):
        assert (got[b, :, n[b]:] == 7).all() and (got_lse[b, :, n[b]:] == 7).all()
        r, m, g = ref[b, :, :n[b]], mag[b, :, :n[b]], got[b, :, :n[b]]
        assert torch.equal(torch.isnan(r), torch.isnan(g)), b
        bad = (g - r).abs() > (2.0 ** -8 + 2.0 ** -12) * m + 2.0 ** -8 * r.abs()
        assert not bad.any(), (b, bad.nonzero()[:4], float((g - r).abs().nan_to_num().max()))
        rl, gl = ref_lse[b, :, :n[b]], got_lse[b, :, :n[b]]
        assert torch.equal(torch.isinf(rl), torch.isinf(gl)) and torch.equal(torch.isnan(rl), torch.isnan(gl))
        assert ((gl - rl).abs().nan_to_num() <= 2.0 ** -12 * (1 + rl.abs().nan_to_num(posinf=0, neginf=0))).all()
    return gpu, dq, past_d, args, o, lse


def draw(seed, B, T, Hq, H, D, page, max_pages):
    g = torch.Generator().manual_seed(seed)
    cache = filled_cache(g, B, H, D, page, max_pages)
    return g, cache, torch.randn(B, Hq, T, D, generator=g).to(torch.bfloat16)


# (B, T, Hq, H, D, page, max_pages, past, n, window)
ATTN = [
    # single tokens: nothing cached before, one, ends of pages and tiles
    (6, 1, 4, 4, 128, 16, 5, [0, 1, 15, 16, 63, 64], None, 0),
    (4, 1, 8, 1, 64, 32, 9, [65, 255, 256, 200], None, 0),
    (2, 1, 16, 1, 128, 64, 16, [1000, 3], None, 0),
    (1, 1, 6, 2, 128, 128, 40, [5000], None, 0),           # split over the keys
    (2, 1, 40, 2, 64, 64, 4, [77, 150], None, 0),          # 20 rows
    (3, 1, 4, 2, 128, 64, 8, [300, 400, 17], [1, 0, 1], 64),
    # a few tokens
    (2, 5, 16, 2, 64, 16, 12, [101, 7], [5, 3], 0),        # 40 rows: tiles of 32 and 8
    (2, 3, 6, 1, 128, 32, 6, [62, 0], None, 10),
    (1, 64, 1, 1, 128, 64, 4, [100], None, 0),             # 64 rows
    # pieces
    (1, 65, 1, 1, 128, 64, 4, [100], None, 0),
    (2, 37, 8, 2, 128, 16, 12, [0, 130], [37, 20], 0),
    (3, 70, 4, 4, 64, 32, 10, [5, 200, 64], [70, 0, 1], 0),
    (1, 130, 12, 2, 64, 64, 12, [500], None, 33),
    (1, 96, 4, 2, 128, 128, 20, [2300], None, 0),          # split over the keys
    (2, 50, 4, 2, 128, 64, 4, [190, 230], None, 0),        # runs past the table's end
]


@pytest.mark.parametrize("case", ATTN, ids=[str(i) for i in range(len(ATTN))])
def test_attention(case):
    B, T, Hq, H, D, page, max_pages, past, n, window = case
    print("case", case, flush=True)
    _, cache, q = draw(1000 + ATTN.index(case), B, T, Hq, H, D, page, max_pages)
    # what no row sees holds NaN: tails of the sequences, pages of nobody
    for b in range(B):
        for t in range(past[b] + (n[b] if n else T), page * max_pages):
            p = int(cache.table[b, t // page])
            cache.k.view(torch.uint8)[p, :, t % page] = 0x7f
            cache.v.view(torch.uint8)[p, :, :, t % page] = 0xff
    free = sorted(set(range(cache.k.shape[0])) - set(cache.table.flatten().tolist()))
    cache.k_scale[free] = math.nan
    cache.v_scale[free] = math.inf
    check_attn(cache, q, past, n or [T] * B, window=window, n_new=n is not None)


@pytest.mark.parametrize("T,Hq", [(1, 4), (4, 8), (80, 2)])
def test_attention_missing_pages(T, Hq):
    """Table entries outside the pool hide their tokens; a row left with none gets 0 and -inf."""
    _, cache, q = draw(5, 3, T, Hq, 2, 64, 16, 12)
    cache.table[0, 1] = -1
    cache.table[0, 4] = cache.k.shape[0]
    cache.table[1] = -5
    cache.table[2, :8] = 1 << 30
    cache.k_scale[0], cache.v_scale[0] = math.nan, math.nan    # page 0, which a missing one must not become
    cache.table[cache.table == 0] = -1
    check_attn(cache, q, [90, 60, 125], [T] * 3)
    check_attn(cache, q, [90, 60, 100], [T] * 3, window=20)


@pytest.mark.parametrize("T,Hq", [(1, 2), (6, 8), (90, 2)])
def test_attention_nan_reaches_only_rows_that_see_it(T, Hq):
    _, cache, q = draw(6, 1, T, Hq, 2, 128, 32, 8)
    past = 40
    for t, f in ((past + T // 2, 3), (past, 77)):
        p = int(cache.table[0, t // 32])
        cache.v.view(torch.uint8)[p, 1, f, t % 32] = 0x7f
    check_attn(cache, q, [past], [T])
    check_attn(cache, q, [past], [T], window=3)
    t = past + T - 1
    cache.k.view(torch.uint8)[int(cache.table[0, t // 32]), 0, t % 32, 5] = 0xff
    check_attn(cache, q, [past], [T])


@pytest.mark.parametrize("T", [1, 70])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 1.5])
def test_attention_scales(T, scale):
    _, cache, q = draw(7, 2, T, 4, 2, 64, 16, 9)
    check_attn(cache, (q * 0.3).to(torch.bfloat16), [60, 20], [T, T], scale=scale)


@pytest.mark.parametrize("T", [1, 70])
@pytest.mark.parametrize("window", [1, 2147479551, 2147483647])
def test_attention_windows_at_the_ends(T, window):
    _, cache, q = draw(9, 2, T, 4, 2, 64, 32, 9)
    check_attn(cache, q, [200, 3], [T, T], window=window)


@pytest.mark.parametrize("T", [1, 5, 70])
def test_attention_token_major_views_and_replays(T):
    """q and o as [B,T,H,D] memory; the same call captured: every replay, between
    eager calls, repeats the eager result bit for bit."""
    _, cache, q = draw(8, 2, T, 8, 2, 128, 64, 40)
    view = lambda x: x.transpose(1, 2).contiguous().transpose(1, 2)  # noqa: E731
    past = [2400, 333]
    gpu, dq, past_d, args, o, lse = check_attn(cache, q, past, [T, T], view=view)
    want, want_lse = o.clone(), lse.clone()
    other = torch.randn_like(dq)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        linrec.kv_attn(gpu, dq, past_d, **args)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        linrec.kv_attn(gpu, dq, past_d, **args)
    for _ in range(4):
        o.fill_(3)
        lse.fill_(3)
        linrec.kv_attn(gpu, other, past_d)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(lse, want_lse)


# ----------------------------------------------------------------- append

def rotate_reference(x, pos, freq, inter):
    """x [H,n,D] in 64 bits turned by pos [n] * freq."""
    x = x.double().clone()
    half = len(freq)
    i = torch.arange(half) * (2 if inter else 1)
    j = i + (1 if inter else half)
    ang = pos.double()[:, None] * freq
    c, s = ang.cos(), ang.sin()
    u, w = x[..., i].clone(), x[..., j].clone()
    x[..., i], x[..., j] = u * c - w * s, w * c + u * s
    return x


def need_scale(x):
    """Least power of two s >= 2^-100 with max|x| <= 448 s, over finite values, per head."""
    amax = torch.where(torch.isfinite(x), x.abs(), 0.0).amax((1, 2))
    return torch.exp2(torch.where(amax > 0, torch.ceil(torch.log2(amax / 448)), -100.0).clamp_min(-100))


def check_append(cache, k, v, past, n, freq, inter, q=None, n_new=True, view=None):
    B, H, T, D = k.shape
    page, max_pages, pages = cache.k.shape[2], cache.table.shape[1], cache.k.shape[0]
    put = (lambda x: x) if view is None else view
    gpu = to_dev(cache)
    before = linrec.KvCache(*(t.clone() for t in cache))
    q_out = None if q is None else put(torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV))
    nd = torch.tensor(n, dtype=torch.int32, device=DEV) if n_new else None
    linrec.kv_append(gpu, put(k.to(DEV)), put(v.to(DEV)), torch.tensor(past, dtype=torch.int32, device=DEV), n_new=nd,
                     inv_freq=None if freq is None else freq.to(DEV), interleaved=inter,
                     q=None if q is None else put(q.to(DEV)), q_out=q_out)
    torch.cuda.synchronize()
    got = linrec.KvCache(*(t.cpu() for t in gpu))
    fr = torch.zeros(0, dtype=torch.float64) if freq is None else freq
    raw = lambda t: t.view(torch.uint8)  # noqa: E731
    want_k, want_v = raw(before.k).clone(), raw(before.v).clone()
    owner, written = {}, set()
    for b in range(B):
        pos = torch.arange(max(past[b], 0), max(past[b], 0) + n[b])
        if q is not None:
            ref = rotate_reference(q[b, :, :n[b]], pos, fr, inter)
            norm = q[b, :, :n[b]].double().norm(dim=-1, keepdim=True)
            out = q_out[b].double().cpu()
            assert ((out[:, :n[b]] - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -21 * norm).all(), b
            assert (out[:, n[b]:] == 7).all()
        new = (rotate_reference(k[b, :, :n[b]], pos, fr, inter), v[b, :, :n[b]].double())
        for blk in range(max(past[b], 0) // page, (int(pos[-1]) // page + 1) if n[b] else 0):
            if blk >= max_pages or not 0 <= int(cache.table[b, blk]) < pages:
                continue
            p = int(cache.table[b, blk])
            if p in owner:
                continue
            owner[p] = (b, blk)
            lo = max(past[b] - blk * page, 0)
            hi = min(past[b] + n[b] - blk * page, page)
            at = slice(blk * page + lo - past[b], blk * page + hi - past[b])
            for x, codes, old, s_got, s_old in (
                    (new[0][:, at], got.k[p], before.k[p], got.k_scale[p], before.k_scale[p]),
                    (new[1][:, at], got.v[p].transpose(1, 2), before.v[p].transpose(1, 2), got.v_scale[p],
                     before.v_scale[p])):
                s = need_scale(x)
                if lo:
                    s = torch.maximum(s, s_old.double())
                assert torch.equal(s_got.double(), s), (b, blk)
                s = s[:, None, None]
                stored = codes.double() * s
                fin = torch.isfinite(x)
                assert torch.equal(torch.isnan(stored[:, lo:hi]), torch.isnan(x))
                norm = torch.where(fin, x, 0.0).norm(dim=-1, keepdim=True)
                lim = 2.0 ** -4 * x.abs() + 2.0 ** -10 * s + 2.0 ** -20 * norm
                assert ((stored[:, lo:hi] - x).abs() <= lim)[fin].all(), (b, blk)
                assert (stored[:, lo:hi].abs() == 448 * s)[torch.isinf(x)].all()
                kept = old.double() * s_old.double()[:, None, None]
                assert ((stored[:, :lo] - kept[:, :lo]).abs() <= 2.0 ** -10 * s).all(), (b, blk)
            written.add(p)
            want_k[p, :, :hi] = raw(got.k)[p, :, :hi]
            want_v[p, :, :, :hi] = raw(got.v)[p, :, :, :hi]
    # nothing else changed: other pages, tokens behind the new ones, other scales
    assert torch.equal(raw(got.k), want_k) and torch.equal(raw(got.v), want_v)
    rest = [p for p in range(pages) if p not in written]
    assert torch.equal(got.k_scale[rest], before.k_scale[rest]) and torch.equal(got.v_scale[rest], before.v_scale[rest])
    return gpu


def freqs(half, base=10000.0):
    return base ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))


# (B, T, Hq, H, D, page, max_pages, past, n, rot, interleaved)
APPEND = [
    (4, 1, 4, 2, 128, 16, 4, [0, 1, 15, 16], None, 128, False),
    (3, 1, 2, 2, 64, 64, 3, [63, 64, 100], [1, 0, 1], 64, True),
    (2, 5, 8, 1, 64, 32, 4, [30, 0], [5, 2], 32, False),
    (2, 100, 4, 2, 128, 16, 12, [7, 33], [100, 61], 32, True),
    (1, 300, 3, 1, 128, 128, 4, [77], None, 64, False),
    (2, 129, 0, 3, 64, 64, 4, [0, 64], None, 0, False),
    (2, 40, 2, 1, 128, 32, 3, [80, 60], None, 16, True),      # runs past the table's end
]


@pytest.mark.parametrize("case", APPEND, ids=[str(i) for i in range(len(APPEND))])
def test_append(case):
    B, T, Hq, H, D, page, max_pages, past, n, rot, inter = case
    print("case", case, flush=True)
    g = torch.Generator().manual_seed(31)
    cache = filled_cache(g, B, H, D, page, max_pages)
    mk = lambda h: torch.randn(B, h, T, D, generator=g).to(torch.bfloat16)  # noqa: E731
    k, v, q = mk(H) * 3, mk(H), mk(Hq) if Hq else None
    freq = freqs(rot // 2) if rot else None
    check_append(cache, k, v, past, n or [T] * B, freq, inter, q, n is not None)
    view = lambda x: x.transpose(1, 2).contiguous().transpose(1, 2)  # noqa: E731
    check_append(cache, k, v, past, n or [T] * B, freq, inter, q, n is not None, view)


def test_append_far_positions():
    """Angles at positions near 2^22: an fp32 product of position and frequency would be off by 0.25."""
    g = torch.Generator().manual_seed(32)
    page, far = 128, (1 << 22) - 3
    cache = filled_cache(g, 1, 1, 64, page, 3)
    table = torch.full((1, far // page + 2), -1, dtype=torch.int32)
    table[0, -2:] = cache.table[0, :2]
    cache = cache._replace(table=table)
    mk = lambda: torch.randn(1, 1, 6, 64, generator=g).to(torch.bfloat16)  # noqa: E731
    check_append(cache, mk(), mk(), [far], [6], freqs(32), False, mk())


def test_append_values_that_are_not_ordinary():
    """NaN, infinities, zeros, the largest and the smallest values; scales at the powers of two."""
    g = torch.Generator().manual_seed(33)
    cache = filled_cache(g, 2, 2, 64, 16, 4)
    k = torch.randn(2, 2, 20, 64, generator=g)
    v = torch.randn(2, 2, 20, 64, generator=g)
    v[0, 0, 2, 5], v[0, 0, 3, 6], v[0, 1, 0, 0] = math.nan, math.inf, -math.inf
    v[1, 0] = 0
    v[1, 1, 16:] = 3.0e38
    k[0, 0, :, :] = 448.0
    k[0, 1, :, :] = 450.0
    k[1, 0, :, :] = 1e-38
    k[1, 1] *= 1e-30
    check_append(cache, k.to(torch.bfloat16), v.to(torch.bfloat16), [0, 32], [20, 20], None, False)


def test_append_pages_missing_or_named_twice():
    g = torch.Generator().manual_seed(34)
    cache = filled_cache(g, 3, 2, 64, 16, 4)
    mk = lambda: torch.randn(3, 2, 40, 64, generator=g).to(torch.bfloat16)  # noqa: E731
    cache.table[0, 1] = -1
    cache.table[1, 0] = cache.table[0, 0]        # sequence 0 comes first
    cache.table[2, 2] = cache.table[2, 0]        # the same sequence, an earlier token first
    cache.table[2, 1] = 1 << 20
    check_append(cache, mk(), mk(), [3, 0, 5], [40, 40, 40], freqs(32), False)


@pytest.mark.parametrize("B,T,page,past", [(70, 500, 16, 9), (2100, 1, 16, 30)])
def test_append_of_very_many_pages(B, T, page, past):
    """Enough pages that their owners are written down first: the same rules for pages
    that are missing or named twice; and every replay of a captured call, its
    workspace full of other bytes, equals the eager one."""
    g = torch.Generator().manual_seed(36)
    cache = filled_cache(g, B, 1, 64, page, (past + T) // page + 2)
    first, last = past // page, (past + T - 1) // page
    cache.table[1, first] = -1
    cache.table[B - 1, first] = cache.table[0, last]
    cache.table[B // 2, last] = cache.table[2, last]
    cache.table[3, last] = cache.table[4, first]
    cache.table[5, last] = cache.k.shape[0]
    mk = lambda: torch.randn(B, 1, T, 64, generator=g).to(torch.bfloat16)  # noqa: E731
    k, v = mk(), mk()
    n = [T if b % 7 else T // 2 for b in range(B)]
    one = check_append(cache, k, v, [past] * B, n, None, False)
    two, nd, pd = to_dev(cache), torch.tensor(n, dtype=torch.int32, device=DEV), torch.full((B,), past, dtype=torch.int32, device=DEV)
    kd, vd = k.to(DEV), v.to(DEV)
    work = torch.empty(8 * cache.k.shape[0], dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        linrec.kv_append(two, kd, vd, pd, n_new=nd, workspace=work)
    for fill in (0, 255, 7):
        for t, c in zip(two, cache):
            t.view(torch.uint8).copy_(c.view(torch.uint8))
        work.fill_(fill)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(one, two):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_append_in_place_queries_and_replays():
    """q_out = q; and a captured append repeats what an eager one leaves."""
    g = torch.Generator().manual_seed(35)
    cache = filled_cache(g, 2, 2, 128, 64, 4)
    mk = lambda h: torch.randn(2, h, 3, 128, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    k, v, q = mk(2), mk(2), mk(4)
    past, freq = torch.tensor([62, 5], dtype=torch.int32, device=DEV), freqs(64).to(DEV)
    one, two = to_dev(cache), to_dev(cache)
    want = linrec.kv_append(one, k, v, past, inv_freq=freq, q=q)
    same = q.clone()
    assert linrec.kv_append(two, k, v, past, inv_freq=freq, q=same, q_out=same) is same
    assert torch.equal(same, want)
    three = to_dev(cache)
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        linrec.kv_append(three, k, v, past, inv_freq=freq, q=q, q_out=out)
    for _ in range(3):
        for t, c in zip(three, cache):
            t.view(torch.uint8).copy_(c.view(torch.uint8))
        out.zero_()
        linrec.kv_append(two, k, v, past, inv_freq=freq)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        for a, b in zip(one, three):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_piece_then_tokens():
    """A prompt in two ragged pieces, then single tokens: append and attend each
    time.  The cache then holds what one append of everything would up to one
    step, and the last token's output is attention over it."""
    g = torch.Generator().manual_seed(36)
    B, H, Hq, D, page = 2, 2, 4, 64, 16
    T = 150
    k, v = (torch.randn(B, H, T, D, generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(B, Hq, T, D, generator=g).to(torch.bfloat16)
    table = torch.randperm(24, generator=g)[:20].view(2, 10).to(torch.int32)
    cache = linrec.kv_cache(24, H, page, D, table.to(DEV))
    freq = freqs(D // 2).to(DEV)
    at = 0
    for n in (70, 77, 1, 1, 1):
        sl = slice(at, at + n)
        past = torch.full((B,), at, dtype=torch.int32, device=DEV)
        qr = linrec.kv_append(cache, k[:, :, sl].to(DEV), v[:, :, sl].to(DEV), past, inv_freq=freq, q=q[:, :, sl].to(DEV))
        o = linrec.kv_attn(cache, qr, past)
        at += n
    torch.cuda.synchronize()
    host = linrec.KvCache(*(t.cpu() for t in cache))
    ref, mag, _ = attn_reference(host, qr.cpu(), [T - 1] * B, [1] * B, D ** -0.5, 0)
    assert ((o.double().cpu() - ref).abs() <= (2.0 ** -8 + 2.0 ** -12) * mag + 2.0 ** -8 * ref.abs()).all()
    for b in range(B):
        K, V, _ = dense(host, b)
        pos = torch.arange(T)
        for got, x in ((K, rotate_reference(k[b], pos, freqs(D // 2), False)), (V, v[b].double())):
            # the smallest step of the page's scale: the scale holds the page's largest value
            s = torch.exp2(torch.ceil(torch.log2(x.abs().amax() / 448)))
            lim = 2.0 ** -4 * x.abs() + 2.0 ** -9 * s + 2.0 ** -20 * x.norm(dim=-1, keepdim=True)
            assert ((got[:, :T] - x).abs() <= lim).all()


@pytest.mark.parametrize("T", [1, 4, 70])
@pytest.mark.parametrize("given", [False, True])
def test_sequences_that_are_not_there(T, given):
    """A negative past: the sequence has no new tokens, n_new or not.  Outputs the
    calls make themselves hold zeros there, whatever their memory held before;
    given ones, the cache and lse stay as they were; the others are as ever."""
    g, cache, q = draw(40, 3, T, 4, 2, 64, 16, 8)
    past, n = [-1, 30, -(1 << 31)], [0, T, 0]
    check_attn(cache, q, past, n, n_new=given)
    k, v = (torch.randn(3, 2, T, 64, generator=g).to(torch.bfloat16) for _ in range(2))
    check_append(cache, k, v, past, n, freqs(16), False, q, given)
    gpu, dq, kd, vd = to_dev(cache), q.to(DEV), k.to(DEV), v.to(DEV)
    past_d = torch.tensor(past, dtype=torch.int32, device=DEV)
    n_d = torch.full((3,), T, dtype=torch.int32, device=DEV) if given else None
    for call in (lambda: linrec.kv_attn(gpu, dq, past_d, n_new=n_d),
                 lambda: linrec.kv_append(gpu, kd, vd, past_d, n_new=n_d, q=dq)):
        for _ in range(8):     # what the allocator hands out next is full of NaN
            torch.full(q.shape, math.nan, dtype=torch.bfloat16, device=DEV)
        out = call()
        torch.cuda.synchronize()
        assert (out[0] == 0).all() and (out[2] == 0).all() and (out[1] != 0).any()


LARGE = [(64, 1, 2, 16), (64, 6, 8, 64), (128, 1, 4, 32), (128, 90, 2, 16), (64, 90, 2, 128), (128, 90, 2, 64), (128, 6, 8, 16)]


@pytest.mark.parametrize("D,T,Hq,page", LARGE)
@pytest.mark.parametrize("exponent", [119, 120, 124, 127])
def test_attention_hidden_values_under_the_largest_scales(D, T, Hq, page, exponent):
    """A code times a scale may pass bf16's range (2^120 * 256, which the append stores
    for the largest bf16 values; 2^127 * 448).  Rows that do not see it are as ever: a page
    behind the last token in the same tile, and tokens behind it in the same page, where
    the first visible one holds 2^118 (times a weight of at most 2^8 that is in range)."""
    _, cache, q = draw(41, 2, T, Hq, 2, D, page, 256 // page)
    past = [37, 100]
    for b in range(2):
        end = past[b] + T                    # the first hidden token
        blk, off = end // page, end % page
        last = (end | 63) // page            # the tile's last page
        for p in range(blk, min(last, cache.table.shape[1] - 1) + 1):
            p_id = int(cache.table[b, p])
            cache.v_scale[p_id] = 2.0 ** exponent
            lo = off if p == blk else 0
            cache.v.view(torch.uint8)[p_id, :, :, :lo] = 0
            cache.v[p_id, :, :, :min(lo, 1)] = torch.tensor(2.0 ** (118 - exponent)).to(F8)
            cache.v.view(torch.uint8)[p_id, :, :, lo:] = 0x7e if b == 0 else 0xfe      # +-448
    check_attn(cache, q, past, [T] * 2)
    check_attn(cache, q, past, [T] * 2, window=21)


@pytest.mark.parametrize("D,T,Hq,page", [c for c in LARGE if c[1] > 1])
@pytest.mark.parametrize("exponent,code", [(120, 0x78), (120, 0xfe), (127, 0x40), (125, 0xd0)])
def test_attention_values_past_bf16_reach_only_rows_that_see_them(D, T, Hq, page, exponent, code):
    """Such a value within the rows' own tokens: rows before it are as ever, and those
    that see it get no finite number in its feature, as from an infinity."""
    _, cache, q = draw(42, 1, T, Hq, 1, D, page, 256 // page)
    past, at, f = 37, 37 + T // 2, 9
    p = int(cache.table[0, at // page])
    cache.v_scale[p] = 2.0 ** exponent
    cache.v.view(torch.uint8)[p] = 0
    cache.v[p, :, :, 0] = torch.tensor(2.0 ** (118 - exponent)).to(F8)
    cache.v.view(torch.uint8)[p, :, f, at % page] = code
    shown = linrec.KvCache(*(t.clone() for t in cache))
    shown.v.view(torch.uint8)[p, :, f, at % page] = 0x7f         # a NaN: the reference's mark
    ref, mag, _ = attn_reference(shown, q, [past], [T], D ** -0.5, 0)
    o = linrec.kv_attn(to_dev(cache), q.to(DEV), torch.tensor([past], dtype=torch.int32, device=DEV)).double().cpu()
    seen = torch.isnan(ref)
    assert seen[:, :, T // 2:, f].all() and not seen[:, :, :T // 2].any()
    assert torch.equal(torch.isfinite(o), ~seen)
    assert ((o - ref).abs() <= (2.0 ** -8 + 2.0 ** -12) * mag + 2.0 ** -8 * ref.abs())[~seen].all()


@pytest.mark.parametrize("D,T,Hq,page", LARGE)
@pytest.mark.parametrize("exponent", [119, 120, 124, 127])
def test_attention_sums_past_fp32_are_not_finite(D, T, Hq, page, exponent):
    """Visible values of 2^123 and more, whose weighted sums may pass fp32's range before
    they are divided: what comes out finite is right."""
    _, cache, q = draw(41, 2, T, Hq, 2, D, page, 256 // page)
    past = [37, 100]
    for b in range(2):
        p = int(cache.table[b, (past[b] + T) // page])
        cache.v_scale[p] = 2.0 ** exponent
        cache.v[p] = (cache.v[p].float().sign() * 2.0 ** min(126 - exponent, 4)).to(F8)
    ref, mag, _ = attn_reference(cache, q, past, [T] * 2, D ** -0.5, 0)
    o = linrec.kv_attn(to_dev(cache), q.to(DEV), torch.tensor(past, dtype=torch.int32, device=DEV)).double().cpu()
    near = (o - ref).abs() <= (2.0 ** -8 + 2.0 ** -12) * mag + 2.0 ** -8 * ref.abs()
    assert (near | ~torch.isfinite(o)).all()


@pytest.mark.parametrize("T,Hq,max_pages", [(1, 4, 8), (1, 2, 60), (6, 8, 8), (90, 2, 8), (90, 2, 60)])
@pytest.mark.parametrize("sign", [1, -1])
def test_attention_scores_past_fp32_are_no_empty_rows(T, Hq, max_pages, sign):
    """A row whose largest scaled score passes fp32's range, upwards or downwards, comes as
    NaN, not as the zeros and -inf of a row that sees nothing; a row of zero scores beside
    it is as ever."""
    _, cache, q = draw(43, 1, T, Hq, 2, 64, 16, max_pages)
    q = q.abs()
    cache.k.view(torch.uint8).bitwise_and_(0x7f).bitwise_or_(0x80 if sign < 0 else 0)   # scores of one sign
    q[:, 0] = 0
    past = max_pages * 16 - T - 3
    q_d, past_d = q.to(DEV), torch.tensor([past], dtype=torch.int32, device=DEV)
    lse = torch.empty(1, Hq, T, device=DEV)
    o = linrec.kv_attn(to_dev(cache), q_d, past_d, scale=2.0 ** 127, lse=lse).double().cpu()
    ref, mag, ref_lse = attn_reference(cache, q, [past], [T], 2.0 ** 127, 0)
    assert (sign * ref_lse[:, 1:] > 2.0 ** 128).all()
    assert torch.isnan(o[:, 1:]).all() and torch.isnan(lse[:, 1:]).all()
    assert ((o - ref).abs() <= (2.0 ** -8 + 2.0 ** -12) * mag + 2.0 ** -8 * ref.abs())[:, 0].all()
    assert ((lse.double().cpu() - ref_lse).abs() <= 2.0 ** -12 * (1 + ref_lse.abs()))[:, 0].all()


# (B, T, Hq, H, D, page, max_pages, past): odd numbers of rows, several splits
ODD = [(1, 1, 1, 1, 128, 64, 64, [4000]), (1, 1, 1, 1, 64, 16, 64, [1000]), (1, 3, 1, 1, 128, 32, 40, [1200]),
       (3, 1, 5, 1, 64, 128, 16, [2000, 0, 700]), (1, 129, 3, 3, 128, 64, 20, [1100]), (1, 67, 1, 1, 64, 16, 90, [1300])]


@pytest.mark.parametrize("case", ODD, ids=[str(i) for i in range(len(ODD))])
def test_attention_splits_of_an_odd_number_of_rows(case):
    """The parts of every split lie on 16-byte boundaries; the workspace is used to its end
    and no further."""
    B, T, Hq, H, D, page, max_pages, past = case
    _, cache, q = draw(44, B, T, Hq, H, D, page, max_pages)
    c = linrec._kv_desc(cache, B)
    need = linrec._lib().linrec_kv_attn_workspace_bytes(linrec.ctypes.byref(c), B, T, Hq)
    rows = B * T * Hq
    per = -(-rows * (D + 2) // 4) * 16
    assert need % per == 0 and need // per > 1
    work = torch.full((need + 256,), 0x5a, dtype=torch.uint8, device=DEV)
    check_attn(cache, q, past, [T] * B, workspace=work)
    assert (work[need:] == 0x5a).all() and (work[:need - 16] != 0x5a).any()


def test_captured_calls_that_make_their_outputs():
    """Outputs made within a capture are cleared by every replay, whatever was left in
    their memory, between eager calls that make theirs."""
    g, cache, q = draw(45, 3, 2, 4, 2, 64, 16, 8)
    k, v = (torch.randn(3, 2, 2, 64, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    gpu, dq, past = to_dev(cache), q.to(DEV), torch.tensor([-1, 30, 5], dtype=torch.int32, device=DEV)

    freq = freqs(16).to(DEV)

    def both():
        qr = linrec.kv_append(gpu, k, v, past, q=dq, inv_freq=freq)
        return qr, linrec.kv_attn(gpu, qr, past)

    want = both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for _ in range(4):
        for t in out:
            t.fill_(math.nan)
        graph.replay()
        again = both()
        torch.cuda.synchronize()
        for a, b, c in zip(out, want, again):
            assert torch.equal(a, b) and torch.equal(c, b) and (a[0] == 0).all()
