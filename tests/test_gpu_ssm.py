"""The short causal convolution and the selective state-space scan on the GPU
against the 64-bit definition (ssm_reference).

Tolerances, with u = 2^-24 and every error measured against the sum of the
absolute values of an output's terms:
 - convolution: a term passes at most K + 2 additions and products; silu adds an
   exponential (off by |p| u in its argument, which e^-|p| outweighs: below 1 u of
   the value, and 2 u of its own), a reciprocal (2 u) and 3 products: 16 u bounds
   a value.  Sums over tokens add their adds one after another over at most 32
   tokens in a lane, 256 in a workgroup and the workgroups in order: at most
   T B + 300 additions, so (B T + 332) u.
 - scan: a term of h_t passes at most T steps, each a product, an addition and a
   gate; a gate a = exp2(d A') is off by 2 u and by |d A| (4 u + the step's 16 u)
   of itself (the exponential, its two reciprocals and seven products of softplus,
   exp(-|v|) by |v| u <= 16 u of the values here).  Summed over a path the latter
   is 20 u sum |d A|, and a path that decays by L = sum |d A| weighs exp(-L): at
   most 20 u L exp(-L) < 8 u of the undecayed term; the path's own majorant counts
   exp(-L) only, so L <= 12 is allowed for by 20 * 12 u = 240 u and terms behind
   that are e^-12 of a majorant that holds undecayed ones.  So (5 T + 300) u, and
   for a sum over tokens and batch or over channels as many additions more.
 - rounding to the output type: half a step, 2^-8 of the value in bf16, 2^-24 in
   fp32.
"""
import pytest
import torch

import ssm_reference as ref
from state_passing_amd import linrec

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def half_step(t):
    return torch.finfo(t.dtype).eps / 2


def close(name, got, want, bound, terms):
    """|got - want| <= terms u bound, and the output's own rounding."""
    got64, want = got.detach().to("cpu", torch.float64), want.reshape(got.shape)
    tol = terms * U * bound.reshape(got.shape) * (1 + 2.0 ** -7) + half_step(got) * want.abs() + 1e-37
    off = (got64 - want).abs()
    assert torch.isfinite(got64).all(), name
    bad = off > tol
    assert not bad.any(), (name, (off / tol).max().item(), int(bad.sum()), bad.nonzero()[0].tolist())


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rows(g, B, T, C, dtype, scale=1.0, of=1):
    """[B,T,C] rows that begin at 16 bytes, a slice of rows `of` times as wide."""
    pad = -(-C // 8) * 8
    t = (torch.randn(B, T, of * pad, generator=g) * scale).to(dtype).to(DEV)
    return t[..., (of - 1) * pad:(of - 1) * pad + C]


# ----------------------------------------------------------------- convolution

def conv_inputs(B, T, C, K, dtype, seed=0, bias=True, state=True, of=1):
    g = gen(seed)
    s = dict(x=rows(g, B, T, C, dtype, of=of), w=(torch.randn(C, K, generator=g) * 0.6).to(DEV))
    s["bias"] = (torch.randn(C, generator=g) * 0.2).to(DEV) if bias else None
    s["state"] = torch.randn(B, K - 1, C, generator=g).to(DEV) if state else None
    s["dy"], s["dstate"] = rows(g, B, T, C, dtype), torch.randn(B, K - 1, C, generator=g).to(DEV)
    return s


CONV = [   # B, T, C, K, dtype, out dtype, act, n_new
    (1, 1, 8, 4, BF, None, "silu", None), (1, 1, 1, 2, F32, None, None, None), (2, 2, 24, 4, BF, F32, "silu", None),
    (2, 3, 7, 4, F32, None, "silu", None), (3, 7, 13, 3, BF, None, "silu", [7, 0, 2]), (1, 8, 64, 2, BF, None, None, None),
    (2, 9, 130, 4, F32, None, "silu", [1, 9]), (2, 31, 520, 3, BF, F32, None, [40, -3]), (1, 33, 1000, 4, BF, None, "silu", None),
    (4, 65, 72, 4, F32, None, None, [65, 64, 1, 33]), (1, 300, 257, 2, BF, None, "silu", [299]), (2, 1027, 8, 4, BF, None, "silu", [1027, 3]),
    (1, 2050, 3, 3, F32, None, "silu", None), (1, 4133, 2048, 4, BF, None, "silu", None),
]


@pytest.mark.parametrize("B,T,C,K,dtype,out,act,n", CONV)
def test_conv_forward_and_backward(B, T, C, K, dtype, out, act, n):
    s = conv_inputs(B, T, C, K, dtype, seed=T + C, bias=T % 2 == 1, state=C % 3 != 0, of=2 if C % 2 else 1)
    n_new = None if n is None else torch.tensor(n, dtype=torch.int32, device=DEV)
    args = dict(act=act, n_new=n_new, out_dtype=out)
    y, state = linrec.conv_fwd(s["x"], s["w"], s["bias"], s["state"], **args)
    dx, dw, dbias, dstate = linrec.conv_bwd(s["x"], s["w"], s["bias"], s["state"], s["dy"], s["dstate"], **args)
    torch.cuda.synchronize()
    plain = dict(x=s["x"], w=s["w"], bias=s["bias"], state=s["state"], act=act, n_new=n, dy=s["dy"], dstate=s["dstate"])
    want, most = ref.conv(**plain), ref.conv(**plain, absolute=True)
    long = B * T + 332
    assert y.dtype == dx.dtype == (out or dtype)
    close("y", y, want["y"], most["y"], 16)
    close("state_out", state, want["state_out"], most["state_out"], 0)
    close("dx", dx, want["dx"], most["dx"], 16)
    close("dstate_in", dstate, want["dstate_in"], most["dstate_in"], 16)
    close("dw", dw, want["dw"], most["dw"], long)
    if s["bias"] is None:
        assert dbias is None
    else:
        close("dbias", dbias, want["dbias"], most["dbias"], long)


def test_conv_pieces_are_the_whole():
    s = conv_inputs(2, 150, 40, 4, F32, seed=5)
    x, dy = s["x"], s["dy"]
    y, end = linrec.conv_fwd(x, s["w"], s["bias"], s["state"])
    full = linrec.conv_bwd(x, s["w"], s["bias"], s["state"], dy, s["dstate"])
    cuts, st, entering = [0, 1, 3, 60, 60, 61, 150], s["state"].clone(), []
    for a, b in zip(cuts, cuts[1:]):
        entering.append(st.clone())
        part, st = linrec.conv_fwd(x[:, a:b], s["w"], s["bias"], st, state_out=st)   # in place
        assert torch.equal(part, y[:, a:b])
    assert torch.equal(st, end)
    dst, dw, db = s["dstate"].clone(), 0, 0
    for i in reversed(range(len(cuts) - 1)):
        a, b = cuts[i], cuts[i + 1]
        dx, w1, b1, dst = linrec.conv_bwd(x[:, a:b], s["w"], s["bias"], entering[i], dy[:, a:b], dst, dstate_in=dst)
        dw, db = dw + w1, db + b1
        # a sum of at most 4 terms is grouped otherwise where a cut parts it
        assert b == a or (dx - full[0][:, a:b]).abs().max() <= 16 * U * full[0].abs().max()
    for got, want in ((dst, full[3]), (dw, full[1]), (db, full[2])):
        assert (got - want).abs().max() <= 1000 * U * want.abs().max()


def test_conv_rows_behind_stay():
    s = conv_inputs(3, 40, 24, 4, BF, seed=2)
    n = torch.tensor([40, 0, 17], dtype=torch.int32, device=DEV)
    x, dy = s["x"].clone(), s["dy"].clone()
    for b, k in enumerate(n.tolist()):
        x[b, k:], dy[b, k:] = float("nan"), float("inf")
    y, dx = torch.full_like(x, 7.0), torch.full_like(x, 5.0)
    _, state = linrec.conv_fwd(x, s["w"], s["bias"], s["state"], n_new=n, y=y)
    _, dw, db, ds = linrec.conv_bwd(x, s["w"], s["bias"], s["state"], dy, s["dstate"], n_new=n, dx=dx)
    for t in (state, dw, db, ds):
        assert torch.isfinite(t).all()
    for b, k in enumerate(n.tolist()):
        assert (y[b, k:] == 7.0).all() and (dx[b, k:] == 5.0).all()
        assert torch.isfinite(y[b, :k]).all() and torch.isfinite(dx[b, :k]).all()
    assert torch.equal(state[1], s["state"][1]) and torch.equal(ds[1], s["dstate"][1])


@pytest.mark.parametrize("B,T,C,K,dtype", [(1, 1, 8, 4, BF), (5, 1, 1000, 4, BF), (3, 4, 13, 3, F32), (70, 2, 264, 2, BF)])
def test_conv_step(B, T, C, K, dtype):
    s = conv_inputs(B, T, C, K, dtype, seed=B)
    slots = torch.randperm(B + 4, generator=gen(B))[:B].to(torch.int32).to(DEV)
    pool = torch.randn(B + 4, K - 1, C, generator=gen(1)).to(DEV)
    before = pool.clone()
    y = linrec.conv_step(s["x"], s["w"], s["bias"], pool, slots=slots)
    want, state = linrec.conv_fwd(s["x"], s["w"], s["bias"], before[slots.long()])
    assert torch.equal(y, want) and torch.equal(pool[slots.long()], state)
    rest = torch.ones(B + 4, dtype=torch.bool)
    rest[slots.long().cpu()] = False
    assert torch.equal(pool[rest.to(DEV)], before[rest.to(DEV)])
    pool = before[:B].clone()
    assert torch.equal(linrec.conv_step(s["x"], s["w"], s["bias"], pool), linrec.conv_fwd(s["x"], s["w"], s["bias"], before[:B].clone())[0])


# ----------------------------------------------------------------- scan

def scan_inputs(B, T, C, N, G=1, dtype=BF, seed=0, D=True, z=True, bias=True, state=True, softplus=True, of=1):
    g = gen(seed)
    s = dict(x=rows(g, B, T, C, dtype, of=of))
    s["A"] = (-torch.arange(1, N + 1) * torch.exp(0.3 * torch.randn(C, N, generator=g))).to(DEV)
    proj = torch.randn(B, T, 2, G, N, generator=g).to(dtype).to(DEV)
    s["B"], s["C"] = proj[:, :, 0].transpose(1, 2), proj[:, :, 1].transpose(1, 2)
    if softplus:
        s["dt"] = rows(g, B, T, C, dtype, 0.5)
        s["dt_bias"] = (torch.rand(C, generator=g) * 4 - 6).to(DEV) if bias else None
    else:
        s["dt"] = rows(g, B, T, C, dtype, 0.02).abs_()
        s["dt_bias"] = (torch.rand(C, generator=g) * 0.02).to(DEV) if bias else None
    s["D"] = torch.randn(C, generator=g).to(DEV) if D else None
    s["z"] = rows(g, B, T, C, dtype, of=of) if z else None
    s["h_in"] = (torch.randn(B, C, N, generator=g) * 0.5).to(DEV) if state else None
    s["softplus"] = softplus
    grad = dict(dy=rows(g, B, T, C, dtype), dh_out=(torch.randn(B, C, N, generator=g) * 0.3).to(DEV))
    return s, grad


def run(s, grad, n_new=None, out=None, **kw):
    first = [s[k] for k in ("x", "dt", "A", "B", "C")]
    layer = {k: s[k] for k in ("D", "z", "dt_bias", "softplus")}
    y, h_out, saved = linrec.scan_fwd(*first, s["h_in"], n_new=n_new, save=True, out_dtype=out, **layer)
    r = linrec.scan_bwd(*first, saved, grad["dy"], grad["dh_out"], n_new=n_new, out_dtype=out, **layer, **kw)
    return dict(y=y, h_out=h_out, **r._asdict())


def check(s, grad, got, B, T, C, n=None):
    want, most = (ref.scan(**s, **grad, n_new=n, absolute=a) for a in (False, True))
    path, tokens, group = 5 * T + 300, B * T, C
    terms = dict(y=path, h_out=path, dx=2 * path, ddt=2 * path, dB=2 * path + group, dC=2 * path + group, dh_in=2 * path,
                 dA=2 * path + tokens, dD=path + tokens, ddt_bias=2 * path + tokens, dz=path)
    for k, t in terms.items():
        if got.get(k) is not None:
            close(k, got[k], want[k], most[k], t)


SCAN = [   # B, T, C, N, G, dtype, out, n_new, options
    (1, 1, 8, 16, 1, BF, None, None, {}), (1, 1, 1, 8, 1, F32, None, None, dict(z=False)),
    (2, 2, 24, 64, 1, BF, F32, None, dict(D=False)), (2, 7, 13, 16, 1, F32, None, None, dict(bias=False)),
    (3, 8, 64, 32, 1, BF, None, [8, 0, 3], {}), (1, 9, 70, 16, 1, BF, None, None, dict(softplus=False)),
    (2, 31, 72, 16, 1, F32, None, [31, 50], dict(z=False, D=False, bias=False)), (2, 32, 130, 8, 1, BF, F32, None, {}),
    (1, 33, 136, 64, 1, F32, None, None, {}), (2, 65, 48, 32, 2, F32, None, None, dict(of=2)),
    (3, 40, 96, 16, 4, BF, None, [40, -1, 1], dict(of=2)), (2, 129, 24, 16, 1, BF, None, [129, 128], dict(state=False)),
    (1, 300, 200, 16, 1, BF, None, None, {}), (2, 513, 33, 8, 1, F32, None, [513, 200], {}),
    (1, 700, 16, 64, 2, BF, None, [640], dict(softplus=False)), (1, 1000, 40, 32, 1, F32, None, None, dict(z=False)),
]


@pytest.mark.parametrize("B,T,C,N,G,dtype,out,n,options", SCAN)
def test_scan_forward_and_backward(B, T, C, N, G, dtype, out, n, options):
    s, grad = scan_inputs(B, T, C, N, G, dtype, seed=T + N, **options)
    n_new = None if n is None else torch.tensor(n, dtype=torch.int32, device=DEV)
    got = run(s, grad, n_new, out)
    torch.cuda.synchronize()
    assert got["y"].dtype == got["dx"].dtype == got["dB"].dtype == (out or dtype)
    assert (got["dz"] is None) == (s["z"] is None) and (got["dD"] is None) == (s["D"] is None)
    check(s, grad, got, B, T, C, n)


@pytest.mark.parametrize("N", [8, 16, 32, 64])
@pytest.mark.parametrize("dtype,out", [(BF, None), (BF, F32), (F32, None)])
def test_scan_without_a_gate(N, dtype, out):
    """Its backward is a kernel of its own, of every number of states and type; a segmented piece, a group's end."""
    B, T, C, n = 2, 170, 520 // N + 11, [170, 97]
    s, grad = scan_inputs(B, T, C, N, dtype=dtype, seed=N, z=False)
    got = run(s, grad, torch.tensor(n, dtype=torch.int32, device=DEV), out)
    torch.cuda.synchronize()
    assert got["dz"] is None
    check(s, grad, got, B, T, C, n)


@pytest.mark.parametrize("N,dtype", [(16, BF), (64, F32), (8, BF), (32, F32)])
def test_scan_pieces_are_the_whole(N, dtype):
    B, T, C = 2, 330, 24
    s, grad = scan_inputs(B, T, C, N, 1, dtype, seed=9)
    cuts, h, kept = [0, 5, 37, 37, 200, 330], s["h_in"].clone(), []
    layer = {k: s[k] for k in ("D", "dt_bias", "softplus")}

    def part(a, b):
        return [s[k][:, a:b] for k in ("x", "dt")] + [s["A"]] + [s[k][:, :, a:b] for k in ("B", "C")], dict(layer, z=s["z"][:, a:b])

    y = torch.empty_like(s["x"])
    for a, b in zip(cuts, cuts[1:]):
        first, rest = part(a, b)
        _, h, saved = linrec.scan_fwd(*first, h, h_out=h, y=y[:, a:b], save=True, **rest)
        kept.append(saved)
    got = dict(y=y, h_out=h)
    g = grad["dh_out"].clone()
    sums, grads = {}, {}
    for i in reversed(range(len(cuts) - 1)):
        a, b = cuts[i], cuts[i + 1]
        first, rest = part(a, b)
        r = linrec.scan_bwd(*first, kept[i], grad["dy"][:, a:b], g, dh_in=g, **rest)._asdict()
        for k in ("dA", "dD", "ddt_bias"):
            sums[k] = sums.get(k, 0) + r[k]
        for k in ("dx", "ddt", "dz"):
            grads.setdefault(k, torch.empty_like(s["x"]))[:, a:b] = r[k]
        for k in ("dB", "dC"):
            grads.setdefault(k, torch.empty(B, 1, T, N, dtype=dtype, device=DEV))[:, :, a:b] = r[k]
    check(s, grad, dict(got, dh_in=g, **sums, **grads), B, T, C)


def test_scan_rows_behind_stay():
    B, T, C, N = 3, 50, 24, 16
    s, grad = scan_inputs(B, T, C, N, seed=4)
    n = torch.tensor([50, 0, 21], dtype=torch.int32, device=DEV)
    clean = run(s, grad, n)
    for t in (s["x"], s["dt"], s["z"], grad["dy"]):
        for b, k in enumerate(n.tolist()):
            t[b, k:] = float("nan")
    for t in (s["B"], s["C"]):
        for b, k in enumerate(n.tolist()):
            t[b, :, k:] = float("inf")
    new = {k: torch.full((B, T, C), 3.0, dtype=BF, device=DEV) for k in ("dx", "ddt", "dz")}
    new |= {k: torch.full((B, 1, T, N), 3.0, dtype=BF, device=DEV) for k in ("dB", "dC")}
    got = run(s, grad, n, **new)
    for k, t in got.items():
        if k in new:
            for b, m in enumerate(n.tolist()):
                at = (b, slice(m, None)) if t.dim() == 3 else (b, slice(None), slice(m, None))
                live = (b, slice(0, m)) if t.dim() == 3 else (b, slice(None), slice(0, m))
                assert (t[at] == 3.0).all() and torch.equal(t[live], clean[k][live]), k
        else:
            assert torch.equal(t, clean[k]), k   # NaN would not be equal
    assert torch.equal(got["h_out"][1], s["h_in"][1]) and torch.equal(got["dh_in"][1], grad["dh_out"][1])


@pytest.mark.parametrize("B,T,C,N,G,dtype", [(1, 1, 8, 16, 1, BF), (5, 1, 1000, 16, 1, BF), (3, 4, 40, 64, 2, F32),
                                             (70, 2, 264, 8, 1, BF), (9, 1, 66, 32, 3, F32)])
def test_scan_step(B, T, C, N, G, dtype):
    if G == 3:
        C = 72
    s, _ = scan_inputs(B, T, C, N, G, dtype, seed=B)
    first = [s[k] for k in ("x", "dt", "A", "B", "C")]
    layer = {k: s[k] for k in ("D", "z", "dt_bias", "softplus")}
    slots = torch.randperm(B + 4, generator=gen(B))[:B].to(torch.int32).to(DEV)
    pool = torch.randn(B + 4, C, N, generator=gen(1)).to(DEV)
    before = pool.clone()
    y = linrec.scan_step(*first, pool, slots=slots, **layer)
    s["h_in"] = before[slots.long()]
    want, most = ref.scan(**s), ref.scan(**s, absolute=True)
    close("y", y, want["y"], most["y"], 5 * T + 300)
    close("S", pool[slots.long()], want["h_out"], most["h_out"], 5 * T + 300)
    rest = torch.ones(B + 4, dtype=torch.bool)
    rest[slots.long().cpu()] = False
    assert torch.equal(pool[rest.to(DEV)], before[rest.to(DEV)])


def test_steps_skip_bad_and_repeated_slots():
    B, C, N, K = 6, 40, 16, 4
    s, _ = scan_inputs(B, 2, C, N, seed=3)
    c = conv_inputs(B, 2, C, K, BF, seed=3)
    slots = torch.tensor([2, -1, 2, 9, 0, 1], dtype=torch.int32, device=DEV)   # entries 1, 2 and 3 are skipped
    keep = torch.tensor([True, False, False, False, True, True], device=DEV)
    S, W = torch.randn(4, C, N, device=DEV), torch.randn(4, K - 1, C, device=DEV)
    S0, W0 = S.clone(), W.clone()
    first = [s[k] for k in ("x", "dt", "A", "B", "C")]
    layer = {k: s[k] for k in ("D", "z", "dt_bias", "softplus")}
    y = linrec.scan_step(*first, S, slots=slots, **layer)
    v = linrec.conv_step(c["x"], c["w"], c["bias"], W, slots=slots)
    assert (y[~keep] == 0).all() and (v[~keep] == 0).all()
    at = slots[keep].long()
    few = [t[keep] if t.shape[0] == B and t is not s["A"] else t for t in first]
    S1, W1 = S0[at].clone(), W0[at].clone()
    assert torch.equal(y[keep], linrec.scan_step(*few, S1, **dict(layer, z=s["z"][keep])))
    assert torch.equal(v[keep], linrec.conv_step(c["x"][keep], c["w"], c["bias"], W1))
    assert torch.equal(S[at], S1) and torch.equal(W[at], W1)
    assert torch.equal(S[3], S0[3]) and torch.equal(W[3], W0[3])


def test_empty_pieces():
    s, grad = scan_inputs(2, 5, 16, 16)
    first = [s["x"][:, :0], s["dt"][:, :0], s["A"], s["B"][:, :, :0], s["C"][:, :, :0]]
    layer = dict(D=s["D"], z=s["z"][:, :0], dt_bias=s["dt_bias"])
    y, h, saved = linrec.scan_fwd(*first, s["h_in"], save=True, **layer)
    r = linrec.scan_bwd(*first, saved, grad["dy"][:, :0], grad["dh_out"], **layer)
    assert y.shape == (2, 0, 16) and torch.equal(h, s["h_in"]) and torch.equal(r.dh_in, grad["dh_out"])
    for t in (r.dA, r.dD, r.ddt_bias):
        assert (t == 0).all()
    assert linrec.scan_step(*first, h, **layer).shape == (2, 0, 16)
    c = conv_inputs(2, 5, 16, 4, BF)
    y, st = linrec.conv_fwd(c["x"][:, :0], c["w"], c["bias"], c["state"])
    dx, dw, db, ds = linrec.conv_bwd(c["x"][:, :0], c["w"], c["bias"], c["state"], c["dy"][:, :0], c["dstate"])
    assert torch.equal(st, c["state"]) and torch.equal(ds, c["dstate"]) and (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_hidden_steps_leave_the_state(dtype):
    """A raw step of -inf, or of the type's lowest value, is a step of 0: the token changes
    no state and gets no gradient through its step; its output is that of the state before."""
    B, T, C, N = 2, 45, 24, 16
    s, grad = scan_inputs(B, T, C, N, 1, dtype, seed=14)
    hidden = torch.zeros(T, dtype=torch.bool)
    hidden[[0, 7, 8, 31, 32, 44]] = True
    s["dt"][0, hidden.to(DEV)] = float("-inf")
    s["dt"][1, hidden.to(DEV)] = torch.finfo(dtype).min
    got = run(s, grad)
    check(s, grad, got, B, T, C)
    assert (got["ddt"][:, hidden.to(DEV)] == 0).all()
    few = dict(s, **{k: s[k][:, ~hidden.to(DEV)] for k in ("x", "dt", "z")}, **{k: s[k][:, :, ~hidden.to(DEV)] for k in ("B", "C")})
    few_y, few_h, _ = linrec.scan_fwd(*(few[k] for k in ("x", "dt", "A", "B", "C")), few["h_in"],
                                      **{k: few[k] for k in ("D", "z", "dt_bias")})
    assert torch.equal(few_y, got["y"][:, ~hidden.to(DEV)]) and torch.equal(few_h, got["h_out"])


def test_values_that_are_not_finite_stay_with_their_channel():
    """An infinite or NaN input spoils its own channel from its token on, and the gradients
    that sum over it; other channels and sequences, and the tokens before, keep their values."""
    B, T, C, N = 2, 70, 24, 16
    s, grad = scan_inputs(B, T, C, N, 1, BF, seed=15)
    clean = run(s, grad)
    c = conv_inputs(B, T, C, 4, BF, seed=15)
    cy, cs = linrec.conv_fwd(c["x"], c["w"], c["bias"], c["state"])
    cg = linrec.conv_bwd(c["x"], c["w"], c["bias"], c["state"], c["dy"], c["dstate"])
    for bad in (float("inf"), float("nan")):
        x = s["x"].clone()
        x[0, 40, 5] = bad
        got = run(dict(s, x=x), grad)
        rest = [k for k in range(C) if k != 5]
        for k in ("y", "dx", "ddt", "dz"):
            assert torch.equal(got[k][1], clean[k][1]) and torch.equal(got[k][0][:, rest], clean[k][0][:, rest]), k
        assert torch.equal(got["y"][0, :40], clean["y"][0, :40]) and not torch.isfinite(got["y"][0, 41:, 5]).any()
        for k in ("dA", "dD", "ddt_bias"):
            assert torch.equal(got[k][rest], clean[k][rest]), k
        assert torch.equal(got["dB"][1], clean["dB"][1]) and torch.equal(got["h_out"][0][rest], clean["h_out"][0][rest])
        x = c["x"].clone()
        x[0, T - 1, 5] = bad          # the last one: nothing behind it
        y, st = linrec.conv_fwd(x, c["w"], c["bias"], c["state"])
        dx, dw, db, ds = linrec.conv_bwd(x, c["w"], c["bias"], c["state"], c["dy"], c["dstate"])
        assert torch.equal(y[0, :T - 1], cy[0, :T - 1]) and torch.equal(y[1], cy[1]) and torch.equal(y[0][:, rest], cy[0][:, rest])
        assert torch.equal(dx[0, :T - 4], cg[0][0, :T - 4]) and torch.equal(dx[0][:, rest], cg[0][0][:, rest])
        assert torch.equal(dx[1], cg[0][1]) and torch.equal(dw[rest], cg[1][rest]) and torch.equal(ds, cg[3])


def test_broadcast_inputs():
    """One sequence's inputs for the whole batch, one projection for all groups: their gradients come entry by entry."""
    B, T, C, N, G = 3, 40, 32, 16, 2
    s, grad = scan_inputs(B, T, C, N, G, F32, seed=8)
    s["x"], s["dt"] = (s[k][:1].expand(B, -1, -1) for k in ("x", "dt"))
    s["B"] = s["B"][:, :1].expand(-1, G, -1, -1)
    check(s, grad, run(s, grad), B, T, C)
    c = conv_inputs(B, T, C, 4, F32, seed=8)
    x = c["x"][:1].expand(B, -1, -1)
    y, _ = linrec.conv_fwd(x, c["w"], c["bias"], c["state"])
    y1, _ = linrec.conv_fwd(x.contiguous(), c["w"], c["bias"], c["state"])
    assert torch.equal(y, y1)


def test_far_apart_sequences():
    """Offsets past 2^31 elements."""
    T, C, N = 40, 64, 16
    far = (1 << 31) + 64
    store = torch.zeros(far + T * C, dtype=BF, device=DEV)
    s, grad = scan_inputs(2, T, C, N, seed=6)
    want = run(s, grad)
    wide = lambda: store.as_strided((2, T, C), (far, C, 1))  # noqa: E731
    for k in ("x", "dt", "z"):
        view = wide()
        view.copy_(s[k])
        got = run(dict(s, **{k: view}), grad)
        for name in want:
            assert torch.equal(got[name], want[name]), (k, name)
    y = wide()
    first = [s[k] for k in ("x", "dt", "A", "B", "C")]
    linrec.scan_fwd(*first, s["h_in"], y=y, **{k: s[k] for k in ("D", "z", "dt_bias")})
    assert torch.equal(y, want["y"])
    c = conv_inputs(2, T, C, 4, BF, seed=6)
    view = wide()
    view.copy_(c["x"])
    assert torch.equal(linrec.conv_fwd(view, c["w"], c["bias"], c["state"])[0], linrec.conv_fwd(c["x"], c["w"], c["bias"], c["state"])[0])
    a = linrec.conv_bwd(view, c["w"], c["bias"], c["state"], c["dy"], c["dstate"])
    for p, q in zip(a, linrec.conv_bwd(c["x"], c["w"], c["bias"], c["state"], c["dy"], c["dstate"])):
        assert torch.equal(p, q)


def test_gradients_by_differences():
    """<dy, y> + <dh_out, h_out> in fp32 moves as its gradients say: central
    differences along a random direction.  The loss' curvature leaves a relative
    error of eps^2 times third derivatives, its rounding about 300 u |loss terms| / eps."""
    B, T, C, N = 2, 70, 24, 16
    s, grad = scan_inputs(B, T, C, N, 1, F32, seed=12)
    r = run(s, grad)
    g = gen(3)

    def loss(v):
        first = [v[k] for k in ("x", "dt", "A", "B", "C")]
        y, h, _ = linrec.scan_fwd(*first, v["h_in"], D=v["D"], z=v["z"], dt_bias=v["dt_bias"])
        return (y.double() * grad["dy"].double()).sum() + (h.double() * grad["dh_out"].double()).sum()

    names = dict(x="dx", dt="ddt", A="dA", B="dB", C="dC", D="dD", z="dz", dt_bias="ddt_bias", h_in="dh_in")
    eps = 2.0 ** -7
    for k, dk in names.items():
        way = (torch.randn(s[k].shape, generator=g) / s[k].numel() ** 0.5).to(DEV)
        up, down = (loss(dict(s, **{k: s[k] + sign * eps * way})) for sign in (1, -1))
        slope = (r[dk].double() * way.double()).sum()
        scale = (r[dk].double().norm() * way.double().norm())
        assert abs((up - down) / (2 * eps) - slope) <= 2e-3 * scale, k
