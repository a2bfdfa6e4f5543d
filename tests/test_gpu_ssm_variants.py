"""The kernels that the causal convolution's and the scan's calls choose between (long
runs, types, taps, numbers of states, token steps with and without each option), and
how parameters' gradients are added up over workgroups."""
import pytest
import torch

import ssm_reference as ref
from state_passing_amd import linrec
from test_gpu_ssm import BF, DEV, F32, U, check, close, conv_inputs, gen, half_step, scan_inputs
from test_gpu_ssm import run as scan_run

pytestmark = pytest.mark.gpu


def whole(g, most, *shape):
    """Whole numbers 0 .. most in fp32 on the GPU."""
    return torch.randint(0, most + 1, shape, generator=g).float().to(DEV)


def test_convolution_sums_over_workgroups_are_exact():
    """dw and dbias of whole numbers: a workgroup's 1024 tokens add up to less than 2^24, exactly, so what
    comes is the exact sum over the 128 workgroups, rounded once (added in fp32 they would round at 2^24)."""
    g, T, C, K = torch.Generator().manual_seed(1), 131072, 8, 4
    d = linrec._CONV(1, T, C, K, 0, linrec.F32, linrec.F32)
    assert linrec._lib().linrec_conv_bwd_workspace_bytes(d) == 4 * ((K - 1) * C + 128 * (K + 1) * C)
    x, dy, w = whole(g, 1, 1, T, C), whole(g, 2 ** 14 - 1, 1, T, C), torch.randn(C, K, generator=g).to(DEV)
    _, dw, dbias, _ = linrec.conv_bwd(x, w, torch.zeros(C, device=DEV), None, dy, act=None)
    x, dy = x[0].cpu().double(), dy[0].cpu().double()
    want = torch.stack([(dy[K - 1 - k:] * x[:T - (K - 1 - k)]).sum(0) for k in range(K)], 1)
    assert want.min() > 2 ** 25
    assert torch.equal(dw.cpu(), want.float()) and torch.equal(dbias.cpu(), dy.sum(0).float())


def test_scan_sums_over_segments_are_exact():
    """dD and ddt_bias likewise: gates of exp(-1000) = 0 leave ddt = x dy (c and b pick one state), whole numbers
    whose sum over a segment's 128 tokens is exact; 256 segments."""
    g, T, C, N = torch.Generator().manual_seed(2), 32768, 64, 16
    d = linrec._SCAN(1, T, C, N, 1, 0, linrec.F32, linrec.F32)
    assert linrec._lib().linrec_scan_fwd_workspace_bytes(d) == 4 * 256 * C * (N + 1)
    x, dy = whole(g, 1, 1, T, C), whole(g, 2 ** 17 - 1, 1, T, C)
    one = torch.zeros(1, 1, T, N, device=DEV)
    one[..., 3] = 1
    A, ones = torch.full((C, N), -1000.0, device=DEV), torch.ones(C, device=DEV)
    first = (x, torch.zeros_like(x), A, one, one)
    rest = dict(D=ones, dt_bias=ones, softplus=False)
    r = linrec.scan_bwd(*first, linrec.scan_fwd(*first, save=True, **rest)[2], dy, **rest)
    want = (x[0].cpu().double() * dy[0].cpu().double()).sum(0)
    assert want.min() > 2 ** 29
    assert torch.equal(r.dD.cpu(), want.float()) and torch.equal(r.ddt_bias.cpu(), want.float())
    assert (r.dA == 0).all()


# ----------------------------------------------------------------- convolution

TYPES = [(BF, None), (BF, F32), (F32, None)]


def conv64(x, w, bias, state, act, n, dy, dstate):
    """The definition in 64 bits on the GPU: (name, value, sum of the terms' absolute values)."""
    x, w, bias, state, dy, dstate = (t.double() for t in (x, w, bias, state, dy, dstate))
    B, T, C = x.shape
    K = w.shape[1]
    live = (torch.arange(T, device=DEV) < n[:, None])[..., None]
    full = torch.cat([state, x], 1)
    p, m = bias.expand(B, T, C).clone(), bias.abs().expand(B, T, C).clone()
    for k in range(K):
        p += w[:, k] * full[:, k:k + T]
        m += (w[:, k] * full[:, k:k + T]).abs()
    s = 1 / (1 + torch.exp(-p))
    yield "y", torch.where(live, p * s if act else p, 0.0), torch.where(live, 1.1 * m if act else m, 0.0)   # silu's slope: at most 1.1
    d = torch.where(live, dy * (s + p * s * (1 - s)) if act else dy, 0.0)
    dm = torch.where(live, dy.abs() * (s * (1 + p.abs()) + m / 2) if act else dy.abs(), 0.0)                # and its own: 1/2
    del p, m, s
    last = (n[:, None] + torch.arange(K - 1, device=DEV))[..., None].expand(B, K - 1, C)
    yield "state_out", full.gather(1, last), torch.zeros_like(state)
    g, gm = torch.zeros_like(full), torch.zeros_like(full)
    g.scatter_(1, last, dstate)
    gm.scatter_(1, last, dstate.abs())
    dw, dwm = torch.zeros_like(w), torch.zeros_like(w)
    for k in range(K):
        g[:, k:k + T] += w[:, k] * d
        gm[:, k:k + T] += w[:, k].abs() * dm
        dw[:, k], dwm[:, k] = (d * full[:, k:k + T]).sum((0, 1)), (dm * full[:, k:k + T].abs()).sum((0, 1))
    yield "dx", torch.where(live, g[:, K - 1:], 0.0), gm[:, K - 1:]
    yield "dstate_in", g[:, :K - 1], gm[:, :K - 1]
    yield "dw", dw, dwm
    yield "dbias", d.sum((0, 1)), dm.sum((0, 1))


def conv_run(B, T, C, K):
    """Tokens a lane of the backward, from its workspace's size."""
    vecs = -(-C // 4)
    shift = min(6, (vecs - 1).bit_length())
    words = linrec._lib().linrec_conv_bwd_workspace_bytes(linrec._CONV(B, T, C, K, 0, linrec.F32, linrec.F32)) // 4
    groups = (words - B * (K - 1) * C) // (B * (K + 1) * C)
    return next(run for run in (64, 8) if groups == -(-T // (run * (256 >> shift))))


@pytest.mark.parametrize("act", ["silu", None])
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("dtype,out", TYPES)
@pytest.mark.parametrize("B,T,C,run", [(5, 3303, 2050, 64), (3, 300, 22, 8)], ids=["long", "short"])
def test_every_convolution(B, T, C, run, dtype, out, K, act):
    """Every kernel of the convolution's pieces.  Tolerances in u = 2^-24 of the terms' absolute values: 16 for a
    value (K + 1 sums and products, an exponential, a reciprocal, three products); a parameter's gradient adds a
    lane's `run` terms in fp32, and is rounded once a workgroup (the sums over both are in 64 bits)."""
    assert conv_run(B, T, C, K) == run
    # the forward's runs of 32, from 131072 runs on
    lanes = lambda v: B * -(-(-(-C // v)) // 64) * 64  # noqa: E731
    assert (lanes(4 if dtype is F32 else 8) * -(-T // 32) >= 131072) == (run == 64)
    g = torch.Generator(device=DEV).manual_seed(K)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    pad = -(-C // 8) * 8
    x, dy = (r(B, T, pad).to(dtype)[..., :C] for _ in range(2))
    w, bias, state, dstate = r(C, K) * 0.6, r(C) * 0.2, r(B, K - 1, C), r(B, K - 1, C)
    n = torch.tensor([T, T - 1, 2, 0, T // 2][:B], device=DEV)
    rest = dict(act=act, n_new=n.int(), out_dtype=out)
    y, end = linrec.conv_fwd(x, w, bias, state, **rest)
    dx, dw, dbias, dstart = linrec.conv_bwd(x, w, bias, state, dy, dstate, **rest)
    got = dict(y=y, state_out=end, dx=dx, dstate_in=dstart, dw=dw, dbias=dbias)
    terms = dict(y=16, dx=16, dstate_in=16, state_out=0, dw=18 + run, dbias=18 + run)
    for name, want, most in conv64(x, w, bias, state, act, n, dy, dstate):
        t = got[name]
        tol = terms[name] * U * most * (1 + 2.0 ** -7) + half_step(t) * want.abs() + 1e-37
        off = (t.double() - want).abs()
        assert torch.isfinite(t).all() and (off <= tol).all(), (name, (off / tol).max().item())


@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("act", ["silu", None])
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("dtype,out", TYPES)
def test_every_convolution_step(dtype, out, K, act, bias):
    B, T, C = 4, 3, 37
    s = conv_inputs(B, T, C, K, dtype, seed=K, bias=bias)
    slots = torch.tensor([5, 0, 3, 1], dtype=torch.int32, device=DEV)
    pool = torch.randn(6, K - 1, C, generator=gen(2)).to(DEV)
    before = pool.clone()
    y = linrec.conv_step(s["x"], s["w"], s["bias"], pool, act=act, slots=slots, out_dtype=out)
    assert y.dtype == (out or dtype)
    plain = dict(x=s["x"], w=s["w"], bias=s["bias"], state=before[slots.long()], act=act)
    want, most = ref.conv(**plain), ref.conv(**plain, absolute=True)
    close("y", y, want["y"], most["y"], 16)
    assert torch.equal(pool[slots.long()].cpu().double(), want["state_out"])
    assert torch.equal(pool[[2, 4]], before[[2, 4]])


# ----------------------------------------------------------------- scan

FORMS = [dict(), dict(z=False), dict(softplus=False), dict(D=False, bias=False), dict(z=False, D=False, bias=False, softplus=False)]


@pytest.mark.parametrize("form", FORMS, ids=["all", "no gate", "plain step", "no D, bias", "none"])
@pytest.mark.parametrize("N,G", [(8, 1), (16, 2), (32, 1), (64, 2)])
@pytest.mark.parametrize("dtype,out", TYPES)
def test_every_scan_step(dtype, out, N, G, form):
    B, T, C = 4, 2, 80 if G == 2 else 75
    s, _ = scan_inputs(B, T, C, N, G, dtype, seed=N, state=False, **form)
    slots = torch.tensor([5, 0, 3, 1], dtype=torch.int32, device=DEV)
    pool = torch.randn(6, C, N, generator=gen(2)).to(DEV)
    before = pool.clone()
    y = linrec.scan_step(*(s[k] for k in ("x", "dt", "A", "B", "C")), pool, D=s["D"], z=s["z"], dt_bias=s["dt_bias"],
                         softplus=s["softplus"], slots=slots, out_dtype=out)
    assert y.dtype == (out or dtype)
    s["h_in"] = before[slots.long()]
    want, most = ref.scan(**s), ref.scan(**s, absolute=True)
    close("y", y, want["y"], most["y"], 5 * T + 300)
    close("S", pool[slots.long()], want["h_out"], most["h_out"], 5 * T + 300)
    assert torch.equal(pool[[2, 4]], before[[2, 4]])


@pytest.mark.parametrize("N", [8, 16, 32, 64])
@pytest.mark.parametrize("dtype,out", TYPES)
def test_every_gated_scan(dtype, out, N):
    """Its backward is a kernel of its own, of every number of states and type; a segmented piece, a group's end."""
    B, T, C, n = 2, 170, 520 // N + 11, [170, 97]
    s, grad = scan_inputs(B, T, C, N, dtype=dtype, seed=N)
    got = scan_run(s, grad, torch.tensor(n, dtype=torch.int32, device=DEV), out)
    check(s, grad, got, B, T, C, n)


@pytest.mark.parametrize("N", [8, 16, 32, 64])
def test_scan_walks_that_are_not_split(N):
    """With 320 workgroups from the batch alone a piece is walked whole: three of the sequences against 64 bits."""
    B, T, C = 330, 100, 16
    words = linrec._lib().linrec_scan_fwd_workspace_bytes(linrec._SCAN(B, T, C, N, 1, 1, linrec.BF16, linrec.BF16))
    assert words == 0
    s, grad = scan_inputs(B, T, C, N, seed=N + 1)
    n = [T - b % 7 for b in range(B)]
    got = scan_run(s, grad, torch.tensor(n, dtype=torch.int32, device=DEV))
    for b in (0, 160, B - 1):
        one = lambda v: {k: t[b:b + 1] if isinstance(t, torch.Tensor) and t.shape[0] == B else t for k, t in v.items()}  # noqa: E731
        mine = {k: t for k, t in one(got).items() if k not in ("dA", "dD", "ddt_bias")}
        check(one(s), one(grad), mine, 1, T, C, n[b:b + 1])


# ----------------------------------------------------------------- ends of the ranges

def first_of(s):
    return [s[k] for k in ("x", "dt", "A", "B", "C")]


def test_the_most_sequences():
    """32767 of them: three equal the calls of their own, forward, backward and as tokens of a pool."""
    B, T, C, N = 32767, 3, 8, 8
    at = torch.tensor([0, 12345, B - 1], device=DEV)
    s, grad = scan_inputs(B, T, C, N, seed=1)
    some = lambda v: {k: t[at].contiguous() if isinstance(t, torch.Tensor) and t.shape[0] == B else t for k, t in v.items()}  # noqa: E731
    n = torch.randint(0, T + 1, (B,), generator=gen(4), dtype=torch.int32).to(DEV)
    got, want = scan_run(s, grad, n), scan_run(some(s), some(grad), n[at])
    for k, t in want.items():
        if k not in ("dA", "dD", "ddt_bias"):
            assert torch.equal(got[k][at], t), k
    rest = {k: s[k] for k in ("D", "dt_bias")}
    S, slots = torch.randn(B, C, N, generator=gen(5)).to(DEV), torch.randperm(B, generator=gen(6)).to(torch.int32).to(DEV)
    mine = S[slots[at].long()].clone()
    y = linrec.scan_step(*first_of(s), S, z=s["z"], slots=slots, **rest)
    few = some(s)
    assert torch.equal(y[at], linrec.scan_step(*first_of(few), mine, z=few["z"], **rest)) and torch.equal(S[slots[at].long()], mine)
    c = conv_inputs(B, T, C, 4, BF, seed=2)
    few = some(c)
    for a, b in zip(linrec.conv_fwd(c["x"], c["w"], c["bias"], c["state"], n_new=n),
                    linrec.conv_fwd(few["x"], c["w"], c["bias"], few["state"], n_new=n[at])):
        assert torch.equal(a[at], b)
    a = linrec.conv_bwd(c["x"], c["w"], c["bias"], c["state"], c["dy"], c["dstate"], n_new=n)
    b = linrec.conv_bwd(few["x"], c["w"], c["bias"], few["state"], few["dy"], few["dstate"], n_new=n[at])
    assert torch.equal(a[0][at], b[0]) and torch.equal(a[3][at], b[3])
    W = torch.randn(B, 3, C, generator=gen(7)).to(DEV)
    mine = W[slots[at].long()].clone()
    y = linrec.conv_step(c["x"], c["w"], c["bias"], W, slots=slots)
    assert torch.equal(y[at], linrec.conv_step(few["x"], c["w"], c["bias"], mine)) and torch.equal(W[slots[at].long()], mine)


@pytest.mark.parametrize("C,G,N", [(1 << 20, 1, 8), (65535 * 8, 65535, 8), (1 << 20, 2, 64)])
def test_the_most_channels_and_groups(C, G, N):
    """The last channels (of the last group) equal a call of their own."""
    T, few = 2, 8
    s, grad = scan_inputs(1, T, C, N, G, seed=1)

    def last(v):
        out = {}
        for k, t in v.items():
            if k in ("B", "C"):
                t = t[:, -1:]
            elif k in ("A", "D", "dt_bias"):
                t = t[-few:]
            elif k in ("h_in", "dh_out"):
                t = t[:, -few:].contiguous()
            elif isinstance(t, torch.Tensor):
                t = t[..., -few:]
            out[k] = t
        return out

    got, want = scan_run(s, grad), scan_run(last(s), last(grad))
    for k in ("y", "dx", "ddt", "dz"):
        assert torch.equal(got[k][..., -few:], want[k]), k
    for k in ("h_out", "dh_in"):
        assert torch.equal(got[k][:, -few:], want[k]), k
    for k in ("dA", "dD", "ddt_bias"):
        assert torch.equal(got[k][-few:], want[k]), k
    if C // G == few:
        assert torch.equal(got["dB"][:, -1:], want["dB"]) and torch.equal(got["dC"][:, -1:], want["dC"])
    if G > 2:
        return
    c = conv_inputs(1, T, C, 4, BF, seed=2)
    part = {k: t[-few:] if k in ("w", "bias") else t[..., -few:].contiguous() for k, t in c.items()}
    order = ("x", "w", "bias", "state")
    assert torch.equal(linrec.conv_fwd(*(c[k] for k in order))[0][..., -few:], linrec.conv_fwd(*(part[k] for k in order))[0])
    order += ("dy", "dstate")
    a, b = linrec.conv_bwd(*(c[k] for k in order)), linrec.conv_bwd(*(part[k] for k in order))
    assert torch.equal(a[0][..., -few:], b[0]) and torch.equal(a[1][-few:], b[1]) and torch.equal(a[2][-few:], b[2])
