"""GPU tests of the elementwise gated recurrence (linrec_diag_fwd / _bwd)
against the token-by-token recurrence in 64 bits on the CPU, and of its
gradients against differences.

Tolerances.  One token's step rounds a few times: the gate (exp2 of a rounded
product, below 2^-21 for the gates drawn, |g| <= 2, and for g <= -2 the gate is
small), the product and the sum; 2^-20 of the largest value per step covers
them.  An error lives as long as the state does, M = 1 / (1 - a_max) tokens at
most (or the piece), so |error| <= 2^-20 M max|value|.  Outputs in bf16 add
half a step, 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

from state_passing_amd import linrec

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def reference(g, x, h_in, dh, dh_out, mix):
    """(h, h_out, dg, dx, dh_in, G) in 64 bits."""
    g, x, h = g.double(), x.double(), h_in.double()
    a = g.exp()
    w = -torch.expm1(g) if mix else torch.ones_like(g)
    hs, prev = torch.zeros_like(x), torch.zeros_like(x)
    for t in range(x.shape[1]):
        prev[:, t] = h
        h = torch.where(a[:, t] == 0, 0.0, a[:, t] * h) + w[:, t] * x[:, t]
        hs[:, t] = h
    R, G = dh_out.double(), torch.zeros_like(x)
    for t in range(x.shape[1] - 1, -1, -1):
        G[:, t] = dh[:, t].double() + R
        R = a[:, t] * G[:, t]
    dg = a * G * (prev - x if mix else prev)
    return hs, h, dg, w * G, R, G


def draw(seed, B, T, C, dtype, slow=8.0):
    """Gates of channels that remember from 2 to 2^slow tokens."""
    gen = torch.Generator().manual_seed(seed)
    rate = torch.exp2(-1 - (slow - 1) * torch.rand(C, generator=gen))
    g = -(rate * (0.5 + torch.rand(B, T, C, generator=gen)))
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return g.to(dtype), r(B, T, C).to(dtype), r(B, C), r(B, T, C).to(dtype), r(B, C)


def compare(name, got, ref, lim):
    got = got.double().cpu()
    half = 2.0 ** -8 * ref.abs() if name in BF_OUT else 0.0
    bad = (got - ref).abs() - half > lim
    assert not bad.any() and not torch.isnan(got).any(), (name, float((got - ref).abs().max()), float(lim), bad.nonzero()[:3])


BF_OUT = set()


def check(g, x, h_in, dh, dh_out, mix, out=None, view=lambda t: t, null=False):
    ref = reference(g, x, torch.zeros_like(h_in) if null else h_in, dh, torch.zeros_like(dh_out) if null else dh_out, mix)
    form = "mix" if mix else "plain"
    d = lambda t: view(t.to(DEV))  # noqa: E731
    hin, dho = (None, None) if null else (h_in.to(DEV), dh_out.to(DEV))
    h, h_out, st = linrec.diag_fwd(d(g), d(x), hin, form=form, out_dtype=out)
    dg, dx, dh_in = linrec.diag_bwd(d(g), d(x), st, d(dh), dho, form=form, out_dtype=out)
    torch.cuda.synchronize()
    bf = h.dtype == BF
    BF_OUT.clear()
    if bf:
        BF_OUT.update(("h", "dg", "dx"))
    T = g.shape[1]
    a_max = float(g.double().exp().max()) if T else 0.0
    M = min(T, 1 / (1 - a_max)) if a_max < 1 else T
    eps = 2.0 ** -20 * max(M, 1)
    hm = max(float(ref[0].abs().max()), float(h_in.abs().max()), float(x.double().abs().max()))
    gm = max(float(ref[5].abs().max()), float(dh_out.abs().max()))
    compare("h", h, ref[0], eps * hm)
    compare("h_out", h_out, ref[1], eps * hm)
    compare("dx", dx, ref[3], eps * gm)
    compare("dh_in", dh_in, ref[4], eps * gm)
    compare("dg", dg, ref[2], 4 * eps * gm * hm)
    return h, h_out, dg, dx, dh_in


CASES = [
    # B, T, C, dtype, mix, out
    (3, 1, 8, BF, True, None), (2, 1, 1000, F32, False, None), (1, 5, 64, BF, False, None),
    (2, 8, 513 * 8, BF, True, None), (1, 9, 24, F32, True, None), (2, 63, 64, BF, True, F32),
    (1, 255, 72, BF, False, None), (2, 256, 128, F32, True, None), (3, 257, 40, BF, True, None),
    (1, 512, 136, BF, False, F32), (1, 1000, 32, F32, False, None), (2, 4099, 96, BF, True, None),
    (1, 5000, 200, F32, True, None), (40, 300, 8, BF, False, None),
    # many chains of segments at once, their lengths multiples of the look-back window
    (2, 4096, 1024, F32, False, None), (6, 2304, 512, BF, True, None),
]


@pytest.mark.parametrize("case", CASES, ids=[f"{c[0]}x{c[1]}x{c[2]}" for c in CASES])
def test_forward_and_backward(case):
    B, T, C, dtype, mix, out = case
    print("case", case, flush=True)
    check(*draw(T, B, T, C, dtype), mix, out)


def test_no_carries_given():
    check(*draw(3, 2, 300, 64, BF), True, null=True)
    check(*draw(3, 2, 4, 64, BF), False, null=True)


@pytest.mark.parametrize("C", [1, 7, 13, 67])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_channel_counts_that_end_inside_a_vector(C, dtype):
    """Rows padded to 16 bytes; what lies in the padding is neither read (NaN) nor written."""
    N = 8 if dtype == BF else 4
    pad = -C % N + N
    g, x, h_in, dh, dh_out = draw(C, 2, 300, C, dtype)
    wide = lambda t: torch.nn.functional.pad(t, (0, pad), value=float("nan"))[..., :C]  # noqa: E731
    check(g, x, h_in, dh, dh_out, True, view=wide)
    out = torch.full((2, 300, C + pad), 5.0, dtype=dtype, device=DEV)
    h, _, st = linrec.diag_fwd(wide(g.to(DEV)), wide(x.to(DEV)), form="mix", h=out[..., :C])
    assert (out[..., C:] == 5).all()
    outs = [torch.full((2, 300, C + pad), 5.0, dtype=dtype, device=DEV) for _ in range(2)]
    linrec.diag_bwd(wide(g.to(DEV)), wide(x.to(DEV)), st, wide(dh.to(DEV)), form="mix", dg=outs[0][..., :C], dx=outs[1][..., :C])
    assert all((o[..., C:] == 5).all() for o in outs)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strides_and_aliases(dtype):
    """Token-major memory ([T,B,C]); gradients written over the inputs."""
    B, T, C = 3, 600, 64
    g, x, h_in, dh, dh_out = draw(11, B, T, C, dtype)
    tb = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    want = check(g, x, h_in, dh, dh_out, True, view=tb)
    gd, xd, dd, h, r = (t.to(DEV) for t in (g, x, dh, h_in, dh_out))
    _, _, st = linrec.diag_fwd(gd, xd, h, form="mix", h_out=h)
    assert torch.equal(h, want[1])
    linrec.diag_bwd(gd, xd, st, dd, r, form="mix", dg=gd, dx=dd, dh_in=r)
    assert torch.equal(gd, want[2]) and torch.equal(dd, want[3]) and torch.equal(r, want[4])


@pytest.mark.parametrize("mix", [False, True])
def test_gates_at_the_ends(mix):
    """g = -inf forgets everything before the token; g = 0 keeps all; tiny |g|."""
    g, x, h_in, dh, dh_out = draw(12, 2, 700, 16, F32)
    g[:, 100] = -torch.inf
    g[0, 300:400, :8] = 0.0
    g[1, :, 8:] = -1e-7
    g[1, 500] = -200.0
    ref = reference(g, x, h_in, dh, dh_out, mix)
    form = "mix" if mix else "plain"
    h, h_out, st = linrec.diag_fwd(g.to(DEV), x.to(DEV), h_in.to(DEV), form=form)
    dg, dx, dh_in = linrec.diag_bwd(g.to(DEV), x.to(DEV), st, dh.to(DEV), dh_out.to(DEV), form=form)
    BF_OUT.clear()
    eps = 2.0 ** -20 * 700
    hm, gm = float(ref[0].abs().max()), float(ref[5].abs().max())
    for n, t, r, lim in (("h", h, ref[0], hm), ("h_out", h_out, ref[1], hm), ("dg", dg, ref[2], 4 * gm * hm),
                         ("dx", dx, ref[3], gm), ("dh_in", dh_in, ref[4], gm)):
        compare(n, t, r, eps * lim)
    if mix:   # 1 - a of the tiny gates keeps its relative precision
        # dx = (1 - a) G: G is off by eps max|G| whatever its own size (a sum that may
        # cancel), so the bound on dx / (1 - a) is absolute
        w = -np.expm1(float(g[1, 0, 8]))
        got, G = dx.double().cpu()[1, :100, 8:] / w, ref[5][1, :100, 8:]
        assert ((got - G).abs() <= eps * gm).all()


def test_pieces_equal_one_pass():
    """Odd pieces chained through h_out -> h_in and dh_in -> dh_out."""
    B, T, C = 2, 1900, 48
    g, x, h_in, dh, dh_out = draw(13, B, T, C, F32)
    want = check(g, x, h_in, dh, dh_out, True)
    gd, xd, dd = (t.to(DEV) for t in (g, x, dh))
    cuts, h, sts, hs = [0, 1, 8, 300, 557, 557, 1900], h_in.to(DEV), [], []
    for i, j in zip(cuts, cuts[1:]):
        o, h, st = linrec.diag_fwd(gd[:, i:j], xd[:, i:j], h, form="mix")
        hs.append(o)
        sts.append(st)
    r, gs, xs = dh_out.to(DEV), [], []
    for n in reversed(range(len(sts))):
        sl = slice(cuts[n], cuts[n + 1])
        a, b, r = linrec.diag_bwd(gd[:, sl], xd[:, sl], sts[n], dd[:, sl], r, form="mix")
        gs.insert(0, a)
        xs.insert(0, b)
    got = (torch.cat(hs, 1), h, torch.cat(gs, 1), torch.cat(xs, 1), r)
    eps = 2.0 ** -18 * 256        # twice the bound of either
    for a, b in zip(got, want):
        assert float((a - b).abs().max()) <= eps * max(1.0, float(b.abs().max()) ** 2)


def test_gradients_against_differences():
    """Central differences of the GPU's own forward, in fp32 with a step of 2^-6:
    the loss is a sum over 37 * 8 terms, each rounded to 2^-24 of values of a few
    units, over a step of 2^-5: noise below 2^-24 * 300 * 8 * 32 = 5e-3; the
    third-derivative term is below step^2 * |value| = 3e-3."""
    B, T, C = 1, 37, 8
    g, x, h_in, dh, dh_out = draw(14, B, T, C, F32, slow=4.0)
    run = lambda g, x, h: linrec.diag_fwd(g.to(DEV), x.to(DEV), h.to(DEV), form="mix")  # noqa: E731

    def loss(g, x, h):
        o, e, _ = run(g, x, h)
        return float((o.double().cpu() * dh.double()).sum() + (e.double().cpu() * dh_out.double()).sum())

    st = run(g, x, h_in)[2]
    grads = linrec.diag_bwd(g.to(DEV), x.to(DEV), st, dh.to(DEV), dh_out.to(DEV), form="mix")
    e = 2.0 ** -6
    rng = np.random.default_rng(0)
    for which, t in ((0, g), (1, x), (2, h_in)):
        for _ in range(12):
            at = tuple(int(rng.integers(n)) for n in t.shape)
            p, m = [u.clone() for u in (g, x, h_in)], [u.clone() for u in (g, x, h_in)]
            p[which][at] += e
            m[which][at] -= e
            diff = (loss(*p) - loss(*m)) / (2 * e)
            assert abs(diff - float(grads[which][at])) <= 1.5e-2 + 1e-2 * abs(diff), (which, at)


def test_empty_piece_passes_the_carry():
    z = torch.empty(2, 0, 16, device=DEV)
    h_in = torch.randn(2, 16, device=DEV)
    h, h_out, st = linrec.diag_fwd(z, z, h_in)
    assert torch.equal(h_out, h_in) and h.shape == z.shape
    assert torch.equal(linrec.diag_bwd(z, z, st, z, h_in)[2], h_in)
    assert (linrec.diag_fwd(z, z)[1] == 0).all()


@pytest.mark.parametrize("T", [3, 200, 1500])
def test_replays_and_streams(T):
    """Captured forward and backward with their own workspaces: every replay, with
    eager calls between, equals the eager results bit for bit; so does a call on
    another stream."""
    g, x, h_in, dh, dh_out = (t.to(DEV) for t in draw(15, 2, T, 64, BF))
    h, e, st = linrec.diag_fwd(g, x, h_in, form="mix")
    back = linrec.diag_bwd(g, x, st, dh, dh_out, form="mix")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        h2, e2, st2 = linrec.diag_fwd(g, x, h_in, form="mix")
        back2 = linrec.diag_bwd(g, x, st2, dh, dh_out, form="mix")
    side.synchronize()
    assert torch.equal(h, h2) and torch.equal(e, e2) and all(torch.equal(a, b) for a, b in zip(back, back2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h3, e3, st3 = linrec.diag_fwd(g, x, h_in, form="mix")
        back3 = linrec.diag_bwd(g, x, st3, dh, dh_out, form="mix")
    for _ in range(3):
        for t in (h3, e3, *back3):
            t.zero_()
        linrec.diag_fwd(g.flip(1).contiguous(), x, h_in)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, h3) and torch.equal(e, e3) and all(torch.equal(a, b) for a, b in zip(back, back3))


def test_two_calls_at_once():
    """Calls of many segments on two streams, each with its own workspace, in flight
    together: every result equals that of the call made alone, bit for bit."""
    sets = [[t.to(DEV) for t in draw(20 + i, 2, 5000 - 700 * i, 1024, BF)] for i in range(2)]

    def both(s):
        g, x, h_in, dh, dh_out = s
        h, e, st = linrec.diag_fwd(g, x, h_in, form="mix")
        return (h, e, *linrec.diag_bwd(g, x, st, dh, dh_out, form="mix"))

    want = [both(s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(4):
        got = []
        for s, stream in zip(sets, streams):
            with torch.cuda.stream(stream):
                got.append(both(s))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for w, g in zip(want, got) for a, b in zip(w, g))
