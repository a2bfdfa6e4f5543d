"""Pieces of the selective scan that are split into segments, against the walk
token by token in 64 bits: states that grow, states and gradients that are still
zero, and the most segments that a call makes.

Tolerances come from the walk itself.  Steps are given as they are (no softplus, no
bias), so d is exact, and with u = 2^-24 a token's gate exp2(d A') is off by 2 u and
by 3 u |d A|; where a segment's gates are taken together, the sum of its steps is off
by a rounding a token and its exponential is squared, so with S tokens a segment
(S + 6) u |d A| and 2 u a token bound either way.  Beside the state h runs the sum of
its terms' absolute values M and a bound E on its error,
    M_t = a M + |d x b|,   E_t = a E + ((2 + (S + 6) |d A|) a M + M_t + 3 |d x b|) u
(a fused product and sum, three products of the added term), and the same for the
gradients from behind.  Products of two inexact values add their errors crosswise;
terms in u^2 are covered by 1 part in 64.  Sums over N states or C channels add N u or
C u of their terms; dA's S tokens follow each other in a segment, 256 segments behind
them.
"""
import pytest
import torch

from state_passing_amd import linrec

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
F64 = torch.float64


def segments(B, T, C, N):
    """How many segments a forward of one group makes, from its workspace's size."""
    d = linrec._SCAN(B, T, C, N, 1, 0, linrec.F32, linrec.F32)
    words = linrec._lib().linrec_scan_fwd_workspace_bytes(d) // 4
    return max(words // (B * C * (N + 1)), 1)


def walk(x, d, A, Bm, Cm, h0, dy, g0, S):
    """Values, and bounds on their errors, of one sequence: x, d, dy: [T,C], A: [C,N], Bm, Cm: [T,N], h0, g0: [C,N]."""
    T, C = x.shape
    N = A.shape[1]
    want, err = {}, {}
    h, M, E = h0, h0.abs(), torch.zeros_like(h0)
    kept = []
    gate, loose = torch.exp(d[:, :, None] * A), 2 + (S + 6) * (d[:, :, None] * A).abs()
    y, ey = torch.zeros(T, C, dtype=F64), torch.zeros(T, C, dtype=F64)
    for t in range(T):
        kept.append((h, M, E))
        a, u = gate[t], (d[t] * x[t])[:, None] * Bm[t]
        h, aM = a * h + u, a * M
        M = aM + u.abs()
        E = a * E + (loose[t] * aM + M + 3 * u.abs()) * U
        y[t] = (h * Cm[t]).sum(-1)
        ey[t] = ((E + N * U * M) * Cm[t].abs()).sum(-1)
    kept.append((h, M, E))
    want["y"], err["y"], want["h_out"], err["h_out"] = y, ey, h, E
    for k in ("dx", "ddt"):
        want[k], err[k] = torch.zeros(T, C, dtype=F64), torch.zeros(T, C, dtype=F64)
    for k in ("dB", "dC"):
        want[k], err[k] = torch.zeros(T, N, dtype=F64), torch.zeros(T, N, dtype=F64)
    want["dA"], err["dA"] = torch.zeros_like(A), torch.zeros_like(A)
    g, Mg, Eg = g0, g0.abs(), torch.zeros_like(g0)
    for t in reversed(range(T)):
        a, e, u = gate[t], dy[t][:, None], (d[t] * x[t])[:, None]
        (hb, Mb, Eb), (hn, Mn, En) = kept[t], kept[t + 1]
        up = e * Cm[t]
        g, Mg = g + up, Mg + up.abs()
        Eg = Eg + (Mg + up.abs()) * U
        want["dC"][t], err["dC"][t] = (e * hn).sum(0), (e.abs() * (En + (C + 3) * U * Mn)).sum(0)
        want["dB"][t], err["dB"][t] = (u * g).sum(0), (u.abs() * (Eg + (C + 3) * U * Mg)).sum(0)
        du, edu = (g * Bm[t]).sum(-1), ((Eg + (N + 2) * U * Mg) * Bm[t].abs()).sum(-1)
        want["dx"][t], err["dx"][t] = du * d[t], (edu + U * du.abs()) * d[t].abs()
        g, aM = a * g, a * Mg
        Eg = a * Eg + (loose[t] * aM + aM) * U
        Mg = aM
        q, Mq = g * hb, Mg * Mb
        Eq = Mg * Eb + Eg * Mb + U * Mq
        want["ddt"][t] = (q * A).sum(-1) + du * x[t]
        err["ddt"][t] = ((Eq + (N + 6) * U * Mq) * A.abs()).sum(-1) + (edu + 2 * U * du.abs()) * x[t].abs()
        want["dA"] += q * d[t][:, None]
        err["dA"] += (Eq + (S + 260) * U * Mq) * d[t].abs()[:, None]
    want["dh_in"], err["dh_in"] = g, Eg
    return want, err


def run(x, d, A, Bm, Cm, h0, dy, g0):
    """The same sequence through the library, by the names of walk()."""
    up = lambda t: None if t is None else t.float().to(DEV)  # noqa: E731

    def rows(t):   # that begin at 16 bytes
        return torch.nn.functional.pad(up(t), (0, -t.shape[1] % 4))[None, :, :t.shape[1]]

    first = (rows(x), rows(d), up(A), up(Bm)[None, None], up(Cm)[None, None])
    h0, g0 = (None if t is None else up(t)[None] for t in (h0, g0))
    y, h, saved = linrec.scan_fwd(*first, h0, softplus=False, save=True)
    r = linrec.scan_bwd(*first, saved, rows(dy), g0, softplus=False)
    got = dict(y=y[0], h_out=h[0], dx=r.dx[0], ddt=r.ddt[0], dB=r.dB[0, 0], dC=r.dC[0, 0], dA=r.dA, dh_in=r.dh_in[0])
    torch.cuda.synchronize()
    return {k: t.to("cpu", F64) for k, t in got.items()}


def check(got, want, err):
    for k, w in want.items():
        assert torch.isfinite(got[k]).all(), k
        tol = err[k] * (1 + 1 / 64) + w.abs() * U + 1e-37
        off = (got[k] - w).abs()
        assert (off <= tol).all(), (k, (off / tol).max().item(), (off > tol).nonzero()[0].tolist())


def inputs(T, C, N, seed):
    """In fp32's values."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(F64)  # noqa: E731
    rate = (0.2 + 0.8 * torch.rand(C, N, generator=g)).to(F64)
    return r, rate


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("N,C", [(16, 24), (64, 5), (8, 3)])
def test_a_zero_state_does_not_grow(sign, N, C):
    """Gates above 1 (a positive A, or negative steps), whose product over a segment passes fp32's
    range: states that nothing has entered yet stay zero, and so do gradients from behind."""
    T, S = 300, 64
    assert segments(1, T, C, N) == 5
    r, rate = inputs(T, C, N, N)
    A = (sign * 20 * rate).float().to(F64)
    d = torch.full((T, C), sign * 0.15, dtype=torch.float32).to(F64)          # 0.6 to 3 a token, up to 192 a segment
    x, dy = torch.zeros(T, C, dtype=F64), torch.zeros(T, C, dtype=F64)
    x[-20:], dy[:20] = r(20, C), r(20, C)
    zero = torch.zeros(C, N, dtype=F64)
    args = (x, d, A, r(T, N), r(T, N))
    want, err = walk(*args, zero, dy, zero, S)
    assert all(torch.isfinite(t).all() for t in want.values())
    got = run(*args, None, dy, None)
    check(got, want, err)
    assert (got["y"][:-20] == 0).all() and (got["dx"][20:] == 0).all() and (got["dB"][20:] == 0).all()
    assert (got["h_out"] != 0).all() and (got["dh_in"] != 0).all()


def test_a_small_state_grows_across_a_segment():
    """One segment multiplies a state (a gradient) by more than fp32 holds, and the product fits again."""
    T, C, N, S = 300, 24, 16, 64
    assert segments(1, T, C, N) == 5
    r, rate = inputs(T, C, N, 1)
    A = (14 + rate).float().to(F64)
    d = torch.zeros(T, C, dtype=F64)
    d[64:128] = 0.1                                                            # exp(91) to exp(96) in the second segment
    x, dy = torch.zeros(T, C, dtype=F64), torch.zeros(T, C, dtype=F64)
    h0 = (1e-30 * r(C, N)).float().to(F64)
    d = d.float().to(F64)
    args = (x, d, A, r(T, N), r(T, N))
    # no gradient from behind here, and no state in the other call: their product would pass fp32's range
    zero = torch.zeros(C, N, dtype=F64)
    want, err = walk(*args, h0, dy, zero, S)
    got = run(*args, h0, dy, None)
    check(got, want, err)
    assert (got["h_out"].abs() > 1e3).any()
    want, err = walk(*args, zero, dy, h0, S)
    check(run(*args, None, dy, h0), want, err)


@pytest.mark.parametrize("C,N,T,S,count", [(8, 8, 16377, 64, 256), (136, 8, 12279, 96, 128), (70, 16, 8190, 64, 128), (16, 64, 5000, 64, 79)])
def test_the_most_segments(C, N, T, S, count):
    """As many segments as a call makes (a workgroup each, and two), with states that live for one to ten or
    more segments, so that every segment counts in those behind it."""
    assert segments(1, T, C, N) == count and -(-T // S) == count
    r, rate = inputs(T, C, N, T)
    A = (-2 * 10.0 ** (-1.3 * rate)).float().to(F64)                 # -1.1 to -0.1, a hundredth of it a token
    d = (0.02 * torch.rand(T, C, generator=torch.Generator().manual_seed(3))).to(F64)
    args = (r(T, C), d, A, r(T, N), r(T, N), r(C, N), r(T, C), r(C, N))
    want, err = walk(*args, S)
    check(run(*args), want, err)
