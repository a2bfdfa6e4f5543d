"""A state-space layer as a model runs it: projection, causal convolution, the
projections of the step and of b and c, the scan, the gate and a projection back;
a prompt in pieces of its own lengths, then token after token from pools of
states, eagerly and captured; and a training step whose gradients are checked
against automatic differentiation of the formulas in 64 bits."""
import pytest
import torch

from state_passing_amd import linrec

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
B, M, C, N, K, R = 3, 32, 48, 16, 4, 8   # sequences, model width, channels, states, taps, width of the step's projection
PIECES, TOKENS = (37, 70), 6
T = sum(PIECES) + TOKENS


def layer(dtype=torch.float64, device="cpu"):
    g = torch.Generator().manual_seed(21)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    p = dict(inp=r(M, 2 * C) * M ** -0.5, w=r(C, K) * 0.5, bias=r(C) * 0.1, low=r(C, R + 2 * N) * C ** -0.5, step=r(R, C) * R ** -0.5,
             dt_bias=r(C) * 0.5 - 3.0, A=-torch.arange(1, N + 1) * torch.exp(0.2 * r(C, N)), D=1 + 0.1 * r(C), back=r(C, M) * C ** -0.5)
    return {k: v.to(device, dtype) for k, v in p.items()}


def tokens(n=T):
    return torch.randn(B, n, M, generator=torch.Generator().manual_seed(5), dtype=torch.float64)


def project(p, u):
    """x and z of the layer, then what the scan takes of the convolved x."""
    both = torch.matmul(u, p["inp"])
    return both[..., :C], both[..., C:]


def low(p, x):
    v = torch.matmul(x, p["low"])
    return torch.matmul(v[..., :R], p["step"]), v[..., R:R + N].unsqueeze(1), v[..., R + N:].unsqueeze(1)


def piece(p, u, conv, h, n_new=None, save=False):
    x, z = project(p, u)
    y, conv = linrec.conv_fwd(x, p["w"], p["bias"], conv, n_new=n_new)
    dt, b, c = low(p, y)
    o, h, saved = linrec.scan_fwd(y, dt, p["A"], b, c, h, D=p["D"], z=z, dt_bias=p["dt_bias"], n_new=n_new, save=save)
    return torch.matmul(o, p["back"]), conv, h, (x, z, y, dt, b, c, o, saved)


def token(p, u, conv, h, slots):
    x, z = project(p, u)
    y = linrec.conv_step(x, p["w"], p["bias"], conv, slots=slots)
    dt, b, c = low(p, y)
    return torch.matmul(linrec.scan_step(y, dt, p["A"], b, c, h, D=p["D"], z=z, dt_bias=p["dt_bias"], slots=slots), p["back"])


def plain(p, u):
    """The formulas in torch, differentiable: token by token."""
    n, t = u.shape[0], u.shape[1]
    x, z = project(p, u)
    full = torch.cat([x.new_zeros(n, K - 1, C), x], 1)
    pre = p["bias"] + sum(p["w"][:, k] * full[:, k:k + t] for k in range(K))
    y = pre / (1 + torch.exp(-pre))
    dt, b, c = low(p, y)
    d = torch.logaddexp(dt + p["dt_bias"], torch.zeros_like(dt))
    h, out = x.new_zeros(n, C, N), []
    for i in range(t):
        h = torch.exp(d[:, i, :, None] * p["A"]) * h + (d[:, i] * y[:, i])[..., None] * b[:, :, i]
        o = (h * c[:, :, i]).sum(-1) + p["D"] * y[:, i]
        out.append(o * z[:, i] / (1 + torch.exp(-z[:, i])))
    return torch.matmul(torch.stack(out, 1), p["back"]), full[:, t:], h


# Six stages follow each other, each off by at most (5 T + 300) 2^-24 of the sum of its
# terms' absolute values (T < 128: 940 2^-24), and those sums are within a factor of 5 of
# the largest value of a stage: 6 * 940 * 5 * 2^-24 < 2^-9 of the largest value.
BAR = 2.0 ** -9


def near(got, want, name):
    off = (got.detach().double().cpu() - want).abs().max()
    assert off <= BAR * want.abs().max(), (name, float(off / want.abs().max()))


def test_pieces_of_their_own_lengths_then_tokens():
    p, u = layer(torch.float32, DEV), tokens()
    lengths = torch.tensor([[37, 70], [37, 31], [20, 70]])   # the second and third end pieces early
    want = []
    for b, n in enumerate(lengths.tolist()):
        mine = torch.cat([u[b, :n[0]], u[b, 37:37 + n[1]], u[b, 107:]])
        want.append(plain(layer(), mine[None]))
    x = u.float().to(DEV)
    conv = h = None
    at, got = 0, [[] for _ in range(B)]
    for i, n in enumerate(PIECES):
        n_new = lengths[:, i].to(torch.int32).to(DEV)
        o, conv, h, _ = piece(p, x[:, at:at + n], conv, h, n_new)
        for b in range(B):
            got[b].append(o[b, :lengths[b, i]])
        at += n
    # the states go into pools, entries in another order
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device=DEV)
    cpool, hpool = torch.randn(5, K - 1, C, device=DEV), torch.randn(5, C, N, device=DEV)
    cpool[slots.long()], hpool[slots.long()] = conv, h
    for t in range(at, T):
        o = token(p, x[:, t:t + 1], cpool, hpool, slots)
        for b in range(B):
            got[b].append(o[b])
    for b in range(B):
        near(torch.cat(got[b]), want[b][0][0], f"outputs {b}")
        near(cpool[slots[b].long()], want[b][1][0], "convolution's state")
        near(hpool[slots[b].long()], want[b][2][0], "scan's state")


def test_a_training_step():
    ref = {k: v.requires_grad_() for k, v in layer().items()}
    u = tokens()
    ru = u.clone().requires_grad_()
    up = torch.randn(B, T, M, generator=torch.Generator().manual_seed(8), dtype=torch.float64)
    plain(ref, ru)[0].mul(up).sum().backward()

    p, x = layer(torch.float32, DEV), u.float().to(DEV)
    out, conv, h, (xc, z, y, dt, b, c, o, saved) = piece(p, x, None, None, save=True)
    do = up.float().to(DEV)
    flat = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
    g = {"back": flat(o).t() @ flat(do)}
    r = linrec.scan_bwd(y, dt, p["A"], b, c, saved, torch.matmul(do, p["back"].t()), D=p["D"], z=z, dt_bias=p["dt_bias"])
    g |= {"A": r.dA, "D": r.dD, "dt_bias": r.ddt_bias}
    mid = torch.matmul(y, p["low"][:, :R])
    g["step"] = flat(mid).t() @ flat(r.ddt)
    dv = torch.cat([torch.matmul(r.ddt, p["step"].t()), r.dB[:, 0], r.dC[:, 0]], -1)
    g["low"] = flat(y).t() @ flat(dv)
    dx, g["w"], g["bias"], _ = linrec.conv_bwd(xc, p["w"], p["bias"], None, r.dx + torch.matmul(dv, p["low"].t()))
    both = torch.cat([dx, r.dz], -1)
    g["inp"] = flat(x).t() @ flat(both)
    near(torch.matmul(both, p["inp"].t()), ru.grad, "input")
    for k, t in g.items():
        near(t, ref[k].grad, k)


def test_a_captured_token_advances_the_pools():
    p, x = layer(torch.float32, DEV), tokens().float().to(DEV)
    slots = torch.tensor([1, 3, 0], dtype=torch.int32, device=DEV)
    pools = [torch.randn(4, K - 1, C, device=DEV), torch.rand(4, C, N, device=DEV)]
    twin = [t.clone() for t in pools]
    u = x[:, :1].clone()
    token(p, u, *[t.clone() for t in pools], slots)   # the library's first products choose their kernels
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = token(p, u, *twin, slots)
    for a, b in zip(pools, twin):                      # capturing ran nothing
        assert torch.equal(a, b)
    for t in range(TOKENS):
        u.copy_(x[:, t:t + 1])
        want = token(p, x[:, t:t + 1].clone(), *pools, slots)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), t
        for a, b in zip(pools, twin):
            assert torch.equal(a, b), t


def pieces_of(seed, t=300, dtype=torch.bfloat16):
    """What a forward and backward of both operators read, and the pair as one call."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(dtype).to(DEV)  # noqa: E731
    f = lambda *s: torch.randn(*s, generator=g).to(DEV)  # noqa: E731
    s = dict(x=r(B, t, C), dt=r(B, t, C), b=r(B, 1, t, N), c=r(B, 1, t, N), z=r(B, t, C), dy=r(B, t, C), A=-f(C, N).abs(),
             bias=f(C) - 3, w=f(C, K), n=torch.tensor([t, t // 3, 0], dtype=torch.int32, device=DEV))

    def call(workspace=None):
        first = (s["x"], s["dt"], s["A"], s["b"], s["c"])
        rest = dict(z=s["z"], dt_bias=s["bias"], n_new=s["n"])
        y, h, saved = linrec.scan_fwd(*first, save=True, workspace=workspace, **rest)
        grads = [t for t in linrec.scan_bwd(*first, saved, s["dy"], workspace=workspace, **rest) if t is not None]
        v, e = linrec.conv_fwd(s["x"], s["w"], n_new=s["n"])
        back = linrec.conv_bwd(s["x"], s["w"], None, None, s["dy"], n_new=s["n"], workspace=workspace)
        return [y, h, *grads, v, e, *(t for t in back if t is not None)]

    return s, call


def test_captured_steps_replay():
    """Two captured steps over one workspace, replayed by turns with eager work between, give the eager step's bits."""
    work = torch.empty(8 << 20, dtype=torch.uint8, device=DEV)
    made = []
    for seed in (1, 2):
        s, call = pieces_of(seed)
        call(work)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call(work)
        made.append((s, call, graph, out))
    fresh = torch.Generator().manual_seed(50)
    for turn in range(3):
        for s, call, graph, out in made:
            for k in ("x", "dt", "dy", "z"):
                s[k].copy_(torch.randn(s[k].shape, generator=fresh))
            s["n"].copy_(torch.randint(0, 301, (B,), generator=fresh))
            work.random_(0, 255)
            graph.replay()
            torch.cuda.synchronize()
            want = call()
            for i, (a, b) in enumerate(zip(out, want)):
                assert torch.equal(a, b), (turn, i)


def test_two_streams_at_once():
    """Calls in flight on two streams, each with its own memory, equal the calls made alone."""
    made = [pieces_of(seed, 1000) for seed in (3, 4)]
    want = [call() for _, call in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    got = [[], []]
    for _ in range(4):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(made[i][1]())
    torch.cuda.synchronize()
    for i in range(2):
        for run in got[i]:
            for a, b in zip(run, want[i]):
                assert torch.equal(a, b)


@pytest.mark.parametrize("C_,t", [(16, 5000), (24, 4100)])
def test_many_segments(C_, t):
    """Pieces split over as many segments as a call makes: the whole against its halves."""
    g = torch.Generator().manual_seed(t)
    r = lambda *s: torch.randn(*s, generator=g).to(DEV)  # noqa: E731
    x, dt, z, dy, b, c = r(1, t, C_), r(1, t, C_), r(1, t, C_), r(1, t, C_), r(1, 1, t, 8), r(1, 1, t, 8)
    A, bias, h0, e = -r(C_, 8).abs() * 4, r(C_) - 4, r(1, C_, 8), r(1, C_, 8)
    y, h, saved = linrec.scan_fwd(x, dt, A, b, c, h0, z=z, dt_bias=bias, save=True)
    full = linrec.scan_bwd(x, dt, A, b, c, saved, dy, e, z=z, dt_bias=bias)
    m = t // 2 + 3
    cut = [(slice(0, m), slice(None, m)), (slice(m, t), slice(m, None))]
    carry, kept = h0, []
    for sl, _ in cut:
        yp, carry, sv = linrec.scan_fwd(x[:, sl], dt[:, sl], A, b[:, :, sl], c[:, :, sl], carry, z=z[:, sl], dt_bias=bias, save=True)
        kept.append(sv)
        # states of one sequence of tokens, joined at other places: each path of gates is off by a
        # few roundings a token
        assert (yp - y[:, sl]).abs().max() <= 5 * t * 2.0 ** -24 * y.abs().max()
    assert (carry - h).abs().max() <= 5 * t * 2.0 ** -24 * h.abs().max()
    grad, dA = e, 0
    for (sl, _), sv in zip(reversed(cut), reversed(kept)):
        part = linrec.scan_bwd(x[:, sl], dt[:, sl], A, b[:, :, sl], c[:, :, sl], sv, dy[:, sl], grad, z=z[:, sl], dt_bias=bias)
        grad, dA = part.dh_in, dA + part.dA
        for k in ("dx", "ddt", "dz"):
            whole = getattr(full, k)
            assert (getattr(part, k) - whole[:, sl]).abs().max() <= 5 * t * 2.0 ** -24 * whole.abs().max(), k
    assert (grad - full.dh_in).abs().max() <= 5 * t * 2.0 ** -24 * full.dh_in.abs().max()
    assert (dA - full.dA).abs().max() <= 6 * t * 2.0 ** -24 * full.dA.abs().max()


def test_a_large_batch_is_its_sequences():
    """The variants of large calls (long runs of the convolution, walks that are not
    split) against the same sequences one call each."""
    g = torch.Generator(device=DEV).manual_seed(31)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    n_, t, c_ = 17, 1040, 2056
    x, dy = r(n_, t, c_).bfloat16(), r(n_, t, c_).bfloat16()
    w, bias, st, dst = r(c_, 4), r(c_), r(n_, 3, c_), r(n_, 3, c_)
    n = torch.randint(t // 2, t + 1, (n_,), generator=g, device=DEV, dtype=torch.int32)
    n[3], n[4] = 0, 2
    y, end = linrec.conv_fwd(x, w, bias, st, n_new=n)
    dx, dw, db, ds = linrec.conv_bwd(x, w, bias, st, dy, dst, n_new=n)
    dw1, db1 = torch.zeros_like(dw, dtype=torch.float64), torch.zeros_like(db, dtype=torch.float64)
    for b in range(n_):
        at = slice(b, b + 1)
        y1, end1 = linrec.conv_fwd(x[at], w, bias, st[at], n_new=n[at])
        dx1, *sums, ds1 = linrec.conv_bwd(x[at], w, bias, st[at], dy[at], dst[at], n_new=n[at])
        assert torch.equal(y[at], y1) and torch.equal(end[at], end1) and torch.equal(dx[at], dx1) and torch.equal(ds[at], ds1), b
        dw1 += sums[0]
        db1 += sums[1]
    # at most 100 additions follow each other (a run, a workgroup, the workgroups), on terms whose absolute values add
    # up to about 30 times the largest sum: 3000 2^-24 of it, below n_ t
    for got, want in ((dw, dw1), (db, db1)):
        assert (got - want).abs().max() <= n_ * t * 2.0 ** -24 * want.abs().max()
    n_, t, c_ = 21, 150, 1016                      # 16 workgroups a sequence
    x, dt, z, dy = (r(n_, t, c_) for _ in range(4))
    b, c = r(n_, 1, t, N), r(n_, 1, t, N)
    A, dt_bias, D, h0, e = -r(c_, N).abs() * 8, r(c_) - 4, r(c_), r(n_, c_, N), r(n_, c_, N)
    n = torch.randint(1, t + 1, (n_,), generator=g, device=DEV, dtype=torch.int32)
    rest = dict(D=D, dt_bias=dt_bias)
    y, h, saved = linrec.scan_fwd(x, dt, A, b, c, h0, z=z, n_new=n, save=True, **rest)
    full = linrec.scan_bwd(x, dt, A, b, c, saved, dy, e, z=z, n_new=n, **rest)
    sums = {k: 0 for k in ("dA", "dD", "ddt_bias")}
    # paths of gates joined at other places: a few roundings a token
    near_ = lambda a, b, k: (a - b).abs().max() <= 6 * t * 2.0 ** -24 * b.abs().max() or pytest.fail(k)  # noqa: E731
    for i in range(n_):
        at = slice(i, i + 1)
        first = (x[at], dt[at], A, b[at], c[at])
        y1, h1, saved1 = linrec.scan_fwd(*first, h0[at], z=z[at], n_new=n[at], save=True, **rest)
        part = linrec.scan_bwd(*first, saved1, dy[at], e[at], z=z[at], n_new=n[at], **rest)
        near_(y[at], y1, "y")
        near_(h[at], h1, "h_out")
        for k in ("dx", "ddt", "dz", "dB", "dC", "dh_in"):
            near_(getattr(full, k)[at], getattr(part, k), k)
        sums = {k: v + getattr(part, k).double() for k, v in sums.items()}
    for k, v in sums.items():
        near_(getattr(full, k), v, k)
