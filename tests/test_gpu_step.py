"""GPU tests of the single-token step (linrec_step) against the recurrence in
64 bits on the CPU, and against the chunked forward it continues.

Tolerance: every product and sum is fp32.  With d_k <= 128 terms a sum is off by
at most (d_k + 8) 2^-24 of the sum of its terms' magnitudes, and so is what is
built on it; the magnitudes are carried through the same formulas.  bf16 outputs
add half a step, 2^-8 of the value."""
import pytest
import torch

from state_passing_amd import linrec

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def reference(q, k, v, a, beta, S, slots):
    """(o, S, |o| bound, |S| bound) in 64 bits.  a, beta: [B,H,T]."""
    B, H, T, _ = q.shape
    S, mag = S.double().clone(), S.double().abs()
    o = torch.zeros(*v.shape, dtype=torch.float64)
    om = torch.zeros_like(o)
    seen = set()
    for b in range(B):
        s = b if slots is None else int(slots[b])
        if not 0 <= s < S.shape[0] or s in seen:
            continue
        seen.add(s)
        for t in range(T):
            qq, kk, vv = (x[b, :, t].double() for x in (q, k, v))
            at = a[b, :, t].double()[:, None]
            u, um = vv, vv.abs()
            if beta is not None:
                bt = beta[b, :, t].double()[:, None]
                u = bt * (vv - at * torch.einsum("hk,hkv->hv", kk, S[s]))
                um = bt * (vv.abs() + at * torch.einsum("hk,hkv->hv", kk.abs(), mag[s]))
            S[s] = at[..., None] * S[s] + kk[..., None] * u[:, None]
            mag[s] = at[..., None] * mag[s] + kk.abs()[..., None] * um[:, None]
            o[b, :, t] = torch.einsum("hk,hkv->hv", qq, S[s])
            om[b, :, t] = torch.einsum("hk,hkv->hv", qq.abs(), mag[s])
    return o, S, om, mag


def draw(seed, B, H, T, dk, dv, n, dtype):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(dtype)  # noqa: E731
    return dict(q=unit(r(B, H, T, dk)), k=unit(r(B, H, T, dk)), v=r(B, H, T, dv).to(dtype),
                S=0.3 * r(n, H, dk, dv), beta=torch.sigmoid(r(B, H, T)), a=0.9 + 0.1 * torch.sigmoid(r(B, H, T)),
                head=0.8 + 0.2 * torch.rand(H, generator=g))


def check(x, kind, delta, slots=None, out=None, view=lambda t: t):
    B, H, T, dk = x["q"].shape
    a = {"none": torch.ones(B, H, T), "head": x["head"][None, :, None].expand(B, H, T), "token": x["a"]}[kind]
    decay = {"none": None, "head": x["head"], "token": x["a"]}[kind]
    beta = x["beta"] if delta else None
    o, S, om, Sm = reference(x["q"], x["k"], x["v"], a, beta, x["S"], slots)
    d = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    Sd = d(x["S"])
    got = linrec.step(view(d(x["q"])), view(d(x["k"])), view(d(x["v"])), d(decay), Sd, beta=d(beta), slots=d(slots),
                      out_dtype=out)
    torch.cuda.synchronize()
    eps = (dk + 8) * 2.0 ** -24 * (T + 1) * 2
    half = 2.0 ** -8 * o.abs() if got.dtype == BF else 0.0
    assert ((got.double().cpu() - o).abs() <= eps * om + half).all()
    assert ((Sd.double().cpu() - S).abs() <= eps * Sm).all()
    skipped = [b for b in range(B) if om[b].abs().max() == 0]
    assert (got[skipped] == 0).all()
    return got, Sd


@pytest.mark.parametrize("kind", ["none", "head", "token"])
@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("dk,dv,dtype", [(128, 128, BF), (64, 64, BF), (64, 128, BF), (128, 64, BF), (64, 64, F32)])
def test_step(kind, delta, dk, dv, dtype):
    check(draw(dk + dv, 2, 3, 1, dk, dv, 2, dtype), kind, delta)
    check(draw(dk + dv, 1, 2, 5, dk, dv, 3, dtype), kind, delta, out=F32)


@pytest.mark.parametrize("B,H", [(1, 1), (5, 2), (70, 8), (300, 2)])
@pytest.mark.parametrize("delta", [False, True])
def test_slots(B, H, delta):
    """States by slot: in any order, outside the pool (skipped), named twice (the first counts)."""
    x = draw(B, B, H, 2, 64, 128, B + 2, BF)
    g = torch.Generator().manual_seed(B)
    slots = torch.randperm(B + 2, generator=g)[:B].to(torch.int32)
    check(x, "token", delta, slots)
    if B > 4:
        slots[1], slots[2], slots[4] = -1, B + 2, slots[0]
        slots[B - 1] = slots[3]
        before = x["S"].clone()
        _, S = check(x, "token", delta, slots)
        used = set(slots.tolist())
        rest = [i for i in range(B + 2) if i not in used]
        assert torch.equal(S.cpu()[rest], before[rest])


def test_token_major_views():
    view = lambda t: t.transpose(1, 2).contiguous().transpose(1, 2)  # noqa: E731
    check(draw(9, 3, 4, 2, 128, 128, 3, BF), "token", True, view=view)
    check(draw(9, 3, 4, 1, 128, 128, 3, BF), "token", False, view=view)


@pytest.mark.parametrize("delta", [False, True])
def test_continues_a_piece(delta):
    """The chunked forward over 100 tokens, then steps, against one forward over all."""
    B, H, T, d = 2, 3, 107, 128
    x = draw(21, B, H, T, d, d, B, BF)
    dev = {n: t.to(DEV) for n, t in x.items()}
    cut = lambda i, j: [dev[n][:, :, i:j] for n in ("q", "k", "v")]  # noqa: E731
    dec = lambda i, j: dev["a"][:, :, i:j]  # noqa: E731
    if delta:
        whole, S_all, _ = linrec.delta_fwd(*cut(0, T), dev["beta"], dec(0, T), out_dtype=F32)
        _, S, _ = linrec.delta_fwd(*cut(0, 100), dev["beta"][:, :, :100], dec(0, 100))
    else:
        whole, S_all, _ = linrec.fwd(*cut(0, T), dec(0, T), out_dtype=F32)
        _, S, _ = linrec.fwd(*cut(0, 100), dec(0, 100))
    for i, j in ((100, 101), (101, 102), (102, 107)):
        o = linrec.step(*cut(i, j), dec(i, j), S, beta=dev["beta"][:, :, i:j] if delta else None, out_dtype=F32)
        # the chunked kernels hold the 2e-2 bar of bf16 activations against the oracle
        scale = float(whole.square().mean().sqrt())
        assert float((o - whole[:, :, i:j]).abs().max()) <= 2e-2 * scale
    assert float((S - S_all).abs().max()) <= 2e-2 * float(S_all.square().mean().sqrt())


def test_replay_advances_the_state():
    """A captured step reads and writes the state it was given: n replays are n tokens."""
    x = draw(22, 4, 2, 1, 128, 128, 6, BF)
    dev = {n: t.to(DEV) for n, t in x.items()}
    slots = torch.tensor([5, 0, 3, -1], dtype=torch.int32, device=DEV)
    S1, S2 = dev["S"].clone(), dev["S"].clone()
    o2 = torch.empty_like(dev["v"])
    args = (dev["q"], dev["k"], dev["v"], dev["a"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        linrec.step(*args, S2, beta=dev["beta"], slots=slots, o=o2)
    assert torch.equal(S2, dev["S"])
    for _ in range(4):
        o1 = linrec.step(*args, S1, beta=dev["beta"], slots=slots)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(S1, S2) and torch.equal(o1, o2)


def test_skipped_sequence_of_very_many_tokens():
    """2^25 + 1 tokens of 64 columns: 2^31 + 64 outputs, every one of them zeroed."""
    T = 2 ** 25 + 1
    x = torch.ones(1, 1, T, 64, dtype=BF, device=DEV)
    o = torch.full_like(x, 5.0)
    S = torch.ones(2, 1, 64, 64, device=DEV)
    linrec.step(x, x, x, None, S, slots=torch.tensor([-1], dtype=torch.int32, device=DEV), o=o)
    torch.cuda.synchronize()
    # (in parts: a reduction over the whole would count in 64 bits anyway, but holds a copy)
    assert not any(bool(p.any()) for p in o.view(-1).split(2 ** 28))
    assert (S == 1).all()
