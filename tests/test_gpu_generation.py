"""The operators together, as a hybrid model runs them: a prompt in pieces through
the chunked layer, the delta rule, the elementwise recurrence and the cached
attention, then token after token through the step, the recurrence, the append
and the attention -- eagerly and as one captured graph whose replays advance
every state in place."""
import pytest
import torch

from state_passing_amd import linrec

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
B, H, Hkv, D, C, PAGE = 2, 4, 2, 64, 96, 16
PIECES, TOKENS = (37, 20), 6
T = sum(PIECES) + TOKENS


def inputs():
    g = torch.Generator().manual_seed(77)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    bf = lambda x: x.to(torch.bfloat16).to(DEV)  # noqa: E731
    return dict(q=bf(unit(r(B, H, T, D))), k=bf(unit(r(B, H, T, D))), v=bf(r(B, H, T, D)),
                a=(0.9 + 0.1 * torch.sigmoid(r(B, H, T))).to(DEV), beta=torch.sigmoid(r(B, H, T)).to(DEV),
                g=bf(-0.2 * torch.rand(B, T, C, generator=g)), x=bf(r(B, T, C)),
                aq=bf(r(B, H, T, D)), ak=bf(r(B, Hkv, T, D)), av=bf(r(B, Hkv, T, D)))


class State:
    def __init__(self):
        self.S = torch.zeros(B, H, D, D, device=DEV)
        self.Sd = torch.zeros(B, H, D, D, device=DEV)
        self.h = torch.zeros(B, C, device=DEV)
        table = torch.arange(B * 5, dtype=torch.int32).view(5, B).t().contiguous().to(DEV)
        self.cache = linrec.kv_cache(B * 5, Hkv, PAGE, D, table)
        self.past = torch.zeros(B, dtype=torch.int32, device=DEV)
        self.freq = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).to(DEV)

    def all(self):
        return [self.S, self.Sd, self.h, self.past, *(t.view(torch.uint8) for t in self.cache[:2]), *self.cache[2:4]]


def attend(st, m, sl):
    q = linrec.kv_append(st.cache, m["ak"][:, :, sl], m["av"][:, :, sl], st.past, inv_freq=st.freq, q=m["aq"][:, :, sl])
    o = linrec.kv_attn(st.cache, q, st.past)
    st.past.add_(sl.stop - sl.start)
    return o


def prompt(st, m):
    out, at = [], 0
    for n in PIECES:
        sl = slice(at, at + n)
        qkv = [m[x][:, :, sl] for x in "qkv"]
        o1, _, _ = linrec.fwd(*qkv, m["a"][:, :, sl], st.S, S_out=st.S)
        o2, _, _ = linrec.delta_fwd(*qkv, m["beta"][:, :, sl], m["a"][:, :, sl], st.Sd, S_out=st.Sd)
        o3, _, _ = linrec.diag_fwd(m["g"][:, sl], m["x"][:, sl], st.h, h_out=st.h, form="mix")
        out.append((o1, o2, o3, attend(st, m, sl)))
        at += n
    return out


def token(st, m, sl):
    qkv = [m[x][:, :, sl] for x in "qkv"]
    o1 = linrec.step(*qkv, m["a"][:, :, sl], st.S)
    o2 = linrec.step(*qkv, m["a"][:, :, sl], st.Sd, beta=m["beta"][:, :, sl])
    o3, _, _ = linrec.diag_fwd(m["g"][:, sl], m["x"][:, sl], st.h, h_out=st.h, form="mix")
    return o1, o2, o3, attend(st, m, sl)


def test_pieces_then_tokens_equal_one_pass():
    m, st = inputs(), State()
    parts = prompt(st, m)
    for t in range(sum(PIECES), T):
        parts.append(token(st, m, slice(t, t + 1)))
    got = [torch.cat([p[i] for p in parts], 1 if i == 2 else 2).float() for i in range(4)]
    one = State()
    qkv = [m[x] for x in "qkv"]
    want = [linrec.fwd(*qkv, m["a"], one.S, S_out=one.S, out_dtype=torch.float32)[0],
            linrec.delta_fwd(*qkv, m["beta"], m["a"], one.Sd, S_out=one.Sd, out_dtype=torch.float32)[0],
            linrec.diag_fwd(m["g"], m["x"], one.h, h_out=one.h, form="mix", out_dtype=torch.float32)[0],
            attend(one, m, slice(0, T)).float()]
    rms = lambda x: float(x.float().square().mean().sqrt())  # noqa: E731
    # the 2e-2 bar of bf16 activations on the two layers, beside the outputs' own rounding
    for i in (0, 1):
        assert ((got[i] - want[i]).abs() <= 2.0 ** -8 * want[i].abs() + 2e-2 * rms(want[i])).all(), i
    # the recurrence is fp32 inside: both sides round only their outputs (2^-8)
    assert ((got[2] - want[2]).abs() <= 2.0 ** -8 * want[2].abs() + 2.0 ** -16 * float(want[2].abs().max())).all()
    for a, b, tol in ((st.S, one.S, 2e-2), (st.Sd, one.Sd, 2e-2), (st.h, one.h, 2.0 ** -16)):
        assert float((a - b).abs().max()) <= tol * max(rms(b), float(b.abs().max()) if tol < 1e-3 else 0)
    # a page filled piece by piece may have grown its scale on the way: a stored value then
    # was rounded under a smaller scale first, off by one more smallest step (2^-10 of the
    # final scale); scales end the same, for they hold the same largest values
    for i in (2, 3):
        assert torch.equal(st.cache[i], one.cache[i])
    for i in (0, 1):
        diff = (st.cache[i].float() - one.cache[i].float()).abs()
        assert float(diff.max()) <= 2.0 ** -9


def test_a_captured_token_advances_every_state():
    m, st = inputs(), State()
    prompt(st, m)
    twin = State()
    for a, b in zip(twin.all(), st.all()):
        a.copy_(b)
    first = sum(PIECES)
    slot = {n: t[:, :, :1].clone() if n not in "gx" else t[:, :1].clone() for n, t in m.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = token(twin, slot, slice(0, 1))
    for a, b in zip(twin.all(), st.all()):        # capturing ran nothing
        assert torch.equal(a, b)
    for t in range(first, T):
        sl = slice(t, t + 1)
        want = token(st, m, sl)
        for n, s in slot.items():
            s.copy_(m[n][:, sl] if n in "gx" else m[n][:, :, sl])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), t
        for a, b in zip(twin.all(), st.all()):
            assert torch.equal(a, b), t
