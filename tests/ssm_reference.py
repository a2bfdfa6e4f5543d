"""The short causal convolution and the selective state-space scan in 64 bits on
the CPU, token by token, forward and backward, written from their formulas; and
for each output a bound on how much its terms add up to in absolute value (the
same sums over absolute values), which rounding errors are measured against.
"""
import torch

F64 = torch.float64


def f64(t):
    return None if t is None else t.detach().to("cpu", F64)


def sig(p):
    return 1.0 / (1.0 + torch.exp(-p))


def counts(n_new, B, T):
    return [T] * B if n_new is None else [min(max(int(n), 0), T) for n in n_new]


def conv(x, w, bias=None, state=None, act="silu", n_new=None, dy=None, dstate=None, absolute=False):
    """A dict of y, state_out and, with dy, dx, dw, dbias, dstate_in (rows that are not there: zeros)."""
    x, w, bias, state, dy, dstate = map(f64, (x, w, bias, state, dy, dstate))
    B, T, C = x.shape
    K = w.shape[1]
    signed = dict(x=x, w=w, bias=bias, state=state)
    if absolute:
        w = w.abs()
    out = dict(y=torch.zeros_like(x), state_out=torch.zeros(B, K - 1, C, dtype=F64))
    if dy is not None:
        out |= dict(dx=torch.zeros_like(x), dw=torch.zeros_like(w), dbias=torch.zeros(C, dtype=F64),
                    dstate_in=torch.zeros(B, K - 1, C, dtype=F64))
    for b, n in enumerate(counts(n_new, B, T)):
        def before(v):
            return torch.zeros(K - 1, C, dtype=F64) if v is None else v[b]
        full = torch.cat([before(signed["state"]), signed["x"][b, :n]])
        there = full.abs() if absolute else full
        p = torch.zeros(n, C, dtype=F64) if bias is None else bias.expand(n, C).clone()
        m = p.abs()
        for k in range(K):
            p = p + signed["w"][:, k] * full[k:k + n]
            m = m + (signed["w"][:, k] * full[k:k + n]).abs()
        s = sig(p)
        if act:   # the slope of silu is at most 1.1: an error of p is one of y
            out["y"][b, :n] = 1.1 * m if absolute else p * s
        else:
            out["y"][b, :n] = m if absolute else p
        out["state_out"][b] = there[n:]
        if dy is not None:
            d = dy[b, :n].abs() if absolute else dy[b, :n].clone()
            if act:   # and its second derivative at most 1/2
                d = d * (s * (1 + p.abs()) + m / 2) if absolute else d * (s + p * s * (1 - s))
            g = torch.zeros_like(full)
            if dstate is not None:
                g[n:] += dstate[b].abs() if absolute else dstate[b]
            for k in range(K):
                g[k:k + n] += w[:, k] * d
                out["dw"][:, k] += (d * there[k:k + n]).sum(0)
            out["dbias"] += d.sum(0)
            out["dx"][b, :n], out["dstate_in"][b] = g[K - 1:], g[:K - 1]
    return out


def scan(x, dt, A, B, C, h_in=None, D=None, z=None, dt_bias=None, softplus=True, n_new=None, dy=None, dh_out=None,
         absolute=False):
    """A dict of y, h_out and, with dy, the gradients by scan_bwd's names (rows that are not there: zeros)."""
    x, dt, A, Bp, Cp, h_in, D, z, dt_bias, dy, dh_out = map(f64, (x, dt, A, B, C, h_in, D, z, dt_bias, dy, dh_out))
    nb, T, ch = x.shape
    G, N = Bp.shape[1], Bp.shape[3]
    per = ch // G
    mag = torch.abs if absolute else (lambda t: t)
    raw = dt + (0.0 if dt_bias is None else dt_bias)
    d_all = torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw
    slope = sig(raw) if softplus else torch.ones_like(raw)
    out = dict(y=torch.zeros_like(x), h_out=torch.zeros(nb, ch, N, dtype=F64))
    if dy is not None:
        out |= dict(dx=torch.zeros_like(x), ddt=torch.zeros_like(x), dA=torch.zeros_like(A), dB=torch.zeros_like(Bp),
                    dC=torch.zeros_like(Cp), dh_in=torch.zeros(nb, ch, N, dtype=F64), dD=torch.zeros(ch, dtype=F64),
                    dz=torch.zeros_like(x), ddt_bias=torch.zeros(ch, dtype=F64))
    skip = torch.zeros(ch, dtype=F64) if D is None else mag(D)
    for b, n in enumerate(counts(n_new, nb, T)):
        h = torch.zeros(ch, N, dtype=F64) if h_in is None else mag(h_in[b])
        xs, ds = mag(x[b, :n]), d_all[b, :n]
        Bs, Cs = (mag(p[b, :, :n]).repeat_interleave(per, 0) for p in (Bp, Cp))   # [ch, n, N]
        if z is None:
            gate, dgate = torch.ones_like(xs), torch.zeros_like(xs)
        else:
            zs = z[b, :n]
            q = sig(zs)
            gate = mag(zs * q)
            dgate = q * (1 + zs.abs()) if absolute else q * (1 + zs * (1 - q))
        hs = [h]
        ys = torch.zeros_like(xs)
        for t in range(n):
            h = torch.exp(ds[t][:, None] * A) * h + mag(ds[t] * xs[t])[:, None] * Bs[:, t]
            hs.append(h)
            ys[t] = (Cs[:, t] * h).sum(-1) + skip * xs[t]
        out["y"][b, :n], out["h_out"][b] = ys * gate, h
        if dy is None:
            continue
        dys = mag(dy[b, :n])
        g = torch.zeros(ch, N, dtype=F64) if dh_out is None else mag(dh_out[b])
        out["dz"][b, :n] = dys * ys * dgate
        for t in reversed(range(n)):
            e = dys[t] * gate[t]
            Gt = g + Cs[:, t] * e[:, None]
            u = mag(ds[t] * xs[t])
            out["dC"][b, :, t] = (e[:, None] * hs[t + 1]).view(G, per, N).sum(1)
            out["dB"][b, :, t] = (Gt * u[:, None]).view(G, per, N).sum(1)
            du = (Gt * Bs[:, t]).sum(-1)
            g = torch.exp(ds[t][:, None] * A) * Gt
            qt = g * hs[t]
            out["dA"] += qt * mag(ds[t])[:, None]
            dd = ((qt * mag(A)).sum(-1) + du * xs[t]) * slope[b, t]
            out["dx"][b, t] = e * skip + du * mag(ds[t])
            out["ddt"][b, t] = dd
            out["dD"] += e * xs[t]
            out["ddt_bias"] += dd
        out["dh_in"][b] = g
    return out
