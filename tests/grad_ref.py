"""Plain 64-bit forms (CPU, torch double) of the gated delta rule's gradients:
the recurrence token by token and its reverse.

    S_d = a S,  e = v - S_d k,  S' = S_d + (b e) k^T,  o = S' q
"""
import torch

F64 = torch.float64


def forward(q, k, v, b, g, S, every=None):
    """One sequence [L, H, ..], S [H, dv, dk]: (o, steps); steps: the (S, S_d, e, S') of every token.  every: a
    function of (token count, state) that may replace the state (the quantization at a boundary)."""
    out, steps = [], []
    for t in range(v.shape[0]):
        Sd = S * g[t].exp()[:, None, None]
        e = v[t] - (Sd * k[t][:, None, :]).sum(-1)
        Sn = Sd + (b[t][:, None] * e)[:, :, None] * k[t][:, None, :]
        out.append((Sn * q[t][:, None, :]).sum(-1))
        steps.append((S, Sd, e, Sn))
        S = Sn if every is None else every(t + 1, Sn)
    return (torch.stack(out) if out else torch.zeros_like(v)), steps, S


def backward(q, k, v, b, g, steps, do, R):
    dq, dk, dv, db, dg = (torch.zeros_like(x) for x in (q, k, v, b, g))
    for t in range(v.shape[0] - 1, -1, -1):
        S, Sd, e, Sn = steps[t]
        dq[t] = (do[t][:, :, None] * Sn).sum(1)
        R = R + do[t][:, :, None] * q[t][:, None, :]
        Rk = (R * k[t][:, None, :]).sum(-1)
        db[t] = (Rk * e).sum(-1)
        de = b[t][:, None] * Rk
        dv[t] = de
        dk[t] = b[t][:, None] * (e[:, :, None] * R).sum(1) - (de[:, :, None] * Sd).sum(1)
        R = R - de[:, :, None] * k[t][:, None, :]
        dg[t] = (R * Sd).sum((-1, -2))
        R = R * g[t].exp()[:, None, None]
    return dq, dk, dv, db, dg, R


def grad(q, k, v, b, g, cu, do, lens=None, S0=None, dS=None, states=None):
    """The packed operator: (dq, dk, dv, db, dg, dS0); rows outside the sequences are 0.  states: [n_bounds, H, dv,
    dk], what the chunks after the first of each sequence start from."""
    T, H, dk = k.shape
    dv = v.shape[2]
    q, k, v, b, g, do = (x.to(F64).cpu() for x in (q, k, v, b, g, do))
    cu = [int(x) for x in cu]
    outs = [torch.zeros_like(x) for x in (q, k, v, b, g)]
    d0, at = [], 0
    zero = torch.zeros(H, dv, dk, dtype=F64)
    for n in range(len(cu) - 1):
        L = cu[n + 1] - cu[n] if lens is None else int(lens[n])
        r = slice(cu[n], cu[n] + L)
        every = None
        if states is not None:
            def every(t, S, at=at):
                return states[at + t // 64 - 1].to(F64).cpu() if t % 64 == 0 else S
        x = (q[r], k[r], v[r], b[r], g[r])
        _, steps, _ = forward(*x, zero if S0 is None else S0[n].to(F64).cpu(), every)
        got = backward(*x, steps, do[r], zero if dS is None else dS[n].to(F64).cpu())
        for o, y in zip(outs, got):
            o[r] = y
        d0.append(got[5])
        at += -(-L // 64)
    return (*outs, torch.stack(d0))
