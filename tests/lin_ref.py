"""Plain 64-bit forms of the linear-attention block's operators (CPU, torch
double): the recurrence token by token, its reverse, the block norms by
torch's differentiation of the formulas, the E4M3 codes by exact rounding."""
import torch

F64 = torch.float64


def seq_fwd(q, k, v, g, S0):
    """q, k [L, H, dk], v [L, H, dv], g [L, H], S0 [H, dv, dk]: o, states after every token (S0 first)."""
    S, out, states = S0.clone(), [], [S0.clone()]
    for t in range(v.shape[0]):
        S = S * g[t].exp()[:, None, None] + v[t][:, :, None] * k[t][:, None, :]
        states.append(S)
        out.append((S * q[t][:, None, :]).sum(-1))
    return (torch.stack(out) if out else torch.zeros_like(v)), states


def seq_bwd(q, k, v, g, states, do, dS):
    dq, dk, dv, dg = (torch.zeros_like(x) for x in (q, k, v, g))
    R = dS.clone()
    for t in range(v.shape[0] - 1, -1, -1):
        dq[t] = (do[t][:, :, None] * states[t + 1]).sum(1)
        R = R + do[t][:, :, None] * q[t][:, None, :]
        dk[t] = (v[t][:, :, None] * R).sum(1)
        dv[t] = (R * k[t][:, None, :]).sum(-1)
        R = R * g[t].exp()[:, None, None]
        dg[t] = (R * states[t]).sum((-1, -2))
    return dq, dk, dv, dg, R


def lin(q, k, v, g, cu, S0=None, do=None, dS=None):
    """The packed operator in 64 bits: (o, S) or, with do, (dq, dk, dv, dg, dS0);
    rows outside the sequences are 0."""
    T, Hk, dk = k.shape
    H, dv = v.shape[1], v.shape[2]
    q, k = (x.to(F64).cpu().repeat_interleave(H // Hk, 1) for x in (q, k))
    v = v.to(F64).cpu()
    gg = g.to(F64).cpu().expand(T, H)
    cu = [int(x) for x in cu]
    zero = torch.zeros(H, dv, dk, dtype=F64)
    if do is None:
        o, S = torch.zeros(T, H, dv, dtype=F64), []
        for n in range(len(cu) - 1):
            r = slice(cu[n], cu[n + 1])
            o[r], st = seq_fwd(q[r], k[r], v[r], gg[r], zero if S0 is None else S0[n].to(F64).cpu())
            S.append(st[-1])
        return o, torch.stack(S)
    do = do.to(F64).cpu()
    dq, dkk, dvv, dg = (torch.zeros_like(x) for x in (q, k, v, gg.clone()))
    d0 = []
    for n in range(len(cu) - 1):
        r = slice(cu[n], cu[n + 1])
        _, st = seq_fwd(q[r], k[r], v[r], gg[r], zero if S0 is None else S0[n].to(F64).cpu())
        dq[r], dkk[r], dvv[r], dg[r], d = seq_bwd(q[r], k[r], v[r], gg[r], st, do[r],
                                                  zero if dS is None else dS[n].to(F64).cpu())
        d0.append(d)
    dq, dkk = (x.reshape(T, Hk, H // Hk, dk).sum(2) for x in (dq, dkk))
    return dq, dkk, dvv, (dg.sum(0) if g.dim() == 1 else dg), torch.stack(d0)


def _none_abs(x):
    return None if x is None else x.abs()


def lin_abs(q, k, v, g, cu, S0=None, do=None, dS=None):
    """The same sums with every factor's absolute value: what rounding errors are relative to."""
    return lin(q.abs(), k.abs(), v.abs(), g, cu, _none_abs(S0), _none_abs(do), _none_abs(dS))


def pack(x):
    """(values code * scale, scales): s = fl32(amax / 448), 1 where not positive; nearest E4M3 to fl32(x / s)."""
    x = x.to(F64).cpu()
    R, D = x.shape
    out, scales = torch.empty_like(x), []
    for c in range(0, D, 64):
        p = x[:, c:c + 64]
        s = (p.abs().amax(-1, keepdim=True) / 448).float().to(F64)
        s = torch.where(s > 0, s, torch.ones_like(s))
        y = (p / s).float().to(F64).clamp(-448, 448)
        _, e = torch.frexp(y)                       # |y| in [2^(e-1), 2^e)
        ulp = torch.ldexp(torch.ones_like(y), torch.clamp(e - 1, min=-6) - 3)
        out[:, c:c + 64] = (torch.round(y / ulp) * ulp).mul(s).float().to(F64)
        scales.append(s)
    return out, torch.cat(scales, 1)


def norm(f, w_post, z, act, res, res_scale, w_pre, eps):
    y = f / torch.sqrt(f.pow(2).mean(-1, keepdim=True) + eps) * w_post
    if z is not None:
        y = y * (torch.sigmoid(z) if act == "sigmoid" else z * torch.sigmoid(z))
    x = res_scale * y + (0 if res is None else res)
    h = None if w_pre is None else x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps) * w_pre
    return x, h
