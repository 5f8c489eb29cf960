"""Plain 64-bit form (CPU, torch double) of the distillation loss, straight from its definition, row by row and entry
by entry; gradients by torch's differentiation of it."""
import math

import torch

F64 = torch.float64


def losses(z, ids, top, lse=None, targets=None, h=1.0, kd_weight=1.0, ce_weight=0.0, ignore=-100):
    """(loss [R], stats [R, 4]) of logits z [R, V] in double (with gradient where z has one)."""
    R, V = z.shape
    out, stats = [], []
    for r in range(R):
        if targets is not None and int(targets[r]) == ignore:
            out.append(z[r, 0].detach() * 0 if torch.isfinite(z[r, 0]) else torch.zeros((), dtype=F64))
            stats.append(torch.zeros(4, dtype=F64))
            continue
        zh = z[r] / h
        kept = [j for j in range(ids.shape[1]) if int(ids[r, j]) >= 0]
        t = torch.stack([top[r, j].to(F64) / h for j in kept]) if kept else torch.zeros(0, dtype=F64)
        c = lse[r].to(F64) if lse is not None else (t.logsumexp(0) if kept else torch.tensor(-math.inf, dtype=F64))
        zlse = zh.logsumexp(0)
        kd, mass = torch.zeros((), dtype=F64), 0.0
        for i, j in enumerate(kept):
            lp = t[i] - c
            p = math.exp(lp) if t[i] > -math.inf else 0.0
            mass += p
            if p > 0:
                kd = kd + p * (lp - (zh[int(ids[r, j])] - zlse))
        last = torch.zeros((), dtype=F64)
        if lse is not None:
            off = torch.ones(V, dtype=torch.bool)
            off[[int(ids[r, j]) for j in kept]] = False
            rest = max(0.0, 1.0 - mass)
            if off.any():
                last = zh[off].logsumexp(0)
                if rest > 0:
                    kd = kd + rest * (math.log(rest) - (last - zlse))
            else:
                last = torch.tensor(-math.inf, dtype=F64)
        loss, first = kd_weight * kd, torch.zeros((), dtype=F64)
        if targets is not None:
            first = z[r].logsumexp(0)
            loss = loss + ce_weight * (first - z[r, int(targets[r])])
        out.append(loss)
        stats.append(torch.stack([first.detach(), zlse.detach(), c, last.detach()]))
    return torch.stack(out), torch.stack(stats)


def grads(z, ids, top, d_loss, **kw):
    """(loss, stats, dz) in double."""
    z = z.detach().to(F64).cpu().clone().requires_grad_()
    loss, stats = losses(z, ids, top, **kw)
    if not loss.requires_grad:
        return loss, stats, torch.zeros_like(z)
    w = torch.ones_like(loss) if d_loss is None else d_loss.to(F64).cpu()
    dz, = torch.autograd.grad((loss * w).sum(), z)
    return loss.detach(), stats, dz
