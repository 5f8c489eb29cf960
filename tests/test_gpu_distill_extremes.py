"""Distillation on the GPU at the ends of its range: masked vocabularies, far logits, values that are not finite.

The reference forms everything from differences of a row's logits in 64 bits, so that it holds for logits of any size.
Tolerances.  A logsumexp's sum is within 2^-15 of itself (derived in test_gpu_distill.py; an argument (v - max) c / h
has two roundings more, |x| 2^-23 for |x| < 17 where e^x counts), and the rest of a row's values is formed in fp64: a
loss is within (kd_weight + ce_weight) 2^-14 + 2^-23 of itself.  A probability is within 2^-15 for the sum and |y| 1.5 *
2^-23 < 2^-16 for its argument y > -87 of itself, so a gradient's value within 2^-14 of its terms' magnitudes, with
bf16 2^-8 of itself more.
"""
import math

import pytest
import torch

from fp8_state_qat_amd import api

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
INF, NAN = float("inf"), float("nan")


def lse(y):
    m = y.max().detach()
    return m + (y - m).exp().sum().log() if m > -INF else m


def reference(d):
    """(loss [R], dz [R, V], magnitudes of the gradient's terms [R, V]) in double."""
    h, wk, wc = (float(torch.tensor(d["kw"][n], dtype=F32)) for n in ("temperature", "kd_weight", "ce_weight"))  # as passed
    z0 = d["z"].to(F64)
    R, V = z0.shape
    loss, dz, mag = torch.zeros(R, dtype=F64), torch.zeros(R, V, dtype=F64), torch.zeros(R, V, dtype=F64)
    for r in range(R):
        z = z0[r].clone().requires_grad_()
        top = z.max().detach()
        y = (z - top) / h
        on = d["ids"][r] >= 0
        ids, t = d["ids"][r][on].long(), d["top"][r][on].to(F64) / h
        c = lse(t) if d["lse"] is None else d["lse"][r].to(F64)
        p = (t - c).exp()
        total = lse(y)
        kd = (p * (t - c - (y[ids] - total))).sum() if len(ids) else torch.zeros((), dtype=F64)
        a, b = abs(float(d["d_loss"][r])) * wk / h, abs(float(d["d_loss"][r])) * wc
        mag[r] = a * (y - total).exp().detach()
        mag[r].index_add_(0, ids, a * p)
        if d["lse"] is not None:
            off = torch.ones(V, dtype=torch.bool)
            off[ids] = False
            rest = max(0.0, 1.0 - float(p.sum()))
            if off.any() and rest > 0:
                last = lse(y[off])
                kd = kd + rest * (math.log(rest) - (last - total))
                mag[r][off] += a * rest * (y[off] - y[off].max()).exp().detach() / (y[off] - y[off].max()).exp().sum().item()
        out = wk * kd
        if d["targets"] is not None:
            k = int(d["targets"][r])
            x = z - top
            out = out + wc * (lse(x) - x[k])
            mag[r] += b * torch.softmax(x, 0).detach()
            mag[r, k] += b
        loss[r] = out.detach()
        dz[r], = torch.autograd.grad(out * float(d["d_loss"][r]), z)
    return loss, dz, mag


def make(z, ids, dtype, tail, ce=True, h=1.0, seed=0):
    """The teacher's logits: 3 of every row, spread by chance; targets among the kept."""
    gen = torch.Generator().manual_seed(seed)
    R, K = ids.shape
    d = dict(z=z.to(dtype), ids=ids.int(), top=2 * torch.randn(R, K, generator=gen))
    d["lse"] = (torch.logsumexp(d["top"].double() / h, 1) + 0.4).float() if tail else None
    d["targets"] = ids[:, 0].long() if ce else None
    d["d_loss"] = torch.rand(R, generator=gen) + 0.25
    d["kw"] = dict(temperature=h, kd_weight=0.75, ce_weight=0.25 if ce else 0.0)
    return d


def run(d):
    """(losses of both calls, gradients of both)."""
    x = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in d.items()}
    kw = dict(teacher_lse=x["lse"], targets=x["targets"], **d["kw"])
    a = x["z"], x["ids"], x["top"]
    loss, stats = api.distill_fwd(*a, **kw)
    back = api.distill_bwd(*a, stats, x["d_loss"], **kw)
    both, grad = api.distill_fwd_bwd(*a, x["d_loss"], **kw)
    for out in (x["z"].clone(), x["z"].clone()):      # in place
        api.distill_bwd(out, x["ids"], x["top"], stats, x["d_loss"], out=out, **kw)
        assert torch.equal(out, back) or not torch.isfinite(back).all()
    return (loss.cpu(), both.cpu()), (back.cpu(), grad.cpu()), stats.cpu()


def check(d, far=0.0):
    """far: the logsumexps' magnitude, of which a probability may be off by 2^-22 times itself more."""
    loss, dz, mag = reference(d)
    losses, grads, stats = run(d)
    wanted = loss.float()
    tol = (d["kw"]["kd_weight"] + d["kw"]["ce_weight"]) * 2.0 ** -14 + 2.0 ** -23 * loss.abs()
    for got in losses:
        ok = (got == wanted) | ((got.double() - loss).abs() <= tol)
        assert ok.all(), (got, wanted)
    for name, g in zip(("backward", "both"), grads):
        err = (g.double() - dz).abs()
        bound = (2.0 ** -14 + 2.0 ** -22 * far) * mag + (2.0 ** -8 * dz.abs() if g.dtype == BF else 0) + 1e-36
        bad = ~(err <= bound)
        assert not bad.any(), f"{name}: {bad.nonzero()[:5].tolist()}, worst {float((err / bound).max()):.3g}"
    return losses, grads, stats


def random_ids(R, V, K, lo=0):
    gen = torch.Generator().manual_seed(V)
    return torch.stack([lo + torch.randperm(V - lo, generator=gen)[:K] for _ in range(R)])


# ---------------------------------------------------------------- far logits
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("V,h", [(301, 1.0), (700, 2.0), (5003, 1.0), (40000, 0.5)])
def test_far_logits_beside_each_other(dtype, tail, V, h):
    """Logits whose neighbours differ in size and sign; the largest in even and in odd columns."""
    z = torch.randn(6, V, generator=torch.Generator().manual_seed(V))
    z[0, 0::2], z[0, 1::2] = -30000.0, -20000.0
    z[1, 1::2], z[1, 0::2] = -30000.0, -20000.0
    z[2, 101] = z[3, 100] = 20000.0
    z[4] *= 9000.0
    z[5, 0::2] -= 25000.0
    check(make(z, random_ids(6, V, 3), dtype, tail, h=h), far=45000.0 / min(h, 1.0))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [40, 5003])
@pytest.mark.parametrize("value", [INF, NAN])
def test_a_logit_that_is_not_finite_makes_its_row_nan(dtype, V, value):
    z = torch.randn(4, V, generator=torch.Generator().manual_seed(V))
    z[1, 6] = z[2, 7] = value
    for h in (1.0, 2.0):
        alone(make(z, random_ids(4, V, 3, lo=9), dtype, False, h=h), (0, 3))


def alone(d, good):
    losses, grads, _ = run(d)
    r = torch.zeros(len(d["z"]), dtype=torch.bool)
    r[list(good)] = True
    for x in losses:
        assert torch.isfinite(x[r]).all() and torch.isnan(x[~r]).all(), x
    for g in grads:
        assert torch.isfinite(g[r]).all() and torch.isnan(g[~r]).all(), torch.isnan(g).sum(1)


# ---------------------------------------------------------------- masks of finite values
def masked(V, values, kept):
    """A row for each value and mask: a run of columns to the end, an octet and a run, all but a few columns."""
    z = torch.randn(3 * len(values), V, generator=torch.Generator().manual_seed(V))
    for i, m in enumerate(values):
        z[3 * i, V // 3:] = m
        z[3 * i + 1, 8:16] = z[3 * i + 1, 24:V // 2] = m
        z[3 * i + 2, :kept] = z[3 * i + 2, kept + 12:] = m
    return z


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("h", [0.7, 1.0, 2.0, 3.0])
@pytest.mark.parametrize("V", [60, 511, 700, 9001, 66000, 140003])
def test_masked_by_finite_values(dtype, tail, h, V):
    """Ranges of columns at the type's lowest value and others that stand for it."""
    values = [torch.finfo(dtype).min, -1e30, -1e10, -1e9]
    kept = 24 if V == 60 else V // 2 - 6
    z = masked(V, values, kept)
    R = len(z)
    ids = torch.stack([torch.tensor([0, 1, 17]) if r % 3 < 2 else torch.tensor([kept, kept + 5, kept + 9])
                       for r in range(R)])
    losses, grads, stats = check(make(z, ids, dtype, tail, h=h))
    assert torch.isfinite(stats).all()


# ---------------------------------------------------------------- values that are not finite, beside a rest
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("ce", [False, True])
@pytest.mark.parametrize("h", [1.0, 2.0, 3.0])
@pytest.mark.parametrize("value", [INF, NAN])
def test_a_logit_that_is_not_finite_beside_a_rest(dtype, ce, h, value):
    """In a kept column, in all of them, in the target's, in others."""
    V = 700
    z = torch.randn(6, V, generator=torch.Generator().manual_seed(3))
    ids = random_ids(6, V, 3, lo=20)
    z[1, ids[1, 1]] = value
    z[2, ids[2]] = value
    z[3, 6] = z[4, 7] = value
    alone(make(z, ids, dtype, True, ce, h), (0, 5))


# ---------------------------------------------------------------- a rest without any value
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("h", [1.0, 2.0, 3.0])
@pytest.mark.parametrize("level", [-100.0, -600.0, 100.0])
def test_every_column_that_is_not_kept_is_masked(dtype, h, level):
    """By -inf: their gradient is 0.  What of p is kept sums to 1, so that no mass is left for the rest."""
    V = 700
    z = torch.full((4, V), -INF)
    ids = random_ids(4, V, 3)
    for r in range(4):
        z[r, ids[r]] = level + torch.randn(3, generator=torch.Generator().manual_seed(r))
    d = make(z, ids, dtype, True, h=h)
    d["lse"] = (torch.logsumexp(d["top"].double() / h, 1) - 0.01).float()
    _, grads, _ = check(d)
    for g in grads:
        assert (g[torch.isinf(d["z"])] == 0).all()


# ---------------------------------------------------------------- rows whose logits are all far
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("V,h", [(301, 1.0), (700, 2.0), (5003, 0.7), (40000, 3.0)])
def test_far_rows(dtype, tail, V, h):
    """A row is as exact far from 0 as near it, also by the backward alone, whose statistics have 24 bits."""
    gen = torch.Generator().manual_seed(V)
    step = 128.0 if dtype == BF else 1.0
    z = torch.stack([at + step * torch.randn(V, generator=gen).round() for at in (2e4, -2e4, 500.0, -1500.0)])
    check(make(z, random_ids(4, V, 3), dtype, tail, h=h))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("V,h", [(60, 1.0), (700, 2.0), (700, 0.7), (9001, 1.0), (40000, 3.0)])
def test_rows_whose_mask_leaves_nothing(dtype, tail, V, h):
    """Every column at one far value: all are alike."""
    low = torch.finfo(dtype).min
    z = torch.stack([torch.full((V,), x) for x in (low, -1e30, -1e9, -3000.0, 1e20, -low)])
    check(make(z, random_ids(6, V, 3), dtype, tail, h=h))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("h", [0.7, 1.0, 2.0, 3.0])
@pytest.mark.parametrize("V", [60, 700, 9001])
def test_a_rest_whose_mask_leaves_nothing(dtype, h, V):
    """All but the kept columns at one far value: the rest's part of the gradient is spread over them alike."""
    low = torch.finfo(dtype).min
    ids = random_ids(4, V, 3)
    z = torch.stack([torch.full((V,), x) for x in (low, -1e30, -1e9, -3000.0)])
    for r in range(4):
        z[r, ids[r]] = torch.randn(3, generator=torch.Generator().manual_seed(r))
    check(make(z, ids, dtype, True, h=h))


# ---------------------------------------------------------------- the teacher's values
@pytest.mark.parametrize("tail", [False, True])
def test_a_teacher_that_is_not_finite_makes_its_row_nan(tail):
    """NaN and +inf among the kept logits or as their logsumexp; entries that are not used are not looked at."""
    V = 300
    z, ids = torch.randn(9, V, generator=torch.Generator().manual_seed(1)), random_ids(9, V, 3)
    d = make(z, ids, F32, tail)
    clean = run(d)
    d["top"][1, 0], d["top"][2, 2] = NAN, INF
    d["top"][3] = NAN
    d["ids"][5, 1] = -1
    plain = run(d)
    d["top"][5, 1] = NAN
    bad = [1, 2, 3]
    if tail:
        d["lse"][6], d["lse"][7], d["lse"][8] = NAN, INF, -INF
        bad += [6, 7, 8]
    good = [r for r in range(9) if r not in bad]
    alone(d, good)
    got = run(d)
    for x, y, p in zip((*got[0], *got[1]), (*clean[0], *clean[1]), (*plain[0], *plain[1])):
        keep = [r for r in good if r != 5]
        assert torch.equal(x[keep], y[keep]) and torch.equal(x[5], p[5])


# ---------------------------------------------------------------- many rows
@pytest.mark.parametrize("dtype,V,h", [(BF, 131075, 2.0), (F32, 70001, 1.0)])
def test_many_rows_of_a_wide_vocabulary(dtype, V, h):
    """More rows than compute units, whose long rows go by fewer threads each; masked columns among them."""
    z = torch.randn(4, V, generator=torch.Generator().manual_seed(V))
    ids = random_ids(4, V, 3)
    z[1, :V // 2] = torch.finfo(dtype).min
    z[1, ids[1]] = 1.0
    d = make(z, ids, dtype, True, h=h)
    loss, _, _ = reference(d)
    x = {n: d[n].cuda().repeat(100, *[1] * (d[n].dim() - 1)) for n in ("z", "ids", "top", "lse", "targets")}
    got, stats = api.distill_fwd(x["z"], x["ids"], x["top"], teacher_lse=x["lse"], targets=x["targets"], **d["kw"])
    got, stats = got.view(100, 4).cpu(), stats.view(100, 4, 4).cpu()
    assert (got == got[0]).all() and (stats == stats[0]).all() and torch.isfinite(stats).all()
    assert ((got[0].double() - loss).abs() <= 2.0 ** -14 + 2.0 ** -23 * loss.abs()).all()


# ---------------------------------------------------------------- the largest sizes
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("off", [0, 1])
def test_the_largest_vocabulary(dtype, tail, off):
    """2^20 columns, the row at any address, 256 kept of which some come twice."""
    V, K = 1 << 20, 256
    z = torch.randn(1, V, generator=torch.Generator().manual_seed(5))
    ids = random_ids(1, V, K)
    ids[0, 100:110], ids[0, 3] = ids[0, 50], V - 1
    d = make(z, ids, dtype, tail, h=2.0)
    loss, dz, mag = reference(d)
    box = torch.zeros(V + 8, dtype=dtype, device="cuda")
    x = box[off:off + V].view(1, V)
    x.copy_(d["z"])
    kw = dict(teacher_lse=None if d["lse"] is None else d["lse"].cuda(), targets=d["targets"].cuda(), **d["kw"])
    a = x, d["ids"].cuda(), d["top"].cuda()
    got, stats = api.distill_fwd(*a, **kw)
    w = d["d_loss"].cuda()
    both, g = api.distill_fwd_bwd(*a, w, **kw)
    back = api.distill_bwd(*a, stats, w, out=x, **kw)
    for v in (got, both):
        assert ((v.double().cpu() - loss).abs() <= 2.0 ** -14 + 2.0 ** -23 * loss.abs()).all()
    for v in (g, back):
        tol = 2.0 ** -14 * mag + (2.0 ** -8 * dz.abs() if dtype == BF else 0) + 1e-36
        assert ((v.double().cpu() - dz).abs() <= tol).all()
    assert (box[:off] == 0).all() and (box[off + V:] == 0).all()


def test_more_rows_than_a_launch_has():
    """2^26 rows of two columns: the rows of the second launch come out as alone."""
    R = (1 << 26) + 70
    gen = torch.Generator(device="cuda").manual_seed(6)
    z = torch.randn(R, 2, generator=gen, device="cuda")
    ids = torch.randint(2, (R, 1), generator=gen, device="cuda").int()
    top, targets = torch.randn(R, 1, generator=gen, device="cuda"), torch.randint(2, (R,), generator=gen, device="cuda")
    loss, g = api.distill_fwd_bwd(z, ids, top, targets=targets, ce_weight=0.5)
    end = [t[-100:].contiguous() for t in (z, ids, top)]
    l1, g1 = api.distill_fwd_bwd(*end, targets=targets[-100:].contiguous(), ce_weight=0.5)
    assert torch.equal(loss[-100:], l1) and torch.equal(g[-100:], g1)
    want = -torch.log_softmax(z[::4096].double(), 1)
    want = want.gather(1, ids[::4096].long()) + 0.5 * want.gather(1, targets[::4096, None])
    assert ((loss[::4096, None].double() - want).abs() <= 2.0 ** -14 + 2.0 ** -23 * want.abs()).all()


# ---------------------------------------------------------------- the ends of the temperature
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tail,h", [(False, 1e-29), (False, 1e-12), (False, 1e-3), (False, 1e3), (False, 1e12),
                                    (False, 9e29), (True, 1e-3), (True, 1e3), (True, 1e12), (True, 9e29)])
def test_cold_and_hot(dtype, tail, h):
    """From one-hot distributions to uniform ones.  (Not a given logsumexp of cold ones: it is fp32, and at 1e12 half a
    step of it is 2^15, so that the p that it stands for are e^(2^15).)"""
    z = torch.randn(4, 700, generator=torch.Generator().manual_seed(9))
    d = make(z, random_ids(4, 700, 3), dtype, tail, h=h)
    d["top"] = d["top"] + torch.tensor([0.0, 5.0, -3.0])
    if tail:   # the logsumexp of the kept, which have nearly all of the mass
        d["lse"] = (torch.logsumexp(d["top"].double() / float(torch.tensor(h)), 1) + 2.0 ** -6).float()
        d["lse"] = torch.maximum(d["lse"], (d["top"].amax(1).double() / float(torch.tensor(h))).float())
    check(d)
