"""Distillation on the GPU against its definition in 64 bits.

Tolerances.  A sum of a row's exponentials has at most 128 terms a thread for each run of the row and 16 tree steps;
these sizes have at most two runs, and an exponential is off by 2^-23 of itself and |x| 2^-23 for its argument's
rounding, where e^x is not below 2^-24 of the sum |x| < 17: (256 + 16) 2^-24 + 18 * 2^-23 < 2^-15.  So a logsumexp is
within 2^-15 + 2^-23 of its magnitude, a loss within (kd_weight + ce_weight) (2^-14 + 2^-22 max |z / h|), and a
probability within 2^-15 + 2^-23 |logsumexp| + |y| 2^-23 of itself, for arguments y up to -100: 2^-14 of it.  A
gradient's value is a sum of at most four such terms, rounded once: 2^-14 of their magnitudes' sum, with bf16 2^-8 of
the value more.
"""
import pytest
import torch

import distill_ref as ref
from fp8_state_qat_amd import api

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def make(R, V, K, dtype, tail=False, ce=True, h=1.0, seed=0, scale=2.0):
    gen = torch.Generator().manual_seed(seed)
    teacher = scale * torch.randn(R, V, generator=gen)
    d = dict(z=(0.8 * teacher + torch.randn(R, V, generator=gen)).to(dtype))
    top, ids = teacher.topk(K, dim=1)
    d["ids"], d["top"] = ids.int(), top
    for r in range(1, R, 3):                      # some teachers kept fewer, in any place
        d["ids"][r, torch.randperm(K, generator=gen)[:K // 2]] = -1
    d["lse"] = torch.logsumexp(teacher.double() / h, 1).float() if tail else None
    d["targets"] = None
    if ce:
        d["targets"] = torch.randint(V, (R,), generator=gen)
        if K:
            d["targets"][::2] = ids[::2, 0]
        if R > 2:
            d["targets"][2] = -100
    d["d_loss"] = torch.rand(R, generator=gen) - 0.3
    d["kw"] = dict(temperature=h, kd_weight=0.75, ce_weight=0.25 if ce else 0.0)
    return d


def kwargs(d):
    return dict(teacher_lse=None if d["lse"] is None else d["lse"].cuda(),
                targets=None if d["targets"] is None else d["targets"].cuda(), **d["kw"])


def want(d):
    kw = d["kw"]
    return ref.grads(d["z"], d["ids"], d["top"], d["d_loss"], lse=d["lse"], targets=d["targets"], h=kw["temperature"],
                     kd_weight=kw["kd_weight"], ce_weight=kw["ce_weight"])


def magnitudes(d):
    """Of a gradient's terms: w (kd_weight / h (q + p + rest's share) + ce_weight (softmax + [target]))."""
    kw, z = d["kw"], d["z"].double()
    R, V = z.shape
    a, b = d["d_loss"].double().abs() * kw["kd_weight"] / kw["temperature"], d["d_loss"].double().abs() * kw["ce_weight"]
    m = a[:, None] * torch.softmax(z / kw["temperature"], 1) + b[:, None] * torch.softmax(z, 1)
    for r in range(R):
        on = d["ids"][r] >= 0
        t = d["top"][r].double() / kw["temperature"]
        c = d["lse"][r].double() if d["lse"] is not None else t[on].logsumexp(0)
        p = (t - c).exp() * on
        m[r].index_add_(0, d["ids"][r].clamp(min=0).long(), a[r] * p)
        if d["lse"] is not None:
            off = torch.ones(V, dtype=torch.bool)
            off[d["ids"][r][on].long()] = False
            m[r][off] += a[r] * (1 - p.sum()).clamp(min=0) * torch.softmax(z[r][off] / kw["temperature"], 0)
        if d["targets"] is not None and d["targets"][r] >= 0:
            m[r, d["targets"][r]] += b[r]
    return m


def check_grad(got, wanted, d, name):
    g = got.double().cpu()
    assert torch.isfinite(g).all(), name
    tol = 2.0 ** -14 * magnitudes(d) + (2.0 ** -8 * wanted.abs() if got.dtype == BF else 0)
    bad = (g - wanted).abs() > tol + 1e-36
    assert not bad.any(), f"{name}: {int(bad.sum())} values, worst {float(((g - wanted).abs() / (tol + 1e-36)).max()):.3g}"


def check_loss(got, wanted, d):
    kw = d["kw"]
    top = (d["z"].double().abs().amax() + d["top"].double().abs().amax() if d["top"].numel() else
           d["z"].double().abs().amax()) / min(1.0, kw["temperature"])
    tol = (kw["kd_weight"] + kw["ce_weight"]) * (2.0 ** -14 + 2.0 ** -22 * float(top))
    assert (got.double().cpu() - wanted).abs().max() <= tol


CASES = [
    # rows, vocab, kept, dtype, rest, cross entropy, temperature
    (1, 1, 1, F32, False, True, 1.0),
    (3, 2, 1, BF, True, True, 2.0),
    (4, 7, 3, F32, True, False, 1.0),
    (5, 8, 0, BF, False, True, 1.0),
    (5, 9, 8, BF, True, True, 1.0),
    (6, 63, 5, BF, False, True, 0.7),
    (3, 64, 16, F32, True, True, 2.0),
    (7, 1003, 16, BF, False, True, 1.0),
    (5, 2047, 100, BF, True, True, 3.0),
    (3, 2048, 8, F32, False, False, 2.0),
    (4, 2049, 65, BF, True, False, 1.0),
    (3, 8191, 256, F32, True, True, 2.0),
    (3, 8300, 20, BF, True, True, 2.0),
    (3, 16385, 20, F32, False, True, 1.0),
    (3, 32761, 64, BF, False, True, 2.0),
    (2, 32800, 64, BF, True, True, 1.0),
    (2, 65537, 33, F32, True, True, 1.0),
    (2, 131072, 64, BF, True, True, 2.0),
    (2, 131075, 64, BF, True, True, 2.0),
    (2, 200001, 12, BF, False, True, 2.0),
]


@pytest.mark.parametrize("R,V,K,dtype,tail,ce,h", CASES)
def test_against_64_bits(R, V, K, dtype, tail, ce, h):
    d = make(R, V, K, dtype, tail, ce, h, seed=V)
    loss, stats, dz = want(d)
    z, ids, top, w = (d[n].cuda() for n in ("z", "ids", "top", "d_loss"))
    kw = kwargs(d)
    got, st = api.distill_fwd(z, ids, top, **kw)
    check_loss(got, loss, d)
    fin = torch.isfinite(stats)
    assert torch.equal(torch.isfinite(st.cpu()), fin)
    assert ((st.double().cpu() - stats)[fin].abs() <= 2.0 ** -15 + 2.0 ** -23 * stats[fin].abs()).all()
    check_grad(api.distill_bwd(z, ids, top, st, w, **kw), dz, d, "backward")
    both, g = api.distill_fwd_bwd(z, ids, top, w, **kw)
    check_loss(both, loss, d)
    check_grad(g, dz, d, "both")
    # in place
    z1, z2 = z.clone(), z.clone()
    assert api.distill_bwd(z1, ids, top, st, w, out=z1, **kw) is z1
    assert torch.equal(z1, api.distill_bwd(z, ids, top, st, w, **kw))
    api.distill_fwd_bwd(z2, ids, top, w, out=z2, **kw)
    assert torch.equal(z2, g)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("off,wide", [(0, 130), (1, 130), (3, 131), (5, 137)])
def test_slices_of_wider_rows(dtype, off, wide):
    """Logits and gradients at any address and stride; what lies between the rows keeps its values."""
    d = make(6, 120, 9, dtype, True, True, 2.0, seed=off)
    box = torch.full((6, wide), float("nan"), dtype=dtype, device="cuda")
    z = box[:, off:off + 120]
    z.copy_(d["z"])
    out_box = torch.full((6, 140), 9.0, dtype=dtype, device="cuda")
    out = out_box[:, 7:127]
    ids, top, w = (d[n].cuda() for n in ("ids", "top", "d_loss"))
    loss, g = api.distill_fwd_bwd(z, ids, top, w, out=out, **kwargs(d))
    plain = api.distill_fwd_bwd(d["z"].cuda(), ids, top, w, **kwargs(d))
    rl, _, dz = want(d)
    check_loss(loss, rl, d)
    check_grad(g, dz, d, "slice")
    check_loss(plain[0], rl, d)
    assert (out_box[:, :7] == 9.0).all() and (out_box[:, 127:] == 9.0).all()
    assert torch.isnan(box[:, :off]).all() and torch.isnan(box[:, off + 120:]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [2101, 28700])
@pytest.mark.parametrize("off,to", [(1, 1), (2, 3), (3, 0)])
def test_slices_of_long_rows(dtype, V, off, to):
    """The same of rows that whole waves go through; with other addresses of the gradient than of the logits."""
    d = make(3, V, 17, dtype, True, True, 2.0, seed=off)
    box = torch.full((3, V + 9), float("nan"), dtype=dtype, device="cuda")
    z = box[:, off:off + V]
    z.copy_(d["z"])
    ids, top, w = (d[n].cuda() for n in ("ids", "top", "d_loss"))
    rl, _, dz = want(d)
    loss, stats = api.distill_fwd(z, ids, top, **kwargs(d))
    check_loss(loss, rl, d)
    for what in ("backward", "both"):
        out_box = torch.full((3, V + 9), 9.0, dtype=dtype, device="cuda")
        out = out_box[:, to:to + V]
        if what == "backward":
            api.distill_bwd(z, ids, top, stats, w, out=out, **kwargs(d))
        else:
            check_loss(api.distill_fwd_bwd(z, ids, top, w, out=out, **kwargs(d))[0], rl, d)
        check_grad(out, dz, d, what)
        assert (out_box[:, :to] == 9.0).all() and (out_box[:, to + V:] == 9.0).all()


@pytest.mark.parametrize("tail", [False, True])
def test_the_same_column_twice_and_every_column(tail):
    d = make(3, 40, 40, F32, tail, True, 1.0, seed=3)
    d["ids"][:] = torch.arange(40).int()
    d["ids"][0, 5:9] = 4                       # five entries of one column, four columns not kept
    d["targets"] = torch.tensor([4, 0, 7])
    d["top"] = torch.randn(3, 40, generator=torch.Generator().manual_seed(1))
    if tail:
        d["lse"] = torch.logsumexp(d["top"].double(), 1).float() + 0.01
    loss, _, dz = want(d)
    z, ids, top, w = (d[n].cuda() for n in ("z", "ids", "top", "d_loss"))
    got, st = api.distill_fwd(z, ids, top, **kwargs(d))
    check_loss(got, loss, d)
    check_grad(api.distill_bwd(z, ids, top, st, w, **kwargs(d)), dz, d, "backward")
    check_grad(api.distill_fwd_bwd(z, ids, top, w, **kwargs(d))[1], dz, d, "both")


@pytest.mark.parametrize("tail", [False, True])
def test_rows_without_kept_entries(tail):
    """No kd: the loss is the cross entropy's."""
    d = make(4, 300, 6, BF, tail, True, 2.0, seed=4)
    d["ids"][0] = -1
    d["ids"][3] = -7
    z, ids, top, w = (d[n].cuda() for n in ("z", "ids", "top", "d_loss"))
    loss, g = api.distill_fwd_bwd(z, ids, top, w, **kwargs(d))
    _, st = api.distill_fwd(z, ids, top, **kwargs(d))
    g2 = api.distill_bwd(z, ids, top, st, w, **kwargs(d))
    zz = d["z"].double()
    for r in (0, 3):
        t = int(d["targets"][r])
        ce = zz[r].logsumexp(0) - zz[r, t]
        assert abs(float(loss[r]) - 0.25 * float(ce)) < 1e-4
        e = torch.softmax(zz[r], 0)
        e[t] -= 1
        e *= 0.25 * float(d["d_loss"][r])
        for x in (g, g2):
            assert ((x[r].double().cpu() - e).abs() <= 2.0 ** -8 * e.abs() + 2.0 ** -14 * (e.abs() + 1e-9)).all()


def test_ignored_rows_are_not_read():
    d = make(5, 500, 6, BF, True, True, 2.0, seed=5)
    d["targets"] = torch.tensor([3, -100, 4, -100, 5])
    clean = api.distill_fwd_bwd(*(d[n].cuda() for n in ("z", "ids", "top", "d_loss")), **kwargs(d))
    d["z"][1] = float("nan")
    d["z"][3, 7] = float("inf")
    d["lse"][1] = float("nan")
    d["d_loss"][3] = float("nan")
    d["ids"][3] = 100000
    args = [d[n].cuda() for n in ("z", "ids", "top", "d_loss")]
    loss, g = api.distill_fwd_bwd(*args, **kwargs(d))
    assert torch.equal(loss, clean[0]) and torch.equal(g, clean[1])
    assert (loss[[1, 3]] == 0).all() and (g[[1, 3]] == 0).all()
    l2, st = api.distill_fwd(*args[:3], **kwargs(d))
    assert (l2[[1, 3]] == 0).all() and (st[[1, 3]] == 0).all()
    g2 = api.distill_bwd(*args[:3], st, args[3], **kwargs(d))
    assert (g2[[1, 3]] == 0).all() and torch.isfinite(g2).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tail", [False, True])
def test_masked_and_extreme_logits(dtype, tail):
    """-inf and the type's lowest value in columns that are neither kept nor targets; a rest far below the kept
    columns; a kept column of -inf."""
    d = make(5, 700, 5, dtype, tail, True, 1.0, seed=6)
    d["targets"] = d["ids"][:, 0].clamp(min=0).long()
    used = [set(d["ids"][r].tolist()) | {int(d["targets"][r])} for r in range(5)]
    for c in range(0, 700, 3):
        if c not in used[0]:
            d["z"][0, c] = float("-inf")
        if c not in used[1]:
            d["z"][1, c] = torch.finfo(dtype).min
    for c in range(700):
        if c not in used[2]:
            d["z"][2, c] -= 150                    # e^-150 of the kept columns' mass
    loss, _, dz = want(d)
    z, ids, top, w = (d[n].cuda() for n in ("z", "ids", "top", "d_loss"))
    got, st = api.distill_fwd(z, ids, top, **kwargs(d))
    check_loss(got[:4], loss[:4], d if not tail else dict(d, kw=dict(d["kw"], kd_weight=2.0)))
    for g in (api.distill_bwd(z, ids, top, st, w, **kwargs(d)), api.distill_fwd_bwd(z, ids, top, w, **kwargs(d))[1]):
        check_grad(g, dz, d, "masked")
        if dtype == BF:
            assert (g[0][torch.isinf(z[0])] == 0).all()
    z2 = z.clone()
    z2[3, int(d["ids"][3, 0])] = float("-inf")
    got, _ = api.distill_fwd(z2, ids, top, **kwargs(d))
    assert got[3] == float("inf") and torch.isfinite(got[[0, 1, 2, 4]]).all()


def test_rows_out_of_contract_are_nan_and_alone():
    d = make(6, 333, 4, F32, True, True, 2.0, seed=7)
    d["targets"] = torch.tensor([1, 333, -1, 2, 3, 4])
    d["ids"][3, 2] = 333
    d["ids"][4, 1] = 1 << 30
    d["z"][5, 9] = float("nan")
    args = [d[n].cuda() for n in ("z", "ids", "top", "d_loss")]
    loss, st = api.distill_fwd(*args[:3], **kwargs(d))
    both, g = api.distill_fwd_bwd(*args, **kwargs(d))
    g2 = api.distill_bwd(*args[:3], st, args[3], **kwargs(d))
    for x in (loss, both):
        assert torch.isfinite(x[0]) and torch.isnan(x[1:]).all()
    for x in (g, g2):
        assert torch.isfinite(x[0]).all() and torch.isnan(x[1:]).all()


def test_without_weights_and_defaults():
    d = make(4, 100, 5, F32, False, False, 1.0, seed=8)
    args = [d[n].cuda() for n in ("z", "ids", "top")]
    d["d_loss"] = torch.ones(4)
    d["kw"] = dict(temperature=1.0, kd_weight=1.0, ce_weight=0.0)
    loss, _, dz = want(d)
    got, st = api.distill_fwd(*args)
    check_loss(got, loss, d)
    check_grad(api.distill_bwd(*args, st), dz, d, "backward")
    check_grad(api.distill_fwd_bwd(*args)[1], dz, d, "both")


def test_no_rows():
    e = torch.empty
    z, ids, top = e(0, 50, device="cuda"), e(0, 4, dtype=torch.int32, device="cuda"), e(0, 4, device="cuda")
    loss, st = api.distill_fwd(z, ids, top)
    assert loss.shape == (0,) and st.shape == (0, 4)
    assert api.distill_bwd(z, ids, top, st).shape == (0, 50) and api.distill_fwd_bwd(z, ids, top)[1].shape == (0, 50)


def test_repeats_bit_for_bit_on_streams_and_in_graphs():
    d = make(40, 5000, 32, BF, True, True, 2.0, seed=9)
    args, kw = [d[n].cuda() for n in ("z", "ids", "top", "d_loss")], kwargs(d)
    first = api.distill_fwd_bwd(*args, **kw)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        other = api.distill_fwd_bwd(*args, **kw)
    again = api.distill_fwd_bwd(*args, **kw)
    torch.cuda.synchronize()
    for x in (other, again):
        assert torch.equal(x[0], first[0]) and torch.equal(x[1], first[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, st = api.distill_fwd(*args[:3], **kw)
        g = api.distill_bwd(*args[:3], st, args[3], **kw)
    for i in range(3):
        fresh = make(40, 5000, 32, BF, True, True, 2.0, seed=30 + i)
        for t, n in zip(args, ("z", "ids", "top", "d_loss")):
            t.copy_(fresh[n])
        kw["teacher_lse"].copy_(fresh["lse"])
        kw["targets"].copy_(fresh["targets"])
        graph.replay()
        torch.cuda.synchronize()
        e1, est = api.distill_fwd(*args[:3], **kw)
        assert torch.equal(loss, e1) and torch.equal(g, api.distill_bwd(*args[:3], est, args[3], **kw))


def test_offsets_past_32_bits():
    """Rows whose byte and element offsets pass 2^32 come out as alone."""
    R, V, K = 40_000, 120_000, 4
    z = torch.empty(R, V, dtype=BF, device="cuda").normal_()
    gen = torch.Generator().manual_seed(0)
    ids = torch.randint(V, (R, K), generator=gen).int().cuda()
    top = torch.randn(R, K, generator=gen).cuda()
    loss, g = api.distill_fwd_bwd(z, ids, top)
    l1, g1 = api.distill_fwd_bwd(z[-3:].contiguous(), ids[-3:].contiguous(), top[-3:].contiguous())
    assert torch.equal(loss[-3:], l1) and torch.equal(g[-3:], g1)
    assert torch.isfinite(loss).all()
