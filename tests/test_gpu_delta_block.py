"""The operators that train gated-delta-rule blocks, run together: by themselves in fp32, and as
examples/linear_block.py uses them.

Tolerances.  By themselves: chunk_fwd and chunk_grad in fp32 accumulate at most 64 products of a chunk and 128 channels
a step, a few 2^-24 each, so that a gradient's values are off by far less than 2^-13 of the largest of their row (the
bound that chunk_grad alone is held to is 2^-16 of the sum of its terms); the losses by 2^-20 of their terms, which are
logits of size 8 and their logarithms.  The model: a gradient against torch's own differentiation in fp64 passes at
most 20 bf16 roundings (rms 2^-9 / sqrt(3)) and 4 E4M3 checkpoints (rms about 2^-4 / sqrt(12)): sqrt(20 * 2^-19.6 + 5 *
2^-11.6) = 0.042.  A state in FP8: a state off by rms 2^-8 rounds to the next code with a chance of about 2^-4, and
that code is 2^-3 away, rms 2^-5 = 0.031.  Together 0.052, held to twice that.  The differentiation is at the
projections that the model's forward had: a first token's output is (q . k) b v, and where q . k happens to be 0.002 the
norm behind it multiplies its gradients by 500, so that rounding q and k to bf16 alone (each is off by 2^-9, their
product by 2^-9 sqrt(2 / 64) = 3e-4, a sixth of it) changes the exact gradient by that sixth.
"""
import os
import sys

import pytest
import torch

from fp8_state_qat_amd import api
from oracle import oracle as orc

import distill_ref
import grad_ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import linear_block as lb  # noqa: E402

pytestmark = pytest.mark.gpu
QDQ = api.GDN_QDQ_CHUNK | api.GDN_QDQ_WRITE


class NoQdq(lb.DeltaConfig):
    qdq = 0


def delta_inputs(gen, T, H, dk, dv):
    def rn(*shape):
        return torch.randn(shape, generator=gen)

    q, k = (torch.nn.functional.normalize(rn(T, H, dk), dim=-1) for _ in range(2))
    return q, k, rn(T, H, dv), torch.rand(T, H, generator=gen), -torch.rand(T, H, generator=gen) * 0.1


@pytest.mark.parametrize("lens,qdq,given", [((130, 1, 64), QDQ, True), ((130, 1, 64), QDQ, False),
                                            ((67, 0, 200), 0, False)])
def test_loss_to_inputs(lens, qdq, given):
    gen = torch.Generator().manual_seed(len(lens) + qdq)
    H, dk, dv, V, K = 2, 64, 64, 97, 6
    T = sum(lens)
    x = delta_inputs(gen, T, H, dk, dv)
    head = torch.randn(H * dv, V, generator=gen) / (H * dv) ** 0.5
    teacher = 3 * torch.randn(T, V, generator=gen)
    top, ids = teacher.topk(K, 1)
    targets = torch.randint(V, (T,), generator=gen)
    targets[3] = -100
    kw = dict(temperature=2.0, kd_weight=4.0, ce_weight=0.5)
    cu = torch.tensor((0, *lens)).cumsum(0).int()
    q, k, v, beta, g = (t.cuda() for t in x)
    bounds = torch.tensor([0] + [-(-n // 64) for n in lens]).cumsum(0).int().cuda()
    debug = {"bound_offsets": bounds, "bound_post": torch.empty(int(bounds[-1]), H, dv, dk, device="cuda")}
    o, _ = api.chunk_fwd(q, k, v, beta, g, cu.cuda(), qdq_flags=qdq, debug=debug)
    logits = o.view(T, -1) @ head.cuda()
    lse = (teacher / 2).logsumexp(1)
    d_loss = torch.full((T,), 1 / T, device="cuda")
    loss, d = api.distill_fwd_bwd(logits, ids.int().cuda(), top.cuda(), d_loss, teacher_lse=lse.cuda(),
                                  targets=targets.cuda(), out=logits, **kw)
    got = api.chunk_grad(q, k, v, beta, g, cu.cuda(), (d @ head.cuda().t()).view_as(v), qdq_flags=qdq,
                         states=debug["bound_post"] if given else None, check_status=True)

    states = debug["bound_post"].cpu() if qdq else None
    ref_o = torch.zeros(T, H, dv, dtype=torch.float64)
    at = 0
    for a, b in zip(cu[:-1].tolist(), cu[1:].tolist()):
        def every(t, S, at=at):
            return states[at + t // 64 - 1].double() if states is not None and t % 64 == 0 else S
        zero = torch.zeros(H, dv, dk, dtype=torch.float64)
        ref_o[a:b] = grad_ref.forward(*(t[a:b].double() for t in x), zero, every)[0]
        at += -(-(b - a) // 64)
    z = ref_o.view(T, -1) @ head.double()
    want_loss, _, dz = distill_ref.grads(z, ids, top, d_loss, lse=lse, targets=targets, h=2.0, kd_weight=4.0,
                                         ce_weight=0.5)
    want = grad_ref.grad(*x, cu, (dz @ head.double().t()).view(T, H, dv), states=states)
    assert (loss.cpu().double() - want_loss).abs().max() < 2.0 ** -20 * 64
    for name, a, b in zip(("dq", "dk", "dv", "dbeta", "dg", "dS0"), got, want):
        tol = 2.0 ** -13 * b.abs().amax(tuple(range(1, b.dim())), keepdim=True) + 2.0 ** -20 * b.abs().max()
        assert ((a.cpu().double() - b).abs() <= tol).all(), name


def plain_logits(cfg, p, tokens, cu, saved):
    """The delta-rule model in p's dtype, token by token, by torch operations; the projections' values are those that
    forward saved, and they and the state's quantization are straight-through."""
    def at(t, value):
        return t + (value.double().cpu().view_as(t) - t.detach())

    def rms(t):
        return t / (t.pow(2).mean(-1, keepdim=True) + cfg.eps).sqrt()

    def unit(t):
        return t / (t.norm(dim=-1, keepdim=True) + 1e-3)

    x = p["embed"][tokens]
    h = rms(x) * p["norm0"]
    for i in range(cfg.layers):
        q, k, v, z = (at(t.reshape(len(tokens), cfg.heads, -1), s)
                      for t, s in zip((h @ p[f"in{i}"]).split(cfg.widths, 1), saved[1 + i]))
        q, k = at(unit(q), saved[1 + i][-1][0]), at(unit(k), saved[1 + i][-1][2])
        g = torch.nn.functional.logsigmoid(h @ p[f"gate{i}"] + 3)
        beta = torch.sigmoid(h @ p[f"beta{i}"])
        o = []
        for a, b in zip(cu[:-1], cu[1:]):
            S = torch.zeros(cfg.heads, cfg.dv, cfg.dk, dtype=x.dtype)
            for t in range(a, b):
                if cfg.qdq and t > a and (t - a) % 64 == 0:
                    S = S + (torch.from_numpy(orc.qdq_states(S.detach().float().numpy())[0]).double() - S.detach())
                S = S * g[t].exp()[:, None, None]
                e = v[t] - (S @ k[t][:, :, None])[..., 0]
                S = S + (beta[t][:, None] * e)[:, :, None] * k[t][:, None, :]
                o.append((S @ q[t][:, :, None])[..., 0])
        y = rms(torch.stack(o)) * p[f"head_norm{i}"] * torch.nn.functional.silu(z)
        x = x + cfg.res_scale * rms(y.flatten(1) @ p[f"out{i}"]) * p[f"post{i}"]
        h = rms(x) * p[f"pre{i}"]
    return h @ p["head"]


@pytest.mark.parametrize("cfg", [NoQdq(), lb.DeltaConfig()], ids=("fp32 state", "fp8 state"))
def test_model_gradients(cfg):
    p = lb.init_params(cfg, seed=3)
    tokens, targets, cu = lb.batch(cfg, (70, 1, 33), torch.Generator().manual_seed(4))
    teacher = lb.best(2 * torch.randn(len(tokens), cfg.vocab, generator=torch.Generator().manual_seed(5)).cuda())
    saved = []
    logits, _ = lb.forward(cfg, p, tokens, cu, saved)
    loss, d = lb.distill_and_grad(logits.to(torch.bfloat16), *teacher, targets)
    got = lb.backward(cfg, p, tokens, cu, saved, d)
    ref = {n: t.double().cpu().requires_grad_() for n, t in p.items()}
    out = plain_logits(cfg, ref, tokens.cpu(), cu.tolist(), saved)
    top, ids, lse = (t.cpu() for t in teacher)
    want, _ = distill_ref.losses(out, ids, top, lse=lse, targets=targets.cpu(), h=2.0, kd_weight=4.0, ce_weight=0.5)
    want.mean().backward()
    assert abs(loss.item() - want.mean().item()) < 2.0 ** -5 * want.mean().item()
    assert sorted(got) == sorted(ref)
    for n, t in ref.items():
        err = (got[n].double().cpu() - t.grad).norm() / t.grad.norm()
        assert err < 0.105, (n, float(err))


def test_distilled_student_decodes():
    big, cfg = lb.Config(), lb.DeltaConfig()
    student, losses = lb.train(cfg, 4, seed=1, teacher=(big, lb.init_params(big)))
    assert all(x == x and abs(x) < 100 for x in losses)
    gen = torch.Generator().manual_seed(5)
    prompts = [lb.batch(cfg, [n], gen)[0] for n in (9, 70, 1)]
    assert torch.isfinite(lb.generate(cfg, student, prompts, 6)[1]).all()
    # without the state's quantization decoding is the packed form, with at most 16 other bf16 roundings a layer
    tokens, logits = lb.generate(NoQdq(), student, prompts, 6)
    for s, t, got in zip(prompts, tokens, logits):
        full = torch.cat([s, t[:-1]])
        cu = torch.tensor([0, len(full)], dtype=torch.int32, device="cuda")
        want = lb.forward(NoQdq(), student, full, cu)[0][len(s) - 1:]
        assert (got - want).abs().max() < 2.0 ** -5.3 * want.abs().max()
