"""examples/linear_block.py: the block's operators run together.

Tolerances.  Gradients against torch's own differentiation of the same model
in fp64.  A bf16 rounding is off by at most 2^-8 / 2 (rms 2^-9 / sqrt(3)) of a
value, an E4M3 checkpoint by at most 2^-4 (rms about 2^-4 / sqrt(12)); a
gradient passes at most 16 bf16 roundings and 4 checkpoints (h, y, f, and o
with z) whose errors are independent, so its relative L2 error is expected
below sqrt(16 * 2^-19.6 + 5 * 2^-11.6) = 0.04; held to twice that.  Decoding
against the packed form: the same model with other roundings of the state
products, at most 16 bf16 roundings a layer: rms 2^-9.8 sqrt(32) of the
logits' size, held to 4 times that (2^-5.3) for the largest of them.
"""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import linear_block as lb  # noqa: E402

pytestmark = pytest.mark.gpu


def plain_logits(cfg, p, tokens, cu):
    """The model in p's dtype, token by token, by torch operations."""
    def rms(t):
        return t / (t.pow(2).mean(-1, keepdim=True) + cfg.eps).sqrt()

    x = p["embed"][tokens]
    h = rms(x) * p["norm0"]
    rep = cfg.heads // cfg.qk_heads
    for i in range(cfg.layers):
        q, k, v, z = (h @ p[f"in{i}"]).split(cfg.widths, 1)
        q, k = (t.reshape(-1, cfg.qk_heads, cfg.dk).repeat_interleave(rep, 1) for t in (q, k))
        v, z = (t.reshape(-1, cfg.heads, cfg.dv) for t in (v, z))
        g = torch.nn.functional.logsigmoid(h @ p[f"gate{i}"] + 3)
        o = []
        for a, b in zip(cu[:-1], cu[1:]):
            S = torch.zeros(cfg.heads, cfg.dv, cfg.dk, dtype=x.dtype)
            for t in range(a, b):
                S = S * g[t].exp()[:, None, None] + v[t][:, :, None] * k[t][:, None, :]
                o.append((S @ q[t][:, :, None])[..., 0])
        y = rms(torch.stack(o)) * p[f"head_norm{i}"] * torch.nn.functional.silu(z)
        x = x + cfg.res_scale * rms(y.flatten(1) @ p[f"out{i}"]) * p[f"post{i}"]
        h = rms(x) * p[f"pre{i}"]
    return h @ p["head"]


def test_gradients():
    cfg = lb.Config()
    p = lb.init_params(cfg, seed=3)
    tokens, targets, cu = lb.batch(cfg, (70, 1, 33), torch.Generator().manual_seed(4))
    saved = []
    logits, _ = lb.forward(cfg, p, tokens, cu, saved)
    _, d = lb.loss_and_grad(logits, targets)
    got = lb.backward(cfg, p, tokens, cu, saved, d)
    ref = {n: t.double().cpu().requires_grad_() for n, t in p.items()}
    out = plain_logits(cfg, ref, tokens.cpu(), cu.tolist())
    torch.nn.functional.cross_entropy(out, targets.cpu()).backward()
    assert sorted(got) == sorted(ref)
    for n, t in ref.items():
        err = (got[n].double().cpu() - t.grad).norm() / t.grad.norm()
        assert err < 0.08, (n, float(err))


def test_training_and_decoding():
    cfg = lb.Config()
    p, losses = lb.train(cfg, 60)
    assert losses[-1] < 0.6 * losses[0]
    gen = torch.Generator().manual_seed(5)
    prompts = [lb.batch(cfg, [n], gen)[0] for n in (9, 70, 1)]
    tokens, logits = lb.generate(cfg, p, prompts, 6)
    for s, t, got in zip(prompts, tokens, logits):
        full = torch.cat([s, t[:-1]])
        cu = torch.tensor([0, len(full)], dtype=torch.int32, device="cuda")
        want = lb.forward(cfg, p, full, cu)[0][len(s) - 1:]
        assert (got - want).abs().max() < 2.0 ** -5.3 * want.abs().max()
