"""A small language model of linear-attention blocks, trained and then decoded.

Shows the block's operators together, as a training loop and a server use them:

  training   lin_attn_fwd / lin_attn_bwd over packed sequences, the gated norm
             of every head's output and the norms around each block
             (block_norm_fwd / block_norm_bwd), activations kept in 8 bits
             between forward and backward (act_pack, checkpoint=True), but for
             what the decays' gradients come from: their terms cancel
  serving    lin_attn_fwd on the prompt, lin_attn_step for every next token

One block, on the residual stream x [T, D] (fp32) and its norm h (bf16):

    q, k, v, z = h W_in          g = log sigmoid(h w_gate + 3)
    o = linear attention(q, k, v, g)
    y = rmsnorm(o) a(z)          per head
    x, h = norm after, residual, norm before the next block (y W_out, x)

    python examples/linear_block.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from fp8_state_qat_amd import api  # noqa: E402

BF16 = torch.bfloat16


class Config:
    vocab, cols, layers = 64, 256, 2
    heads, qk_heads, dk, dv = 4, 2, 64, 64
    res_scale, eps = 1.0, 1e-6

    @property
    def widths(self):
        """Columns of q, k, v and the output gate z in W_in."""
        return [self.qk_heads * self.dk] * 2 + [self.heads * self.dv] * 2


def init_params(cfg, seed=0, device="cuda"):
    gen = torch.Generator().manual_seed(seed)

    def rn(*shape):
        return (torch.randn(shape, generator=gen) / shape[0] ** 0.5).to(device)

    p = {"embed": rn(cfg.vocab, cfg.cols) * cfg.vocab ** 0.5, "head": rn(cfg.cols, cfg.vocab),
         "norm0": torch.ones(cfg.cols, device=device)}
    for i in range(cfg.layers):
        p[f"in{i}"] = rn(cfg.cols, sum(cfg.widths))
        p[f"gate{i}"] = rn(cfg.cols, cfg.heads)
        p[f"out{i}"] = rn(cfg.heads * cfg.dv, cfg.cols)
        p[f"head_norm{i}"] = torch.ones(cfg.dv, device=device)
        p[f"post{i}"] = torch.ones(cfg.cols, device=device)
        p[f"pre{i}"] = torch.ones(cfg.cols, device=device)
    return p


def _mm(a, w):
    return a @ w.to(BF16)


def _first_norm(cfg, p, x):
    """The norm before the first block: the embedding's rows are the whole x."""
    return api.block_norm_fwd(x.to(BF16), p["norm0"], eps=cfg.eps)[0]


def _split(cfg, h, p, i):
    T = h.shape[0]
    q, k, v, z = (t.contiguous() for t in _mm(h, p[f"in{i}"]).split(cfg.widths, 1))
    g = torch.nn.functional.logsigmoid(h.float() @ p[f"gate{i}"] + 3)
    return (q.view(T, cfg.qk_heads, cfg.dk), k.view(T, cfg.qk_heads, cfg.dk), v.view(T, cfg.heads, cfg.dv),
            z.view(T, cfg.heads, cfg.dv), g)


def forward(cfg, p, tokens, cu, saved=None):
    """Logits of packed sequences and the blocks' states; with `saved` (a
    list) what the backward needs is appended to it."""
    x = p["embed"][tokens].float()
    h = _first_norm(cfg, p, x)
    if saved is not None:
        saved.append(x.to(BF16))
    states = []
    for i in range(cfg.layers):
        q, k, v, z, g = _split(cfg, h, p, i)
        o, state = api.lin_attn_fwd(q, k, v, g, cu)
        states.append(state)
        y, _ = api.block_norm_fwd(o, p[f"head_norm{i}"], gate=z, eps=cfg.eps)
        f = _mm(y.view(len(tokens), -1), p[f"out{i}"])
        h8 = api.act_pack(h)
        x, h, f8, _ = api.block_norm_fwd(f, p[f"post{i}"], residual=x, w_pre=p[f"pre{i}"], res_scale=cfg.res_scale,
                                         eps=cfg.eps, checkpoint=True)
        if saved is not None:
            saved.append((q, k, v, z, g, o, h8, api.act_pack(y), f8, x))
    if saved is not None:
        saved.append(api.act_pack(h))
    return _mm(h, p["head"]).float(), states


def backward(cfg, p, tokens, cu, saved, d_logits):
    """Gradients of all parameters from those of the logits."""
    grads = {}
    d_logits = d_logits.to(BF16)

    def into(name, act8, d_out):
        """Weight gradient from an 8-bit activation, and the gradient of that activation."""
        grads[name] = (api.act_unpack(*act8).view(len(tokens), -1).t() @ d_out).float()
        return d_out @ p[name].to(BF16).t()

    d_h = into("head", saved[-1], d_logits)
    d_x = torch.zeros(len(tokens), cfg.cols, device=d_h.device)
    for i in reversed(range(cfg.layers)):
        q, k, v, z, g, o, h8, y8, f8, x = saved[1 + i]
        d_f, _, d_x, grads[f"post{i}"], grads[f"pre{i}"] = api.block_norm_bwd(
            f8, p[f"post{i}"], d_x, d_h=d_h, x=x, w_pre=p[f"pre{i}"], res_scale=cfg.res_scale, eps=cfg.eps)
        d_y = into(f"out{i}", y8, d_f).view_as(v)
        d_o, d_z, _, grads[f"head_norm{i}"], _ = api.block_norm_bwd(o, p[f"head_norm{i}"], d_y, gate=z, eps=cfg.eps,
                                                                    want_residual=False)
        d_q, d_k, d_v, d_g, _ = api.lin_attn_bwd(q, k, v, g, cu, d_o)
        d_in = torch.cat([t.flatten(1) for t in (d_q, d_k, d_v, d_z)], 1)
        d_s = d_g * -torch.expm1(g)                     # d log sigmoid(s) = 1 - sigmoid(s) = 1 - e^g
        d_h = into(f"in{i}", h8, d_in)
        grads[f"gate{i}"] = api.act_unpack(*h8, dtype=torch.float32).t() @ d_s
        d_h = (d_h.float() + d_s @ p[f"gate{i}"].t()).to(BF16)
    d_e, _, _, grads["norm0"], _ = api.block_norm_bwd(saved[0], p["norm0"], d_h, eps=cfg.eps, want_residual=False)
    grads["embed"] = torch.zeros_like(p["embed"]).index_add_(0, tokens, d_x + d_e.float())
    return grads


def loss_and_grad(logits, targets):
    """Mean cross entropy and its gradient, in fp32."""
    logp = logits - logits.logsumexp(1, keepdim=True)
    d = logp.exp()
    d[torch.arange(len(targets), device=d.device), targets] -= 1
    return -logp.gather(1, targets[:, None]).mean(), d / len(targets)


def batch(cfg, lens, gen, device="cuda"):
    """Packed sequences from random first tokens, each next one by a fixed
    random permutation of the vocabulary."""
    after = torch.randperm(cfg.vocab, generator=torch.Generator().manual_seed(0))
    tokens, targets, cu = [], [], [0]
    for n in lens:
        s = [int(torch.randint(cfg.vocab, (1,), generator=gen))]
        while len(s) <= n:
            s.append(int(after[s[-1]]))
        tokens += s[:-1]
        targets += s[1:]
        cu.append(cu[-1] + n)
    return tuple(torch.tensor(t, dtype=d, device=device)
                 for t, d in ((tokens, torch.int64), (targets, torch.int64), (cu, torch.int32)))


def train(cfg, steps, seed=0, lens=(100, 64, 1, 163, 40, 144), lr=3e-3):
    p = init_params(cfg, seed)
    for t in p.values():
        t.grad = torch.zeros_like(t)
    opt = torch.optim.Adam(p.values(), lr=lr)
    gen = torch.Generator().manual_seed(seed + 1)
    losses = []
    for _ in range(steps):
        tokens, targets, cu = batch(cfg, lens, gen)
        saved = []
        logits, _ = forward(cfg, p, tokens, cu, saved)
        loss, d_logits = loss_and_grad(logits, targets)
        for n, g in backward(cfg, p, tokens, cu, saved, d_logits).items():
            p[n].grad.copy_(g)
        opt.step()
        losses.append(loss.item())
    return p, losses


def step(cfg, p, token, states):
    """Logits of one next token for each sequence; the states move on in place."""
    x = p["embed"][token].float()
    h = _first_norm(cfg, p, x)
    for i in range(cfg.layers):
        q, k, v, z, g = _split(cfg, h, p, i)
        o = api.lin_attn_step(q, k, v, g, states[i])
        y, _ = api.block_norm_fwd(o, p[f"head_norm{i}"], gate=z, eps=cfg.eps)
        f = _mm(y.view(len(token), -1), p[f"out{i}"])
        x, h = api.block_norm_fwd(f, p[f"post{i}"], residual=x, w_pre=p[f"pre{i}"], res_scale=cfg.res_scale,
                                  eps=cfg.eps)
    return _mm(h, p["head"]).float()


def generate(cfg, p, prompts, n):
    """n greedy tokens after each prompt (a list of 1-D tensors); also every
    step's logits."""
    cu = torch.tensor([0] + [len(s) for s in prompts], device="cuda").cumsum(0).int()
    logits, states = forward(cfg, p, torch.cat(prompts), cu)
    logits = [logits[cu[1:].long() - 1]]
    out = [logits[0].argmax(1)]
    for _ in range(n - 1):
        logits.append(step(cfg, p, out[-1], states))
        out.append(logits[-1].argmax(1))
    return torch.stack(out, 1), torch.stack(logits, 1)


def main():
    cfg = Config()
    p, losses = train(cfg, int(sys.argv[1]) if len(sys.argv) > 1 else 100)
    for i in range(0, len(losses), 10):
        print(f"step {i:4d}  loss {losses[i]:.3f}")
    gen = torch.Generator().manual_seed(7)
    prompts = [batch(cfg, [n], gen)[0] for n in (9, 70)]
    tokens, _ = generate(cfg, p, prompts, 8)
    for s, t in zip(prompts, tokens):
        print("prompt of", len(s), "ending in", s[-3:].tolist(), "goes on", t.tolist())


if __name__ == "__main__":
    main()
