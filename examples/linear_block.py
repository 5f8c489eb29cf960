"""A small language model of linear-attention blocks, trained and then decoded,
and a student of gated-delta-rule blocks, distilled from it.

Shows the block's operators together, as a training loop and a server use them:

  training   lin_attn_fwd / lin_attn_bwd over packed sequences, the gated norm
             of every head's output and the norms around each block
             (block_norm_fwd / block_norm_bwd), activations kept in 8 bits
             between forward and backward (act_pack, checkpoint=True), but for
             what the decays' gradients come from: their terms cancel
  serving    lin_attn_fwd on the prompt, lin_attn_step for every next token

With DeltaConfig the blocks are the gated delta rule with its state in FP8:
chunk_fwd keeps the states after every chunk, chunk_grad takes them, and
decode_step writes the state in FP8 after every token.  distill() trains such a
model on another's best logits of every token (distill_fwd_bwd).

One block, on the residual stream x [T, D] (fp32) and its norm h (bf16):

    q, k, v, z = h W_in          g = log sigmoid(h w_gate + 3)
    o = linear attention(q, k, v, g)
    y = rmsnorm(o) a(z)          per head
    x, h = norm after, residual, norm before the next block (y W_out, x)

with the delta rule   b = sigmoid(h w_beta)   o = delta rule(q / |q|, k / |k|, v, b, g)

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
    delta, qdq = False, 0

    @property
    def widths(self):
        """Columns of q, k, v and the output gate z in W_in."""
        return [self.qk_heads * self.dk] * 2 + [self.heads * self.dv] * 2


class DeltaConfig(Config):
    layers, qk_heads = 1, 4
    delta, qdq = True, api.GDN_QDQ_CHUNK | api.GDN_QDQ_WRITE


def init_params(cfg, seed=0, device="cuda"):
    gen = torch.Generator().manual_seed(seed)

    def rn(*shape):
        return (torch.randn(shape, generator=gen) / shape[0] ** 0.5).to(device)

    p = {"embed": rn(cfg.vocab, cfg.cols) * cfg.vocab ** 0.5, "head": rn(cfg.cols, cfg.vocab),
         "norm0": torch.ones(cfg.cols, device=device)}
    for i in range(cfg.layers):
        p[f"in{i}"] = rn(cfg.cols, sum(cfg.widths))
        p[f"gate{i}"] = rn(cfg.cols, cfg.heads)
        if cfg.delta:
            p[f"beta{i}"] = rn(cfg.cols, cfg.heads)
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


def _unit(t):
    """Rows divided by their length, and the lengths."""
    n = t.float().norm(dim=-1, keepdim=True) + 1e-3
    return (t.float() / n).to(t.dtype), n


def _unit_bwd(u, n, d):
    """Gradient of _unit's rows from that of its result u."""
    u, d = u.float(), d.float()
    return (d / n - u * (u * d).sum(-1, keepdim=True) / (n - 1e-3).clamp_min(1e-12)).to(BF16)


def _mix(cfg, p, i, h, q, k, v, g, cu, keep):
    """The block's attention: (o, state, what _mix_bwd needs)."""
    if not cfg.delta:
        o, state = api.lin_attn_fwd(q, k, v, g, cu)
        return o, state, None
    (q, nq), (k, nk) = _unit(q), _unit(k)
    beta = torch.sigmoid(h.float() @ p[f"beta{i}"])
    debug = None
    if keep:                                           # the states after every chunk of every sequence
        at = torch.cat([cu[:1], ((cu.diff() + 63) // 64).cumsum(0).int()])
        debug = {"bound_offsets": at,
                 "bound_post": v.new_empty((int(at[-1]), *v.shape[1:], cfg.dk), dtype=torch.float32)}
    o, state = api.chunk_fwd(q, k, v, beta, g, cu, qdq_flags=cfg.qdq, debug=debug)
    return o, state, keep and (q, nq, k, nk, beta, debug["bound_post"])


def _mix_bwd(cfg, p, i, h, q, k, v, g, cu, kept, d_o, grads):
    """Gradients of q, k, v, g, and of h through beta."""
    if not cfg.delta:
        return *api.lin_attn_bwd(q, k, v, g, cu, d_o)[:4], 0.0
    q, nq, k, nk, beta, states = kept
    d_q, d_k, d_v, d_beta, d_g, _ = api.chunk_grad(q, k, v, beta, g, cu, d_o, states=states, qdq_flags=cfg.qdq)
    d_b = d_beta * beta * (1 - beta)
    grads[f"beta{i}"] = h.t() @ d_b
    return _unit_bwd(q, nq, d_q), _unit_bwd(k, nk, d_k), d_v, d_g, d_b @ p[f"beta{i}"].t()


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
        o, state, kept = _mix(cfg, p, i, h, q, k, v, g, cu, saved is not None)
        states.append(state)
        y, _ = api.block_norm_fwd(o, p[f"head_norm{i}"], gate=z, eps=cfg.eps)
        f = _mm(y.view(len(tokens), -1), p[f"out{i}"])
        h8 = api.act_pack(h)
        x, h, f8, _ = api.block_norm_fwd(f, p[f"post{i}"], residual=x, w_pre=p[f"pre{i}"], res_scale=cfg.res_scale,
                                         eps=cfg.eps, checkpoint=True)
        if saved is not None:
            saved.append((q, k, v, z, g, o, h8, api.act_pack(y), f8, x, kept))
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
        q, k, v, z, g, o, h8, y8, f8, x, kept = saved[1 + i]
        h = api.act_unpack(*h8, dtype=torch.float32)
        d_f, _, d_x, grads[f"post{i}"], grads[f"pre{i}"] = api.block_norm_bwd(
            f8, p[f"post{i}"], d_x, d_h=d_h, x=x, w_pre=p[f"pre{i}"], res_scale=cfg.res_scale, eps=cfg.eps)
        d_y = into(f"out{i}", y8, d_f).view_as(v)
        d_o, d_z, _, grads[f"head_norm{i}"], _ = api.block_norm_bwd(o, p[f"head_norm{i}"], d_y, gate=z, eps=cfg.eps,
                                                                    want_residual=False)
        d_q, d_k, d_v, d_g, d_hb = _mix_bwd(cfg, p, i, h, q, k, v, g, cu, kept, d_o, grads)
        d_in = torch.cat([t.flatten(1) for t in (d_q, d_k, d_v, d_z)], 1)
        d_s = d_g * -torch.expm1(g)                     # d log sigmoid(s) = 1 - sigmoid(s) = 1 - e^g
        d_h = into(f"in{i}", h8, d_in)
        grads[f"gate{i}"] = h.t() @ d_s
        d_h = (d_h.float() + d_s @ p[f"gate{i}"].t() + d_hb).to(BF16)
    d_e, _, _, grads["norm0"], _ = api.block_norm_bwd(saved[0], p["norm0"], d_h, eps=cfg.eps, want_residual=False)
    grads["embed"] = torch.zeros_like(p["embed"]).index_add_(0, tokens, d_x + d_e.float())
    return grads


def loss_and_grad(logits, targets):
    """Mean cross entropy and its gradient, in fp32."""
    logp = logits - logits.logsumexp(1, keepdim=True)
    d = logp.exp()
    d[torch.arange(len(targets), device=d.device), targets] -= 1
    return -logp.gather(1, targets[:, None]).mean(), d / len(targets)


def distill_and_grad(logits, top, ids, lse, targets, temperature=2.0, ce_weight=0.5):
    """Mean loss against a teacher's best logits (the others one more outcome)
    and the targets, and its gradient, which takes the logits' place."""
    n = len(targets)
    loss, d = api.distill_fwd_bwd(logits, ids, top, logits.new_full((n,), 1 / n, dtype=torch.float32), teacher_lse=lse,
                                  targets=targets, temperature=temperature, kd_weight=temperature ** 2,
                                  ce_weight=ce_weight, out=logits)
    return loss.mean(), d


def best(logits, k=8, temperature=2.0):
    """What distill_and_grad needs of a teacher: its k best logits, their columns, and the row's logsumexp."""
    top, ids = logits.topk(k, 1)
    return top, ids.int(), (logits / temperature).logsumexp(1)


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


def train(cfg, steps, seed=0, lens=(100, 64, 1, 163, 40, 144), lr=3e-3, teacher=None):
    """Parameters and every step's loss.  teacher: (its config, its parameters)."""
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
        if teacher is None:
            loss, d_logits = loss_and_grad(logits, targets)
        else:
            loss, d_logits = distill_and_grad(logits.to(BF16), *best(forward(*teacher, tokens, cu)[0]), targets)
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
        if cfg.delta:
            beta = torch.sigmoid(h.float() @ p[f"beta{i}"])
            o = api.decode_step(_unit(q)[0], _unit(k)[0], v, beta, g, states[i], qdq=cfg.qdq != 0)
        else:
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


def show(losses):
    for i in range(0, len(losses), 10):
        print(f"step {i:4d}  loss {losses[i]:.3f}")


def main():
    steps = int(sys.argv[1]) if len(sys.argv) > 1 else 100
    cfg, small = Config(), DeltaConfig()
    p, losses = train(cfg, steps)
    show(losses)
    print("a student with its state in FP8")
    student, losses = train(small, steps, seed=1, teacher=(cfg, p))
    show(losses)
    gen = torch.Generator().manual_seed(7)
    prompts = [batch(cfg, [n], gen)[0] for n in (9, 70)]
    for c, q in ((cfg, p), (small, student)):
        tokens, _ = generate(c, q, prompts, 8)
        for s, t in zip(prompts, tokens):
            print("prompt of", len(s), "ending in", s[-3:].tolist(), "goes on", t.tolist())


if __name__ == "__main__":
    main()
