"""Cases of the linear-attention block's operators, with their plain forms.

Operators (the package's entry points):
  lin_attn_fwd   linear attention with a decay for each head over packed
                 sequences, S_t = e^{g_t} S_{t-1} + v_t k_t^T, o_t = S_t q_t
  lin_attn_bwd   its gradients (q, k, v, the log decay, the initial state)
  lin_attn_step  one token for each sequence against a stored state
  block_norm_fwd, block_norm_bwd
                 the norm after a block, its gate, the scaled residual and the
                 norm before the next block, in one pass; the backward can take
                 the block's output and gate as 8-bit checkpoints
  act_pack, act_unpack
                 activations as E4M3 codes with a scale for each 64 columns

`own` false runs the plain form (elementary torch operations); `own` true
makes the package's calls.
"""
import math
import random

import torch

own = False

CHUNK = 64   # tokens of one chunk of the plain form
GROUP = 64   # columns that share a checkpoint scale


def listed():
    return [
        # the first prompt of an interactive session: launch latency counts
        {"name": "prompt_short", "op": "fwd", "seqs": 1, "tokens": 130, "heads": 4, "qk_heads": 4, "dk": 64, "dv": 64,
         "dtype": "bf16", "gate": "head", "even": True, "init": False},
        # packed prompts of unlike lengths (an empty and a one-token one among them) that continue stored states
        {"name": "prompt_ragged_fp32", "op": "fwd", "seqs": 9, "tokens": 5003, "heads": 6, "qk_heads": 2, "dk": 64,
         "dv": 128, "dtype": "fp32", "gate": "token", "even": False, "init": True},
        # one long document: the parallelism has to come from the token axis
        {"name": "prompt_long", "op": "fwd", "seqs": 1, "tokens": 32768, "heads": 16, "qk_heads": 16, "dk": 128,
         "dv": 128, "dtype": "bf16", "gate": "token", "even": True, "init": False},
        # the training batch of the prefill benchmark
        {"name": "train_batch", "op": "bwd", "seqs": 4, "tokens": 16384, "heads": 16, "qk_heads": 16, "dk": 128,
         "dv": 128, "dtype": "bf16", "gate": "token", "even": True, "init": False},
        # packed training documents, shared query/key heads, fixed decays, carried state
        {"name": "train_ragged", "op": "bwd", "seqs": 11, "tokens": 7001, "heads": 8, "qk_heads": 4, "dk": 64,
         "dv": 128, "dtype": "bf16", "gate": "head", "even": False, "init": True},
        # one user's next token
        {"name": "step_one", "op": "step", "seqs": 1, "heads": 16, "qk_heads": 16, "dk": 128, "dv": 128,
         "dtype": "bf16", "gate": "head"},
        # the decode batch of the handoff benchmark
        {"name": "step_batch", "op": "step", "seqs": 256, "heads": 32, "qk_heads": 32, "dk": 128, "dv": 128,
         "dtype": "bf16", "gate": "token"},
        # the norms around a block while decoding a few sequences
        {"name": "norm_step", "op": "norm", "rows": 8, "cols": 2048, "dtype": "bf16", "res": "fp32", "act": "none",
         "residual": True, "pre": True},
        # the gated norm of every head's output in a prompt
        {"name": "norm_heads", "op": "norm", "rows": 262144, "cols": 128, "dtype": "bf16", "res": "bf16", "act": "silu",
         "residual": False, "pre": False},
        # a training step through the norms, the block's output and gate kept in 8 bits
        {"name": "norm_train8", "op": "train", "rows": 16384, "cols": 2048, "dtype": "bf16", "res": "bf16",
         "act": "silu", "residual": True, "pre": True, "ckpt": True},
        # a small activation (a short odd batch) through an 8-bit checkpoint and back
        {"name": "act8_small", "op": "act8", "rows": 333, "cols": 1000, "dtype": "fp32"},
        # a layer's activations of a training batch through an 8-bit checkpoint and back
        {"name": "act8_batch", "op": "act8", "rows": 16384, "cols": 4096, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "step", "norm", "train", "act8"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("fwd", "bwd", "step"):
        heads = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
        share = rng.choice([s for s in (1, 1, 2, 3, 4) if heads % s == 0])
        c = {"op": op, "heads": heads, "qk_heads": heads // share, "dk": rng.choice([64, 128]),
             "dv": rng.choice([64, 128, 128, 192, 256]), "dtype": dtype, "gate": rng.choice(["head", "token"])}
        if op == "step":
            return dict(c, seqs=_log(rng, 1, 256))
        cost = heads * c["dk"] * c["dv"] * (4 if dtype == "fp32" else 1)
        most = min(32768 if op == "fwd" else 16384, 16384 * 16 * 128 * 128 // cost)
        tokens = _log(rng, 1, most)
        seqs = min(_log(rng, 1, 24), max(1, tokens // 8))
        even = rng.random() < 0.3
        tokens = max(seqs, tokens // seqs * seqs) if even else tokens
        return dict(c, seqs=seqs, tokens=tokens, even=even, init=rng.random() < 0.5)
    if op == "act8":
        cols = 8 * _log(rng, 1, 1024)
        return {"op": op, "rows": _log(rng, 1, min(65536, 16384 * 4096 // cols)), "cols": cols, "dtype": dtype}
    per_head = rng.random() < 0.3
    cols = rng.choice([64, 128, 256]) if per_head else 8 * _log(rng, 8, 1024)
    most = 16384 * 2048 // cols // (2 if dtype == "fp32" else 1)
    c = {"op": op, "rows": _log(rng, 1, most), "cols": cols, "dtype": dtype,
         "res": rng.choice(["bf16", "fp32"]) if dtype == "bf16" else "fp32",
         "act": rng.choice(["none", "silu", "sigmoid"]), "residual": not per_head, "pre": not per_head}
    return dict(c, ckpt=rng.random() < 0.5) if op == "train" else c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS, RES_SCALE = 1e-6, 0.5


def _lens(case):
    """Sequence lengths: equal ones, or an uneven split with an empty and a one-token sequence where it has room."""
    n, t = case["seqs"], case["tokens"]
    if case["even"] or n == 1:
        return [t // n] * (n - 1) + [t - t // n * (n - 1)]
    r = random.Random(1000 * t + n)
    w = [r.uniform(0.3, 1.7) for _ in range(n)]
    if n >= 4:
        w[n // 2] = 0.0
    lens = [int(t * x / sum(w)) for x in w]
    if n >= 3 and t >= 2 * n:
        lens[1] = 1
    lens[-1] += t - sum(lens)
    return lens


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    s = dict(case)
    dt = _DT[case["dtype"]]
    if case["op"] in ("fwd", "bwd", "step"):
        N, H, Hk, dk, dv = case["seqs"], case["heads"], case["qk_heads"], case["dk"], case["dv"]
        T = N if case["op"] == "step" else case["tokens"]
        s["q"] = _unit(normal(T, Hk, dk)).to(dt)
        s["k"] = _unit(normal(T, Hk, dk)).to(dt)
        s["v"] = normal(T, H, dv).to(dt)
        if case["gate"] == "head":
            # fixed decays from 1 - 2^-3 to 1 - 2^-9 over the heads, with a little of the seed
            e = 3 + 6 * torch.arange(H, device=dev) / max(1, H - 1) + 0.1 * torch.rand(H, generator=gen, device=dev)
            s["g"] = torch.log1p(-torch.exp2(-e))
        else:
            s["g"] = -0.1 * torch.nn.functional.softplus(normal(T, H))
        if case["op"] == "step":
            s["state"] = normal(N, H, dv, dk)
            return s
        lens = _lens(case)
        s["lens"] = lens
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        s["S0"] = normal(N, H, dv, dk) if case["init"] else None
        if case["op"] == "bwd":
            s["d_o"] = normal(T, H, dv).to(dt)
            s["dS"] = normal(N, H, dv, dk) if case["init"] else None
        return s
    R, D = case["rows"], case["cols"]
    if case["op"] == "act8":
        s["x"] = (normal(R, D) * torch.exp(normal(R, 1))).to(dt)
        return s
    rt = _DT[case["res"]]
    s["f"] = normal(R, D).to(dt)
    s["z"] = normal(R, D).to(dt) if case["act"] != "none" else None
    s["x"] = normal(R, D).to(rt) if case["residual"] else None
    s["w_post"] = 1 + 0.1 * normal(D)
    s["w_pre"] = 1 + 0.1 * normal(D) if case["pre"] else None
    if case["op"] == "train":
        s["d_x"] = normal(R, D).to(rt)
        s["d_h"] = normal(R, D).to(dt) if case["pre"] else None
        # the residual stream that the backward reads is an input of its own: whether the forward's rounding of it
        # to bf16 goes up or down is no part of what the gradients are compared for
        s["x_kept"] = normal(R, D).to(rt) if case["pre"] else None
    return s


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("fwd", "bwd", "step"):
        N, H, Hk, dk, dv = case["seqs"], case["heads"], case["qk_heads"], case["dk"], case["dv"]
        state = 4 * N * H * dk * dv
        if case["op"] == "step":
            gate = 4 * H * (N if case["gate"] == "token" else 1)
            return {"bytes": 2 * state + e * N * (2 * Hk * dk + 2 * H * dv) + gate, "flops": 4 * N * H * dk * dv}
        T = case["tokens"]
        gate = 4 * H * (T if case["gate"] == "token" else 1)
        if case["op"] == "fwd":
            return {"bytes": e * T * (2 * Hk * dk + 2 * H * dv) + gate + state * (2 if case["init"] else 1),
                    "flops": 4 * T * H * dk * dv}
        return {"bytes": e * T * (4 * Hk * dk + 3 * H * dv) + 2 * gate + state * (3 if case["init"] else 1),
                "flops": 10 * T * H * dk * dv}
    n = case["rows"] * case["cols"]
    if case["op"] == "act8":
        groups = case["rows"] * -(-case["cols"] // GROUP)
        return {"bytes": 2 * (e * n + n + 4 * groups), "flops": 4 * n}
    r = 2 if case["res"] == "bf16" else 4
    z, x, h = case["act"] != "none", case["residual"], case["pre"]
    fwd = n * (e * (1 + z + h) + r * (1 + x)) + 4 * case["cols"] * (1 + h)
    if case["op"] == "norm":
        return {"bytes": fwd, "flops": n * (6 + 6 * z + 4 * h)}
    kept = (1 + 4 / GROUP) if case["ckpt"] else e   # a kept value of f or z, as the backward reads it
    bwd = n * (kept * (1 + z) + e * h + r * (1 + h + x) + e * (1 + z)) + 8 * case["cols"] * (1 + h)
    return {"bytes": fwd + bwd + (n * kept * (1 + z) if case["ckpt"] else 0), "flops": n * (20 + 16 * z + 12 * h)}


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _padded(s):
    """Chunked [N, H, chunks, 64, d] fp32 views of the packed inputs, zeros (and gates of 0) past each length."""
    N, H, lens = s["seqs"], s["heads"], s["lens"]
    nc = max(1, -(-max(lens) // CHUNK))
    cu = s["cu"].long()
    at = torch.arange(nc * CHUNK, device=cu.device)[None] + cu[:-1, None]
    ok = at < cu[1:, None]
    at = at.clamp(max=max(0, s["q"].shape[0] - 1))

    def rows(x, heads):
        x = x.float().repeat_interleave(heads // x.shape[1], dim=1)[at] * ok[..., None, None]
        return x.reshape(N, nc, CHUNK, heads, -1).permute(0, 3, 1, 2, 4).contiguous()

    g = s["g"].double()
    g = (g[at] if g.dim() == 2 else g.expand(N, nc * CHUNK, H)) * ok[..., None]
    g = g.reshape(N, nc, CHUNK, H).permute(0, 3, 1, 2)
    return rows, g, (at, ok)


def _unpad(x, where, s, heads):
    N, d = s["seqs"], x.shape[-1]
    flat = x.permute(0, 2, 3, 1, 4).reshape(N, -1, x.shape[1], d)
    out = flat[where[1]]
    return out.reshape(out.shape[0], heads, -1, d).sum(2) if heads != x.shape[1] else out


def _tri(G, strict=False):
    """e^{G_i - G_j} for j <= i, else 0."""
    n = G.shape[-1]
    i = torch.arange(n, device=G.device)
    keep = i[:, None] > i[None] if strict else i[:, None] >= i[None]
    return torch.where(keep, (G[..., :, None] - G[..., None, :]).clamp(max=700).exp(), 0.0)


def _entering(E, before, local, first):
    """State entering every chunk and the one after the last: decayed sums of the chunks' own states."""
    N, H, nc = E.shape
    i = torch.arange(nc, device=E.device)
    # entering chunk c: all c' < c, decayed from the end of c' to the start of c
    M = torch.where(i[:, None] > i[None], (before[..., :, None] - E[..., None, :]).clamp(max=700).exp(), 0.0).float()
    flat = local.reshape(N, H, nc, -1)
    S = M @ flat
    last = ((E[..., -1:] - E).exp().float()[..., None, :] @ flat).reshape(N, H, *local.shape[3:])
    if first is not None:
        S = S + before.exp().float()[..., None] * first.reshape(N, H, 1, -1)
        last = last + E[..., -1].exp().float()[..., None, None] * first
    return S.reshape(local.shape), last


def _plain_fwd(s):
    rows, g, where = _padded(s)
    H = s["heads"]
    q, k, v = rows(s["q"], H), rows(s["k"], H), rows(s["v"], H)
    G = g.cumsum(-1)
    E = G[..., -1].cumsum(-1)
    to_end = (G[..., -1:] - G).exp().float()[..., None]
    local = (v * to_end).transpose(-1, -2) @ k
    S, last = _entering(E, E - G[..., -1], local, s["S0"])
    o = ((q @ k.transpose(-1, -2)) * _tri(G).float()) @ v
    o = o + (q * G.exp().float()[..., None]) @ S.transpose(-1, -2)
    return _unpad(o, where, s, H).to(s["v"].dtype), last


def _plain_bwd(s):
    rows, g, where = _padded(s)
    H, Hk = s["heads"], s["qk_heads"]
    q, k, v, do = rows(s["q"], H), rows(s["k"], H), rows(s["v"], H), rows(s["d_o"], H)
    G = g.cumsum(-1)
    Gc = G[..., -1]
    E = Gc.cumsum(-1)
    eg, to_end = G.exp().float()[..., None], (G[..., -1:] - G).exp().float()[..., None]
    S, last = _entering(E, E - Gc, (v * to_end).transpose(-1, -2) @ k, s["S0"])
    # gradient of the state at every chunk's end: the later chunks' own parts, last chunk first
    F = Gc.flip(-1).cumsum(-1)
    dS, first = _entering(F, F - Gc.flip(-1), ((do * eg).transpose(-1, -2) @ q).flip(2), s["dS"])
    dS = dS.flip(2)
    D = _tri(G).float()
    A, B = (q @ k.transpose(-1, -2)), (do @ v.transpose(-1, -2))
    dq_in, dk_out = eg * (do @ S), to_end * (v @ dS)
    dq = (B * D) @ k + dq_in
    dk = (B * D).transpose(-1, -2) @ q + dk_out
    dv = (A * D).transpose(-1, -2) @ do + to_end * (k @ dS.transpose(-1, -2))
    # log decay of token t: every pair it lies between, j >= t > i
    M = (A * B).double() * _tri(G, strict=True)
    c = (k * dk_out).double().sum(-1)
    r = M.sum(-1) - M.sum(-2) + (q * dq_in).double().sum(-1)
    dg = r.flip(-1).cumsum(-1).flip(-1) + c.cumsum(-1) - c
    dg = dg + (Gc.exp() * (S * dS).double().sum((-1, -2)))[..., None]
    dg = _unpad(dg[..., None], where, s, H)[..., 0]
    dt = s["v"].dtype
    return (_unpad(dq, where, s, Hk).to(dt), _unpad(dk, where, s, Hk).to(dt), _unpad(dv, where, s, H).to(dt),
            (dg.sum(0) if s["g"].dim() == 1 else dg).float(), first)


def _plain_step(s):
    H = s["heads"]
    share = H // s["qk_heads"]
    q, k = (s[n].float().repeat_interleave(share, dim=1) for n in ("q", "k"))
    a = s["g"].exp().expand(s["seqs"], H)
    s["state"].mul_(a[..., None, None]).add_(s["v"].float()[..., :, None] * k[..., None, :])
    return (s["state"] * q[..., None, :]).sum(-1).to(s["v"].dtype), s["state"]


def _act(z, kind):
    """The gate's value and its derivative."""
    p = 1 / (1 + torch.exp(-z))
    return (p, p * (1 - p)) if kind == "sigmoid" else (z * p, p * (1 + z * (1 - p)))


def _rms(x):
    return 1 / ((x * x).mean(-1, keepdim=True) + EPS).sqrt()


def _plain_norm(s):
    f = s["f"].float()
    y = f * _rms(f) * s["w_post"]
    if s["z"] is not None:
        y = y * _act(s["z"].float(), s["act"])[0]
    x = RES_SCALE * y
    if s["x"] is not None:
        x = x + s["x"].float()
    h = (x * _rms(x) * s["w_pre"]).to(s["f"].dtype) if s["w_pre"] is not None else None
    return x.to(_DT[s["res"]]), h


def _plain_norm_bwd(s, x, f, z):
    dxp = s["d_x"].float()
    dw_pre = d_z = None
    if s["w_pre"] is not None:
        x = x.float()
        r = _rms(x)
        xh, t = x * r, s["d_h"].float() * s["w_pre"]
        dxp = dxp + r * (t - xh * (t * xh).mean(-1, keepdim=True))
        dw_pre = (s["d_h"].double() * xh).sum(0).float()
    dy = RES_SCALE * dxp
    r = _rms(f)
    n = f * r
    t = dy
    if z is not None:
        a, da = _act(z, s["act"])
        d_z = (dy * n * s["w_post"] * da).to(s["f"].dtype)
        t = dy * a
    dw_post = (t.double() * n).sum(0).float()
    t = t * s["w_post"]
    d_f = (r * (t - n * (t * n).mean(-1, keepdim=True))).to(s["f"].dtype)
    return d_f, d_z, dxp.to(_DT[s["res"]]) if s["x"] is not None else None, dw_post, dw_pre


def _plain_pack(x):
    """E4M3 values (as floats) and the scales: amax / 448 of each 64 columns, 1 where that is not positive."""
    R, D = x.shape
    groups = -(-D // GROUP)
    p = torch.nn.functional.pad(x.float(), (0, groups * GROUP - D)).reshape(R, groups, GROUP)
    sc = (p.abs().amax(-1).double() / 448).float()
    sc = torch.where(sc > 0, sc, 1.0)
    codes = (p.double() / sc.double()[..., None]).float().clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes.float(), sc


def _plain_unpack(codes, sc, D):
    return (codes * sc[..., None]).reshape(codes.shape[0], -1)[:, :D].contiguous()


def _run_plain(s):
    op = s["op"]
    if op == "fwd":
        return _plain_fwd(s)
    if op == "bwd":
        return _plain_bwd(s)
    if op == "step":
        return _plain_step(s)
    if op == "norm":
        return _plain_norm(s)
    if op == "act8":
        codes, sc = _plain_pack(s["x"])
        return _plain_unpack(codes, sc, s["cols"]).to(s["x"].dtype), sc
    x, h = _plain_norm(s)
    f, z = s["f"].float(), None if s["z"] is None else s["z"].float()
    if s["ckpt"]:
        f = _plain_unpack(*_plain_pack(s["f"]), s["cols"])
        z = None if z is None else _plain_unpack(*_plain_pack(s["z"]), s["cols"])
    return (x, h, *_plain_norm_bwd(s, s["x_kept"], f, z))


# ---------------------------------------------------------------------------
# the package's calls
# ---------------------------------------------------------------------------
def _run_own(s):
    from fp8_state_qat_amd import api
    op = s["op"]
    if op == "fwd":
        return api.lin_attn_fwd(s["q"], s["k"], s["v"], s["g"], s["cu"], initial_state=s["S0"])
    if op == "bwd":
        return api.lin_attn_bwd(s["q"], s["k"], s["v"], s["g"], s["cu"], s["d_o"], initial_state=s["S0"],
                                d_final_state=s["dS"])
    if op == "step":
        return api.lin_attn_step(s["q"], s["k"], s["v"], s["g"], s["state"]), s["state"]
    if op == "act8":
        codes, sc = api.act_pack(s["x"])
        return api.act_unpack(codes, sc, dtype=s["x"].dtype), sc
    kw = dict(gate=s["z"], act=s["act"] if s["z"] is not None else "silu", res_scale=RES_SCALE, eps=EPS)
    res = _DT[s["res"]]
    if op == "norm":
        return api.block_norm_fwd(s["f"], s["w_post"], residual=s["x"], w_pre=s["w_pre"], x_dtype=res, **kw)
    f, z = s["f"], s["z"]
    if s["ckpt"]:
        x, h, f, z = api.block_norm_fwd(f, s["w_post"], residual=s["x"], w_pre=s["w_pre"], x_dtype=res,
                                        checkpoint=True, **kw)
        kw["gate"] = z
    else:
        x, h = api.block_norm_fwd(f, s["w_post"], residual=s["x"], w_pre=s["w_pre"], x_dtype=res, **kw)
    grads = api.block_norm_bwd(f, s["w_post"], s["d_x"], d_h=s["d_h"], x=s["x_kept"], w_pre=s["w_pre"],
                               want_residual=s["residual"], io_dtype=s["f"].dtype, **kw)
    return (x, h, *grads)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits, token by token and row by row
# ---------------------------------------------------------------------------
def _exact_seq(q, k, v, g, S0, do=None, dS=None):
    """One sequence: q, k [L, H, dk], v [L, H, dv], g [L, H]; S [H, dv, dk] in fp64."""
    L, H, dv = v.shape
    S = S0.clone()
    a = g.exp()
    o = torch.empty_like(v)
    before = [] if do is not None else None
    keep = 64   # states kept: every 64th, the others computed again from it
    for t in range(L):
        if before is not None and t % keep == 0:
            before.append(S.clone())
        S.mul_(a[t, :, None, None]).addcmul_(v[t, :, :, None], k[t, :, None, :])
        if do is None:
            o[t] = (S @ q[t, :, :, None])[..., 0]
    if do is None:
        return o, S
    dq, dk, dvv, dg = (torch.empty_like(x) for x in (q, k, v, g))
    R = dS.clone()
    for c in range((L - 1) // keep, -1, -1):
        t0, t1 = c * keep, min(L, c * keep + keep)
        states = [before[c]]
        for t in range(t0, t1):
            states.append(states[-1] * a[t, :, None, None] + v[t, :, :, None] * k[t, :, None, :])
        for t in range(t1 - 1, t0 - 1, -1):
            prev, now = states[t - t0], states[t - t0 + 1]
            dq[t] = (do[t, :, None, :] @ now)[:, 0]
            R.addcmul_(do[t, :, :, None], q[t, :, None, :])
            dk[t] = (v[t, :, None, :] @ R)[:, 0]
            dvv[t] = (R @ k[t, :, :, None])[..., 0]
            R.mul_(a[t, :, None, None])
            dg[t] = (R * prev).sum((-1, -2))
    return dq, dk, dvv, dg, R


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("fwd", "bwd", "step"):
        H, Hk = case["heads"], case["qk_heads"]
        if case["op"] != "step" and sum(_lens(case)) * (1 if case["op"] == "fwd" else 4) > 70000:
            return None
        q, k = (s[n].double().repeat_interleave(H // Hk, dim=1) for n in ("q", "k"))
        v, T = s["v"].double(), s["v"].shape[0]
        g = s["g"].double().expand(T, H)
        if case["op"] == "step":
            S = s["state"].double() * g.exp()[..., None, None] + v[..., :, None] * k[..., None, :]
            return (S @ q[..., None])[..., 0], S
        parts, at = [], 0
        for n, L in enumerate(s["lens"]):
            sl = slice(at, at + L)
            at += L
            zero = torch.zeros(H, case["dv"], case["dk"], dtype=torch.float64, device=q.device)
            S0 = zero if s["S0"] is None else s["S0"][n].double()
            if case["op"] == "fwd":
                parts.append(_exact_seq(q[sl], k[sl], v[sl], g[sl], S0))
            else:
                dS = zero if s["dS"] is None else s["dS"][n].double()
                parts.append(_exact_seq(q[sl], k[sl], v[sl], g[sl], S0, s["d_o"][sl].double(), dS))
        if case["op"] == "fwd":
            return torch.cat([p[0] for p in parts]), torch.stack([p[1] for p in parts])
        dq, dk, dv, dg = (torch.cat([p[i] for p in parts]) for i in range(4))
        dq, dk = (x.reshape(T, Hk, H // Hk, -1).sum(2) for x in (dq, dk))
        return dq, dk, dv, dg.sum(0) if s["g"].dim() == 1 else dg, torch.stack([p[4] for p in parts])
    if case["op"] == "act8":
        return _exact_pack(s["x"].double())
    f, z = s["f"].double(), None if s["z"] is None else s["z"].double()
    w = s["w_post"].double()
    gate = (lambda u: torch.sigmoid(u)) if case["act"] == "sigmoid" else (lambda u: u * torch.sigmoid(u))
    if case["op"] == "norm":
        return _exact_norm(s, f, z, w, gate)
    x, h = _exact_norm(s, f, z, w, gate)
    if case["ckpt"]:
        f = _exact_pack(f)[0]
        z = None if z is None else _exact_pack(z)[0]
    # gradients by torch's own differentiation of the formulas in 64 bits
    f, w = f.requires_grad_(), w.clone().requires_grad_()
    leaves = [f, w]
    y = f / torch.sqrt(f.pow(2).mean(-1, keepdim=True) + EPS) * w
    if z is not None:
        z = z.requires_grad_()
        leaves.append(z)
        y = y * gate(z)
    dxp = s["d_x"].double()
    d_pre = None
    if s["w_pre"] is not None:
        xk, wp = s["x_kept"].double().requires_grad_(), s["w_pre"].double().requires_grad_()
        hk = xk / torch.sqrt(xk.pow(2).mean(-1, keepdim=True) + EPS) * wp
        gx, d_pre = torch.autograd.grad(hk, (xk, wp), s["d_h"].double())
        dxp = dxp + gx
    grads = torch.autograd.grad(RES_SCALE * y, leaves, dxp)
    return (x, h, grads[0], grads[2] if z is not None else None, dxp if s["x"] is not None else None, grads[1], d_pre)


def _exact_norm(s, f, z, w, gate):
    y = f / torch.sqrt(f.pow(2).mean(-1, keepdim=True) + EPS) * w
    if z is not None:
        y = y * gate(z)
    x = RES_SCALE * y + (0 if s["x"] is None else s["x"].double())
    if s["w_pre"] is None:
        return x, None
    return x, x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + EPS) * s["w_pre"].double()


def _exact_pack(x):
    """The nearest E4M3 value to x / s (ties to even) times s; s and x / s in 32 bits by definition."""
    R, D = x.shape
    out, scales = torch.empty_like(x), []
    for c in range(0, D, GROUP):
        p = x[:, c:c + GROUP]
        sc = (p.abs().amax(-1, keepdim=True) / 448).float().double()
        sc = torch.where(sc > 0, sc, 1.0)
        y = (p / sc).float().double().clamp(-448, 448)
        e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
        e = torch.where(torch.exp2(e) > y.abs().clamp(min=2.0 ** -6), e - 1, e)
        e = torch.where(torch.exp2(e + 1) <= y.abs(), e + 1, e)
        ulp = torch.exp2(e - 3)
        out[:, c:c + GROUP] = torch.round(y / ulp) * ulp * sc
        scales.append(sc)
    return out, torch.cat(scales, 1)
