"""Cases of the operators that train a model of gated-delta-rule blocks, with
their plain forms.

Operators (the package's entry points):
  chunk_grad       every gradient of the chunked gated delta rule (q, k, v,
                   beta, the log-gate, the initial state), identity
                   straight-through at the state's quantization; the states of
                   the forward's 64-token boundaries are recomputed or given
  distill_fwd      distillation from a teacher's top logits and cross entropy,
                   a loss for each row of logits
  distill_bwd      the gradient of the logits from the losses' gradients
  distill_fwd_bwd  both in one call, where the losses' gradients are known

`own` false runs the plain form (elementary torch operations); `own` true
makes the package's calls.
"""
import math
import random

import torch

own = False

CHUNK = 64   # tokens of one chunk


def listed():
    return [
        # one short document: launch latency counts
        {"name": "grad_short", "op": "grad", "seqs": 1, "tokens": 130, "heads": 2, "dk": 64, "dv": 64, "dtype": "bf16",
         "even": True, "states": "recompute", "init": False, "pad": False},
        # packed documents of unlike lengths with padded segments that continue stored states, quantized states kept
        {"name": "grad_ragged_qat", "op": "grad", "seqs": 9, "tokens": 5003, "heads": 6, "dk": 64, "dv": 128,
         "dtype": "bf16", "even": False, "states": "given", "init": True, "pad": True},
        # the training batch of the prefill benchmark
        {"name": "grad_train", "op": "grad", "seqs": 4, "tokens": 16384, "heads": 16, "dk": 128, "dv": 128,
         "dtype": "bf16", "even": True, "states": "recompute", "init": False, "pad": False},
        # the same batch in shorter sequences, quantization-aware: the quantized states kept by the forward
        {"name": "grad_train_qat", "op": "grad", "seqs": 16, "tokens": 16384, "heads": 16, "dk": 128, "dv": 128,
         "dtype": "bf16", "even": True, "states": "given", "init": False, "pad": False},
        # one long document: few chains, many chunks
        {"name": "grad_long", "op": "grad", "seqs": 1, "tokens": 8192, "heads": 16, "dk": 128, "dv": 128,
         "dtype": "bf16", "even": True, "states": "recompute", "init": False, "pad": False},
        # fp32 inputs, as a reference run of the training has them
        {"name": "grad_fp32", "op": "grad", "seqs": 3, "tokens": 1501, "heads": 4, "dk": 128, "dv": 128,
         "dtype": "fp32", "even": False, "states": "recompute", "init": True, "pad": False},
        # validation loss of a small odd batch, rest of the vocabulary as one more outcome, labels mixed in
        {"name": "distill_fwd_small", "op": "fwd", "rows": 33, "vocab": 4099, "topk": 8, "dtype": "fp32", "tail": True,
         "ce": True, "temperature": 1.0},
        # validation loss of a training batch
        {"name": "distill_fwd_batch", "op": "fwd", "rows": 16384, "vocab": 32000, "topk": 64, "dtype": "bf16",
         "tail": False, "ce": True, "temperature": 2.0},
        # gradient with an odd vocabulary, rest as one more outcome
        {"name": "distill_bwd_odd", "op": "bwd", "rows": 1000, "vocab": 50001, "topk": 20, "dtype": "fp32",
         "tail": True, "ce": True, "temperature": 1.0},
        # gradient of a training batch from the losses' gradients
        {"name": "distill_bwd_batch", "op": "bwd", "rows": 16384, "vocab": 32000, "topk": 64, "dtype": "bf16",
         "tail": False, "ce": False, "temperature": 2.0},
        # loss and gradient of a short batch over a small vocabulary
        {"name": "distill_step_small", "op": "both", "rows": 512, "vocab": 1003, "topk": 16, "dtype": "bf16",
         "tail": False, "ce": True, "temperature": 1.0},
        # loss and gradient of a training step over a wide vocabulary
        {"name": "distill_step_wide", "op": "both", "rows": 4096, "vocab": 131072, "topk": 64, "dtype": "bf16",
         "tail": True, "ce": True, "temperature": 2.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["grad", "grad", "grad", "fwd", "bwd", "both"])
    if op == "grad":
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        c = {"op": op, "heads": rng.choice([1, 2, 3, 4, 6, 8, 12, 16]), "dk": rng.choice([64, 128]),
             "dv": rng.choice([64, 128, 128, 192, 256]), "dtype": dtype}
        cost = c["heads"] * c["dk"] * c["dv"] * (16 if dtype == "fp32" else 1)
        tokens = _log(rng, 1, min(8192, 8192 * 16 * 128 * 128 // cost))
        seqs = min(_log(rng, 1, 24), max(1, tokens // 8))
        even = rng.random() < 0.3
        tokens = max(seqs, tokens // seqs * seqs) if even else tokens
        return dict(c, seqs=seqs, tokens=tokens, even=even, states=rng.choice(["recompute", "given"]),
                    init=rng.random() < 0.5, pad=rng.random() < 0.3)
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    vocab = _log(rng, 100, 131072)
    most = 16384 * 16000 // vocab // (2 if dtype == "fp32" else 1)
    return {"op": op, "rows": _log(rng, 1, min(16384, most)), "vocab": vocab, "topk": min(_log(rng, 1, 128), vocab // 2),
            "dtype": dtype, "tail": rng.random() < 0.5, "ce": rng.random() < 0.5,
            "temperature": rng.choice([1.0, 1.0, 2.0, 0.7])}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
KD_WEIGHT, CE_WEIGHT, IGNORE = 0.75, 0.25, -100


def _lens(case):
    """(segment lengths, valid lengths): equal segments, or an uneven split with an empty and a one-token segment
    where it has room; with padding some segments are longer than their sequences."""
    n, t = case["seqs"], case["tokens"]
    if case["even"] or n == 1:
        seg = [t // n] * (n - 1) + [t - t // n * (n - 1)]
    else:
        r = random.Random(1000 * t + n)
        w = [r.uniform(0.3, 1.7) for _ in range(n)]
        if n >= 4:
            w[n // 2] = 0.0
        seg = [int(t * x / sum(w)) for x in w]
        if n >= 3 and t >= 2 * n:
            seg[1] = 1
        seg[-1] += t - sum(seg)
    if not case["pad"]:
        return seg, list(seg)
    return seg, [max(0, x - x // 5) if i % 2 == 0 else x for i, x in enumerate(seg)]


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def _quantized(S):
    """The state with a scale amax / 448 for each 64 value rows, to the nearest E4M3 value and back."""
    p = S.reshape(*S.shape[:-2], S.shape[-2] // 64, 64, S.shape[-1])
    sc = p.abs().amax((-1, -2), keepdim=True) / 448
    sc = torch.where(sc > 0, sc, 1.0)
    return ((p / sc).clamp(-448, 448).to(torch.float8_e4m3fn).float() * sc).reshape(S.shape)


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    s = dict(case)
    dt = _DT[case["dtype"]]
    if case["op"] == "grad":
        N, T, H, dk, dv = (case[n] for n in ("seqs", "tokens", "heads", "dk", "dv"))
        s["q"] = (_unit(normal(T, H, dk)) * dk ** -0.5).to(dt)
        s["k"] = _unit(normal(T, H, dk)).to(dt)
        s["v"] = normal(T, H, dv).to(dt)
        s["beta"] = torch.sigmoid(normal(T, H))
        s["g"] = -0.1 * torch.nn.functional.softplus(normal(T, H))
        s["d_o"] = normal(T, H, dv).to(dt)
        seg, lens = _lens(case)
        cu = [0]
        for n in seg:
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev) if case["pad"] else None
        s["len_list"] = lens
        s["S0"] = normal(N, H, dv, dk) if case["init"] else None
        s["dS"] = normal(N, H, dv, dk) if case["init"] else None
        s["kept"] = None
        if case["states"] == "given":
            p = _Packed(s, torch.float32)
            S = p.forward(_quantized)[:, :, 1:]    # the states after every chunk, quantized, of every sequence in turn
            s["kept"] = torch.cat([S[n, :, :-(-L // CHUNK)].transpose(0, 1) for n, L in enumerate(lens)])
        return s
    R, V, K = case["rows"], case["vocab"], case["topk"]
    teacher = 2.5 * normal(R, V)
    s["logits"] = (0.8 * teacher + 1.5 * normal(R, V)).to(dt)
    top, ids = teacher.topk(K, dim=1)
    # teachers that kept fewer: every seventh row half of them (one at least), the others marked -1
    few = (torch.arange(R, device=dev) % 7 == 3)[:, None] & (torch.arange(K, device=dev) >= max(1, K // 2))[None]
    s["ids"] = torch.where(few, -1, ids).to(torch.int32)
    s["top"] = top
    s["lse"] = torch.logsumexp(teacher.double() / case["temperature"], 1).float() if case["tail"] else None
    s["targets"] = None
    if case["ce"]:
        t = torch.where(torch.rand(R, generator=gen, device=dev) < 0.7, ids[:, 0],
                        torch.randint(V, (R,), generator=gen, device=dev))
        s["targets"] = torch.where(torch.arange(R, device=dev) % 11 == 5, IGNORE, t)
    if case["op"] != "fwd":
        s["d_loss"] = (0.5 + torch.rand(R, generator=gen, device=dev)) / R
    if case["op"] == "bwd":
        s["stats"] = _stats(s)
    return s


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "grad":
        N, T, H, dk, dv = (case[n] for n in ("seqs", "tokens", "heads", "dk", "dv"))
        T = sum(_lens(case)[1])
        chunks = sum(-(-n // CHUNK) for n in _lens(case)[1])
        state = 4 * H * dv * dk
        given = case["states"] == "given"
        data = e * T * H * (4 * dk + 3 * dv) + 16 * T * H
        states = state * (N * (3 if case["init"] else 1) + (chunks if given else 0))
        # products of a chunk with the state (64 x dk x dv): K S, K dS, the reverse update's two, dO S, Y S, U dS (and
        # the forward update where it is recomputed); of 64 x 64 with dk or dv columns, half of them in the triangle
        big = 7 + (0 if given else 1)
        flops = chunks * H * (2 * 64 * dk * dv * big + 64 * 64 * (6 * dv + 6 * dk))
        return {"bytes": data + states, "flops": flops}
    R, V, K = case["rows"], case["vocab"], case["topk"]
    passes = 1 if case["op"] == "fwd" else 2
    small = R * (8 * K + (4 if case["tail"] else 0) + (8 if case["ce"] else 0) + 24)
    exps = (1 if case["temperature"] == 1.0 or not case["ce"] else 2) * (2 if case["op"] == "both" else 1)
    return {"bytes": passes * R * V * e + small, "flops": R * V * (4 * exps + 2)}


# ---------------------------------------------------------------------------
# the plain forms: the gated delta rule
#
# Chunk of 64 tokens, G_r the sum of the log-gates up to token r, D_rs = e^(G_r - G_s) for s <= r, S the state entering
# it, B_rs = D_rs k_r.k_s (s < r), M = (I + B diag(beta))^-1:
#   E = M (V - e^G K S^T),  U = beta E,  S' = e^(G_C) S + U^T (e^(G_C - G) K),  O = e^G Q S^T + (D Q K^T) U
# ---------------------------------------------------------------------------
class _Packed:
    """[N, H, chunks, 64, ..] views of the packed inputs, zeros past each length, and the chunks' matrices."""

    def __init__(self, s, dt):
        N, H, lens = s["seqs"], s["heads"], s["len_list"]
        self.s, self.dt = s, dt
        self.nc = max(1, -(-max(lens) // CHUNK))
        cu = s["cu"].long()
        at = torch.arange(self.nc * CHUNK, device=cu.device)[None] + cu[:-1, None]
        end = (cu[:-1] + torch.tensor(lens, device=cu.device))[:, None]
        self.ok = at < end
        self.at = at.clamp(max=max(0, s["q"].shape[0] - 1))
        self.q, self.k, self.v = (self.rows(s[n]) for n in ("q", "k", "v"))
        self.beta = self.rows(s["beta"][..., None])
        g = torch.where(self.ok[..., None], s["g"].double()[self.at], 0.0)
        G = g.reshape(N, self.nc, CHUNK, H).permute(0, 3, 1, 2).cumsum(-1)
        self.eG = G.exp().to(dt)[..., None]                       # e^G
        self.eL = (G[..., -1:] - G).exp().to(dt)[..., None]       # e^(G_C - G)
        self.eC = G[..., -1].exp().to(dt)[..., None, None]        # e^(G_C)
        i = torch.arange(CHUNK, device=cu.device)
        self.low = i[:, None] >= i[None]
        self.strict = i[:, None] > i[None]
        self.D = torch.where(self.low, (G[..., :, None] - G[..., None, :]).clamp(max=0).exp(), 0.0).to(dt)
        kk = self.k @ self.k.transpose(-1, -2)
        self.B = torch.where(self.strict, self.D * kk, 0.0)
        # forward substitution, row by row
        A = self.B * self.beta.transpose(-1, -2)
        M = torch.eye(CHUNK, dtype=dt, device=cu.device).expand_as(A).clone()
        for r in range(1, CHUNK):
            M[..., r, :r] = -(A[..., r, None, :r] @ M[..., :r, :r])[..., 0, :]
        self.M = M

    def rows(self, x):
        N, H = self.s["seqs"], self.s["heads"]
        x = torch.where(self.ok[..., None, None], x[self.at].to(self.dt), 0.0)
        return x.reshape(N, self.nc, CHUNK, H, -1).permute(0, 3, 1, 2, 4).contiguous()

    def unpad(self, x, like):
        """Back to packed rows, zeros in padding."""
        N = self.s["seqs"]
        flat = x.permute(0, 2, 3, 1, 4).reshape(N, self.nc * CHUNK, x.shape[1], x.shape[-1])
        out = torch.zeros((*like.shape[:2], x.shape[-1]), dtype=x.dtype, device=x.device)
        out[self.at[self.ok]] = flat[self.ok]
        return out.reshape(like.shape).to(like.dtype)

    def first(self):
        s = self.s
        if s["S0"] is not None:
            return s["S0"].to(self.dt)
        return torch.zeros(s["seqs"], s["heads"], s["dv"], s["dk"], dtype=self.dt, device=self.q.device)

    def forward(self, quantize=None):
        """The states entering every chunk, and after the last one: [N, H, chunks + 1, dv, dk]."""
        S = self.first()
        out = [S]
        kl = self.k * self.eL
        for c in range(self.nc):
            E = self.M[:, :, c] @ (self.v[:, :, c] - self.eG[:, :, c] * (self.k[:, :, c] @ S.transpose(-1, -2)))
            S = self.eC[:, :, c] * S + (self.beta[:, :, c] * E).transpose(-1, -2) @ kl[:, :, c]
            S = S if quantize is None else quantize(S)
            out.append(S)
        return torch.stack(out, 2)

    def kept(self):
        """The states entering every chunk, from those kept after each."""
        s = self.s
        S = self.first()[:, :, None].repeat(1, 1, self.nc, 1, 1)
        at = 0
        for n, L in enumerate(s["len_list"]):
            c = -(-L // CHUNK)
            if c > 1:
                S[n, :, 1:c] = s["kept"][at:at + c - 1].to(self.dt).transpose(0, 1)
            at += c
        return S


def _plain_grad(s):
    p = _Packed(s, torch.float32)
    S = p.kept() if s["kept"] is not None else p.forward()[:, :, :-1]
    q, k, v, beta, D, B, M = p.q, p.k, p.v, p.beta, p.D, p.B, p.M
    do = p.rows(s["d_o"])
    P = D * (q @ k.transpose(-1, -2))
    PdO = P.transpose(-1, -2) @ do
    Mt = M.transpose(-1, -2)
    kl, kg, qg = k * p.eL, k * p.eG, q * p.eG
    # the states' gradients, last chunk first; dS[c]: of the state after chunk c
    R = s["dS"] if s["dS"] is not None else torch.zeros_like(S[:, :, 0])
    dS, Y = [None] * p.nc, [None] * p.nc
    for c in range(p.nc - 1, -1, -1):
        dS[c] = R
        Y[c] = Mt[:, :, c] @ (beta[:, :, c] * (PdO[:, :, c] + kl[:, :, c] @ R.transpose(-1, -2)))
        R = (p.eC[:, :, c] * R + do[:, :, c].transpose(-1, -2) @ qg[:, :, c]
             - Y[c].transpose(-1, -2) @ kg[:, :, c])
    dS, Y = torch.stack(dS, 2), torch.stack(Y, 2)
    E = M @ (v - kg @ S.transpose(-1, -2))
    bt = beta.transpose(-1, -2)
    dP = do @ E.transpose(-1, -2)                     # of P, without beta
    YE = torch.where(p.strict, Y @ E.transpose(-1, -2), 0.0)
    W = torch.where(p.low, dP * D, 0.0) * bt          # gradient of q.k
    Gk = -D * YE * bt                                 # gradient of k.k
    dq_s = p.eG * (do @ S)
    dk_x = -p.eG * (Y @ S)
    dk_s = p.eL * (E @ dS)                            # without beta
    dq = dq_s + W @ k
    dk = dk_x + beta * dk_s + W.transpose(-1, -2) @ q + Gk @ k + Gk.transpose(-1, -2) @ k
    dbeta = (dP * P).sum(-2)[..., None] - (B * YE).sum(-2)[..., None] + (k * dk_s).sum(-1, keepdim=True)
    # log-gate of token t: all that lies across it
    pair = torch.where(p.strict, (dP * P - B * YE) * bt, 0.0).double()
    own_ = pair.sum(-1) - pair.sum(-2) + (q * dq_s + k * dk_x).double().sum(-1)
    out = (beta * k * dk_s).double().sum(-1)
    dg = own_.flip(-1).cumsum(-1).flip(-1) + out.cumsum(-1) - out
    dg = dg + (p.eC[..., 0, 0] * (S * dS).double().sum((-1, -2)))[..., None]
    return (p.unpad(dq, s["q"]), p.unpad(dk, s["k"]), p.unpad(Y, s["v"]), p.unpad(dbeta, s["beta"]),
            p.unpad(dg[..., None].float(), s["g"]), R)


# ---------------------------------------------------------------------------
# the plain forms: distillation
#
# Row with logits z, kept teacher logits t_j at ids i_j (-1: none), temperature h:
#   p_j = e^(t_j / h - c), c the logsumexp of the kept t / h, or the given one of the whole vocabulary (tail)
#   kd  = sum p_j (ln p_j - ln q_(i_j)), q = softmax(z / h); with tail + p_r ln(p_r / q_r), the rest's two masses
#   ce  = logsumexp(z) - z_target
#   loss = 0.75 kd + 0.25 ce; a row whose target is ignored has none
# stats: logsumexp of z (0 without targets), of z / h, c, and of z / h over the rest (0 without tail)
# ---------------------------------------------------------------------------
def _teacher(s, dt=torch.float64):
    """(p [R, K], c [R], rest [R], index, kept) in 64 bits: 1 - sum p cancels."""
    on = s["ids"] >= 0
    t = torch.where(on, s["top"].to(dt) / s["temperature"], -math.inf)
    c = s["lse"].to(dt) if s["lse"] is not None else torch.logsumexp(t, 1)
    p = torch.where(on, (t - c[:, None]).exp(), 0.0)
    rest = (1 - p.sum(1)).clamp(min=0) if s["lse"] is not None else torch.zeros_like(c)
    return p, c, rest, s["ids"].clamp(min=0).long(), on


def _lse(x):
    m = x.amax(1, keepdim=True)
    return (m + (x - m).exp().sum(1, keepdim=True).log())[:, 0]


def _stats(s):
    """[R, 4] fp32, zeros in ignored rows."""
    z = s["logits"].float()
    _, c, _, ids, on = _teacher(s)
    zh = z / s["temperature"]
    zero = torch.zeros_like(z[:, 0])
    out = [_lse(z) if s["targets"] is not None else zero, _lse(zh), c.float(), zero]
    if s["lse"] is not None:
        out[3] = _lse(_without(zh, ids, on, -math.inf))
    out = torch.stack(out, 1)
    return out if s["targets"] is None else torch.where((s["targets"] == IGNORE)[:, None], 0.0, out)


def _without(x, ids, on, value):
    """x with `value` at the kept ids."""
    r = torch.arange(x.shape[0], device=x.device)[:, None].expand_as(ids)[on]
    x = x.clone()
    x[r, ids[on]] = value
    return x


def _plain_loss(s, stats):
    p, c, rest, ids, on = _teacher(s)
    z = s["logits"]
    zt = z.gather(1, ids).float() / s["temperature"]
    t = torch.where(on, s["top"].double() / s["temperature"], 0.0) - c[:, None]
    kd = torch.where(on, p * (t - (zt - stats[:, 1:2]).double()), 0.0).sum(1)
    if s["lse"] is not None:
        lr = torch.where(rest > 0, rest, 1.0).log()
        kd = kd + rest * (lr - (stats[:, 3] - stats[:, 1]).double())
    loss = KD_WEIGHT * kd
    if s["targets"] is not None:
        used = s["targets"] != IGNORE
        zt = z.gather(1, s["targets"].clamp(min=0)[:, None])[:, 0].float()
        loss = torch.where(used, loss + CE_WEIGHT * (stats[:, 0] - zt), 0.0)
    return loss.float()


def _plain_dlogits(s, stats):
    p, _, rest, ids, on = _teacher(s)
    z = s["logits"].float()
    w = s["d_loss"] if s["targets"] is None else torch.where(s["targets"] != IGNORE, s["d_loss"], 0.0)
    h = s["temperature"]
    a = (KD_WEIGHT / h * w)[:, None]
    r = torch.arange(z.shape[0], device=z.device)[:, None].expand_as(ids)
    if s["lse"] is None:
        d = a * (z / h - stats[:, 1:2]).exp()
    else:
        q_rest = (stats[:, 3] - stats[:, 1]).exp()
        d = a * (z / h - stats[:, 3:4]).exp() * (q_rest - rest.float())[:, None]
        d[r[on], ids[on]] = (a * (z.gather(1, ids) / h - stats[:, 1:2]).exp())[on]
    d.index_put_((r[on], ids[on]), (-a * p.float())[on], accumulate=True)
    if s["targets"] is not None:
        b = CE_WEIGHT * w
        d += b[:, None] * (z - stats[:, 0:1]).exp()
        d[torch.arange(z.shape[0], device=z.device), s["targets"].clamp(min=0)] -= b
        d = torch.where((s["targets"] == IGNORE)[:, None], 0.0, d)
    return d.to(s["logits"].dtype)


def _run_plain(s):
    if s["op"] == "grad":
        return _plain_grad(s)
    if s["op"] == "bwd":
        return _plain_dlogits(s, s["stats"])
    stats = _stats(s)
    loss = _plain_loss(s, stats)
    return (loss, stats) if s["op"] == "fwd" else (loss, _plain_dlogits(s, stats))


# ---------------------------------------------------------------------------
# the package's calls
# ---------------------------------------------------------------------------
def _run_own(s):
    from fp8_state_qat_amd import api
    if s["op"] == "grad":
        return api.chunk_grad(s["q"], s["k"], s["v"], s["beta"], s["g"], s["cu"], s["d_o"], seq_lens=s["lens"],
                              initial_state=s["S0"], states=s["kept"], d_final_state=s["dS"],
                              qdq_flags=0 if s["kept"] is None else api.GDN_QDQ_CHUNK)
    kw = dict(teacher_lse=s["lse"], targets=s["targets"], temperature=s["temperature"], kd_weight=KD_WEIGHT,
              ce_weight=CE_WEIGHT if s["targets"] is not None else 0.0, ignore_index=IGNORE)
    if s["op"] == "fwd":
        return api.distill_fwd(s["logits"], s["ids"], s["top"], **kw)
    if s["op"] == "bwd":
        return api.distill_bwd(s["logits"], s["ids"], s["top"], s["stats"], s["d_loss"], **kw)
    return api.distill_fwd_bwd(s["logits"], s["ids"], s["top"], s["d_loss"], **kw)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits: token by token, and by torch's differentiation of the loss
# ---------------------------------------------------------------------------
def _token(S, a, k, v, b):
    """One token of the gated delta rule: the state after it, the decayed one, the error."""
    Sd = S * a[..., None, None]
    e = v - (Sd @ k[..., None])[..., 0]
    return Sd + (b[..., None] * e)[..., :, None] * k[..., None, :], Sd, e


def _exact_grad(s):
    N, H, lens = s["seqs"], s["heads"], s["len_list"]
    top = max(lens)
    dev = s["q"].device
    f64 = torch.float64
    at = (s["cu"].long()[:-1, None] + torch.arange(max(1, top), device=dev)).clamp(max=max(0, s["q"].shape[0] - 1))
    live = torch.arange(max(1, top), device=dev)[None] < torch.tensor(lens, device=dev)[:, None]

    def rows(x):   # [tokens, N, H, ..]; past a sequence's end zeros: such a token changes nothing
        x = x.to(f64)[at]
        return torch.where(live.reshape(live.shape + (1,) * (x.dim() - 2)), x, 0.0).transpose(0, 1).contiguous()

    q, k, v, b, g, do = (rows(s[n]) for n in ("q", "k", "v", "beta", "g", "d_o"))
    a = g.exp()
    zero = torch.zeros(N, H, s["dv"], s["dk"], dtype=f64, device=dev)
    S = zero if s["S0"] is None else s["S0"].to(f64)
    nc = -(-top // CHUNK)
    entering = []
    if s["kept"] is None:
        for t in range(top):
            if t % CHUNK == 0:
                entering.append(S)
            S = _token(S, a[t], k[t], v[t], b[t])[0]
    else:
        entering = [S.clone() for _ in range(nc)]
        i = 0
        for n, L in enumerate(lens):
            for c in range(-(-L // CHUNK)):
                if c + 1 < nc:
                    entering[c + 1][n] = s["kept"][i].to(f64)
                i += 1
    R = zero if s["dS"] is None else s["dS"].to(f64)
    dq, dk, dv, db, dg = (torch.zeros_like(x) for x in (q, k, v, b, g))
    for c in range(nc - 1, -1, -1):
        t0, t1 = c * CHUNK, min(top, c * CHUNK + CHUNK)
        states, S = [], entering[c]
        for t in range(t0, t1):
            now = _token(S, a[t], k[t], v[t], b[t])
            states.append((S, *now))
            S = now[0]
        for t in range(t1 - 1, t0 - 1, -1):
            prev, S, Sd, e = states.pop()
            dq[t] = (do[t][..., None, :] @ S)[..., 0, :]
            R = R + do[t][..., :, None] * q[t][..., None, :]
            Rk = (R @ k[t][..., None])[..., 0]
            db[t] = (Rk * e).sum(-1)
            de = b[t][..., None] * Rk
            dv[t] = de
            dk[t] = b[t][..., None] * (e[..., None, :] @ R)[..., 0, :] - (de[..., None, :] @ Sd)[..., 0, :]
            R = (R - de[..., :, None] * k[t][..., None, :])
            dg[t] = (R * Sd).sum((-1, -2))
            R = R * a[t][..., None, None]

    def pack(x):
        out = torch.zeros((s["q"].shape[0], *x.shape[2:]), dtype=f64, device=dev)
        out[at[live]] = x.transpose(0, 1)[live]
        return out

    return pack(dq), pack(dk), pack(dv), pack(db), pack(dg), R


def _exact_losses(s, z):
    """Losses and stats of rows of logits z in 64 bits."""
    h = s["temperature"]
    logq = torch.log_softmax(z / h, 1)
    on = s["ids"] >= 0
    ids = s["ids"].clamp(min=0).long()
    t = s["top"].double() / h
    out = torch.zeros(z.shape[0], dtype=z.dtype, device=z.device)
    c = s["lse"].double() if s["lse"] is not None else torch.where(on, t, -math.inf).logsumexp(1)
    logp = t - c[:, None]
    p = torch.where(on, logp.exp(), 0.0)
    kd = (p * torch.where(on, logp - logq.gather(1, ids), 0.0)).sum(1)
    last = torch.zeros_like(out)
    if s["lse"] is not None:
        rest = (1 - p.sum(1)).clamp(min=0)
        mask = torch.zeros_like(z, dtype=torch.bool)
        mask[torch.arange(z.shape[0], device=z.device)[:, None].expand_as(ids)[on], ids[on]] = True
        last = torch.where(mask, -math.inf, z / h).logsumexp(1)
        lq = last - (z / h).logsumexp(1)
        kd = kd + torch.where(rest > 0, rest * (rest.clamp(min=1e-300).log() - lq), 0.0)
    loss = KD_WEIGHT * kd
    first = torch.zeros_like(out)
    if s["targets"] is not None:
        first = z.logsumexp(1)
        used = s["targets"] != IGNORE
        ce = -torch.log_softmax(z, 1).gather(1, s["targets"].clamp(min=0)[:, None])[:, 0]
        loss = torch.where(used, loss + CE_WEIGHT * ce, 0.0)
    stats = torch.stack([first, (z / h).logsumexp(1), c, last], 1)
    if s["targets"] is not None:
        stats = torch.where(used[:, None], stats, 0.0)
    return loss, stats


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "grad":
        return _exact_grad(s)
    # row by row in groups: 64 bits and torch's saved tensors
    step = max(1, (1 << 26) // case["vocab"])
    loss, stats, grads = [], [], []
    for r0 in range(0, case["rows"], step):
        part = {n: x[r0:r0 + step] if isinstance(x, torch.Tensor) else x for n, x in s.items()}
        z = part["logits"].double()
        if case["op"] != "fwd":
            z.requires_grad_()
        a, b = _exact_losses(part, z)
        if case["op"] != "fwd":
            d, = torch.autograd.grad(a, z, part["d_loss"].double())
            grads.append(d)
        loss.append(a.detach())
        stats.append(b.detach())
    if case["op"] == "fwd":
        return torch.cat(loss), torch.cat(stats)
    return torch.cat(grads) if case["op"] == "bwd" else (torch.cat(loss), torch.cat(grads))
