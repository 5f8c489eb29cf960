"""Linear attention on the GPU against the 64-bit recurrence.

Tolerances.  Every output value is a sum of products; `ref_abs` is the same
sum with every factor's absolute value.  The kernels form it in fp32 with
operands of 24 bits (states, dg, fp32 inputs) or 16 bits (two bf16 planes:
the pair weights, and X in o and dv), one fp32 exponential (2 ulp, and its
argument's rounding, below 16 * 2^-24 of a term that counts) and fp32 sums of at most 192 terms a
chunk (error below 2^-24 sqrt(192) of the sum of magnitudes for errors that
do not line up), then round once to the output's type:
  fp32 outputs: |err| <= 2^-19 ref_abs
  bf16 outputs: |err| <= 2^-8 |ref| + 2^-14 ref_abs
dg differs in that the pairs of a chunk enter two sums that cancel where they
do not straddle the token: its errors are relative to the largest dg_abs of
the sequence's head, 2^-19 of it.
"""
import pytest
import torch

import lin_ref as ref
from fp8_state_qat_amd import _lib, api

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def make(lens, H, Hk, dk, dv, dtype, gate="token", init=True, seed=0, gaps=(0, 0), scale=0.1):
    g0 = torch.Generator().manual_seed(seed)

    def rn(*s):
        return torch.randn(s, generator=g0)

    T, N = sum(lens) + sum(gaps), len(lens)
    cu = [gaps[0]]
    for n in lens:
        cu.append(cu[-1] + n)
    d = dict(q=rn(T, Hk, dk) / dk ** 0.5, k=rn(T, Hk, dk) / dk ** 0.5, v=rn(T, H, dv), do=rn(T, H, dv))
    d = {n: x.to(dtype) for n, x in d.items()}
    d["g"] = -scale * torch.nn.functional.softplus(rn(T, H)) if gate == "token" else -scale * torch.rand(H, generator=g0)
    d["S0"] = rn(N, H, dv, dk) if init else None
    d["dS"] = rn(N, H, dv, dk) if init else None
    d["cu"] = torch.tensor(cu, dtype=torch.int32)
    return d


def dev(d):
    return {n: None if x is None else x.cuda() for n, x in d.items()}


def close(got, want, mag, name):
    got, want = got.double().cpu(), want.double()
    assert torch.isfinite(got).all(), name
    tol = 2.0 ** -19 * mag
    if name.endswith("bf16"):
        tol = 2.0 ** -8 * want.abs() + 2.0 ** -14 * mag
    bad = (got - want).abs() > tol + 1e-30
    assert not bad.any(), f"{name}: {int(bad.sum())} values, worst {float((got - want).abs().max()):.3g}"


def tag(t):
    return "bf16" if t.dtype == BF else "fp32"


def check_fwd(d):
    x = dev(d)
    o, S = api.lin_attn_fwd(x["q"], x["k"], x["v"], x["g"], x["cu"], initial_state=x["S0"], check_status=True)
    a = (d["q"], d["k"], d["v"], d["g"], d["cu"], d["S0"])
    (ro, rS), (mo, mS) = ref.lin(*a), ref.lin_abs(*a)
    rows = slice(int(d["cu"][0]), int(d["cu"][-1]))
    close(o[rows], ro[rows], mo[rows], "o " + tag(o))
    close(S, rS, mS, "state fp32")
    return o, S


def check_bwd(d):
    x = dev(d)
    got = api.lin_attn_bwd(x["q"], x["k"], x["v"], x["g"], x["cu"], x["do"], initial_state=x["S0"],
                           d_final_state=x["dS"], check_status=True)
    a = (d["q"], d["k"], d["v"], d["g"], d["cu"], d["S0"], d["do"], d["dS"])
    want, mag = ref.lin(*a), list(ref.lin_abs(*a))
    mag[3] = mag[3].amax() if mag[3].dim() == 1 else mag[3].amax(0, keepdim=True)
    rows = slice(int(d["cu"][0]), int(d["cu"][-1]))
    for i, name in enumerate(("dq", "dk", "dv", "dg", "d_initial_state")):
        g, w, m = got[i], want[i], mag[i]
        if i < 3 or (i == 3 and g.dim() == 2):
            g, w = g[rows], w[rows]
            m = m[rows] if i < 3 else m
        close(g, w, m, f"{name} {tag(g)}")
    return got


SHAPES = [
    # lens, H, Hk, dk, dv, dtype, gate, init
    ([1], 1, 1, 64, 64, BF, "token", False),
    ([130], 4, 4, 64, 64, BF, "head", False),
    ([0, 1, 63, 64, 65], 2, 2, 128, 128, BF, "token", True),
    ([0, 1, 63, 64, 65], 2, 1, 64, 128, F32, "token", True),
    ([257, 0, 129], 6, 2, 64, 192, BF, "token", True),
    ([200, 3], 4, 1, 128, 256, BF, "head", True),
    ([333], 3, 3, 128, 64, F32, "head", True),
    ([70, 141], 2, 2, 128, 128, F32, "token", False),
    ([600, 515], 2, 2, 128, 128, BF, "token", True),     # several segments and stored states a sequence
]


@pytest.mark.parametrize("lens,H,Hk,dk,dv,dtype,gate,init", SHAPES)
def test_fwd(lens, H, Hk, dk, dv, dtype, gate, init):
    check_fwd(make(lens, H, Hk, dk, dv, dtype, gate, init))


@pytest.mark.parametrize("lens,H,Hk,dk,dv,dtype,gate,init", SHAPES)
def test_bwd(lens, H, Hk, dk, dv, dtype, gate, init):
    check_bwd(make(lens, H, Hk, dk, dv, dtype, gate, init, seed=1))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_whole_sequence_segments(dtype):
    """Enough (sequence, head) pairs for one segment a sequence; long ones hold several groups of stored states."""
    lens = [1, 0, 300, 64] + [5] * 126
    d = make(lens, 4, 2, 64, 64, dtype, "token", True, seed=2)
    check_fwd(d)
    check_bwd(d)


def test_rows_outside_the_sequences():
    """NaN in rows before, after and (as an empty sequence's) between: no influence, and nothing written there."""
    d = make([70, 0, 40], 2, 2, 64, 64, BF, gaps=(5, 9), seed=3)
    for n in ("q", "k", "v", "do", "g"):
        d[n][:5] = float("nan")
        d[n][-9:] = float("nan")
    x = dev(d)
    out = torch.full_like(x["v"], 3.0)
    api.lin_attn_fwd(x["q"], x["k"], x["v"], x["g"], x["cu"], initial_state=x["S0"], out=out)
    check_fwd(d)
    bufs = dict(dq=torch.full_like(x["q"], 3.0), dk=torch.full_like(x["k"], 3.0), d_v=torch.full_like(x["v"], 3.0),
                dg=torch.full_like(x["g"], 3.0))
    api.lin_attn_bwd(x["q"], x["k"], x["v"], x["g"], x["cu"], x["do"], initial_state=x["S0"],
                     d_final_state=x["dS"], **bufs)
    check_bwd(d)
    for t in (out, *bufs.values()):
        assert (t[:5] == 3.0).all() and (t[-9:] == 3.0).all() and (t[5:-9] != 3.0).any()


def test_rows_outside_with_shared_heads():
    """The same where dq, dk and dg pass through partial sums (shared heads, two value tiles)."""
    d = make([70, 40], 4, 2, 64, 256, BF, gaps=(5, 9), seed=4)
    x = dev(d)
    bufs = dict(dq=torch.full_like(x["q"], 3.0), dk=torch.full_like(x["k"], 3.0), dg=torch.full_like(x["g"], 3.0))
    api.lin_attn_bwd(x["q"], x["k"], x["v"], x["g"], x["cu"], x["do"], initial_state=x["S0"],
                     d_final_state=x["dS"], **bufs)
    for t in bufs.values():
        assert (t[:5] == 3.0).all() and (t[-9:] == 3.0).all() and (t[5:-9] != 3.0).any()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decays_at_the_ends(dtype):
    """No decay at all, decays that leave nothing within a token, and a reset (-inf)."""
    d = make([150, 90], 3, 3, 64, 64, dtype, seed=5)
    d["g"][:, 0] = 0.0
    d["g"][:, 1] = -60.0
    d["g"][::7, 2] = float("-inf")
    x = dev(d)
    o, S = api.lin_attn_fwd(x["q"], x["k"], x["v"], x["g"], x["cu"], initial_state=x["S0"])
    b = api.lin_attn_bwd(x["q"], x["k"], x["v"], x["g"], x["cu"], x["do"], initial_state=x["S0"],
                         d_final_state=x["dS"])
    a = (d["q"], d["k"], d["v"], d["g"].clamp(min=-1e4), d["cu"], d["S0"])
    (ro, rS), (mo, mS) = ref.lin(*a), ref.lin_abs(*a)
    close(o, ro, mo, "o " + tag(o))
    close(S, rS, mS, "state fp32")
    a = (*a, d["do"], d["dS"])
    want, mag = ref.lin(*a), list(ref.lin_abs(*a))
    # a reset's straddling pairs are 0 while the chunk's sums that cancel are not: relative to all heads' largest
    mag[3] = mag[3].amax().expand_as(mag[3])
    for i in range(5):
        close(b[i], want[i], mag[i], f"grad {i} {tag(b[i])}")


def test_bad_cu_seqlens_write_nothing():
    d = dev(make([64, 64], 2, 2, 64, 64, BF, seed=6))
    for bad in ([0, 100, 90], [-1, 64, 128], [0, 64, 129]):
        cu = torch.tensor(bad, dtype=torch.int32).cuda()
        out, S = torch.full_like(d["v"], 3.0), torch.full_like(d["S0"], 3.0)
        with pytest.raises(_lib.GdnError) as e:
            api.lin_attn_fwd(d["q"], d["k"], d["v"], d["g"], cu, out=out, final_state=S, check_status=True)
        assert e.value.status == _lib.GDN_ERR_INVALID_ARG
        assert (out == 3.0).all() and (S == 3.0).all()
        for g in (d["g"], d["g"][0].contiguous()):
            bufs = [torch.full_like(t, 3.0) for t in (d["q"], d["k"], d["v"], g, d["S0"])]
            with pytest.raises(_lib.GdnError):
                api.lin_attn_bwd(d["q"], d["k"], d["v"], g, cu, d["do"], dq=bufs[0], dk=bufs[1], d_v=bufs[2],
                                 dg=bufs[3], d_initial_state=bufs[4], check_status=True)
            assert all((t == 3.0).all() for t in bufs)


def test_no_tokens():
    d = dev(make([0, 0], 2, 1, 64, 64, BF, seed=7))
    o, S = api.lin_attn_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], initial_state=d["S0"], check_status=True)
    assert o.numel() == 0 and torch.equal(S, d["S0"])
    for g in (d["g"], torch.zeros(2, device="cuda")):
        b = api.lin_attn_bwd(d["q"], d["k"], d["v"], g, d["cu"], d["do"], d_final_state=d["dS"], check_status=True)
        assert torch.equal(b[4], d["dS"]) and not b[3].any()


def test_many_sequences():
    """More sequences than a wave scans at once."""
    d = make([(7 * i) % 5 for i in range(200)], 1, 1, 64, 64, BF, seed=8)
    check_fwd(d)
    check_bwd(d)


def test_repeatable_bit_for_bit_and_on_another_stream():
    d = dev(make([300, 90], 4, 2, 128, 256, BF, seed=9))

    def run():
        f = api.lin_attn_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], initial_state=d["S0"])
        return f + api.lin_attn_bwd(d["q"], d["k"], d["v"], d["g"], d["cu"], d["do"], initial_state=d["S0"],
                                    d_final_state=d["dS"])

    a = run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = run()
    s.synchronize()
    for x, y in zip(a, b):
        assert torch.equal(x, y)


@pytest.mark.parametrize("gate", ["token", "head"])
def test_graph_replays(gate):
    d = dev(make([200, 40], 2, 1, 64, 128, BF, gate, seed=10))
    ws = torch.empty(api.lin_attn_workspace_bytes(2, 2, 1, 64, 128, 240, gate_per_token=gate == "token", backward=True),
                     dtype=torch.uint8, device="cuda")
    run = lambda: api.lin_attn_bwd(d["q"], d["k"], d["v"], d["g"], d["cu"], d["do"], initial_state=d["S0"],  # noqa: E731
                                   d_final_state=d["dS"], workspace=ws)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for i in range(3):
        d["v"].copy_(torch.randn_like(d["v"]))
        for t in out:
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for x, y in zip(got, run()):
            assert torch.equal(x, y), i


def test_offsets_past_32_bits():
    """A long prompt ahead: rows whose byte and element offsets pass 2^32 and 2^31 come out as alone."""
    H, dk, dv, T, n = 16, 64, 256, 540_000, 100
    q, k = (torch.empty(T, H, dk, dtype=BF, device="cuda").normal_() / 8 for _ in range(2))
    v = torch.empty(T, H, dv, dtype=BF, device="cuda").normal_()
    g = torch.full((H,), -0.05, device="cuda")
    o, S = api.lin_attn_fwd(q, k, v, g, torch.tensor([0, T - n, T], dtype=torch.int32, device="cuda"))
    a = [x[T - n:].cpu() for x in (q, k, v)]
    cu = [0, n]
    (ro, rS), (mo, mS) = ref.lin(*a, g.cpu(), cu), ref.lin_abs(*a, g.cpu(), cu)
    close(o[T - n:], ro, mo, "o bf16")
    close(S[1:], rS, mS, "state fp32")


STEPS = [(1, 1, 1, 64, 64, BF, "head"), (3, 6, 2, 64, 192, F32, "token"), (2, 16, 16, 128, 128, BF, "head"),
         (5, 4, 1, 128, 256, BF, "token"), (160, 4, 4, 128, 64, F32, "token"), (130, 4, 2, 64, 128, BF, "token")]


@pytest.mark.parametrize("N,H,Hk,dk,dv,dtype,gate", STEPS)
def test_step(N, H, Hk, dk, dv, dtype, gate):
    d = make([1] * N, H, Hk, dk, dv, dtype, gate, True, seed=11)
    x = dev(d)
    S = x["S0"].clone()
    o = api.lin_attn_step(x["q"], x["k"], x["v"], x["g"], S)
    a = (d["q"], d["k"], d["v"], d["g"], d["cu"], d["S0"])
    (ro, rS), (mo, mS) = ref.lin(*a), ref.lin_abs(*a)
    close(o, ro, mo, "o " + tag(o))
    close(S, rS, mS, "state fp32")
    # the same token as a packed prompt of one-token sequences
    o2, S2 = api.lin_attn_fwd(x["q"], x["k"], x["v"], x["g"], x["cu"], initial_state=x["S0"])
    close(o2, ro, mo, "o " + tag(o))
    close(S2, rS, mS, "state fp32")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("name", ["q", "k", "v"])
def test_non_finite_values_do_not_reach_earlier_tokens(dtype, name):
    """An infinity or a NaN reaches what the recurrence says: from its token on, its value row (v), all rows (k),
    or its token alone (q); everything else keeps its bits."""
    lens = [150, 70, 40]
    d = dev(make(lens, 2, 1 if name != "v" else 2, 64, 128, dtype, seed=12))
    args = (d["g"], d["cu"])
    o0, S0 = api.lin_attn_fwd(d["q"], d["k"], d["v"], *args, initial_state=d["S0"])
    for t, col, x in ((37, 5, float("inf")), (63, 17, float("nan")), (149, 40, float("-inf")), (150, 3, float("nan")),
                      (219, 63, float("inf"))):
        n, end = (0, 150) if t < 150 else (1, 220)
        b = d[name].clone()
        b[t, 0, col] = x
        o, S = api.lin_attn_fwd(*(b if m == name else d[m] for m in ("q", "k", "v")), *args, initial_state=d["S0"])
        hit = torch.zeros_like(o0, dtype=torch.bool)
        hit_S = torch.zeros_like(S0, dtype=torch.bool)
        if name == "v":
            hit[t:end, 0, col] = True
            hit_S[n, 0, col] = True
        elif name == "k":
            hit[t:end] = True
            hit_S[n, :, :, col] = True
        else:
            hit[t] = True
        assert not torch.isfinite(o[hit]).any(), (t, col)
        assert torch.equal(o[~hit], o0[~hit]), (t, col)
        assert not torch.isfinite(S[hit_S]).any() and torch.equal(S[~hit_S], S0[~hit_S]), (t, col)
