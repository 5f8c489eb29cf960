"""What a token of the linear-attention backward can reach: gradients of the
log decays on the scale of their own chunk, and values that are not finite.

Tolerance of dg.  With i >= t > j the pairs that token t lies between,
dg_abs_t is the sum of their magnitudes.  A pair's product is off by at most
2^-19 of its magnitude (two fp32 sums of up to 192 terms, 2^-24 sqrt(192)
each, and the weight's exponential, 16 * 2^-24).  A chunk forms dg of its 64
tokens from sums over all its pairs, those that do not lie across a token
cancelling: every pair of the chunk lies across one of its tokens, so their
magnitudes add up to at most the sum of the chunk's dg_abs, 64 times its
largest, and none exceeds that largest.  Errors that do not line up then add
up to at most sqrt(64) * 2^-19 = 2^-16 of the largest dg_abs of the chunk (of
this sequence and head).  For one decay a head these add up over the chunks,
and the result is rounded once to fp32 (2^-24).
"""
import pytest
import torch

import lin_ref as ref
from fp8_state_qat_amd import api
from test_gpu_lin import BF, F32, close, dev, make

pytestmark = pytest.mark.gpu

# Sequences that are walked whole: enough (sequence, head) pairs to fill the card without cutting them.
FILL = [1] * 127


def chunk_largest(x, cu):
    """Largest |x| of the 64-token chunk (of a sequence) that a row lies in, for each head."""
    out = x.abs().clone()
    for a, b in zip(cu[:-1], cu[1:]):
        for c in range(a, b, 64):
            r = slice(c, min(b, c + 64))
            out[r] = out[r].amax(0, keepdim=True)
    return out


def grads(d):
    x = dev(d)
    return api.lin_attn_bwd(x["q"], x["k"], x["v"], x["g"], x["cu"], x["do"], initial_state=x["S0"],
                            d_final_state=x["dS"], check_status=True)


def check_dg(d):
    a = (d["q"], d["k"], d["v"], d["g"].clamp(min=-1e4), d["cu"], d["S0"], d["do"], d["dS"])
    T = d["v"].shape[0]
    per_token = list(a)
    per_token[3] = a[3].expand(T, -1).contiguous()
    want, mag = ref.lin(*a)[3], ref.lin_abs(*per_token)[3]
    cu = [int(x) for x in d["cu"]]
    tol = 2.0 ** -16 * chunk_largest(mag, cu)
    if d["g"].dim() == 1:
        first = torch.zeros(T, 1, dtype=torch.bool)
        for s, e in zip(cu[:-1], cu[1:]):
            first[s:e:64] = True
        tol = (tol * first).sum(0) + 2.0 ** -24 * want.abs()
    else:
        tol = tol + 2.0 ** -24 * want.abs()
    got = grads(d)[3].double().cpu()
    assert torch.isfinite(got).all()
    bad = (got - want).abs() > tol + 1e-30
    assert not bad.any(), (int(bad.sum()), [int(i) for i in bad.nonzero()[0]],
                           float(((got - want).abs() / (tol + 1e-30)).max()))
    return got


SHAPES = [
    # lens, H, Hk, dk, dv, dtype, gate, init
    ([1], 1, 1, 64, 64, BF, "token", False),
    ([0, 1, 63, 64, 65, 300], 2, 2, 128, 128, BF, "token", True),
    ([0, 1, 63, 64, 65, 300], 2, 1, 64, 128, F32, "token", True),
    ([257, 0, 129], 6, 2, 64, 192, BF, "token", True),
    ([333], 3, 3, 128, 64, F32, "head", True),
    ([200, 3], 4, 1, 128, 256, BF, "head", False),
    ([300] + FILL, 4, 4, 64, 64, BF, "token", True),
    ([300] + FILL, 4, 2, 128, 128, F32, "token", True),
    ([700, 515], 64, 64, 64, 64, BF, "token", True),        # segments of several chunks
]


@pytest.mark.parametrize("lens,H,Hk,dk,dv,dtype,gate,init", SHAPES)
def test_dg_on_the_scale_of_its_chunk(lens, H, Hk, dk, dv, dtype, gate, init):
    check_dg(make(lens, H, Hk, dk, dv, dtype, gate, init, seed=21))


@pytest.mark.parametrize("lens", [[256] + FILL, [256]])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("name", ["k", "v", "q", "do"])
def test_outliers_do_not_reach_other_chunks(lens, dtype, name):
    """One row 2^27 times the others, past several chunks of one walk: dg of the chunks that the row does not
    reach keeps its own scale."""
    d = make(lens, 4, 4, 64, 128, dtype, seed=22)
    d[name][130] *= 2.0 ** 27
    check_dg(d)


@pytest.mark.parametrize("lens", [[250, 90] + FILL, [250, 90]])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_strong_decays_are_judged_on_their_own(lens, dtype):
    """No decay, one that leaves e^-60 a token, and mixed ones: each head's dg on the scale of its own sums."""
    d = make(lens, 4, 4, 64, 64, dtype, seed=23)
    d["g"][:, 0] = 0.0
    d["g"][:, 1] = -60.0
    d["g"][::9, 2] = -30.0
    d["g"][::64, 3] = -100.0
    check_dg(d)


@pytest.mark.parametrize("lens", [[250, 90] + FILL, [250, 90]])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_resets_have_no_gradient(lens, dtype):
    """The derivative of e^g at g = -inf is 0, as is that of a log decay whose e^g is 0 in fp32: exactly."""
    d = make(lens, 4, 2, 64, 64, dtype, seed=25)
    d["g"][::7, 2] = float("-inf")
    d["g"][::5, 1] = -200.0
    d["g"][:, 3] = float("-inf")
    got = check_dg(d)
    assert not got[::7, 2].any() and not got[::5, 1].any() and not got[:, 3].any() and got[:, 2].any()
    d["g"] = torch.tensor([-0.1, float("-inf"), -0.05, -300.0])
    got = check_dg(d)
    assert not got[1] and not got[3] and got[0] and got[2]


@pytest.mark.parametrize("lens", [[150, 90] + FILL, [150, 90]])
@pytest.mark.parametrize("gate", ["token", "head"])
def test_strong_decays_keep_fp32(lens, gate):
    """Outputs that only far tokens or the initial state reach, through decays of e^-15 to e^-60, keep fp32's
    precision: 2^-19 of their magnitudes, as test_gpu_lin.py has it for every fp32 output."""
    d = make(lens, 4, 4, 64, 64, F32, gate, seed=26)
    d["g"] = 10 * d["g"] - 1.5
    T = d["v"].shape[0]
    far = torch.arange(T) % 24 == 23
    far[:30] = False
    d["k"][~far] = 0
    d["do"][torch.arange(T) % 24 != 11] = 0
    x = dev(d)
    o, S = api.lin_attn_fwd(x["q"], x["k"], x["v"], x["g"], x["cu"], initial_state=x["S0"])
    a = (d["q"], d["k"], d["v"], d["g"], d["cu"], d["S0"])
    (ro, rS), (mo, mS) = ref.lin(*a), ref.lin_abs(*a)
    close(o, ro, mo, "o fp32")
    close(S, rS, mS, "state fp32")
    want, mag, got = ref.lin(*a, d["do"], d["dS"]), ref.lin_abs(*a, d["do"], d["dS"]), grads(d)
    for i, name in ((0, "dq"), (1, "dk"), (2, "dv"), (4, "d_initial_state")):
        close(got[i], want[i], mag[i], f"{name} fp32")
    # the step: one token whose state only decays
    x["v"][:1] = 0
    n, g = 1, torch.tensor([[-15.3, -33.7, -58.9, -71.3]])
    S = x["S0"][:1].clone()
    api.lin_attn_step(x["q"][:n], x["k"][:n], x["v"][:n], g.cuda(), S)
    want = d["S0"][:1].double() * g.double().exp()[..., None, None]
    close(S, want, want.abs(), "step's state fp32")


def reach(d, name, t, H, Hk, h):
    """Rows of (dq, dk, dv, dg) and heads, and of d_initial_state, that an infinity or a NaN in row t, head h of an
    input may reach: those of the recurrence, and the chunk of 64 tokens around t."""
    cu = [int(x) for x in d["cu"]]
    n = max(i for i in range(len(cu) - 1) if cu[i] <= t)
    a, b = cu[n], cu[n + 1]
    c0 = a + (t - a) // 64 * 64
    c1 = min(b, c0 + 64)
    back, ahead, chunk = slice(a, c1), slice(c0, b), slice(c0, c1)
    rows = {"q": (chunk, back, back, back), "do": (chunk, back, back, back), "k": (ahead, chunk, chunk, ahead),
            "v": (ahead, chunk, chunk, ahead), "g": (ahead, back, back, slice(a, b))}[name]
    share = H // Hk
    heads = range(share * h, share * h + share) if name in "qk" else [h]
    return n, rows, list(heads), sorted({x // share for x in heads}), name in ("q", "do", "g")


@pytest.mark.parametrize("lens", [[150, 300, 70], [150, 300, 70] + FILL])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("name", ["q", "k", "v", "do", "g"])
def test_non_finite_values_stay_in_their_reach(lens, dtype, name):
    """An infinity or a NaN reaches what the recurrence says and its chunk; every other gradient, other sequences and
    other heads among them, keeps its bits."""
    H, Hk = 4, 2
    d = make(lens, H, Hk, 64, 128, dtype, seed=24)
    clean = [x.cpu() for x in grads(d)]
    assert all(torch.isfinite(x).all() for x in clean)
    for t, h, x in ((37, 0, float("inf")), (149, 1, float("nan")), (150, 0, float("nan")), (150 + 200, 1, float("-inf")),
                    (519, 1, float("nan"))):
        if name == "g" and x == float("-inf"):
            x = float("nan")                    # -inf is a reset, nothing that spreads
        e = dict(d, **{name: d[name].clone()})
        if name == "g":
            e["g"][t, h] = x
        else:
            e[name][t, h, 5] = x
        got = [y.cpu() for y in grads(e)]
        n, rows, heads, qk_heads, start = reach(d, name, t, H, Hk, h)
        for i, what in enumerate(("dq", "dk", "dv", "dg")):
            hit = torch.zeros_like(clean[i], dtype=torch.bool)
            sub = hit[rows[i]]
            sub[:, qk_heads if i < 2 else heads] = True
            assert torch.equal(got[i][~hit], clean[i][~hit]), (what, name, t, x)
        hit = torch.zeros_like(clean[4], dtype=torch.bool)
        if start:
            hit[n, heads] = True
        assert torch.equal(got[4][~hit], clean[4][~hit]), ("d_initial_state", name, t, x)
        assert not all(torch.isfinite(y).all() for y in got)


def test_backward_offsets_past_32_bits():
    """A long prompt ahead: rows whose byte and element offsets pass 2^32 and 2^31, also in the partial sums of dq and
    dk over two value tiles and in the stored states, come out as alone."""
    H, Hk, dk, dv, T, n = 16, 16, 64, 256, 540_000, 100
    q, k = (torch.empty(T, Hk, dk, dtype=BF, device="cuda").normal_() / 8 for _ in range(2))
    v, do = (torch.empty(T, H, dv, dtype=BF, device="cuda").normal_() for _ in range(2))
    g = -0.1 * torch.rand(T, H, device="cuda")
    got = api.lin_attn_bwd(q, k, v, g, torch.tensor([0, T - n, T], dtype=torch.int32, device="cuda"), do,
                           check_status=True)
    a = [x[T - n:].cpu() for x in (q, k, v, g)]
    args = (*a, [0, n], None, do[T - n:].cpu(), None)
    want, mag = ref.lin(*args), ref.lin_abs(*args)
    for i, name in enumerate(("dq bf16", "dk bf16", "dv bf16")):
        close(got[i][T - n:], want[i], mag[i], name)
    close(got[4][1:], want[4], mag[4], "d_initial_state fp32")
    err = (got[3][T - n:].double().cpu() - want[3]).abs()
    assert not (err > 2.0 ** -16 * chunk_largest(mag[3], [0, n]) + 2.0 ** -24 * want[3].abs()).any()
