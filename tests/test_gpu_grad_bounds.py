"""Gradients of the gated delta rule on the GPU at the borders that the calls document."""
import pytest
import torch

from fp8_state_qat_amd import GdnError, api
from fp8_state_qat_amd._lib import GDN_QDQ_CHUNK
from test_gpu_grad import BF, F32, NAMES, bounds, close, dev, make, n_bounds, run, want

pytestmark = pytest.mark.gpu


def test_padding_of_more_than_2_24_rows_gets_zeros():
    """Rows whose elements pass 2^31 in one segment."""
    T, L, dk, dv = (1 << 24) + 70, 65, 128, 64
    d = make([L], 1, dk, dv, BF, [L], False, False, seed=31)
    x = {m: torch.zeros((T, *d[m].shape[1:]), dtype=d[m].dtype, device="cuda") for m in ("q", "k", "v", "beta", "g", "d_o")}
    for m, t in x.items():
        t[:L] = d[m].cuda()
    outs = {n: torch.full_like(x[m], 7.0) for n, m in (("dq", "q"), ("dk", "k"), ("d_v", "v"), ("d_beta", "beta"), ("dg", "g"))}
    cu, lens = (torch.tensor(t, dtype=torch.int32, device="cuda") for t in ([0, T], [L]))
    got = api.chunk_grad(x["q"], x["k"], x["v"], x["beta"], x["g"], cu, x["d_o"], seq_lens=lens, check_status=True, **outs)
    alone = run(d)
    for name, a, b in zip(NAMES, got, alone):
        if name == "dS0":
            assert torch.equal(a, b)
            continue
        assert torch.equal(a[:L], b), name
        for i in range(L, T, 1 << 21):
            assert (a[i:i + (1 << 21)] == 0).all(), (name, i)


@pytest.mark.parametrize("dk,dtype", [(64, BF), (128, BF), (128, F32)])
def test_the_last_given_state_of_a_sequence_reaches_nothing(dk, dtype):
    d = make([70, 0, 200, 64], 2, dk, 64, dtype, [70, 0, 190, 64], seed=32)
    nb = n_bounds(d)
    states = torch.randn(sum(nb), 2, 64, dk, generator=torch.Generator().manual_seed(33))
    plain = run(d, states.cuda())
    for n in (0, 2, 3):
        states[sum(nb[:n + 1]) - 1] = float("nan")
    for name, a, b in zip(NAMES, run(d, states.cuda()), plain):
        assert torch.equal(a, b), name


@pytest.mark.parametrize("dk,dtype", [(64, BF), (128, BF), (64, F32), (128, F32)])
def test_the_forward_run_again_shares_the_call_s_status(dk, dtype):
    """Index arrays out of contract write nothing and are reported; the same workspace serves the next call; no tokens."""
    d = make([130, 64], 2, dk, 64, dtype, seed=34)
    x = dev(d)
    plain = run(d, qdq_flags=GDN_QDQ_CHUNK)
    ws = torch.empty(api.chunk_grad_workspace_bytes(2, 2, dk, 64, 194, dtype, GDN_QDQ_CHUNK), dtype=torch.uint8,
                     device="cuda")
    outs = dict(dq=x["q"], dk=x["k"], d_v=x["v"], d_beta=x["beta"], dg=x["g"], d_initial_state=x["S0"])
    outs = {m: torch.full_like(t, 3.0) for m, t in outs.items()}
    for bad in ([0, 130, 100], [0, 64, 500], [-1, 64, 100]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        with pytest.raises(GdnError, match="out of contract"):
            api.chunk_grad(x["q"], x["k"], x["v"], x["beta"], x["g"], cu, x["d_o"], initial_state=x["S0"],
                           qdq_flags=GDN_QDQ_CHUNK, workspace=ws, check_status=True, **outs)
        for m, t in outs.items():
            assert (t == 3.0).all(), m
    got = run(d, qdq_flags=GDN_QDQ_CHUNK, workspace=ws)
    for name, a, b in zip(NAMES, got, plain):
        assert torch.equal(a, b), name
    e = make([0, 0], 2, dk, 64, dtype, seed=35)
    got = run(e, qdq_flags=GDN_QDQ_CHUNK)
    assert got[0].shape == (0, 2, dk) and torch.equal(got[5], e["dS"].cuda())


# Norms of errors.  States, their gradients, d_v before its rounding, d_beta and dg take terms of 24 bits and sums in
# fp32: a product of at most 64 tokens and 128 channels is off by sqrt(192) 2^-24 of its terms' norm, for errors of
# random signs, and a path from the inputs to an output has at most five such products: sqrt(5 * 192) 2^-24 < 2^-19.
# (Terms of 16 bits would be off by 2^-17 / sqrt(3) each.)  With fp32 inputs the other gradients are as exact.
@pytest.mark.parametrize("dk,dv,dtype,given", [(64, 64, BF, False), (128, 128, BF, False), (64, 128, BF, True),
                                               (128, 192, BF, True), (64, 64, F32, False), (128, 128, F32, True)])
def test_terms_of_24_bits(dk, dv, dtype, given):
    d = make([700, 130], 2, dk, dv, dtype, seed=36)
    states = torch.randn(sum(n_bounds(d)), 2, dv, dk, generator=torch.Generator().manual_seed(37)) if given else None
    got, wanted = run(d, None if states is None else states.cuda()), want(d, states)
    for name, g, w in zip(NAMES, got, wanted):
        if g.dtype == F32:
            err = float((g.double().cpu() - w).norm() / w.norm())
            assert err < 2.0 ** -19, (name, err)


# A bf16 value of a sum that is off by e is off from the rounded sum's border by more than half a step only where the
# sum lies within e of it, which has a chance of 2 e over the step, 2^-8 of the value: with e = 2^-19 (above) the excess
# over half a step is in norm 2^-19 sqrt(2 * 2^-19 / 2^-8) = 2^-24 of the values', held to 4 times that.  (Terms of 16
# bits: sqrt(5) 2^-17, an excess of 2^-20.)
@pytest.mark.parametrize("dk,dv,given", [(64, 64, False), (128, 128, False), (64, 128, True), (128, 192, True)])
def test_bf16_gradients_are_sums_of_24_bits_rounded_once(dk, dv, given):
    d = make([700, 130], 2, dk, dv, BF, seed=38)
    states = torch.randn(sum(n_bounds(d)), 2, dv, dk, generator=torch.Generator().manual_seed(39)) if given else None
    got, wanted = run(d, None if states is None else states.cuda()), want(d, states)
    for name, g, w in zip(NAMES[:3], got, wanted):
        half = torch.ldexp(torch.ones_like(w), torch.frexp(w).exponent - 9)   # of a value's step, 2^-7 of its power of 2
        excess = ((g.double().cpu() - w).abs() - half).clamp(min=0)
        assert float(excess.norm() / w.norm()) < 2.0 ** -22, (name, float(excess.norm() / w.norm()))


@pytest.mark.parametrize("dk,dtype", [(64, BF), (128, F32)])
def test_dg_is_0_where_a_decay_is_0_in_fp32(dk, dtype):
    """e^g is 0 below 2^-150: g <= -103.97208, and 2^-149 from the next value on."""
    d = make([130], 2, dk, 64, dtype, seed=40)
    d["g"][7], d["g"][70], d["g"][71], d["g"][100] = -103.98, -103.99, -104.5, -103.97209
    assert float(torch.tensor(-103.97209).exp()) == 0
    got = run(d)[4]
    assert (got[[7, 70, 71, 100]] == 0).all(), got[[7, 70, 71, 100]]
    assert (got[[6, 8, 69, 72]] != 0).all()


# Every term across a token that keeps e^-20 of the state has that factor; it is off by 2^-20 of itself at most (three
# operands of 24 bits, sums in fp32 of at most 128 terms of random signs, decays to a few 2^-24), and what is not across
# the token cancels in 64 bits: of a chunk's sums of at most 2^7, 2^-46, against e^-20 = 2^-28.9: 2^-17.  Held to 2^-15.
@pytest.mark.parametrize("dk,dtype,given", [(64, BF, False), (128, BF, True), (64, F32, True), (128, F32, False)])
def test_dg_of_tokens_that_forget_nearly_all(dk, dtype, given):
    d = make([200, 64], 2, dk, 64, dtype, seed=41)
    at = [0, 5, 70, 127, 128, 199, 220]
    d["g"][at] = -20.0
    states = torch.randn(sum(n_bounds(d)), 2, 64, dk, generator=torch.Generator().manual_seed(42)) if given else None
    got, wanted = run(d, None if states is None else states.cuda())[4].cpu().double(), want(d, states)[4]
    err = (got - wanted)[at].norm() / wanted[at].norm()
    assert err < 2.0 ** -15, (float(err), got[at], wanted[at])


# In norm: a rounding is off by 2^-24 / sqrt(3) in the mean of squares, at a mean mantissa of 1.4 by 2^-25.3; a sum of n
# terms of random signs rounds partial sums of n / 2 of them in the mean; dg is made of three products of 64 tokens and
# 128 channels (S, R, and theirs), its own sums are fp64: sqrt(3 * 96) 2^-25.3 = 2^-21.2.
@pytest.mark.parametrize("seg,dk,dv,dtype", [([632], 64, 64, F32), ([700], 64, 128, BF), ([300, 333], 128, 64, BF)])
def test_dg_is_as_exact_as_its_terms(seg, dk, dv, dtype):
    d = make(seg, 4, dk, dv, dtype, init=False, fin=False, seed=43)
    err = (run(d)[4].cpu().double() - want(d)[4]).norm() / want(d)[4].norm()
    assert err < 2.0 ** -21, float(err)


@pytest.mark.parametrize("dk,dtype,given", [(64, BF, False), (128, BF, True), (64, F32, True), (128, F32, False)])
def test_resets(dk, dtype, given):
    """Log-gates of -inf: alone, at a chunk's first and last token, several in a row, at a sequence's first."""
    d = make([200, 70], 2, dk, 64, dtype, seed=44)
    at = [0, 7, 63, 64, 100, 101, 102, 199, 200]
    d["g"][at] = -float("inf")
    d["g"][150, 0] = -float("inf")
    states = torch.randn(sum(n_bounds(d)), 2, 64, dk, generator=torch.Generator().manual_seed(45)) if given else None
    got, wanted = run(d, None if states is None else states.cuda()), want(d, states)
    close(got, wanted, bounds(d, states), dtype)
    assert (got[4][at] == 0).all() and got[4][150, 0] == 0
    assert (got[5][:, :] == 0).all()     # nothing reaches the initial states


def test_thousands_of_short_sequences():
    """Sequences of 0 to 3 tokens, more than one scan's workgroup counts at a time."""
    gen = torch.Generator().manual_seed(46)
    seg = torch.randint(0, 4, (3000,), generator=gen).tolist()
    d = make(seg, 1, 64, 64, BF, seed=47)
    got, wanted = run(d), want(d)
    close(got, wanted, bounds(d), BF)
