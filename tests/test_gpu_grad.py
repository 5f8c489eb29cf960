"""All gradients of the gated delta rule on the GPU against the token recurrence in 64 bits.

Tolerances.  With unit keys and beta in (0, 1) a token's step is a contraction, so that an error made in a chunk is
not enlarged by the later ones, and a chunk's own triangular solve keeps vectors within the norms of the recurrence.
An output is a sum of products of two vectors whose errors are relative to their norms: with S, R the largest
Frobenius norms of a state and of a state's gradient over the sequence and head, e, y, o the largest norms of a
token's error, value gradient and output gradient,
    |dq| <= o S,  |dk| <= y S + e R,  |dv| <= R + o,  |dbeta| <= R e,  |dg| <= S R,  |dS0| <= R.
bf16 inputs: operands of 16 bits, each rounding and each dropped product of low parts at most 2^-17; a path from the
inputs to an output has at most five products of two such operands, 3 roundings each: 15 * 2^-17 < 2^-13 of the
bound.  fp32 inputs: at most 128 terms a sum on the matrix unit, (128 + 15) * 2^-24 a product, five of them: 2^-14
at worst; held to 2^-16, as sums of random signs stay a factor of their root below.  Stored bf16 outputs add a
rounding: 2^-8 of the value.
"""
import pytest
import torch

import grad_ref as ref
from fp8_state_qat_amd import GdnError, api
from fp8_state_qat_amd._lib import GDN_QDQ_CHUNK, GDN_QDQ_WRITE

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAMES = ("dq", "dk", "dv", "dbeta", "dg", "dS0")


def make(seg, H, dk, dv, dtype, lens=None, init=True, fin=True, seed=0, gate=0.1, tail=0):
    """Packed inputs on the CPU; tail: rows behind the last segment."""
    gen = torch.Generator().manual_seed(seed)
    T = sum(seg) + tail

    def rn(*s):
        return torch.randn(*s, generator=gen)

    def unit(x):
        return x / x.norm(dim=-1, keepdim=True)

    N = len(seg)
    d = dict(q=(unit(rn(T, H, dk)) * dk ** -0.5).to(dtype), k=unit(rn(T, H, dk)).to(dtype), v=rn(T, H, dv).to(dtype),
             beta=torch.sigmoid(rn(T, H)), g=-gate * torch.nn.functional.softplus(rn(T, H)), d_o=rn(T, H, dv).to(dtype))
    d["cu"] = torch.tensor([0] + seg).cumsum(0).int()
    d["lens"] = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    d["S0"] = rn(N, H, dv, dk) if init else None
    d["dS"] = rn(N, H, dv, dk) if fin else None
    return d


def dev(d):
    return {k: None if x is None else x.cuda() for k, x in d.items()}


def run(d, states=None, **kw):
    x = dev(d)
    return api.chunk_grad(x["q"], x["k"], x["v"], x["beta"], x["g"], x["cu"], x["d_o"], seq_lens=x["lens"],
                          initial_state=x["S0"], d_final_state=x["dS"], states=states, check_status=True, **kw)


def want(d, states=None):
    return ref.grad(d["q"], d["k"], d["v"], d["beta"], d["g"], d["cu"], d["d_o"], d["lens"], d["S0"], d["dS"], states)


def bounds(d, states=None):
    """The norms' bounds of every output, per sequence and head, spread over its rows."""
    T, H, dk = d["k"].shape
    out = [torch.zeros(T, H, 1), torch.zeros(T, H, 1), torch.zeros(T, H, 1), torch.zeros(T, H), torch.zeros(T, H)]
    last, at = [], 0
    cu = d["cu"].tolist()
    for n in range(len(cu) - 1):
        L = cu[n + 1] - cu[n] if d["lens"] is None else int(d["lens"][n])
        r = slice(cu[n], cu[n] + L)
        q, k, v, b, g, do = (d[m][r].double() for m in ("q", "k", "v", "beta", "g", "d_o"))
        zero = torch.zeros(H, v.shape[2], dk, dtype=torch.float64)
        every = None
        if states is not None:
            def every(t, S, at=at):
                return states[at + t // 64 - 1].double().cpu() if t % 64 == 0 else S
        _, steps, _ = ref.forward(q, k, v, b, g, zero if d["S0"] is None else d["S0"][n].double(), every)
        R = zero if d["dS"] is None else d["dS"][n].double()
        S = torch.stack([zero.flatten(1).norm(dim=1)] + [s[3].flatten(1).norm(dim=1) for s in steps] +
                        [s[0].flatten(1).norm(dim=1) for s in steps]).amax(0)
        e = torch.stack([zero[:, :, 0].norm(dim=1)] + [s[2].norm(dim=1) for s in steps]).amax(0)
        o = do.norm(dim=2).amax(0) if L else torch.zeros(H).double()
        Rm = R.flatten(1).norm(dim=1)
        y = torch.zeros(H).double()
        for t in range(L - 1, -1, -1):
            R = R + do[t][:, :, None] * q[t][:, None, :]
            Rk = (R * k[t][:, None, :]).sum(-1)
            Rm = torch.maximum(Rm, R.flatten(1).norm(dim=1))
            y = torch.maximum(y, Rk.norm(dim=1))
            R = (R - (b[t][:, None] * Rk)[:, :, None] * k[t][:, None, :]) * g[t].exp()[:, None, None]
        out[0][r] = (o * S).float()[None, :, None]
        out[1][r] = (y * S + e * Rm).float()[None, :, None]
        out[2][r] = (Rm + o).float()[None, :, None]
        out[3][r] = (Rm * e).float()[None]
        out[4][r] = (S * Rm).float()[None]
        last.append(Rm)
        at += -(-L // 64)
    return (*out, torch.stack(last)[:, :, None, None])


def close(got, wanted, bound, dtype):
    u = 2.0 ** -13 if dtype == BF else 2.0 ** -16
    for name, g, w, b in zip(NAMES, got, wanted, bound):
        g = g.cpu()
        assert torch.isfinite(g).all(), name
        tol = u * b.double() + (2.0 ** -8 * w.abs() if g.dtype == BF else 0)
        bad = (g.double() - w).abs() > tol + 1e-30
        assert not bad.any(), f"{name}: {int(bad.sum())} values, worst {float((g.double() - w).abs().max()):.3g}"


SHAPES = [
    # segments, valid lengths, heads, dk, dv, dtype, initial, final
    ([1], None, 1, 64, 64, BF, False, False),
    ([2], None, 1, 128, 64, BF, True, True),
    ([63], None, 2, 64, 64, BF, False, True),
    ([64], None, 1, 128, 128, BF, True, False),
    ([65], None, 3, 64, 128, BF, True, True),
    ([0, 1, 130, 0, 64, 17], None, 2, 64, 64, BF, True, True),
    ([70, 129, 5], [70, 100, 0], 2, 128, 192, BF, True, True),
    ([200, 64], [190, 64], 3, 64, 256, BF, False, True),
    ([333], None, 2, 128, 256, BF, True, True),
    ([1], None, 1, 128, 128, F32, True, True),
    ([64, 0, 65], None, 2, 64, 64, F32, True, True),
    ([150, 31], [129, 31], 2, 128, 64, F32, False, True),
    ([130], None, 1, 64, 192, F32, True, False),
    ([100, 70], [65, 70], 1, 128, 256, F32, True, True),
]


@pytest.mark.parametrize("seg,lens,H,dk,dv,dtype,init,fin", SHAPES)
def test_against_64_bits(seg, lens, H, dk, dv, dtype, init, fin):
    d = make(seg, H, dk, dv, dtype, lens, init, fin, seed=len(seg) + dv)
    close(run(d), want(d), bounds(d), dtype)


def n_bounds(d):
    cu = d["cu"].tolist()
    L = [b - a for a, b in zip(cu, cu[1:])] if d["lens"] is None else d["lens"].tolist()
    return [-(-x // 64) for x in L]


@pytest.mark.parametrize("dk,dv,dtype", [(64, 64, BF), (128, 128, BF), (64, 192, BF), (128, 256, BF), (64, 128, F32),
                                         (128, 128, F32)])
def test_given_states(dk, dv, dtype):
    """States of any origin: what every chunk after a sequence's first starts from."""
    d = make([70, 0, 200, 64], 2, dk, dv, dtype, [70, 0, 190, 64], seed=5)
    gen = torch.Generator().manual_seed(9)
    states = torch.randn(sum(n_bounds(d)), 2, dv, dk, generator=gen)
    close(run(d, states.cuda()), want(d, states), bounds(d, states), dtype)


@pytest.mark.parametrize("dk,dv,dtype,given", [(64, 64, BF, False), (128, 128, BF, False), (128, 64, BF, True),
                                               (64, 128, F32, False), (128, 64, F32, True)])
def test_many_sequences(dk, dv, dtype, given):
    """More chains than compute units, whose workgroups are wider: the bits that a sequence gives alone."""
    seg = [(7 * i * i + 1) % 131 for i in range(40)]
    d = make(seg, 4, dk, dv, dtype, seed=11)
    nb = n_bounds(d)
    states = torch.randn(sum(nb), 4, dv, dk, generator=torch.Generator().manual_seed(12)) if given else None
    got = run(d, None if states is None else states.cuda())
    close(got, want(d, states), bounds(d, states), dtype)
    for n in (0, 3, 39):
        r, at = slice(int(d["cu"][n]), int(d["cu"][n + 1])), sum(nb[:n])
        one = {m: None if x is None else x[n:n + 1] if m in ("S0", "dS") else x[r] for m, x in d.items() if m != "cu"}
        one["cu"] = torch.tensor([0, seg[n]], dtype=torch.int32)
        alone = run(one, None if states is None else states[at:at + nb[n]].cuda())
        for name, x, y in zip(NAMES, got, alone):
            assert torch.equal(x[n:n + 1] if name == "dS0" else x[r], y), (n, name)


@pytest.mark.parametrize("dk,dtype", [(64, BF), (128, BF), (64, F32), (128, F32)])
@pytest.mark.parametrize("flags", [GDN_QDQ_CHUNK, GDN_QDQ_CHUNK | GDN_QDQ_WRITE])
def test_quantized_forward(dk, dtype, flags):
    """Recomputed with the state's QDQ: the bits that the forward's own recorded states give, and their gradients."""
    d = make([130, 64, 200], 2, dk, 64, dtype, [130, 60, 200], seed=6)
    x = dev(d)
    nb = n_bounds(d)
    offs = torch.tensor([0] + nb).cumsum(0).int().cuda()
    post = torch.zeros(sum(nb), 2, 64, dk, device="cuda")
    api.chunk_fwd(x["q"], x["k"], x["v"], x["beta"], x["g"], x["cu"], seq_lens=x["lens"], initial_state=x["S0"],
                  qdq_flags=flags, debug=dict(bound_offsets=offs, bound_post=post))
    given = run(d, post, qdq_flags=flags)
    again = run(d, qdq_flags=flags)
    for name, a, b in zip(NAMES, given, again):
        assert torch.equal(a, b), name
    close(again, want(d, post), bounds(d, post), dtype)


def test_write_flag_changes_nothing():
    d = make([130], 1, 64, 64, BF)
    for a, b in zip(run(d), run(d, qdq_flags=GDN_QDQ_WRITE)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_padding_is_not_read_and_rows_behind_are_left(dtype):
    """NaN in padding and behind the last segment reaches nothing; padding gets zeros, the rows behind keep theirs."""
    d = make([100, 64, 3], 2, 64, 64, dtype, [70, 0, 3], seed=7, tail=9)
    clean = run(d)
    live = torch.zeros(176, dtype=torch.bool)
    for a, n in ((0, 70), (100, 0), (164, 3)):
        live[a:a + n] = True
    for m in ("q", "k", "v", "beta", "g", "d_o"):
        d[m][~live] = float("nan")
    x = dev(d)
    outs = [torch.full_like(x[m], 7.0) for m in ("q", "k", "v", "beta", "g")]
    got = run(d, dq=outs[0], dk=outs[1], d_v=outs[2], d_beta=outs[3], dg=outs[4])
    for name, a, b in zip(NAMES, got, clean):
        if name == "dS0":
            assert torch.equal(a, b)
            continue
        assert torch.equal(a[live.cuda()], b[live.cuda()]), name
        assert (a[:167][~live[:167].cuda()] == 0).all(), name
        assert (a[167:] == 7.0).all(), name


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strong_and_absent_decays(dtype):
    """Log-gates from 0 to -200 a token, some tokens that forget everything (e^g = 0: no gradient)."""
    d = make([200], 2, 64, 64, dtype, seed=8)
    gen = torch.Generator().manual_seed(3)
    d["g"] = -torch.rand(200, 2, generator=gen) * 10 ** (3 * torch.rand(200, 2, generator=gen) - 1)
    d["g"][17] = 0.0
    d["g"][100, 0] = -1e5
    d["g"][101:140, 1] = -60.0
    got = run(d)
    close(got, want(d), bounds(d), dtype)
    assert float(got[4][100, 0]) == 0.0


def test_zero_beta_and_zero_keys():
    d = make([130], 2, 64, 64, BF, seed=10)
    d["beta"][::3] = 0.0
    d["beta"][64:100, 1] = 0.0
    d["k"][5] = 0.0
    close(run(d), want(d), bounds(d), BF)


def test_repeats_bit_for_bit_also_at_once_on_two_streams():
    d = make([300, 65, 1], 3, 128, 128, BF, seed=11)
    first = run(d)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(3):
                outs.append(run(d))
    torch.cuda.synchronize()
    for o in outs:
        for name, a, b in zip(NAMES, first, o):
            assert torch.equal(a, b), name


@pytest.mark.parametrize("flags", [0, GDN_QDQ_CHUNK])
def test_captured_and_replayed(flags):
    d = make([200, 64], 2, 128, 64, BF, seed=12)
    x = dev(d)
    ws = torch.empty(api.chunk_grad_workspace_bytes(2, 2, 128, 64, 264, qdq_flags=flags), dtype=torch.uint8,
                     device="cuda")

    def call():
        return api.chunk_grad(x["q"], x["k"], x["v"], x["beta"], x["g"], x["cu"], x["d_o"], initial_state=x["S0"],
                              d_final_state=x["dS"], workspace=ws, qdq_flags=flags)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for i in range(3):
        fresh = make([200, 64], 2, 128, 64, BF, seed=20 + i)
        for m in ("q", "k", "v", "beta", "g", "d_o", "S0", "dS"):
            x[m].copy_(fresh[m])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for name, a, b in zip(NAMES, got, run(fresh, qdq_flags=flags)):
            assert torch.equal(a, b), (i, name)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("what", ["q", "k", "v", "d_o"])
def test_what_is_not_finite_stays_in_its_sequence_and_head(what, dtype):
    d = make([70, 130, 40], 2, 64, 128, dtype, [70, 129, 40], seed=21)
    plain = run(d)
    d[what] = d[what].clone()
    d[what][70 + 100, 1, 5] = float("inf")
    got = run(d)
    assert not torch.isfinite(got[0][70:199, 1].float()).all() or not torch.isfinite(got[1][70:199, 1].float()).all()
    for name, x, y in zip(NAMES, got, plain):
        if name == "dS0":
            assert torch.equal(x[[0, 2]], y[[0, 2]]) and torch.equal(x[1, 0], y[1, 0]), name
        else:
            assert torch.equal(x[:70], y[:70]) and torch.equal(x[199:], y[199:]), name
            assert torch.equal(x[70:199, 0], y[70:199, 0]), name


@pytest.mark.parametrize("bad", [[0, 50, 40], [0, 64, 200], [-1, 64, 100]])
def test_bad_index_arrays_write_nothing(bad):
    d = make([64, 36], 1, 64, 64, BF, seed=13)
    x = dev(d)
    cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
    outs = dict(dq=x["q"], dk=x["k"], d_v=x["v"], d_beta=x["beta"], dg=x["g"], d_initial_state=x["S0"])
    outs = {m: torch.full_like(t, 3.0) for m, t in outs.items()}
    with pytest.raises(GdnError, match="out of contract"):
        api.chunk_grad(x["q"], x["k"], x["v"], x["beta"], x["g"], cu, x["d_o"], initial_state=x["S0"],
                       check_status=True, **outs)
    for m, t in outs.items():
        assert (t == 3.0).all(), m


def test_too_few_states_write_nothing():
    d = make([64, 136], 1, 64, 64, BF, seed=14)
    x = dev(d)
    dq = torch.full_like(x["q"], 3.0)
    for n in (3, 0):
        with pytest.raises(GdnError, match="out of contract"):
            api.chunk_grad(x["q"], x["k"], x["v"], x["beta"], x["g"], x["cu"], x["d_o"], dq=dq, check_status=True,
                           states=torch.zeros(n, 1, 64, 64, device="cuda"))
        assert (dq == 3.0).all()


def test_no_tokens():
    d = make([0, 0], 2, 64, 64, BF, seed=15)
    got = run(d)
    assert got[0].shape == (0, 2, 64) and torch.equal(got[5], d["dS"].cuda())


def test_offsets_past_32_bits():
    """A long document ahead: rows, stored states and records whose byte offsets pass 2^32 come out as alone."""
    H, dk, dv, T, n = 16, 128, 128, 300_000, 100
    gen = torch.Generator(device="cuda").manual_seed(0)

    def rn(*s):
        return torch.randn(*s, generator=gen, device="cuda")

    q, k, v, do = (torch.empty(T, H, dk, dtype=BF, device="cuda") for _ in range(4))
    for t in (q, k, v, do):
        for i in range(0, T, 50_000):
            t[i:i + 50_000] = rn(min(50_000, T - i), H, dk) / 11.3
    beta, g = torch.sigmoid(rn(T, H)), -0.1 * torch.rand(T, H, generator=gen, device="cuda")
    cu = torch.tensor([0, T - n, T], dtype=torch.int32, device="cuda")
    got = api.chunk_grad(q, k, v, beta, g, cu, do)
    alone = api.chunk_grad(*(t[T - n:].contiguous() for t in (q, k, v, beta, g)),
                           torch.tensor([0, n], dtype=torch.int32, device="cuda"), do[T - n:].contiguous())
    for name, a, b in zip(NAMES, got, alone):
        assert torch.equal(a[1:] if name == "dS0" else a[T - n:], b), name
    assert all(torch.isfinite(t).all() for t in got)
