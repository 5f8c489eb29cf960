"""Block norms and 8-bit activations on the GPU against 64 bits.

Tolerances.  A row sum of D fp32 squares is off by at most 2^-24 (D / TPR + 12)
of itself (TPR threads a row, at most 32 values a thread and 12 tree steps): 44 * 2^-24, half of it in the
root; with the products around it an output's value is within 2^-18 of the sum of its terms' magnitudes
(the gate's exponential adds a few 2^-24, a gate argument up to 8 times as much), then rounded
once: fp32 |err| <= 2^-18 mag, bf16 2^-8 |ref| + 2^-18 mag.  The weights'
gradients are sums over the rows: 2^-18 of their magnitudes' sum.  Codes and
scales are exact.
"""
import pytest
import torch

import lin_ref as ref
from fp8_state_qat_amd import api

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def close(got, want, mag, name):
    w = want.double()
    got_c = got.double().cpu()
    assert torch.isfinite(got_c).all(), name
    tol = 2.0 ** -18 * mag + (2.0 ** -8 * w.abs() if got.dtype == BF else 0)
    bad = (got_c - w).abs() > tol + 1e-30
    assert not bad.any(), f"{name}: {int(bad.sum())} values, worst {float((got_c - w).abs().max()):.3g}"


CASES = [
    # rows, cols, io, x, act, residual, pre, checkpoint
    (1, 1, F32, F32, None, False, False, False),
    (3, 8, BF, BF, "silu", True, True, True),
    (5, 64, BF, F32, "sigmoid", False, False, False),
    (300, 128, BF, BF, "silu", False, False, True),
    (70, 256, F32, F32, "silu", True, True, True),
    (9, 72, BF, BF, "sigmoid", True, True, True),
    (7, 77, BF, F32, "silu", True, True, True),        # rows off 16-byte steps
    (1, 512, BF, BF, None, True, True, False),
    (33, 1000, F32, F32, "sigmoid", True, True, True),
    (13, 1001, F32, F32, "silu", True, False, False),
    (8, 2048, BF, F32, None, True, True, False),
    (1300, 2056, BF, BF, "silu", True, True, True),
    (4, 8192, BF, BF, "silu", True, True, True),
    (3, 9000, F32, F32, "sigmoid", True, True, False),
    (2, 16384, BF, BF, "silu", True, True, True),
    (2, 16383, BF, BF, "silu", True, True, True),
]


def make(rows, cols, io, xt, act, residual, pre, seed=0):
    gen = torch.Generator().manual_seed(seed)

    def rn(dt=F32):
        return torch.randn(rows, cols, generator=gen).to(dt)

    d = dict(f=rn(io), z=rn(io) if act else None, res=rn(xt) if residual else None, d_x=rn(xt),
             d_h=rn(io) if pre else None, xk=rn(xt) if pre else None)
    d["w_post"] = 1 + 0.1 * torch.randn(cols, generator=gen)
    d["w_pre"] = 1 + 0.1 * torch.randn(cols, generator=gen) if pre else None
    return d


def values(pair):
    codes, scales = pair
    s = scales.double().cpu().repeat_interleave(64, -1)[..., :codes.shape[-1]]
    return (codes.float().cpu().double() * s).float().double()


@pytest.mark.parametrize("rows,cols,io,xt,act,residual,pre,ckpt", CASES)
def test_fwd_bwd(rows, cols, io, xt, act, residual, pre, ckpt):
    d = make(rows, cols, io, xt, act, residual, pre)
    x = {n: None if t is None else t.cuda() for n, t in d.items()}
    rs, eps = 0.5, 1e-6
    kw = dict(gate=x["z"], act=act or "silu", res_scale=rs, eps=eps)
    got = api.block_norm_fwd(x["f"], x["w_post"], residual=x["res"], w_pre=x["w_pre"], x_dtype=xt, checkpoint=ckpt,
                             **kw)
    f, z, res, wp, we = (None if d[n] is None else d[n].double() for n in ("f", "z", "res", "w_post", "w_pre"))
    rx, rh = ref.norm(f, wp, z, act, res, rs, we, eps)
    mag = (rx - (0 if res is None else res)).abs() * 8 + (0 if res is None else res.abs())
    close(got[0], rx, mag, "x")
    if pre:
        close(got[1], rh, mag / torch.sqrt(rx.pow(2).mean(-1, keepdim=True) + eps) * we.abs() + rh.abs(), "h")
    else:
        assert got[1] is None
    fg, zg = x["f"], x["z"]
    if ckpt:
        fg, zg = got[2], got[3]
        for have, src in ((fg, f), (zg, z)):
            if src is None:
                assert have is None
                continue
            want, sc = ref.pack(src)
            assert torch.equal(values(have), want) and torch.equal(have[1].cpu().double(), sc)
        f, z = values(fg), None if z is None else values(zg)
    kw["gate"] = zg
    b = api.block_norm_bwd(fg, x["w_post"], x["d_x"], d_h=x["d_h"], x=x["xk"], w_pre=x["w_pre"],
                           want_residual=residual, io_dtype=io, **kw)
    # the gradients: torch's differentiation of the formulas in 64 bits
    leaves = [t.clone().requires_grad_() for t in (f, wp)] + ([z.clone().requires_grad_()] if z is not None else [])
    y, _ = ref.norm(leaves[0], leaves[1], leaves[2] if z is not None else None, act, None, 1.0, None, eps)
    dxp, mx = d["d_x"].double(), d["d_x"].double().abs()
    if pre:
        xk = d["xk"].double().requires_grad_()
        w2 = we.clone().requires_grad_()
        _, h = ref.norm(torch.ones(1, 1, dtype=torch.float64), torch.ones(1, dtype=torch.float64), None, None, xk, 0.0,
                        w2, eps)
        gx, gw = torch.autograd.grad(h, (xk, w2), d["d_h"].double())
        dxp = dxp + gx
        xk = xk.detach()
        r = 1 / torch.sqrt(xk.pow(2).mean(-1, keepdim=True) + eps)
        t = (d["d_h"].double() * we).abs()
        mx = mx + r * (t + (xk * r).abs() * (t * (xk * r).abs()).mean(-1, keepdim=True))
        close(b[4], gw, (d["d_h"].double() * xk * r).abs().sum(0), "dw_pre")
    else:
        assert b[4] is None
    grads = torch.autograd.grad(rs * y, leaves, dxp)
    r = 1 / torch.sqrt(f.pow(2).mean(-1, keepdim=True) + eps)
    n = (f * r).abs()
    a = 1.0 if z is None else (torch.sigmoid(z) if act == "sigmoid" else (z * torch.sigmoid(z)).abs())
    u = rs * mx * a * wp.abs() * 4
    close(b[0], grads[0], r * (u + n * (u * n).mean(-1, keepdim=True)), "d_f")
    close(b[3], grads[1], (rs * mx * a * 4 * n).sum(0), "dw_post")
    if z is not None:
        close(b[1], grads[2], rs * mx * n * wp.abs() * 8, "d_gate")
    else:
        assert b[1] is None
    if residual:
        close(b[2], dxp, mx, "d_residual")
    else:
        assert b[2] is None


def test_misaligned_rows_and_zero_rows():
    """A contiguous tensor whose start is off 16 bytes takes the general layout; a row of zeros stays finite."""
    base = torch.randn(6 * 64 + 1, device="cuda").to(BF)
    f = base[1:].view(6, 64)
    f[2] = 0
    w = torch.ones(64, device="cuda")
    x, _ = api.block_norm_fwd(f, w)
    x2, _ = api.block_norm_fwd(f.clone(), w)
    want, _ = ref.norm(f.double().cpu(), w.double().cpu(), None, None, None, 1.0, None, 1e-6)
    close(x, want, want.abs(), "x")
    close(x2, want, want.abs(), "x")
    assert not x[2].any()
    d = api.block_norm_bwd(f, w, x)
    assert torch.isfinite(d[0]).all()


def test_no_rows():
    f, w = torch.empty(0, 64, dtype=BF, device="cuda"), torch.ones(64, device="cuda")
    x, h, c, z = api.block_norm_fwd(f, w, w_pre=w, checkpoint=True)
    assert x.shape == h.shape == (0, 64) and z is None
    d = api.block_norm_bwd(f, w, x, d_h=h, x=x, w_pre=w)
    assert not d[3].any() and not d[4].any()
    assert api.act_unpack(*api.act_pack(f)).shape == (0, 64)


def test_norm_repeatable_other_stream_and_graph():
    d = {n: None if t is None else t.cuda() for n, t in make(3000, 256, BF, BF, "silu", True, True).items()}
    run = lambda: api.block_norm_bwd(d["f"], d["w_post"], d["d_x"], d_h=d["d_h"], x=d["xk"], w_pre=d["w_pre"],  # noqa: E731
                                     gate=d["z"])
    a = run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = run()
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for _ in range(3):
        d["f"].copy_(torch.randn_like(d["f"]))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert all(torch.equal(x, y) for x, y in zip(got, run()))


@pytest.mark.parametrize("rows,cols,dtype", [(1, 1, F32), (3, 7, BF), (5, 64, BF), (4, 65, F32), (333, 1000, F32),
                                             (17, 1032, BF), (2, 8192, BF)])
def test_act_round_trip(rows, cols, dtype):
    gen = torch.Generator().manual_seed(cols)
    x = (torch.randn(rows, cols, generator=gen) * torch.exp(4 * torch.randn(rows, 1, generator=gen))).to(dtype)
    x[0, :cols // 2] = 0
    want, sc = ref.pack(x)
    codes, s = api.act_pack(x.cuda())
    assert torch.equal(s.cpu().double(), sc) and torch.equal(values((codes, s)), want)
    for dt in (F32, BF):
        assert torch.equal(api.act_unpack(codes, s, dtype=dt).cpu(), want.float().to(dt))


def test_act_extremes():
    """Ties, the largest and smallest magnitudes, scales in the subnormal range, zeros; a NaN stays in its place."""
    tiny = 2.0 ** -149
    x = torch.zeros(5, 64)
    x[0, :6] = torch.tensor([448.0, 17.0, 19.0, -17.0, 2.0 ** -9, 2.0 ** -10])     # scale 1: ties to even
    x[1, :3] = torch.tensor([3.4e38, -3.4e38, 1.0])
    x[2, :3] = torch.tensor([tiny * 627, tiny * 300, -tiny])                       # scale: one subnormal step
    x[3, :2] = torch.tensor([tiny * 100, 0.0])                                     # amax / 448 rounds to 0
    x[4, :2] = torch.tensor([float("nan"), 2.0])
    codes, s = api.act_pack(x.cuda())
    want, sc = ref.pack(x[:4])
    assert torch.equal(s[:4].cpu().double(), sc) and torch.equal(values((codes[:4], s[:4])), want)
    v = api.act_unpack(codes, s, dtype=F32).cpu()[4]
    assert v[0].isnan() and v[1] == 2.0 and not v[2:].any()


def test_act_past_32_bits():
    rows, cols = 270_000, 8192
    x = torch.empty(rows, cols, dtype=BF, device="cuda").normal_()
    codes, s = api.act_pack(x)
    want, sc = ref.pack(x[-3:])
    assert torch.equal(s[-3:].cpu().double(), sc) and torch.equal(values((codes[-3:], s[-3:])), want)
    assert torch.equal(api.act_unpack(codes, s)[-3:].cpu(), want.float().to(BF))


@pytest.mark.parametrize("cols", [2 ** 31 - 8, 2 ** 31 - 1])
def test_act_one_row_of_most_columns(cols):
    x = torch.empty(1, cols, dtype=BF, device="cuda").normal_()
    codes, s = api.act_pack(x)
    tail = 2 ** 31 - 256
    want, sc = ref.pack(x[:, tail:])
    assert s.shape == (1, 2 ** 25) and torch.equal(s[:, -4:].cpu().double(), sc)
    assert torch.equal(values((codes[:, tail:], s[:, -4:])), want)
    assert torch.equal(api.act_unpack(codes, s)[:, tail:].cpu(), want.float().to(BF))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_act_more_groups_than_one_launch_takes(dtype):
    """Four threads a group: from 2^30 groups on a launch would pass 2^32 threads."""
    rows = 2 ** 30 + 70
    x = torch.zeros(rows, 1, dtype=dtype, device="cuda")
    at = torch.tensor([0, 5, 2 ** 30 - 65, 2 ** 30 - 64, 2 ** 30 - 63, 2 ** 30, rows - 1], device="cuda")
    x[at, 0] = torch.randn(len(at), device="cuda").to(dtype)
    codes, s = api.act_pack(x)
    want, sc = ref.pack(x[at])
    assert torch.equal(s[at].cpu().double(), sc) and torch.equal(values((codes[at], s[at])), want)
    assert (s != 1).sum() == (sc != 1).sum()
    back = api.act_unpack(codes, s, dtype=dtype)
    assert torch.equal(back[at].cpu(), want.float().to(dtype)) and back.count_nonzero() == len(at)


@pytest.mark.parametrize("rows,cols", [(2 ** 29 + 45, 8), (2 ** 23 + 3, 513)])
def test_norm_more_rows_than_one_launch_takes(rows, cols):
    """8 and 512 threads a row: the rows on both sides of 2^32 threads, residual, gate and checkpoints among them."""
    f = torch.zeros(rows, cols, dtype=BF, device="cuda")
    border = 2 ** 29 - 32 if cols == 8 else 2 ** 23 - 1
    at = torch.tensor([0, border - 1, border, border + 1, rows - 1], device="cuda")
    gen = torch.Generator().manual_seed(cols)
    fv, zv = (torch.randn(len(at), cols, generator=gen).to(BF) for _ in range(2))
    f[at] = fv.cuda()
    w = 1 + 0.1 * torch.randn(cols, generator=gen)
    x, h, (fc, fs), _ = api.block_norm_fwd(f, w.cuda(), residual=f, w_pre=w.cuda(), checkpoint=True)
    d, w = fv.double(), w.double()
    rx, rh = ref.norm(d, w, None, None, d, 1.0, w, 1e-6)
    mag = (rx - d).abs() * 8 + d.abs()
    close(x[at], rx, mag, "x")
    close(h[at], rh, mag / torch.sqrt(rx.pow(2).mean(-1, keepdim=True) + 1e-6) * w.abs() + rh.abs(), "h")
    want, sc = ref.pack(fv)
    assert torch.equal(values((fc[at], fs[at])), want) and torch.equal(fs[at].cpu().double(), sc)
    assert x.count_nonzero() == x[at].count_nonzero() and h.count_nonzero() == h[at].count_nonzero()
    del x, h, fc, fs
    f.zero_()
    f[at] = zv.cuda()
    x, _ = api.block_norm_fwd(f, w.float().cuda(), gate=f)
    d = zv.double()
    rx, _ = ref.norm(d, w, d, "silu", None, 1.0, None, 1e-6)
    close(x[at], rx, rx.abs() * 8, "gated x")
    assert x.count_nonzero() == x[at].count_nonzero()


@pytest.mark.parametrize("rows,cols", [(2 ** 20 + 3, 1032), (2 ** 20 + 3, 513), (2 ** 22 + 77, 64)])
def test_norm_weight_gradients_of_many_rows(rows, cols):
    """Rows that are all alike, whose sums' roundings line up: the weights' gradients stay within 2^-18 of the sums
    (at most 32 rows are added in fp32, 2^-19; a term's own rounding is 2^-19.3 as above)."""
    gen = torch.Generator().manual_seed(rows + cols)
    one, dx, dh = (torch.randn(1, cols, generator=gen).to(BF) for _ in range(3))
    w = 1 + 0.1 * torch.randn(cols, generator=gen)
    f, d_x, d_h = (t.cuda().expand(rows, cols).contiguous() for t in (one, dx, dh))
    got = api.block_norm_bwd(f, w.cuda(), d_x, d_h=d_h, x=f, w_pre=w.cuda(), want_residual=False)
    f, d_x, d_h, w = one.double(), dx.double(), dh.double(), w.double()
    r = 1 / torch.sqrt(f.pow(2).mean() + 1e-6)
    n, t = f * r, d_h * w
    d = d_x + r * (t - n * (t * n).mean())
    mag = (d_x.abs() + r * (t.abs() + n.abs() * (t * n).abs().mean())) * n.abs()
    close(got[3], rows * (d * n)[0], rows * mag[0], "dw_post")
    close(got[4], rows * (d_h * n)[0], rows * (d_h * n).abs()[0], "dw_pre")


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_gate_far_from_zero(dtype, act):
    """Gates of -103 to 103.  With f = w = 1 the outputs are the gate's value and, in d_gate, its derivative times n
    = 1.  Either is a product of at most 12 fp32 roundings whatever z is (fp32: 2^-20 of it, of p (1 + |z| (1 - p))
    for silu's derivative, whose sum cancels), and below 2^-126 a few subnormal steps times |z|; bf16's exponential
    adds |z| 2^-23, then the output's rounding."""
    z = torch.linspace(-103, 103, 64 * 64).view(64, 64).to(dtype)
    f, w = torch.ones(64, 64, dtype=dtype), torch.ones(64)
    x, _ = api.block_norm_fwd(f.cuda(), w.cuda(), gate=z.cuda(), act=act, eps=1e-30)
    # dy = n = w = 1: the gradient of the gate is a'(z)
    dz = api.block_norm_bwd(f.cuda(), w.cuda(), f.cuda(), gate=z.cuda(), act=act, eps=1e-30, want_residual=False)[1]
    d = z.double()
    p, q = torch.sigmoid(d), torch.sigmoid(-d)
    pairs = ((x, p, p), (dz, p * q, p * q)) if act == "sigmoid" else \
        ((x, d * p, (d * p).abs()), (dz, p * (1 + d * q), p * (1 + d.abs() * q)))
    for got, want, mag in pairs:
        tol = 2.0 ** -20 * mag + 2.0 ** -146 * (1 + d.abs())
        if dtype == BF:
            tol = tol + d.abs() * 2.0 ** -23 * mag + 2.0 ** -8 * want.abs() + 2.0 ** -133
        bad = (got.double().cpu() - want).abs() > tol
        assert not bad.any(), (int(bad.sum()), z[bad][:4].tolist(), got.cpu()[bad][:4].tolist(), want[bad][:4].tolist())
