"""Linear attention, block norms and 8-bit activations without a GPU: the
64-bit references against differences, the binding's checks of types and
shapes, and the C ABI's refusals (before any device is touched)."""
import ctypes

import pytest
import torch

import lin_ref as ref
from fp8_state_qat_amd import _lib, api
from fp8_state_qat_amd._lib import GdnLin, GdnNorm

P = ctypes.c_void_p
FAKE = 0x10000


# ---------------------------------------------------------------- references
def test_lin_reference_gradients_against_differences():
    """Central differences of the 64-bit forward: error h^2 f''' / 6 + 2^-53 |L| / h ~ 1e-9 at h = 1e-5."""
    torch.manual_seed(0)
    T, H, Hk, dk, dv, cu = 7, 2, 1, 3, 4, [0, 0, 5, 7]
    a = [torch.randn(T, Hk, dk), torch.randn(T, Hk, dk), torch.randn(T, H, dv), -torch.rand(T, H),
         torch.randn(3, H, dv, dk)]
    a = [x.double() for x in a]
    do, dS = torch.randn(T, H, dv).double(), torch.randn(3, H, dv, dk).double()

    def loss(q, k, v, g, S0):
        o, S = ref.lin(q, k, v, g, cu, S0)
        return float((o * do).sum() + (S * dS).sum())

    grads = ref.lin(*a[:4], cu, a[4], do, dS)
    for i, want in enumerate(grads):
        flat = a[i].reshape(-1)
        for j in range(0, flat.numel(), max(1, flat.numel() // 7)):
            keep, h = float(flat[j]), 1e-5
            flat[j] = keep + h
            up = loss(*a)
            flat[j] = keep - h
            down = loss(*a)
            flat[j] = keep
            assert abs((up - down) / (2 * h) - float(want.reshape(-1)[j])) < 1e-7


def test_pack_reference_is_e4m3():
    """Where torch's own conversion is exact arithmetic on the same quotients, the values agree bit for bit."""
    torch.manual_seed(1)
    x = torch.randn(9, 130) * torch.exp(3 * torch.randn(9, 1))
    x[3] = 0.0
    vals, sc = ref.pack(x)
    for c in range(3):
        s = sc[:, c:c + 1]
        code = (x.double()[:, 64 * c:64 * c + 64] / s).float().clamp(-448, 448).to(torch.float8_e4m3fn)
        assert torch.equal(vals[:, 64 * c:64 * c + 64], (code.double() * s).float().double())


# ---------------------------------------------------------------- binding
T, H, HK, DK, DV, N = 20, 4, 2, 64, 128, 2
BF = torch.bfloat16


def _lin(**over):
    a = dict(q=torch.zeros(T, HK, DK, dtype=BF), k=torch.zeros(T, HK, DK, dtype=BF),
             v=torch.zeros(T, H, DV, dtype=BF), g=torch.zeros(T, H),
             cu=torch.tensor([0, 5, T], dtype=torch.int32))
    a.update({k: over.pop(k) for k in list(over) if k in a})
    return (a["q"], a["k"], a["v"], a["g"], a["cu"]), over


LIN_BAD = [
    (dict(q=torch.zeros(T, HK, DK)), "q"), (dict(q=torch.zeros(T, H, DK, dtype=BF)), "q"),
    (dict(k=torch.zeros(T, DK, dtype=BF)), "k"), (dict(k=torch.zeros(T, HK, DK, dtype=torch.float16)), "dtype"),
    (dict(v=torch.zeros(T + 1, H, DV, dtype=BF)), "v"), (dict(v=torch.zeros(T, H, DV)), "v"),
    (dict(g=torch.zeros(T, H, dtype=torch.float64)), "g"), (dict(g=torch.zeros(H + 1)), "g"),
    (dict(g=torch.zeros(T, HK)), "g"), (dict(cu=torch.tensor([0], dtype=torch.int32)), "cu_seqlens"),
    (dict(cu=torch.tensor([0, 5, T])), "cu_seqlens"),
    (dict(initial_state=torch.zeros(N, H, DK, DV)), "initial_state"),
    (dict(q=torch.zeros(HK, T, DK, dtype=BF).transpose(0, 1)), "contiguous"),
]


@pytest.mark.parametrize("over,what", LIN_BAD + [(dict(out=torch.zeros(T, H, DV)), "out"),
                                                 (dict(final_state=torch.zeros(N + 1, H, DV, DK)), "final_state"),
                                                 ({}, "device tensor"), (dict(g=torch.zeros(H)), "device tensor")])
def test_lin_fwd_refusals(over, what):
    a, kw = _lin(**over)
    with pytest.raises(ValueError, match=what):
        api.lin_attn_fwd(*a, **kw)


@pytest.mark.parametrize("over,what", LIN_BAD + [(dict(d_o=torch.zeros(T, H, DV)), "d_o"), (dict(d_o=None), "d_o"),
                                                 (dict(d_final_state=torch.zeros(N, H, DV, DV)), "d_final_state"),
                                                 (dict(dg=torch.zeros(T, H + 1)), "dg"),
                                                 (dict(dq=torch.zeros(T, H, DK, dtype=BF)), "dq"),
                                                 ({}, "device tensor")])
def test_lin_bwd_refusals(over, what):
    a, kw = _lin(**over)
    d_o = kw.pop("d_o") if "d_o" in kw else torch.zeros(T, H, DV, dtype=BF)
    with pytest.raises(ValueError, match=what):
        api.lin_attn_bwd(*a, d_o, **kw)


@pytest.mark.parametrize("state,o,what", [
    (None, None, "state"), (torch.zeros(T, H, DK, DV), None, "state"),
    (torch.zeros(T, H, DV, DK), torch.zeros(T, H, DV), "o must be"), (torch.zeros(T, H, DV, DK), None, "device tensor"),
])
def test_lin_step_refusals(state, o, what):
    a, _ = _lin()
    with pytest.raises(ValueError, match=what):
        api.lin_attn_step(*a[:4], state, o=o)


R, C = 3, 72


@pytest.mark.parametrize("kw,what", [
    (dict(w_post=torch.ones(C + 1)), "w_post"), (dict(w_post=None), "w_post"),
    (dict(gate=torch.zeros(R, C)), "gate"), (dict(act="relu"), "act"), (dict(residual=torch.zeros(R, C + 8)), "residual"),
    (dict(w_pre=torch.ones(C, dtype=BF)), "w_pre"), (dict(x_dtype=torch.float16), "dtypes"), ({}, "device tensor"),
])
def test_norm_fwd_refusals(kw, what):
    kw = dict(dict(w_post=torch.ones(C)), **kw)
    with pytest.raises(ValueError, match=what):
        api.block_norm_fwd(torch.zeros(R, C, dtype=BF), kw.pop("w_post"), **kw)


@pytest.mark.parametrize("over,what", [
    (dict(d_x=None), "d_x"), (dict(d_x=torch.zeros(R, C + 1)), "d_x"), (dict(w_pre=torch.ones(C)), "w_pre needs"),
    (dict(gate=(torch.zeros(R, C).to(torch.float8_e4m3fn), torch.ones(R, 2))), "both"),
    (dict(f=(torch.zeros(R, C).to(torch.float8_e4m3fn), torch.ones(R, 1)), io_dtype=BF), "scales"),
    (dict(f=(torch.zeros(R, C).to(torch.float8_e4m3fn), torch.ones(R, 2))), "io_dtype"),
    (dict(f=(torch.zeros(R, C).to(torch.uint8), torch.ones(R, 2)), io_dtype=BF), "codes"), ({}, "device tensor"),
])
def test_norm_bwd_refusals(over, what):
    a = dict(dict(f=torch.zeros(R, C, dtype=BF), w_post=torch.ones(C), d_x=torch.zeros(R, C, dtype=BF)), **over)
    with pytest.raises(ValueError, match=what):
        api.block_norm_bwd(a.pop("f"), a.pop("w_post"), a.pop("d_x"), **a)


@pytest.mark.parametrize("f", [None, [1.0], "f"])
def test_norm_bwd_refuses_what_is_no_tensor(f):
    with pytest.raises(ValueError, match="f must be a tensor"):
        api.block_norm_bwd(f, torch.ones(C), torch.zeros(R, C, dtype=BF))


def test_act_refusals():
    x = torch.zeros(R, C)
    codes = x.to(torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        api.act_pack(x.half())
    with pytest.raises(ValueError, match="contiguous"):
        api.act_pack(x.t())
    with pytest.raises(ValueError, match="device tensor"):
        api.act_pack(x)
    with pytest.raises(ValueError, match="scales"):
        api.act_unpack(codes, torch.ones(R, 1))
    with pytest.raises(ValueError, match="dtype"):
        api.act_unpack(codes, torch.ones(R, 2), dtype=torch.float16)
    with pytest.raises(ValueError, match="device tensor"):
        api.act_unpack(codes, torch.ones(R, 2))


def test_columns_past_32_bits_are_refused():
    """A column count that would wrap in the library's 32-bit field (2^32 + 64 as 64) is refused, not cut."""
    wide = lambda dt, *s: torch.empty(*s, dtype=dt, device="meta")  # noqa: E731
    for cols in (1 << 31, (1 << 32) + 64):
        x, w = wide(BF, 1, cols), wide(torch.float32, cols)
        codes, scales = wide(torch.float8_e4m3fn, 1, cols), wide(torch.float32, 1, -(-cols // 64))
        for call in (lambda: api.act_pack(x), lambda: api.act_unpack(codes, scales),
                     lambda: api.block_norm_fwd(x, w), lambda: api.block_norm_bwd(x, w, x),
                     lambda: api.block_norm_bwd((codes, scales), w, x, io_dtype=BF)):
            with pytest.raises(ValueError, match="columns"):
                call()


# ---------------------------------------------------------------- C ABI
def _shape(**kw):
    return GdnLin(**dict(dict(n_seqs=2, n_heads=4, qk_heads=2, dk=64, dv=128, io_dtype=1, gate_per_token=1,
                              total_tokens=100), **kw))


LIN_SHAPES = [
    (dict(n_seqs=0), 1), (dict(n_heads=0), 1), (dict(qk_heads=3), 1), (dict(qk_heads=0), 1), (dict(dv=96), 1),
    (dict(dv=0), 1), (dict(dv=320), 2), (dict(dk=32), 2), (dict(dk=96), 2), (dict(io_dtype=2), 1),
    (dict(gate_per_token=2), 1), (dict(total_tokens=-1), 1), (dict(total_tokens=1 << 31), 2), (dict(n_seqs=70000), 2),
    (dict(n_heads=1 << 22, qk_heads=1), 2),
]


def _fwd(shape, q=FAKE, cu=FAKE, init=None, fin=FAKE, ws=FAKE, ws_bytes=None):
    L = _lib.lib()
    if ws_bytes is None:
        ws_bytes = L.gdn_lin_attn_fwd_workspace_bytes(ctypes.byref(shape))
    return L.gdn_lin_attn_fwd(ctypes.byref(shape), P(q), P(FAKE), P(FAKE), P(FAKE), P(cu), P(init), P(FAKE), P(fin),
                              P(ws), ws_bytes, None)


def _bwd(shape, q=FAKE, dg=FAKE, d0=FAKE, dfin=None, ws=FAKE, ws_bytes=None):
    L = _lib.lib()
    if ws_bytes is None:
        ws_bytes = L.gdn_lin_attn_bwd_workspace_bytes(ctypes.byref(shape))
    return L.gdn_lin_attn_bwd(ctypes.byref(shape), P(q), P(FAKE), P(FAKE), P(FAKE), P(FAKE), P(FAKE), None, P(dfin),
                              P(FAKE), P(FAKE), P(FAKE), P(dg), P(d0), P(ws), ws_bytes, None)


@pytest.mark.parametrize("kw,status", LIN_SHAPES)
def test_lin_rejects_bad_shapes(kw, status):
    s = _shape(**kw)
    assert _lib.lib().gdn_lin_attn_fwd_workspace_bytes(ctypes.byref(s)) == 0
    assert _lib.lib().gdn_lin_attn_bwd_workspace_bytes(ctypes.byref(s)) == 0
    assert _fwd(s, ws_bytes=1 << 40) == status and _lib.last_error()
    assert _bwd(s, ws_bytes=1 << 40) == status and _lib.last_error()


def test_lin_rejects_launches_past_32_bits_of_threads():
    """A launch takes fewer than 2^32 threads: more (sequence, head) pairs are refused, not left to the launch."""
    L = _lib.lib()
    most = dict(n_seqs=32768, total_tokens=32768, dk=64, dv=64, gate_per_token=0)   # 4 threads for 64 + 64 columns
    bwd = L.gdn_lin_attn_bwd_workspace_bytes
    assert bwd(ctypes.byref(_shape(**most, n_heads=255, qk_heads=255))) > 0
    s = _shape(**most, n_heads=256, qk_heads=256)
    assert bwd(ctypes.byref(s)) == 0 and _bwd(s, ws_bytes=1 << 50) == 2 and "threads" in _lib.last_error()
    fwd = L.gdn_lin_attn_fwd_workspace_bytes                                        # 4 threads for 64 columns
    assert fwd(ctypes.byref(s)) > 0 and fwd(ctypes.byref(_shape(**most, n_heads=511, qk_heads=511))) > 0
    s = _shape(**most, n_heads=512, qk_heads=512)
    assert fwd(ctypes.byref(s)) == 0 and _fwd(s, ws_bytes=1 << 50) == 2 and "threads" in _lib.last_error()
    step = _shape(n_seqs=1 << 20, total_tokens=1 << 20, n_heads=16, qk_heads=16, dv=64)   # 256 threads for 64 rows
    assert L.gdn_lin_attn_step(ctypes.byref(step), *[P(FAKE)] * 7) == 2 and "threads" in _lib.last_error()


def test_lin_rejects_null_misaligned_and_short_workspaces():
    s = _shape()
    for kw in (dict(q=0), dict(q=FAKE + 8), dict(ws=0), dict(ws=FAKE + 16), dict(ws_bytes=16)):
        assert _fwd(s, **kw) == 1, kw
        assert _bwd(s, **kw) == 1, kw
    assert _fwd(s, cu=0) == 1 and _fwd(s, fin=0) == 1 and _fwd(s, init=FAKE, fin=FAKE) == 1
    assert _bwd(s, dg=0) == 1 and _bwd(s, d0=0) == 1 and _bwd(s, dfin=FAKE, d0=FAKE) == 1
    L = _lib.lib()
    assert L.gdn_lin_attn_fwd(None, *[P(FAKE)] * 9, 0, None) == 1
    step = _shape(total_tokens=2)
    assert L.gdn_lin_attn_step(ctypes.byref(s), *[P(FAKE)] * 7) == 1      # total_tokens != n_seqs
    assert L.gdn_lin_attn_step(ctypes.byref(step), None, *[P(FAKE)] * 6) == 1
    assert L.gdn_lin_attn_step(ctypes.byref(step), P(FAKE + 4), *[P(FAKE)] * 6) == 1


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 1), (dict(cols=0), 1), (dict(cols=16385), 2), (dict(io_dtype=3), 1), (dict(x_dtype=-1), 1),
    (dict(io_dtype=0, x_dtype=1), 2), (dict(act=2), 1), (dict(eps=0.0), 1), (dict(eps=float("nan")), 1),
])
def test_norm_rejects_bad_shapes(kw, status):
    s = GdnNorm(**dict(dict(rows=3, cols=64, io_dtype=1, x_dtype=1, act=0, res_scale=1.0, eps=1e-6), **kw))
    L = _lib.lib()
    assert L.gdn_block_norm_bwd_workspace_bytes(ctypes.byref(s)) == 0
    f = [P(FAKE)] * 7 + [None] * 4
    assert L.gdn_block_norm_fwd(ctypes.byref(s), *f, None) == status


def test_norm_rejects_null_and_misaligned():
    s = ctypes.byref(GdnNorm(3, 64, 1, 1, 0, 1.0, 1e-6))
    L = _lib.lib()

    def fwd(f=FAKE, gate=None, w_pre=None, h=None, fc=None, fs=None, zc=None, zs=None, x=FAKE):
        return L.gdn_block_norm_fwd(s, P(f), P(gate), None, P(FAKE), P(w_pre), P(x), P(h), P(fc), P(fs), P(zc), P(zs),
                                    None)

    for kw in (dict(f=0), dict(f=FAKE + 1), dict(x=0), dict(w_pre=FAKE), dict(h=FAKE), dict(fc=FAKE), dict(fs=FAKE),
               dict(zc=FAKE, zs=FAKE), dict(gate=FAKE, fc=FAKE, fs=FAKE)):
        assert fwd(**kw) == 1, kw
    need = L.gdn_block_norm_bwd_workspace_bytes(s)

    def bwd(f=FAKE, fs=None, z=None, zs=None, w_pre=None, x=None, dz=None, dwp=None, ws=FAKE, n=need):
        return L.gdn_block_norm_bwd(s, P(f), P(fs), P(z), P(zs), P(FAKE), P(w_pre), P(x), P(FAKE), None, P(FAKE),
                                    P(dz), None, P(FAKE), P(dwp), P(ws), n, None)

    for kw in (dict(f=0), dict(f=FAKE + 1), dict(z=FAKE), dict(dz=FAKE), dict(zs=FAKE), dict(w_pre=FAKE),
               dict(w_pre=FAKE, dwp=FAKE), dict(z=FAKE, dz=FAKE, fs=FAKE), dict(ws=0), dict(ws=FAKE + 4), dict(n=8)):
        assert bwd(**kw) == 1, kw


def test_act_rejects_null_and_misaligned():
    L = _lib.lib()
    for fn, order in ((L.gdn_act_pack, "xdcs"), (L.gdn_act_unpack, "csxd")):
        def call(x=FAKE, d=1, c=FAKE, s=FAKE, rows=3, cols=64):
            v = dict(x=P(x), d=d, c=P(c), s=P(s))
            return fn(*[v[o] for o in order], rows, cols, None)
        assert call(x=0) == 1 and call(x=FAKE + 1) == 1 and call(c=0) == 1 and call(s=FAKE + 2) == 1
        assert call(d=5) == 1 and call(rows=-1) == 1 and call(cols=0) == 1
        assert call(rows=1 << 31) == 2
