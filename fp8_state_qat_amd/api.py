"""torch-facing binding of the C ABI: argument marshalling only.

Every function takes device tensors (torch is used for device memory and the
current stream), checks their dtypes, shapes and contiguity against the
call's contract, turns them into pointers and sizes, and calls one entry
point of libgdn.so on torch's current stream.  All arithmetic runs in the
HIP kernels.  A tensor of the wrong shape raises ValueError before anything
is launched: the kernels trust the sizes they are given.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import GDN_BF16, GDN_F32, GDN_QDQ_CHUNK, GDN_QDQ_WRITE, GdnDebug, GdnDistill, GdnLin, GdnNorm, GdnShape

_DT = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16}


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dev(t, name, dtype=None, shape=None):
    """Check that t (if given) is a contiguous tensor of this dtype and exact
    shape.  Whether it lives on the device is checked by _on_device, after
    every tensor of the call has passed these checks."""
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _on_device(**tensors):
    """Every given tensor lives on the current device."""
    dev = None
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a device tensor")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the other tensors on {dev}")
    if dev is not None:
        _current(dev.index)


def _current(dev):
    """The kernels run on the current device and its stream: tensors of another
    one are refused."""
    now = torch._C._cuda_getDevice()
    if dev != now:
        raise ValueError(f"the tensors are on cuda:{dev}, the current device is cuda:{now}")


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _shape(N, H, dk, dv, T, io_dt, o_dt, per_channel, flags, grid=0):
    return GdnShape(N, H, dk, dv, T, _DT[io_dt], _DT[o_dt], 1 if per_channel else 0, int(flags), int(grid))


def _offsets_total(offs, N, name):
    """Host copy of a device [N + 1] offsets tensor (debug records only);
    returns its last entry, the record's first dimension."""
    _dev(offs, name, torch.int32, (N + 1,))
    _on_device(**{name: offs})
    return int(offs[-1].item())


def chunk_workspace_bytes(N, H, dk, dv, T, io_dtype=torch.bfloat16, qdq_flags=0):
    """Device workspace gdn_chunk_fwd needs for this shape (bytes)."""
    shape = _shape(N, H, dk, dv, T, io_dtype, io_dtype, False, qdq_flags)
    n = _lib.lib().gdn_chunk_fwd_workspace_bytes(ctypes.byref(shape))
    if n == 0:
        _lib.check(_lib.GDN_ERR_INVALID_ARG)
    return n


def workspace_status(workspace):
    """gdn_workspace_status: synchronizes torch's current stream and raises
    GdnError when the call that last used this workspace found its index
    arrays out of contract (GDN_ERR_INVALID_ARG) or had a bounded wait run out
    (GDN_ERR_DEVICE)."""
    _dev(workspace, "workspace", torch.uint8)
    _on_device(workspace=workspace)
    _lib.check(_lib.lib().gdn_workspace_status(_ptr(workspace), _stream()))


def chunk_fwd(q, k, v, beta, g, cu_seqlens, *, seq_lens=None, prefix_lens=None,
              initial_state=None, qdq_flags=GDN_QDQ_CHUNK | GDN_QDQ_WRITE, o_dtype=None,
              out=None, final_state=None, workspace=None, debug=None, check_status=False, noalloc=False,
              gate_grid_log2=0):
    """gdn_chunk_fwd.  q, k: [T, H, dk]; v: [T, H, dv] (fp32 or bf16); beta:
    [T, H] fp32; g: [T, H] or [T, H, dk] fp32; cu_seqlens: [N+1] int32;
    seq_lens, prefix_lens: [N] int32 or None; initial_state: [N, H, dv, dk]
    fp32 or None.
    workspace: optional uint8 device tensor of at least
    chunk_workspace_bytes(...) bytes (allocated here when None).
    debug: optional dict with device tensors bound_offsets ([N+1] int32),
    bound_pre, bound_post ([n_bounds, H, dv, dk] fp32), scales ([n_bounds, H,
    dv/64]), w_pre, w_post ([n_bounds, H, 64, dk] fp32, W of each chunk before
    and after its QDQ, with GDN_QDQ_W in qdq_flags), suffix_offsets ([N+1]
    int32), suffix_pre, suffix_post ([n_suffix, H, dv, dk] fp32, the state
    after each recurrent suffix token before and after its QDQ),
    status ([1] int32: receives the call's status word on the stream),
    torch.cuda.Event objects kernel_start, kernel_end (recorded around the
    sequential state kernel) and/or schedule (GDN_SCHEDULE_AUTO, _SPLIT or
    _FUSED: the per-chunk solve as its own kernel or inside the state
    kernel's launch; _FUSED_NO_PRODUCERS, a test hook whose bounded waits all
    run out).  check_status: read the workspace's status word after the call
    (synchronizes; raises GdnError on a device-side failure).
    noalloc: call gdn_chunk_fwd_noalloc instead, whose workspace is the
    library's static per-GPU scratch (out and final_state must be given, no
    workspace; the status word comes back through debug["status"]).
    gate_grid_log2: 0, or k in 1..24: the log-gates of the recurrent suffix
    rounded to multiples of 2^-k (the log-retention grid).
    Returns (o, final_state)."""
    if noalloc:
        if workspace is not None or check_status:
            raise ValueError("noalloc takes no workspace (pass debug['status'] for the status word)")
        if out is None or final_state is None:
            raise ValueError("noalloc needs out and final_state")
    _dev(k, "k")
    if k.dim() != 3:
        raise ValueError(f"k must be [T, H, dk], got shape {tuple(k.shape)}")
    T, H, dk = k.shape
    _dev(v, "v")
    if v.dim() != 3 or tuple(v.shape[:2]) != (T, H):
        raise ValueError(f"v must be [{T}, {H}, dv], got shape {tuple(v.shape)}")
    dv = v.shape[2]
    _dev(cu_seqlens, "cu_seqlens", torch.int32)
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be [N + 1] with N >= 1")
    N = cu_seqlens.numel() - 1
    if q.dtype != k.dtype or v.dtype != k.dtype or k.dtype not in _DT:
        raise ValueError("q, k, v must share one dtype: float32 or bfloat16")
    if o_dtype is None:
        o_dtype = out.dtype if isinstance(out, torch.Tensor) else k.dtype
    if o_dtype not in _DT:
        raise ValueError("o_dtype must be float32 or bfloat16")
    per_channel = g.dim() == 3
    for name, t, dt, shp in (("q", q, None, (T, H, dk)), ("beta", beta, torch.float32, (T, H)),
                             ("g", g, torch.float32, (T, H, dk) if per_channel else (T, H)),
                             ("seq_lens", seq_lens, torch.int32, (N,)),
                             ("prefix_lens", prefix_lens, torch.int32, (N,)),
                             ("initial_state", initial_state, torch.float32, (N, H, dv, dk))):
        _dev(t, name, dt, shp)
    _dev(out, "out", o_dtype, (T, H, dv))
    _dev(final_state, "final_state", torch.float32, (N, H, dv, dk))
    _dev(q, "q", k.dtype, (T, H, dk))
    _on_device(q=q, k=k, v=v, beta=beta, g=g, cu_seqlens=cu_seqlens, seq_lens=seq_lens,
               prefix_lens=prefix_lens, initial_state=initial_state, out=out, final_state=final_state)
    if out is None:
        out = torch.empty((T, H, dv), dtype=o_dtype, device=k.device)
    if final_state is None:
        final_state = torch.empty((N, H, dv, dk), dtype=torch.float32, device=k.device)
    shape = _shape(N, H, dk, dv, T, k.dtype, o_dtype, per_channel, qdq_flags, gate_grid_log2)
    if not noalloc:
        ws_bytes = _lib.lib().gdn_chunk_fwd_workspace_bytes(ctypes.byref(shape))
        if ws_bytes == 0:
            _lib.check(_lib.GDN_ERR_INVALID_ARG)
        if workspace is None:
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=k.device)
        _dev(workspace, "workspace", torch.uint8)
        _on_device(k=k, workspace=workspace)
        if workspace.dim() != 1:
            raise ValueError("workspace must be a 1-D uint8 tensor")
    dbg = None
    if debug is not None:
        unknown = set(debug) - {"bound_offsets", "bound_pre", "bound_post", "scales", "kernel_start",
                                "kernel_end", "schedule", "w_pre", "w_post", "suffix_offsets",
                                "suffix_pre", "suffix_post", "status"}
        if unknown:
            raise ValueError(f"unknown debug keys {sorted(unknown)}")
        if any(debug.get(key) is not None for key in ("bound_pre", "bound_post", "scales", "w_pre", "w_post")):
            if debug.get("bound_offsets") is None:
                raise ValueError("the per-boundary record needs bound_offsets")
            nb = _offsets_total(debug["bound_offsets"], N, "bound_offsets")
            for key, shp in (("bound_pre", (nb, H, dv, dk)), ("bound_post", (nb, H, dv, dk)),
                             ("scales", (nb, H, dv // 64)), ("w_pre", (nb, H, 64, dk)),
                             ("w_post", (nb, H, 64, dk))):
                _dev(debug.get(key), key, torch.float32, shp)
                _on_device(k=k, **{key: debug.get(key)})
        if debug.get("suffix_pre") is not None or debug.get("suffix_post") is not None:
            if debug.get("suffix_offsets") is None:
                raise ValueError("the suffix record needs suffix_offsets")
            ns = _offsets_total(debug["suffix_offsets"], N, "suffix_offsets")
            for key in ("suffix_pre", "suffix_post"):
                _dev(debug.get(key), key, torch.float32, (ns, H, dv, dk))
                _on_device(k=k, **{key: debug.get(key)})
        _dev(debug.get("status"), "status", torch.int32, (1,))
        _on_device(k=k, status=debug.get("status"))
        evs = []
        for key in ("kernel_start", "kernel_end"):
            ev = debug.get(key)
            if ev is not None and not ev.cuda_event:
                ev.record()  # torch creates its HIP event on first record
            evs.append(None if ev is None else ctypes.c_void_p(ev.cuda_event))
        dbg = GdnDebug(*(_ptr(debug.get(key)) for key in ("bound_offsets", "bound_pre",
                                                          "bound_post", "scales")), *evs,
                       int(debug.get("schedule", _lib.GDN_SCHEDULE_AUTO)),
                       _ptr(debug.get("w_pre")), _ptr(debug.get("w_post")),
                       _ptr(debug.get("suffix_offsets")), _ptr(debug.get("suffix_pre")),
                       _ptr(debug.get("suffix_post")), _ptr(debug.get("status")))
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(cu_seqlens), _ptr(seq_lens), _ptr(prefix_lens),
            _ptr(initial_state), _ptr(out), _ptr(final_state))
    dbg_p = ctypes.byref(dbg) if dbg is not None else None
    if noalloc:
        st = _lib.lib().gdn_chunk_fwd_noalloc(ctypes.byref(shape), *args, dbg_p, _stream())
    else:
        st = _lib.lib().gdn_chunk_fwd(ctypes.byref(shape), *args, _ptr(workspace), workspace.numel(), dbg_p,
                                      _stream())
    _lib.check(st)
    if check_status:
        workspace_status(workspace)
    return out, final_state


def chunk_bwd_dh(q, k, beta, g, cu_seqlens, d_o, *, seq_lens=None, d_final_state=None, dh=None,
                 d_initial_state=None, d_v=None, want_dv=False, workspace=None, qdq_flags=0,
                 check_status=False):
    """gdn_chunk_bwd_dh: gradients of the state entering every 64-token chunk
    (dh [n_bounds, H, dv, dk]) and of the initial state ([N, H, dv, dk]) for
    L = sum o . d_o + <S_L, d_final_state>, identity straight-through QDQ;
    with want_dv (or a d_v tensor) also the gradient of v ([T, H, dv] fp32).
    q, k: [T, H, dk] bf16; d_o: [T, H, dv] bf16; beta, g: [T, H] fp32.
    qdq_flags: those of the forward (with GDN_QDQ_W, the backward of the W-QDQ
    forward: its quantized W enters the state gradient).
    dh: an empty tensor asks for no per-chunk gradient.
    Returns (dh, d_initial_state) or (dh, d_initial_state, d_v)."""
    _dev(k, "k", torch.bfloat16)
    if k.dim() != 3:
        raise ValueError(f"k must be [T, H, dk], got shape {tuple(k.shape)}")
    T, H, dk = k.shape
    _dev(d_o, "d_o", torch.bfloat16)
    if d_o.dim() != 3 or tuple(d_o.shape[:2]) != (T, H):
        raise ValueError(f"d_o must be [{T}, {H}, dv], got shape {tuple(d_o.shape)}")
    dv = d_o.shape[2]
    _dev(cu_seqlens, "cu_seqlens", torch.int32)
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be [N + 1] with N >= 1")
    N = cu_seqlens.numel() - 1
    gshape = (T, H, dk) if g.dim() == 3 else (T, H)
    for name, t, dt, shp in (("q", q, torch.bfloat16, (T, H, dk)), ("beta", beta, torch.float32, (T, H)),
                             ("g", g, torch.float32, gshape), ("seq_lens", seq_lens, torch.int32, (N,)),
                             ("d_final_state", d_final_state, torch.float32, (N, H, dv, dk)),
                             ("d_v", d_v, torch.float32, (T, H, dv))):
        _dev(t, name, dt, shp)
    _on_device(q=q, k=k, beta=beta, g=g, cu_seqlens=cu_seqlens, d_o=d_o, seq_lens=seq_lens,
               d_final_state=d_final_state, d_v=d_v)
    lens = seq_lens if seq_lens is not None else (cu_seqlens[1:] - cu_seqlens[:-1])
    n_bounds = int(((lens.to(torch.int64) + 63) // 64).clamp(min=0).sum().item()) if N else 0
    if dh is None:
        dh = torch.empty((n_bounds, H, dv, dk), dtype=torch.float32, device=k.device)
    if d_initial_state is None:
        d_initial_state = torch.empty((N, H, dv, dk), dtype=torch.float32, device=k.device)
    if want_dv and d_v is None:
        d_v = torch.empty((T, H, dv), dtype=torch.float32, device=k.device)
    if dh.numel():   # an empty tensor asks for no dh output
        _dev(dh, "dh", torch.float32, (n_bounds, H, dv, dk))
    _dev(d_initial_state, "d_initial_state", torch.float32, (N, H, dv, dk))
    _on_device(k=k, dh=dh, d_initial_state=d_initial_state, d_v=d_v)
    shape = _shape(N, H, dk, dv, T, k.dtype, k.dtype, g.dim() == 3, qdq_flags)
    ws_bytes = _lib.lib().gdn_chunk_bwd_workspace_bytes(ctypes.byref(shape))
    if ws_bytes == 0:
        _lib.check(_lib.GDN_ERR_INVALID_ARG)
    if workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=k.device)
    _dev(workspace, "workspace", torch.uint8)
    _on_device(k=k, workspace=workspace)
    st = _lib.lib().gdn_chunk_bwd_dh(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(beta), _ptr(g),
                                     _ptr(cu_seqlens), _ptr(seq_lens), _ptr(d_o), _ptr(d_final_state),
                                     _ptr(dh) if dh.numel() else None, _ptr(d_initial_state), _ptr(d_v),
                                     _ptr(workspace), workspace.numel(), _stream())
    _lib.check(st)
    if check_status:
        workspace_status(workspace)
    if d_v is not None:
        return dh, d_initial_state, d_v
    return dh, d_initial_state


def _states_shape(x, name):
    _dev(x, name, torch.float32)
    if x.dim() < 2:
        raise ValueError(f"{name} must be [..., dv, dk]")
    dv, dk = x.shape[-2], x.shape[-1]
    return dv, dk, (x.numel() // (dv * dk) if x.numel() else 0)


def state_qdq(x, out=None, scales=None, want_scales=True):
    """gdn_state_qdq on x [..., dv, dk] fp32.  Returns (out, scales [..., dv/64])."""
    dv, dk, n = _states_shape(x, "x")
    if out is None:
        out = torch.empty_like(x)
    if scales is None and want_scales:
        scales = torch.empty(x.shape[:-2] + (dv // 64,), dtype=torch.float32, device=x.device)
    _dev(out, "out", torch.float32, tuple(x.shape))
    _dev(scales, "scales", torch.float32, tuple(x.shape[:-2]) + (dv // 64,))
    _on_device(x=x, out=out, scales=scales)
    st = _lib.lib().gdn_state_qdq(_ptr(x), _ptr(out), _ptr(scales), n, dv, dk, _stream())
    _lib.check(st)
    return out, scales


def state_qdq_int8(x, out=None, scales=None, want_scales=True):
    """gdn_state_qdq_int8 on x [..., dv, dk] fp32 (blocks of 32 key columns).
    Returns (out, scales [..., dv, dk/32])."""
    dv, dk, n = _states_shape(x, "x")
    if out is None:
        out = torch.empty_like(x)
    if scales is None and want_scales:
        scales = torch.empty(x.shape[:-1] + (dk // 32,), dtype=torch.float32, device=x.device)
    _dev(out, "out", torch.float32, tuple(x.shape))
    _dev(scales, "scales", torch.float32, tuple(x.shape[:-1]) + (dk // 32,))
    _on_device(x=x, out=out, scales=scales)
    st = _lib.lib().gdn_state_qdq_int8(_ptr(x), _ptr(out), _ptr(scales), n, dv, dk, _stream())
    _lib.check(st)
    return out, scales


def decode_step(q, k, v, beta, g, state, *, qdq=True, o=None, o_dtype=None, state_pre=None,
                scales=None, int8=False, active=None, gate_grid_log2=0):
    """gdn_decode_step.  q, k: [N, H, dk]; v: [N, H, dv]; beta: [N, H]; g: [N, H]
    or [N, H, dk]; state [N, H, dv, dk] fp32 updated in place.  int8: the
    per-write QDQ is INT8 block-32 (scales [N, H, dv, dk/32]) instead of FP8
    per tile (scales [N, H, dv/64]).  active: optional [N] int32; sequences
    with active[n] == 0 are left untouched (state, o and the records).
    gate_grid_log2: 0, or k in 1..24: the log-gates rounded to multiples of
    2^-k (the log-retention grid).
    Returns o."""
    _dev(k, "k")
    if k.dim() != 3:
        raise ValueError(f"k must be [N, H, dk], got shape {tuple(k.shape)}")
    N, H, dk = k.shape
    _dev(v, "v")
    if v.dim() != 3 or tuple(v.shape[:2]) != (N, H):
        raise ValueError(f"v must be [{N}, {H}, dv], got shape {tuple(v.shape)}")
    dv = v.shape[2]
    if q.dtype != k.dtype or v.dtype != k.dtype or k.dtype not in _DT:
        raise ValueError("q, k, v must share one dtype: float32 or bfloat16")
    if o_dtype is None:
        o_dtype = o.dtype if isinstance(o, torch.Tensor) else k.dtype
    if o_dtype not in _DT:
        raise ValueError("o_dtype must be float32 or bfloat16")
    per_channel = g.dim() == 3
    sc_shape = (N, H, dv, dk // 32) if (int8 and qdq) else (N, H, dv // 64)
    for name, t, dt, shp in (("q", q, None, (N, H, dk)), ("beta", beta, torch.float32, (N, H)),
                             ("g", g, torch.float32, (N, H, dk) if per_channel else (N, H)),
                             ("state", state, torch.float32, (N, H, dv, dk)),
                             ("state_pre", state_pre, torch.float32, (N, H, dv, dk)),
                             ("scales", scales, torch.float32, sc_shape),
                             ("active", active, torch.int32, (N,))):
        _dev(t, name, dt, shp)
    if state is None:
        raise ValueError("state is required")
    _dev(o, "o", o_dtype, (N, H, dv))
    _on_device(q=q, k=k, v=v, beta=beta, g=g, state=state, state_pre=state_pre, scales=scales,
               active=active, o=o)
    if o is None:
        o = torch.empty((N, H, dv), dtype=o_dtype, device=k.device)
    shape = GdnShape(N, H, dk, dv, N, _DT[k.dtype], _DT[o_dtype], 1 if per_channel else 0,
                     (GDN_QDQ_WRITE if qdq else 0) | (_lib.GDN_QDQ_INT8 if int8 else 0), int(gate_grid_log2))
    st = _lib.lib().gdn_decode_step(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(beta),
                                    _ptr(g), _ptr(active), _ptr(state), _ptr(o), _ptr(state_pre),
                                    _ptr(scales), _stream())
    _lib.check(st)
    return o


# ---------------------------------------------------------------------------
# Linear attention with a decay for each head, block norms, 8-bit activations
#
# A decode step or a short prompt spends more time here than in its kernel, so
# these calls check all their tensors in one walk (_args) and pass plain
# integers to ctypes: a decode step of one sequence, 3 us of which is its
# kernel, takes 9.0 us that way and took 11.2 with a helper for each tensor.
# ---------------------------------------------------------------------------
def _args(*specs):
    """Checks of (name, tensor or None, dtype or None, shape or None), in
    order: type, dtype, shape and contiguity of every tensor first, then that
    all live on the current device.  Returns their addresses (None for no
    tensor)."""
    at = []
    dev, host, other = -1, None, None
    for name, t, dtype, shape in specs:
        if t is None:
            at.append(None)
            continue
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name} must be a torch tensor")
        if dtype is not None and t.dtype is not dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        d = t.get_device()
        if not t.is_cuda:
            host = host or name
        elif dev < 0:
            dev = d
        elif d != dev:
            other = other or (name, d)
        at.append(t.data_ptr())
    if host is not None:
        raise ValueError(f"{host} must be a device tensor")
    if other is not None:
        raise ValueError(f"{other[0]} is on cuda:{other[1]}, the other tensors on cuda:{dev}")
    if dev >= 0:
        _current(dev)
    return at


def _stream_at():
    """torch's current stream as a plain integer (a checked device tensor has
    initialised the device)."""
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _refuse():
    """Raise what the library said about a shape that needs no workspace."""
    _lib.check(_lib.GDN_ERR_INVALID_ARG)


def _scratch(workspace, need, like):
    """Address and bytes of the caller's workspace (checked by the library for
    its size), or of one of `need` bytes; and the tensor that holds it."""
    if need == 0:
        _refuse()
    if workspace is None:
        workspace = like.new_empty(need, dtype=torch.uint8)
        return workspace.data_ptr(), need, workspace
    at = _args(("k", like, None, None), ("workspace", workspace, torch.uint8, None))[1]
    if workspace.dim() != 1:
        raise ValueError("workspace must be a 1-D uint8 tensor")
    return at, workspace.numel(), workspace


def _lin_dims(q, k, v, g):
    """(T, H, Hk, dk, dv) of tensors whose shapes _args checks next."""
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError(f"k must be [T, Hk, dk], got {_what(k)}")
    T, Hk, dk = k.shape
    if k.dtype not in _DT:
        raise ValueError("q, k, v must share one dtype: float32 or bfloat16")
    if not isinstance(v, torch.Tensor) or v.dim() != 3 or v.shape[0] != T:
        raise ValueError(f"v must be [{T}, H, dv], got {_what(v)}")
    for name, t in (("q", q), ("g", g)):
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name} must be a torch tensor")
    return T, v.shape[1], Hk, dk, v.shape[2]


def _what(t):
    return f"shape {tuple(t.shape)}" if isinstance(t, torch.Tensor) else type(t).__name__


def _lin_specs(q, k, v, g, T, H):
    return (("q", q, k.dtype, k.shape), ("k", k, None, None), ("v", v, k.dtype, None),
            ("g", g, torch.float32, (H,) if g.dim() == 1 else (T, H)))


def _lin_seqs(cu_seqlens):
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be a tensor [N + 1] with N >= 1")
    return cu_seqlens.numel() - 1


def lin_attn_workspace_bytes(N, H, Hk, dk, dv, T, io_dtype=torch.bfloat16, gate_per_token=True, backward=False):
    """Device workspace lin_attn_fwd (or lin_attn_bwd) needs for this shape (bytes)."""
    shape = GdnLin(N, H, Hk, dk, dv, _DT[io_dtype], 1 if gate_per_token else 0, T)
    L = _lib.lib()
    n = (L.gdn_lin_attn_bwd_workspace_bytes if backward else L.gdn_lin_attn_fwd_workspace_bytes)(ctypes.byref(shape))
    if n == 0:
        _lib.check(_lib.GDN_ERR_INVALID_ARG)
    return n


def lin_attn_fwd(q, k, v, g, cu_seqlens, *, initial_state=None, out=None, final_state=None, workspace=None,
                 check_status=False):
    """gdn_lin_attn_fwd: S_t = e^{g_t} S_{t-1} + v_t k_t^T, o_t = S_t q_t over
    packed sequences.  q, k: [T, Hk, dk]; v: [T, H, dv] (fp32 or bf16; value
    head h uses query/key head h // (H / Hk)); g: [T, H], or [H] for one decay
    a head, fp32 natural log; cu_seqlens: [N + 1] int32; initial_state:
    [N, H, dv, dk] fp32 or None.  Rows outside every sequence are not written.
    check_status: read the workspace's status word after the call
    (synchronizes; raises GdnError when cu_seqlens is out of contract).
    Returns (o, final_state)."""
    T, H, Hk, dk, dv = _lin_dims(q, k, v, g)
    N = _lin_seqs(cu_seqlens)
    st = (N, H, dv, dk)
    at = _args(*_lin_specs(q, k, v, g, T, H), ("cu_seqlens", cu_seqlens, torch.int32, None),
               ("initial_state", initial_state, torch.float32, st), ("out", out, k.dtype, v.shape),
               ("final_state", final_state, torch.float32, st))
    if out is None:
        out = torch.empty_like(v)
        at[6] = out.data_ptr()
    if final_state is None:
        final_state = v.new_empty(st, dtype=torch.float32)
        at[7] = final_state.data_ptr()
    shape = ctypes.byref(GdnLin(N, H, Hk, dk, dv, _DT[k.dtype], g.dim() - 1, T))
    L = _lib.lib()
    ws, ws_bytes, workspace = _scratch(workspace, L.gdn_lin_attn_fwd_workspace_bytes(shape), k)
    _lib.check(L.gdn_lin_attn_fwd(shape, *at, ws, ws_bytes, _stream_at()))
    if check_status:
        workspace_status(workspace)
    return out, final_state


def lin_attn_bwd(q, k, v, g, cu_seqlens, d_o, *, initial_state=None, d_final_state=None, dq=None, dk=None, d_v=None,
                 dg=None, d_initial_state=None, workspace=None, check_status=False):
    """gdn_lin_attn_bwd: gradients of L = sum o . d_o + <S_final, d_final_state>
    for lin_attn_fwd's inputs.  d_o: as v; d_final_state: [N, H, dv, dk] fp32
    or None (zero).  Returns (dq, dk, dv, dg, d_initial_state): dq, dk, dv in
    the inputs' dtype (dq and dk summed over the heads that share them), dg
    fp32 of g's shape, d_initial_state [N, H, dv, dk] fp32."""
    T, H, Hk, dk_, dv_ = _lin_dims(q, k, v, g)
    N = _lin_seqs(cu_seqlens)
    if d_o is None:
        raise ValueError("d_o is required")
    st = (N, H, dv_, dk_)
    outs = [dq, dk, d_v, dg, d_initial_state]
    at = _args(*_lin_specs(q, k, v, g, T, H), ("cu_seqlens", cu_seqlens, torch.int32, None),
               ("d_o", d_o, k.dtype, v.shape), ("initial_state", initial_state, torch.float32, st),
               ("d_final_state", d_final_state, torch.float32, st), ("dq", dq, k.dtype, k.shape),
               ("dk", dk, k.dtype, k.shape), ("d_v", d_v, k.dtype, v.shape), ("dg", dg, torch.float32, g.shape),
               ("d_initial_state", d_initial_state, torch.float32, st))
    for i, like in enumerate((q, k, v, g)):
        if outs[i] is None:
            outs[i] = torch.empty_like(like)
            at[8 + i] = outs[i].data_ptr()
    if d_initial_state is None:
        outs[4] = v.new_empty(st, dtype=torch.float32)
        at[12] = outs[4].data_ptr()
    shape = ctypes.byref(GdnLin(N, H, Hk, dk_, dv_, _DT[k.dtype], g.dim() - 1, T))
    L = _lib.lib()
    ws, ws_bytes, workspace = _scratch(workspace, L.gdn_lin_attn_bwd_workspace_bytes(shape), k)
    _lib.check(L.gdn_lin_attn_bwd(shape, *at, ws, ws_bytes, _stream_at()))
    if check_status:
        workspace_status(workspace)
    return tuple(outs)


def lin_attn_step(q, k, v, g, state, *, o=None):
    """gdn_lin_attn_step: one token for each sequence.  q, k: [N, Hk, dk]; v:
    [N, H, dv]; g: [N, H] or [H]; state [N, H, dv, dk] fp32 updated in place.
    Returns o [N, H, dv]."""
    N, H, Hk, dk, dv = _lin_dims(q, k, v, g)
    if state is None:
        raise ValueError("state is required")
    at = _args(*_lin_specs(q, k, v, g, N, H), ("state", state, torch.float32, (N, H, dv, dk)),
               ("o", o, k.dtype, v.shape))
    if o is None:
        o = torch.empty_like(v)
        at[5] = o.data_ptr()
    shape = GdnLin(N, H, Hk, dk, dv, _DT[k.dtype], g.dim() - 1, N)
    _lib.check(_lib.lib().gdn_lin_attn_step(ctypes.byref(shape), *at, _stream_at()))
    return o


# ---------------------------------------------------------------------------
# All gradients of the chunked gated delta rule
# ---------------------------------------------------------------------------
def _grad_shape(N, H, dk, dv, T, io_dtype, qdq_flags):
    return GdnShape(N, H, dk, dv, T, _DT[io_dtype], _DT[io_dtype], 0, int(qdq_flags), 0)


def chunk_grad_workspace_bytes(N, H, dk, dv, T, io_dtype=torch.bfloat16, qdq_flags=0, states_given=False):
    """Device workspace chunk_grad needs for this shape (bytes)."""
    shape = _grad_shape(N, H, dk, dv, T, io_dtype, qdq_flags)
    n = _lib.lib().gdn_chunk_grad_workspace_bytes(ctypes.byref(shape), 1 if states_given else 0)
    if n == 0:
        _refuse()
    return n


def chunk_grad(q, k, v, beta, g, cu_seqlens, d_o, *, seq_lens=None, initial_state=None, states=None,
               d_final_state=None, qdq_flags=0, dq=None, dk=None, d_v=None, d_beta=None, dg=None,
               d_initial_state=None, workspace=None, check_status=False):
    """gdn_chunk_grad: every gradient of chunk_fwd over whole sequences for
    L = sum o . d_o + <S_final, d_final_state>, identity straight-through at
    the state's QDQ.  q, k: [T, H, dk]; v, d_o: [T, H, dv] (fp32 or bf16); beta,
    g: [T, H] fp32; cu_seqlens, seq_lens, initial_state: as for chunk_fwd;
    qdq_flags: the forward's (chunk_fwd's default is GDN_QDQ_CHUNK |
    GDN_QDQ_WRITE).  states: the states after every chunk as the forward's
    debug record bound_post has them ([n_bounds, H, dv, dk] fp32); None: they are
    computed again.  check_status: read the workspace's status word after the
    call (synchronizes; raises GdnError when the index arrays are out of
    contract).
    Returns (dq, dk, dv, dbeta, dg, d_initial_state): dq, dk, dv in the inputs'
    dtype, the others fp32; rows of a segment past its length are 0."""
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError(f"k must be [T, H, dk], got {_what(k)}")
    T, H, dk_ = k.shape
    if k.dtype not in _DT:
        raise ValueError("q, k, v must share one dtype: float32 or bfloat16")
    if not isinstance(v, torch.Tensor) or v.dim() != 3 or v.shape[:2] != (T, H):
        raise ValueError(f"v must be [{T}, {H}, dv], got {_what(v)}")
    dv_ = v.shape[2]
    N = _lin_seqs(cu_seqlens)
    for name, t in (("q", q), ("beta", beta), ("g", g), ("d_o", d_o)):
        if t is None:
            raise ValueError(f"{name} is required")
    f32, th, st = torch.float32, (T, H), (N, H, dv_, dk_)
    if states is not None and (not isinstance(states, torch.Tensor) or states.dim() != 4 or
                               states.shape[1:] != (H, dv_, dk_)):
        raise ValueError(f"states must be [n_bounds, {H}, {dv_}, {dk_}], got {_what(states)}")
    outs = [dq, dk, d_v, d_beta, dg, d_initial_state]
    at = _args(("q", q, k.dtype, k.shape), ("k", k, None, None), ("v", v, k.dtype, None), ("beta", beta, f32, th),
               ("g", g, f32, th), ("cu_seqlens", cu_seqlens, torch.int32, None),
               ("seq_lens", seq_lens, torch.int32, (N,)), ("initial_state", initial_state, f32, st),
               ("states", states, f32, None), ("d_o", d_o, k.dtype, v.shape),
               ("d_final_state", d_final_state, f32, st), ("dq", dq, k.dtype, k.shape), ("dk", dk, k.dtype, k.shape),
               ("d_v", d_v, k.dtype, v.shape), ("d_beta", d_beta, f32, th), ("dg", dg, f32, th),
               ("d_initial_state", d_initial_state, f32, st))
    for i, like in enumerate((q, k, v, beta, g)):
        if outs[i] is None:
            outs[i] = torch.empty_like(like)
            at[11 + i] = outs[i].data_ptr()
    if d_initial_state is None:
        outs[5] = v.new_empty(st, dtype=f32)
        at[16] = outs[5].data_ptr()
    shape = ctypes.byref(_grad_shape(N, H, dk_, dv_, T, k.dtype, qdq_flags))
    L = _lib.lib()
    need = L.gdn_chunk_grad_workspace_bytes(shape, 0 if states is None else 1)
    ws, ws_bytes, workspace = _scratch(workspace, need, k)
    if states is not None and at[8] == 0:   # no entries, and so no memory: still given
        at[8] = ws
    at.insert(9, 0 if states is None else states.shape[0])
    _lib.check(L.gdn_chunk_grad(shape, *at, ws, ws_bytes, _stream_at()))
    if check_status:
        workspace_status(workspace)
    return tuple(outs)


_ACT = {"silu": _lib.GDN_ACT_SILU, "sigmoid": _lib.GDN_ACT_SIGMOID}


def _addr(t):
    return None if t is None else t.data_ptr()


def _rows(t, name):
    if not isinstance(t, torch.Tensor) or t.dim() < 1 or t.shape[-1] < 1:
        raise ValueError(f"{name} must be a tensor [..., cols] with cols >= 1")
    if t.shape[-1] >= 1 << 31:     # the library's 32-bit cols would wrap
        raise ValueError(f"{name} must have fewer than 2^31 columns, got {t.shape[-1]}")
    return t.shape[-1], t.numel() // t.shape[-1]


def _norm_shape(rows, cols, io_dtype, x_dtype, act, res_scale, eps):
    if io_dtype not in _DT or x_dtype not in _DT:
        raise ValueError("dtypes must be float32 or bfloat16")
    if act not in _ACT:
        raise ValueError(f"act must be one of {sorted(_ACT)}, got {act!r}")
    return GdnNorm(rows, cols, _DT[io_dtype], _DT[x_dtype], _ACT[act], float(res_scale), float(eps))


def block_norm_fwd(f, w_post, *, gate=None, act="silu", residual=None, res_scale=1.0, w_pre=None, eps=1e-6,
                   x_dtype=None, checkpoint=False):
    """gdn_block_norm_fwd: the norm after a block, its gate, the scaled residual
    and the norm before the next block:
        x = res_scale * (f / rms(f) * w_post * a(gate)) + residual
        h = x / rms(x) * w_pre
    f, gate: [..., cols] fp32 or bf16; act: "silu" or "sigmoid"; residual: as f
    in x_dtype (default: the residual's dtype, else f's); w_post, w_pre: [cols]
    fp32.  Without w_pre h is None.  Returns (x, h); with checkpoint also f and
    the gate as (codes, scales) of act_pack (None without a gate)."""
    cols, rows = _rows(f, "f")
    if x_dtype is None:
        x_dtype = residual.dtype if isinstance(residual, torch.Tensor) else f.dtype
    shape = _norm_shape(rows, cols, f.dtype, x_dtype, act, res_scale, eps)
    if w_post is None:
        raise ValueError("w_post is required")
    at = _args(("f", f, None, None), ("gate", gate, f.dtype, f.shape), ("residual", residual, x_dtype, f.shape),
               ("w_post", w_post, torch.float32, (cols,)), ("w_pre", w_pre, torch.float32, (cols,)))
    x = torch.empty_like(f, dtype=x_dtype)
    h = torch.empty_like(f) if w_pre is not None else None
    fc = zc = (None, None)
    if checkpoint:
        fc = _code_buffers(f)
        zc = _code_buffers(f) if gate is not None else zc
    _lib.check(_lib.lib().gdn_block_norm_fwd(ctypes.byref(shape), *at, x.data_ptr(), _addr(h), _addr(fc[0]),
                                             _addr(fc[1]), _addr(zc[0]), _addr(zc[1]), _stream_at()))
    if checkpoint:
        return x, h, fc, (zc if gate is not None else None)
    return x, h


def _values_or_codes(t, name, dtype):
    """_args' specs of an argument that may be act_pack's pair: (values or
    codes), (scales or None)."""
    if not isinstance(t, tuple):
        return (name, t, dtype, None), (name, None, None, None)
    if len(t) != 2:
        raise ValueError(f"{name} must be a tensor or (codes, scales)")
    codes, scales = t
    cols, _ = _rows(codes, f"{name} codes")
    if scales is None:
        raise ValueError(f"{name} scales are required")
    return ((f"{name} codes", codes, torch.float8_e4m3fn, None),
            (f"{name} scales", scales, torch.float32, codes.shape[:-1] + (-(-cols // 64),)))


def block_norm_bwd(f, w_post, d_x, *, d_h=None, x=None, w_pre=None, gate=None, act="silu", res_scale=1.0, eps=1e-6,
                   want_residual=True, io_dtype=None, workspace=None):
    """gdn_block_norm_bwd: gradients of block_norm_fwd's inputs from d_x and,
    with w_pre, d_h (x is the forward's x).  f and gate are the forward's
    tensors or both its (codes, scales) checkpoints; io_dtype: the dtype of f
    (needed with checkpoints and no d_h).
    Returns (d_f, d_gate, d_residual, d_w_post, d_w_pre), None where the
    forward had no such input (d_residual also without want_residual)."""
    if not isinstance(f, tuple):
        _rows(f, "f")
    if io_dtype is None:
        io_dtype = d_h.dtype if isinstance(d_h, torch.Tensor) else None if isinstance(f, tuple) else f.dtype
        if io_dtype is None:
            raise ValueError("io_dtype is needed with checkpoints and no d_h")
    f_spec, fs_spec = _values_or_codes(f, "f", io_dtype)
    f = f_spec[1]
    cols, rows = _rows(f, "f")
    z_spec = zs_spec = ("gate", None, None, None)
    if gate is not None:
        z_spec, zs_spec = _values_or_codes(gate, "gate", io_dtype)
        if (zs_spec[1] is None) != (fs_spec[1] is None):
            raise ValueError("f and gate must both be tensors or both checkpoints")
        z_spec = z_spec[:3] + (f.shape,)
    if d_x is None:
        raise ValueError("d_x is required")
    if w_post is None:
        raise ValueError("w_post is required")
    if w_pre is not None and (x is None or d_h is None):
        raise ValueError("w_pre needs x and d_h")
    xt = d_x.dtype if isinstance(d_x, torch.Tensor) else None
    at = _args(f_spec, fs_spec, z_spec, zs_spec, ("w_post", w_post, torch.float32, (cols,)),
               ("w_pre", w_pre, torch.float32, (cols,)), ("x", x, xt, f.shape), ("d_x", d_x, None, f.shape),
               ("d_h", d_h, io_dtype, f.shape))
    if w_pre is None:
        at[6] = at[8] = None
    shape = ctypes.byref(_norm_shape(rows, cols, io_dtype, xt, act, res_scale, eps))
    d_f = torch.empty_like(f, dtype=io_dtype)
    d_z = torch.empty_like(d_f) if gate is not None else None
    d_res = torch.empty_like(d_x) if want_residual else None
    dw_post = torch.empty_like(w_post)
    dw_pre = torch.empty_like(w_pre) if w_pre is not None else None
    L = _lib.lib()
    ws, ws_bytes, workspace = _scratch(workspace, L.gdn_block_norm_bwd_workspace_bytes(shape), f)
    _lib.check(L.gdn_block_norm_bwd(shape, *at, d_f.data_ptr(), _addr(d_z), _addr(d_res), dw_post.data_ptr(),
                                    _addr(dw_pre), ws, ws_bytes, _stream_at()))
    return d_f, d_z, d_res, dw_post, dw_pre


def _code_buffers(x):
    return (torch.empty_like(x, dtype=torch.float8_e4m3fn),
            x.new_empty(x.shape[:-1] + (-(-x.shape[-1] // 64),), dtype=torch.float32))


def act_pack(x):
    """gdn_act_pack: x [..., cols] (fp32 or bf16) as E4M3 codes with one fp32
    scale for each 64 columns.  Returns (codes float8_e4m3fn [..., cols],
    scales [..., ceil(cols / 64)])."""
    cols, rows = _rows(x, "x")
    if x.dtype not in _DT:
        raise ValueError("x must be float32 or bfloat16")
    at = _args(("x", x, None, None))
    codes, scales = _code_buffers(x)
    _lib.check(_lib.lib().gdn_act_pack(at[0], _DT[x.dtype], codes.data_ptr(), scales.data_ptr(), rows, cols,
                                       _stream_at()))
    return codes, scales


def act_unpack(codes, scales, *, dtype=torch.bfloat16):
    """gdn_act_unpack: the values code * scale of act_pack's result, in dtype."""
    specs = _values_or_codes((codes, scales), "act", None)
    cols, rows = _rows(codes, "codes")
    if dtype not in _DT:
        raise ValueError("dtype must be float32 or bfloat16")
    at = _args(*specs)
    x = torch.empty_like(codes, dtype=dtype)
    _lib.check(_lib.lib().gdn_act_unpack(*at, x.data_ptr(), _DT[dtype], rows, cols, _stream_at()))
    return x


# ---------------------------------------------------------------------------
# Distillation from a teacher's top logits
# ---------------------------------------------------------------------------
def _matrix(t, name):
    """Rows, columns and row stride of a matrix whose rows are contiguous (a
    slice of a wider one will do)."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.shape[1] < 1:
        raise ValueError(f"{name} must be a tensor [rows, vocab] with vocab >= 1, got {_what(t)}")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    stride = t.stride(0) if rows > 1 else cols
    if stride < cols:
        raise ValueError(f"{name} must have rows that do not overlap")
    if cols >= 1 << 31:    # the library's 32-bit vocab would wrap
        raise ValueError(f"{name} must have fewer than 2^31 columns, got {cols}")
    return rows, cols, stride


_NEW = object()   # a gradient's tensor that is allocated here


def _distill_args(logits, ids, top, teacher_lse, targets, temperature, kd_weight, ce_weight, ignore_index, out, *more):
    """Checked shape, the addresses of ids, top, teacher_lse, targets and of
    `more`, and the gradient's tensor (out, one like the logits, or none)."""
    R, V, stride = _matrix(logits, "logits")
    if out is not None and out is not _NEW and not isinstance(out, torch.Tensor):
        raise ValueError("out must be a torch tensor")
    if logits.dtype not in _DT:
        raise ValueError("logits must be float32 or bfloat16")
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2 or ids.shape[0] != R:
        raise ValueError(f"ids must be [{R}, topk], got {_what(ids)}")
    K = ids.shape[1]
    if K >= 1 << 31:
        raise ValueError(f"ids must have fewer than 2^31 columns, got {K}")
    if top is None:
        raise ValueError("top is required")
    specs = [("ids", ids, torch.int32, None), ("top", top, torch.float32, (R, K)),
             ("teacher_lse", teacher_lse, torch.float32, (R,)), ("targets", targets, torch.int64, (R,)), *more]
    d_stride = V
    if isinstance(out, torch.Tensor):
        d_stride = _matrix(out, "out")[2]
        if out.dtype is not logits.dtype or out.shape != logits.shape:
            raise ValueError(f"out must be {logits.dtype} of shape {tuple(logits.shape)}, got {out.dtype} of "
                             f"shape {tuple(out.shape)}")
        specs.append(("out", out if out.is_contiguous() else out[:1, :1], None, None))
    at = _args(("logits", logits if logits.is_contiguous() else logits[:1, :1], None, None), *specs)
    if out is _NEW:
        out = logits.new_empty(R, V)
    elif out is not None:
        at.pop()
    shape = GdnDistill(R, V, K, _DT[logits.dtype], temperature, kd_weight, ce_weight, ignore_index, stride, d_stride)
    return ctypes.byref(shape), at, out


def distill_fwd(logits, ids, top, *, teacher_lse=None, targets=None, temperature=1.0, kd_weight=1.0, ce_weight=0.0,
                ignore_index=-100):
    """gdn_distill_fwd: kd_weight * kd + ce_weight * ce of every row of logits
    [rows, vocab] (fp32 or bf16; rows contiguous, any row stride).  kd: the
    divergence of the student, softmax(logits / temperature), from the teacher's
    kept logits top [rows, topk] fp32 at columns ids [rows, topk] int32 (negative:
    not used), normalised over them, or with teacher_lse [rows] fp32 (logsumexp of
    the teacher's whole row / temperature) with all other columns as one more
    outcome.  ce: cross entropy against targets [rows] int64 (None: none); a row
    whose target is ignore_index has no loss at all.
    Returns (loss [rows], stats [rows, 4]) in fp32; stats is for distill_bwd."""
    shape, at, _ = _distill_args(logits, ids, top, teacher_lse, targets, temperature, kd_weight, ce_weight,
                                 ignore_index, None)
    loss = top.new_empty(logits.shape[0])
    stats = top.new_empty(logits.shape[0], 4)
    _lib.check(_lib.lib().gdn_distill_fwd(shape, *at, loss.data_ptr(), stats.data_ptr(), _stream_at()))
    return loss, stats


def distill_bwd(logits, ids, top, stats, d_loss=None, *, teacher_lse=None, targets=None, temperature=1.0,
                kd_weight=1.0, ce_weight=0.0, ignore_index=-100, out=None):
    """gdn_distill_bwd: the gradient of distill_fwd's logits for d_loss [rows]
    fp32 (None: 1).  stats: what distill_fwd returned; the other arguments are
    its.  out: as the logits, and may be the logits themselves (they are
    overwritten then).  Returns d_logits."""
    R = logits.shape[0] if isinstance(logits, torch.Tensor) and logits.dim() else 0
    if stats is None:
        raise ValueError("stats is required")
    shape, at, out = _distill_args(logits, ids, top, teacher_lse, targets, temperature, kd_weight, ce_weight,
                                   ignore_index, _NEW if out is None else out,
                                   ("stats", stats, torch.float32, (R, 4)), ("d_loss", d_loss, torch.float32, (R,)))
    _lib.check(_lib.lib().gdn_distill_bwd(shape, *at, out.data_ptr(), _stream_at()))
    return out


def distill_fwd_bwd(logits, ids, top, d_loss=None, *, teacher_lse=None, targets=None, temperature=1.0, kd_weight=1.0,
                    ce_weight=0.0, ignore_index=-100, out=None):
    """gdn_distill_fwd_bwd: distill_fwd's losses and, for d_loss [rows] fp32
    (None: 1), the logits' gradient, reading the logits once.  out: as in
    distill_bwd.  Returns (loss [rows] fp32, d_logits)."""
    R = logits.shape[0] if isinstance(logits, torch.Tensor) and logits.dim() else 0
    shape, at, out = _distill_args(logits, ids, top, teacher_lse, targets, temperature, kd_weight, ce_weight,
                                   ignore_index, _NEW if out is None else out,
                                   ("d_loss", d_loss, torch.float32, (R,)))
    loss = top.new_empty(R)
    _lib.check(_lib.lib().gdn_distill_fwd_bwd(shape, *at, loss.data_ptr(), out.data_ptr(), _stream_at()))
    return loss, out
