"""Binding of the gated delta rule and of the norm and rotation of its queries
and keys (the package's public names; see the header for the formulas).

As in the rest of the binding: arguments are checked, outputs and workspaces
come from PyTorch's allocator, and the library runs on ``stream`` (the current
one by default).  Outputs and workspaces are allocated on that stream too, so
that a workspace is not handed out again before the kernels are done with it.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools

import torch

from . import SSD_BF16, SSD_F32, SsdError, _check, _ptr, lib

DELTA_CU_SEQLENS = 1
NORMS = {"rms": 0, "l2": 1}
_TYPES = {torch.bfloat16: SSD_BF16, torch.float32: SSD_F32}


class QkDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("tokens", "q_stride", "k_stride", "positions")] + \
               [(n, ctypes.c_int32) for n in ("qheads", "kheads", "headdim", "rotary", "interleaved", "norm",
                                              "dtype")] + [("eps", ctypes.c_float)]


class DeltaDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("batch", "seqlen", "nheads", "headdim", "ngroups", "dstate", "nseq",
                                              "q_stride", "k_stride", "v_stride")] + \
               [("dtype", ctypes.c_int32), ("flags", ctypes.c_int32)]


def declare(L):
    """Signatures of the entry points used here (called once, when the library is loaded)."""
    vp, sz, i64, f32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64, ctypes.c_float
    pq, pd = ctypes.POINTER(QkDims), ctypes.POINTER(DeltaDims)
    for name, res, args in (
            ("qk_fwd", ctypes.c_int, [pq] + [vp] * 10),
            ("qk_bwd_workspace_size", sz, [pq]),
            ("qk_bwd", ctypes.c_int, [pq] + [vp] * 14 + [sz, vp]),
            ("delta_saved_size", sz, [pd]),
            ("delta_fwd_workspace_size", sz, [pd]),
            ("delta_bwd_workspace_size", sz, [pd]),
            ("delta_path_name", ctypes.c_char_p, [pd]),
            ("delta_fwd", ctypes.c_int, [pd] + [vp] * 7 + [f32] + [vp] * 3 + [sz, vp, sz, vp]),
            ("delta_bwd", ctypes.c_int, [pd] + [vp] * 5 + [f32, vp, sz] + [vp] * 9 + [sz, vp]),
            ("delta_step", ctypes.c_int, [pd] + [vp] * 5 + [f32, vp, i64, vp, vp, vp])):
        f = getattr(L, "mamba2_ssd_" + name)
        f.argtypes, f.restype = args, res


def make_qk_dims(tokens, qheads, kheads, headdim, rotary=0, positions=0, norm="l2", dtype=torch.bfloat16, eps=1e-6,
                 interleaved=False, q_stride=0, k_stride=0):
    return QkDims(tokens, q_stride, k_stride, positions, qheads, kheads, headdim, rotary, int(interleaved),
                  NORMS[norm], _TYPES[dtype], eps)


def make_delta_dims(batch, seqlen, nheads, headdim, ngroups, dstate, nseq=None, dtype=torch.bfloat16, cu_seqlens=False,
                    q_stride=0, k_stride=0, v_stride=0):
    return DeltaDims(batch, seqlen, nheads, headdim, ngroups, dstate, batch if nseq is None else nseq, q_stride,
                     k_stride, v_stride, _TYPES[dtype], DELTA_CU_SEQLENS if cu_seqlens else 0)


# dims by their values: the sizes of a program's calls are few, and a struct of ten fields costs a few microseconds
_qk_dims = functools.lru_cache(maxsize=256)(make_qk_dims)
_delta_dims = functools.lru_cache(maxsize=256)(make_delta_dims)


def delta_path_name(dims: DeltaDims) -> str:
    """Name of the kernels that these dims run on."""
    return lib().mamba2_ssd_delta_path_name(ctypes.byref(dims)).decode()


def _scope(t, stream):
    """(context, stream handle) in which a call on t's device allocates and launches."""
    if stream is None and t.device.index == torch.cuda.current_device():
        return contextlib.nullcontext(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    s = torch.cuda.current_stream(t.device) if stream is None else stream
    return torch.cuda.stream(s), ctypes.c_void_p(s.cuda_stream)


def _rows(t, name, b, T, dtype, device):
    """t (b, T, heads, d) whose tokens are equally spaced rows, each with its heads side by side: (heads, d, spacing)."""
    if t is None or t.dim() != 4 or t.shape[0] != b or t.shape[1] != T or t.dtype != dtype or t.device != device:
        raise ValueError("%s: expected (%d, %d, heads, d) %s on %s, got %s" %
                         (name, b, T, dtype, device, None if t is None else (tuple(t.shape), t.dtype, t.device)))
    h, d = t.shape[2], t.shape[3]
    if b * T == 0:
        return h, d, 0
    s0, s1, s2, s3 = t.stride()
    if (d > 1 and s3 != 1) or (h > 1 and s2 != d):
        raise ValueError("%s: the heads of a token must lie side by side (strides %s)" % (name, t.stride()))
    if T == 1:
        s1 = s0 if b > 1 else h * d
    elif b > 1 and s0 != T * s1:
        raise ValueError("%s: tokens must be equally spaced over the batch (strides %s)" % (name, t.stride()))
    if b * T > 1 and s1 < h * d:
        raise ValueError("%s: overlapping tokens (strides %s)" % (name, t.stride()))
    return h, d, s1 if b * T > 1 else 0


def _type(t):
    if t.dtype not in _TYPES:
        raise ValueError("expected bf16 or fp32, got %s" % t.dtype)
    return t.dtype


# ---- norm of queries and keys, with rotation --------------------------------

def _qk_args(q, k, wq, wk, cos, sin, positions, norm, eps, interleaved):
    dt, dev = _type(q), q.device
    if q.dim() != 4:
        raise ValueError("q must be (batch, seqlen, heads, headdim)")
    b, T = q.shape[:2]
    hq, d, qs = _rows(q, "q", b, T, dt, dev)
    hk, dk, ks = _rows(k, "k", b, T, dt, dev)
    if dk != d:
        raise ValueError("q and k have different headdim")
    if norm not in NORMS:
        raise ValueError("norm must be 'rms' or 'l2'")
    if (wq is None) != (wk is None):
        raise ValueError("wq and wk are given together or not at all")
    if wq is not None:
        _check(wq, "wq", (d,), torch.float32, dev)
        _check(wk, "wk", (d,), torch.float32, dev)
    rotary = npos = 0
    if cos is not None:
        if cos.dim() != 2 or sin is None or positions is None:
            raise ValueError("cos and sin (positions, rotary / 2) and positions (batch, seqlen) are given together")
        npos, rotary = cos.shape[0], 2 * cos.shape[1]
        _check(cos, "cos", (npos, rotary // 2), torch.float32, dev)
        _check(sin, "sin", (npos, rotary // 2), torch.float32, dev)
        _check(positions, "positions", (b, T), torch.int32, dev)
    elif sin is not None or positions is not None:
        raise ValueError("cos, sin and positions are given together or not at all")
    return _qk_dims(b * T, hq, hk, d, rotary, npos, norm, dt, float(eps), bool(interleaved), qs, ks)


def qk_fwd(q, k, wq=None, wk=None, cos=None, sin=None, positions=None, norm="l2", eps=1e-6, interleaved=False,
           stream=None):
    """(yq, yk): each head's row of q (b,T,Hq,D) and k (b,T,Hk,D) divided by
    the root of its mean ("rms") or summed ("l2") squares plus eps, times wq /
    wk (D, fp32) if given, its first 2 * cos.shape[1] elements turned by the
    angle of the token's position (int32 (b,T) into the fp32 tables cos, sin).
    q and k may be slices of one projection; outputs are packed."""
    dims = _qk_args(q, k, wq, wk, cos, sin, positions, norm, eps, interleaved)
    ctx, st = _scope(q, stream)
    with ctx:
        yq = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        yk = torch.empty(k.shape, dtype=q.dtype, device=q.device)
        rc = lib().mamba2_ssd_qk_fwd(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(wq), _ptr(wk), _ptr(cos), _ptr(sin),
                                     _ptr(positions), _ptr(yq), _ptr(yk), st)
    if rc:
        raise SsdError(rc, "mamba2_ssd_qk_fwd")
    return yq, yk


def qk_bwd(q, k, dyq, dyk, wq=None, wk=None, cos=None, sin=None, positions=None, norm="l2", eps=1e-6,
           interleaved=False, stream=None):
    """dict of dq, dk (in q's dtype, packed) and, with weights, dwq, dwk (fp32) of sum(yq * dyq) + sum(yk * dyk)."""
    dims = _qk_args(q, k, wq, wk, cos, sin, positions, norm, eps, interleaved)
    dt, dev = q.dtype, q.device
    _check(dyq, "dyq", tuple(q.shape), dt, dev)
    _check(dyk, "dyk", tuple(k.shape), dt, dev)
    ctx, st = _scope(q, stream)
    with ctx:
        out = dict(dq=torch.empty(q.shape, dtype=dt, device=dev), dk=torch.empty(k.shape, dtype=dt, device=dev))
        ws = None
        if wq is not None:
            out["dwq"], out["dwk"] = torch.empty_like(wq), torch.empty_like(wk)
            ws = torch.empty(lib().mamba2_ssd_qk_bwd_workspace_size(ctypes.byref(dims)), dtype=torch.uint8, device=dev)
        rc = lib().mamba2_ssd_qk_bwd(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(dyq), _ptr(dyk), _ptr(wq), _ptr(wk),
                                     _ptr(cos), _ptr(sin), _ptr(positions), _ptr(out["dq"]), _ptr(out["dk"]),
                                     _ptr(out.get("dwq")), _ptr(out.get("dwk")), _ptr(ws),
                                     0 if ws is None else ws.numel(), st)
    if rc:
        raise SsdError(rc, "mamba2_ssd_qk_bwd")
    return out


class QkFunction(torch.autograd.Function):
    """(yq, yk) of qk_fwd as a differentiable op; its backward is qk_bwd."""

    @staticmethod
    def forward(ctx, q, k, wq, wk, cos, sin, positions, norm, eps, interleaved):
        ctx.save_for_backward(q, k, wq, wk, cos, sin, positions)
        ctx.how = dict(norm=norm, eps=eps, interleaved=interleaved)
        return qk_fwd(q, k, wq, wk, cos, sin, positions, **ctx.how)

    @staticmethod
    def backward(ctx, dyq, dyk):
        q, k, *rest = ctx.saved_tensors
        g = qk_bwd(q, k, dyq.contiguous(), dyk.contiguous(), *rest, **ctx.how)
        return g["dq"], g["dk"], g.get("dwq"), g.get("dwk"), None, None, None, None, None, None


def qk_norm(q, k, wq=None, wk=None, cos=None, sin=None, positions=None, norm="l2", eps=1e-6, interleaved=False):
    """Differentiable norm and rotation of queries and keys (see qk_fwd)."""
    return QkFunction.apply(q, k, wq, wk, cos, sin, positions, norm, eps, interleaved)


# ---- gated delta rule --------------------------------------------------------

class DeltaSaved:
    """What delta_bwd needs: the forward's inputs and its record."""

    def __init__(self, dims, tensors, scale):
        self.dims = dims
        self.tensors = tensors
        self.scale = scale

    @property
    def final(self):
        """The state after each sequence (nseq, H, P, N) fp32, where the forward was asked for it."""
        return self.tensors["final"]


def _delta_args(q, k, v, g, beta, cu_seqlens, init_states):
    dt, dev = _type(q), q.device
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k (batch, seqlen, groups, dstate) and v (batch, seqlen, heads, headdim) are 4-dimensional")
    b, T = q.shape[:2]
    G, N, qs = _rows(q, "q", b, T, dt, dev)
    Gk, Nk, ks = _rows(k, "k", b, T, dt, dev)
    H, P, vs = _rows(v, "v", b, T, dt, dev)
    if (Gk, Nk) != (G, N):
        raise ValueError("q and k have different shapes")
    if H % G:
        raise ValueError("heads must be a multiple of groups")
    _check(g, "g", (b, T, H), torch.float32, dev)
    _check(beta, "beta", (b, T, H), torch.float32, dev)
    nseq = b
    if cu_seqlens is not None:
        if b != 1 or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
            raise ValueError("cu_seqlens (nseq + 1) goes with one packed row (batch 1)")
        nseq = cu_seqlens.shape[0] - 1
        _check(cu_seqlens, "cu_seqlens", (nseq + 1,), torch.int32, dev)
    if init_states is not None:
        _check(init_states, "init_states", (nseq, H, P, N), torch.float32, dev)
    return _delta_dims(b, T, H, P, G, N, nseq, dt, cu_seqlens is not None, qs, ks, vs)


def _delta_run(q, k, v, g, beta, scale, cu_seqlens, init_states, want_final, want_saved, stream):
    dims = _delta_args(q, k, v, g, beta, cu_seqlens, init_states)
    scale = dims.dstate ** -0.5 if scale is None else float(scale)
    dev, L, at = q.device, lib(), ctypes.byref(dims)
    ctx, st = _scope(q, stream)
    with ctx:
        o = torch.empty(v.shape, dtype=v.dtype, device=dev)
        final = torch.empty((dims.nseq, dims.nheads, dims.headdim, dims.dstate), dtype=torch.float32,
                            device=dev) if want_final else None
        saved = torch.empty(L.mamba2_ssd_delta_saved_size(at), dtype=torch.uint8, device=dev) if want_saved else None
        ws = None if want_saved else torch.empty(L.mamba2_ssd_delta_fwd_workspace_size(at), dtype=torch.uint8, device=dev)
        rc = L.mamba2_ssd_delta_fwd(at, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens),
                                    _ptr(init_states), scale, _ptr(o), _ptr(final), _ptr(saved),
                                    0 if saved is None else saved.numel(), _ptr(ws),
                                    0 if ws is None else ws.numel(), st)
    if rc:
        raise SsdError(rc, "mamba2_ssd_delta_fwd")
    keep = dict(q=q, k=k, g=g, beta=beta, cu_seqlens=cu_seqlens, init=init_states, saved=saved, final=final)
    return o, final, DeltaSaved(dims, keep, scale)


def delta_fwd(q, k, v, g, beta, scale=None, init_states=None, cu_seqlens=None, want_final=False, stream=None):
    """Forward of a training step: (o, saved).  q, k (b,T,G,N) and v (b,T,H,P)
    in bf16 or fp32, possibly slices of wider rows; g (log decay) and beta
    (b,T,H) fp32; init_states (nseq,H,P,N) fp32; cu_seqlens (nseq+1) int32 for
    sequences packed into one row; scale 1/sqrt(N) by default.  The final
    states are saved.final where want_final."""
    o, _, saved = _delta_run(q, k, v, g, beta, scale, cu_seqlens, init_states, want_final, True, stream)
    return o, saved


def delta_prefill(q, k, v, g, beta, scale=None, init_states=None, cu_seqlens=None, stream=None):
    """Forward that keeps nothing for a backward: (o, final states (nseq,H,P,N) fp32)."""
    return _delta_run(q, k, v, g, beta, scale, cu_seqlens, init_states, True, False, stream)[:2]


def delta_bwd(saved: DeltaSaved, dout, dfinal=None, want_dinit=None, stream=None):
    """dict of dq, dk, dv, dg, dbeta (in q's dtype) and, with initial states
    (or want_dinit), dinit (fp32) of sum(o * dout) + sum(final * dfinal)."""
    t, d = saved.tensors, saved.dims
    q, k = t["q"], t["k"]
    dev, dt = q.device, q.dtype
    shape = tuple(q.shape[:2]) + (d.nheads, d.headdim)
    _check(dout, "dout", shape, dt, dev)
    states = (d.nseq, d.nheads, d.headdim, d.dstate)
    if dfinal is not None:
        _check(dfinal, "dfinal", states, torch.float32, dev)
    if want_dinit is None:
        want_dinit = t["init"] is not None
    L, at = lib(), ctypes.byref(d)
    ctx, st = _scope(q, stream)
    with ctx:
        out = dict(dq=torch.empty(q.shape, dtype=dt, device=dev), dk=torch.empty(k.shape, dtype=dt, device=dev),
                   dv=torch.empty(shape, dtype=dt, device=dev), dg=torch.empty(shape[:3], dtype=dt, device=dev),
                   dbeta=torch.empty(shape[:3], dtype=dt, device=dev))
        if want_dinit:
            out["dinit"] = torch.empty(states, dtype=torch.float32, device=dev)
        ws = torch.empty(L.mamba2_ssd_delta_bwd_workspace_size(at), dtype=torch.uint8, device=dev)
        rc = L.mamba2_ssd_delta_bwd(at, _ptr(q), _ptr(k), _ptr(t["g"]), _ptr(t["beta"]), _ptr(t["cu_seqlens"]),
                                    saved.scale, _ptr(t["saved"]), t["saved"].numel(), _ptr(dout), _ptr(dfinal),
                                    _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dg"]),
                                    _ptr(out["dbeta"]), _ptr(out.get("dinit")), _ptr(ws), ws.numel(), st)
    if rc:
        raise SsdError(rc, "mamba2_ssd_delta_bwd")
    return out


def delta_step(q, k, v, g, beta, states, slots=None, scale=None, stream=None):
    """Recurrent form: o (b,T,H,P) of T tokens (one, or a few drafted ones) for
    each of b sequences, whose states (slots,H,P,N) fp32 are updated in place.
    Row i uses states[slots[i]] (slots int32; row i itself without); a slot
    outside the pool marks an idle row (o zero).  Shapes as in delta_fwd."""
    dims = _delta_args(q, k, v, g, beta, None, None)
    n = states.shape[0] if states.dim() == 4 else 0
    _check(states, "states", (n, dims.nheads, dims.headdim, dims.dstate), torch.float32, q.device)
    if slots is not None:
        _check(slots, "slots", (dims.batch,), torch.int32, q.device)
    elif n < dims.batch:
        raise ValueError("fewer states than rows")
    scale = dims.dstate ** -0.5 if scale is None else float(scale)
    ctx, st = _scope(q, stream)
    with ctx:
        o = torch.empty(v.shape, dtype=v.dtype, device=q.device)
        rc = lib().mamba2_ssd_delta_step(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), scale,
                                         _ptr(states), n, _ptr(slots), _ptr(o), st)
    if rc:
        raise SsdError(rc, "mamba2_ssd_delta_step")
    return o


class DeltaFunction(torch.autograd.Function):
    """(o, final states) as a differentiable op: delta_fwd and delta_bwd.
    Gradients come in q's dtype; autograd casts those of g and beta."""

    @staticmethod
    def forward(ctx, q, k, v, g, beta, scale, init_states, cu_seqlens):
        o, final, saved = _delta_run(q, k, v, g, beta, scale, cu_seqlens, init_states, True, True, None)
        ctx.saved = saved
        saved.tensors["final"] = None
        ctx.set_materialize_grads(False)
        return o, final

    @staticmethod
    def backward(ctx, do, dfinal):
        s = ctx.saved
        q, d = s.tensors["q"], s.dims
        if do is None:
            do = torch.zeros(tuple(q.shape[:2]) + (d.nheads, d.headdim), dtype=q.dtype, device=q.device)
        r = delta_bwd(s, do.contiguous(), None if dfinal is None else dfinal.contiguous())
        return r["dq"], r["dk"], r["dv"], r["dg"].float(), r["dbeta"].float(), None, r.get("dinit"), None


def delta(q, k, v, g, beta, scale=None, init_states=None, cu_seqlens=None):
    """Differentiable gated delta rule: (o, final states); see delta_fwd."""
    return DeltaFunction.apply(q, k, v, g, beta, scale, init_states, cu_seqlens)
