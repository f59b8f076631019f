"""Refusals of the gated delta rule and of the query/key norm, through the C
ABI and the binding, without a GPU: every bad argument is answered on the host
before anything is launched (the pointers are fake and never touched)."""
import ctypes

import pytest
import torch

import deterministic_mamba2_ssd_gb300 as ssd

INVALID, WORKSPACE = 1, 3
FAKE = 1 << 20


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    return ssd.lib()


def _delta(L, d, fn="fwd", **over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, beta=FAKE, cu=0, init=0, scale=1.0, o=FAKE, fin=0, saved=FAKE,
             saved_bytes=1 << 60, ws=FAKE, ws_bytes=1 << 60, dout=FAKE, dfinal=0, dq=FAKE, dk=FAKE, dv=FAKE, dg=FAKE,
             dbeta=FAKE, dinit=0, states=FAKE, num_slots=1 << 20, slots=0)
    a.update(over)
    order = {"fwd": "q k v g beta cu init scale o fin saved saved_bytes ws ws_bytes",
             "bwd": "q k g beta cu scale saved saved_bytes dout dfinal dq dk dv dg dbeta dinit ws ws_bytes",
             "step": "q k v g beta scale states num_slots slots o"}[fn]
    return getattr(L, "mamba2_ssd_delta_" + fn)(ctypes.byref(d), *[a[n] for n in order.split()], None)


GOOD = dict(batch=2, seqlen=100, nheads=4, headdim=64, ngroups=2, dstate=128)


@pytest.mark.parametrize("bad", [dict(batch=0), dict(seqlen=-1), dict(nheads=0), dict(nheads=3), dict(headdim=0),
                                 dict(ngroups=0), dict(dstate=0), dict(dstate=257), dict(nseq=3), dict(nseq=0),
                                 dict(q_stride=-1), dict(q_stride=255), dict(v_stride=10), dict(k_stride=1 << 40),
                                 dict(batch=1 << 20, seqlen=1 << 12), dict(nheads=1 << 17, ngroups=1),
                                 dict(headdim=1 << 16)])
def test_delta_rejects_dims(L, bad):
    d = ssd.make_delta_dims(**{**GOOD, **bad})
    assert L.mamba2_ssd_delta_saved_size(ctypes.byref(d)) == 0
    assert L.mamba2_ssd_delta_fwd_workspace_size(ctypes.byref(d)) == 0
    assert L.mamba2_ssd_delta_bwd_workspace_size(ctypes.byref(d)) == 0
    assert ssd.delta_path_name(d) == "invalid"
    for fn in ("fwd", "bwd", "step"):
        assert _delta(L, d, fn) == INVALID


def test_delta_rejects_arguments(L):
    d = ssd.make_delta_dims(**GOOD)
    for name in ("q", "k", "v", "g", "beta", "o"):
        assert _delta(L, d, **{name: 0}) == INVALID
        assert _delta(L, d, **{name: FAKE + 1}) == INVALID
    assert _delta(L, d, scale=float("nan")) == INVALID
    assert _delta(L, d, cu=FAKE) == INVALID             # flag not set
    for name in ("init", "fin", "saved", "ws"):
        assert _delta(L, d, **{name: FAKE + 4}) == INVALID
    assert _delta(L, d, ws=0, saved=0) == INVALID
    need = L.mamba2_ssd_delta_saved_size(ctypes.byref(d))
    assert need > 0 and _delta(L, d, saved_bytes=need - 1) == WORKSPACE
    assert _delta(L, d, saved=0, ws_bytes=L.mamba2_ssd_delta_fwd_workspace_size(ctypes.byref(d)) - 1) == WORKSPACE
    for name in ("q", "k", "g", "beta", "dout", "dq", "dk", "dv", "dg", "dbeta", "saved"):
        assert _delta(L, d, "bwd", **{name: 0}) == INVALID
    assert _delta(L, d, "bwd", saved_bytes=need - 1) == WORKSPACE
    assert _delta(L, d, "bwd", ws_bytes=L.mamba2_ssd_delta_bwd_workspace_size(ctypes.byref(d)) - 1) == WORKSPACE
    for name in ("dfinal", "dinit"):
        assert _delta(L, d, "bwd", **{name: FAKE + 8}) == INVALID
    for name in ("q", "k", "v", "g", "beta", "o", "states"):
        assert _delta(L, d, "step", **{name: 0}) == INVALID
    assert _delta(L, d, "step", num_slots=0) == INVALID
    assert _delta(L, d, "step", num_slots=1) == INVALID   # rows without a slot table need a state each
    assert _delta(L, d, "step", slots=FAKE + 2) == INVALID
    packed = ssd.make_delta_dims(1, 100, 4, 64, 2, 128, nseq=3, cu_seqlens=True)
    assert _delta(L, packed, cu=0) == INVALID
    assert _delta(L, packed, "step", cu=FAKE) == INVALID
    two = ssd.make_delta_dims(2, 100, 4, 64, 2, 128, nseq=3, cu_seqlens=True)
    assert _delta(L, two, cu=FAKE) == INVALID
    d.dtype = 5
    assert _delta(L, d) == INVALID
    d.dtype, d.flags = 1, 2
    assert _delta(L, d) == INVALID


def _qk(L, d, fn="fwd", **over):
    a = dict(q=FAKE, k=FAKE, dyq=FAKE, dyk=FAKE, wq=0, wk=0, cos=FAKE, sin=FAKE, pos=FAKE, oq=FAKE, ok=FAKE, dwq=0,
             dwk=0, ws=FAKE, ws_bytes=1 << 40)
    a.update(over)
    order = "q k wq wk cos sin pos oq ok" if fn == "fwd" else \
        "q k dyq dyk wq wk cos sin pos oq ok dwq dwk ws ws_bytes"
    return getattr(L, "mamba2_ssd_qk_" + fn)(ctypes.byref(d), *[a[n] for n in order.split()], None)


QK = dict(tokens=10, qheads=4, kheads=2, headdim=128, rotary=64, positions=100)


@pytest.mark.parametrize("bad", [dict(tokens=-1), dict(qheads=0), dict(kheads=0), dict(headdim=0), dict(headdim=513),
                                 dict(rotary=63), dict(rotary=130), dict(rotary=-2), dict(positions=0),
                                 dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(q_stride=511),
                                 dict(k_stride=-5)])
def test_qk_rejects_dims(L, bad):
    d = ssd.make_qk_dims(**{**QK, **bad})
    assert _qk(L, d) == INVALID and _qk(L, d, "bwd") == INVALID
    assert L.mamba2_ssd_qk_bwd_workspace_size(ctypes.byref(d)) == 0


def test_qk_rejects_arguments(L):
    d = ssd.make_qk_dims(**QK)
    for name in ("q", "k", "cos", "sin", "pos", "oq", "ok"):
        assert _qk(L, d, **{name: 0}) == INVALID
        assert _qk(L, d, **{name: FAKE + 1}) == INVALID
    assert _qk(L, d, wq=FAKE) == INVALID
    for name in ("dyq", "dyk"):
        assert _qk(L, d, "bwd", **{name: 0}) == INVALID
    assert _qk(L, d, "bwd", dwq=FAKE, dwk=FAKE) == INVALID          # gradients of weights that are not there
    assert _qk(L, d, "bwd", wq=FAKE, wk=FAKE) == INVALID            # weights without their gradients
    need = L.mamba2_ssd_qk_bwd_workspace_size(ctypes.byref(d))
    w = dict(wq=FAKE, wk=FAKE, dwq=FAKE, dwk=FAKE)
    assert _qk(L, d, "bwd", ws_bytes=need - 1, **w) == WORKSPACE
    assert _qk(L, d, "bwd", ws=0, **w) == INVALID
    d.norm = 2
    assert _qk(L, d) == INVALID
    none = ssd.make_qk_dims(**{**QK, "tokens": 0})
    assert _qk(L, none) == 0                                        # no tokens: nothing is launched


def test_binding_rejects(L):
    """Wrong shapes, types and strides raise before the library is called."""
    z = torch.zeros
    q, v, g = z(1, 4, 2, 16), z(1, 4, 4, 8), z(1, 4, 4)
    for call in (
            lambda: ssd.delta_fwd(q.double(), q, v, g, g),
            lambda: ssd.delta_fwd(q[0], q, v, g, g),
            lambda: ssd.delta_fwd(q, q[:, :3], v, g, g),
            lambda: ssd.delta_fwd(q, q, z(1, 4, 3, 8), z(1, 4, 3), z(1, 4, 3)),
            lambda: ssd.delta_fwd(q, q, v, g.bfloat16(), g),
            lambda: ssd.delta_fwd(q, q, v.transpose(2, 3), g, g),
            lambda: ssd.delta_fwd(q, q, v, g, g, init_states=z(1, 4, 16, 8)),
            lambda: ssd.delta_fwd(q, q, v, g, g, cu_seqlens=torch.tensor([0, 4])),
            lambda: ssd.delta_fwd(q, q, v, g, g, cu_seqlens=torch.tensor([0], dtype=torch.int32)),
            lambda: ssd.delta_step(q, q, v, g, g, z(1, 4, 8, 15)),
            lambda: ssd.delta_step(q, q, v, g, g, z(0, 4, 8, 16)),
            lambda: ssd.qk_fwd(q, q, norm="max"),
            lambda: ssd.qk_fwd(q, q, wq=z(16)),
            lambda: ssd.qk_fwd(q, q[..., :8]),
            lambda: ssd.qk_fwd(q, q, cos=z(9, 4)),
            lambda: ssd.qk_fwd(q, q, positions=z(1, 4).int()),
            lambda: ssd.qk_fwd(q.expand(2, 4, 2, 16), q, norm="l2")):
        with pytest.raises(ValueError):
            call()
