"""The oracle of the gated delta rule and of the query/key norm with rotation,
pinned on the CPU: finite differences of its own forward, the chunked form,
closed forms and invariants."""
import numpy as np
import pytest
import torch

import oracle.delta as od
from deterministic_mamba2_ssd_gb300.inputs import make_delta_inputs


def _inputs(**kw):
    d = make_delta_inputs(dtype=torch.float64, **kw)
    return {k: (None if x is None else x.numpy().astype(np.float64) if k != "cu" else x.numpy()) for k, x in d.items()}


@pytest.mark.parametrize("kw", [
    dict(b=2, T=7, H=4, P=3, G=2, N=5, with_init=True, with_dfinal=True),
    dict(b=1, T=9, H=2, P=2, G=1, N=3, seq_lens=(4, 0, 1, 4), with_init=True, with_dfinal=True),
])
def test_gradients_by_differences(kw):
    d = _inputs(seed=5, **kw)
    scale = 0.7

    def loss(x):
        o, fin = od.fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], scale, x["init"], x["cu"])
        return (o * d["dout"]).sum() + (fin * d["dfinal"]).sum()

    r = od.bwd(d["q"], d["k"], d["v"], d["g"], d["beta"], scale, d["dout"], d["init"], d["cu"], d["dfinal"])
    rng = np.random.default_rng(0)
    for name in ("q", "k", "v", "g", "beta", "init"):
        grad = r["d" + name]
        for _ in range(12):
            at = tuple(rng.integers(0, n) for n in grad.shape)
            h = 1e-5
            up, dn = dict(d), dict(d)
            up[name], dn[name] = d[name].copy(), d[name].copy()
            up[name][at] += h
            dn[name][at] -= h
            diff = (loss(up) - loss(dn)) / (2 * h)
            # central differences: h^2 times a third derivative of order 1, and rounding 1e-16 / h
            assert abs(diff - grad[at]) < 1e-7 * max(1.0, np.abs(grad).max()), (name, at)


@pytest.mark.parametrize("chunk", [1, 2, 3, 8, 64])
def test_chunked_form_is_the_recurrence(chunk):
    d = _inputs(b=1, T=21, H=4, P=3, G=2, N=5, seed=1)
    o, _ = od.fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], 0.5)
    assert np.abs(od.chunked_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], 0.5, chunk) - o).max() < 1e-12


def test_closed_forms():
    d = _inputs(b=1, T=6, H=2, P=3, G=2, N=4, seed=2)
    # beta 0: nothing is written, so only the decayed initial state answers
    init = np.ones((1, 2, 3, 4))
    o, fin = od.fwd(d["q"], d["k"], d["v"], d["g"], 0 * d["beta"], 1.0, init)
    dec = np.exp(np.cumsum(d["g"][0], 0))
    assert np.allclose(o[0], dec[:, :, None] * np.einsum("thn,hpn->thp", d["q"][0], init[0]))
    # beta 1, unit key, no decay: the state answers the newest key with its value
    k = d["k"] / np.linalg.norm(d["k"], axis=-1, keepdims=True)
    o, _ = od.fwd(k, k, d["v"], 0 * d["g"], 1 + 0 * d["beta"], 1.0)
    assert np.allclose(o, d["v"])
    # g = -inf forgets everything before the token
    g = d["g"].copy()
    g[:, 3] = -np.inf
    o, _ = od.fwd(d["q"], d["k"], d["v"], g, d["beta"], 1.0, init)
    o2, _ = od.fwd(d["q"][:, 3:], d["k"][:, 3:], d["v"][:, 3:], d["g"][:, 3:], d["beta"][:, 3:], 1.0)
    assert np.allclose(o[:, 3:], o2)


@pytest.mark.parametrize("rms", [True, False])
@pytest.mark.parametrize("inter", [True, False])
def test_qk_gradients_by_differences(rms, inter):
    rng = np.random.default_rng(3)
    x, dz = rng.normal(size=(1, 3, 2, 10)), rng.normal(size=(1, 3, 2, 10))
    w, ang = rng.normal(size=10), rng.normal(size=(7, 3))
    pos = np.array([[5, 0, 2]])

    def z(x, w):
        return od.qk_fwd(x, w, np.cos(ang), np.sin(ang), pos, rms, 1e-3, inter)

    dx, dw = od.qk_bwd(x, dz, w, np.cos(ang), np.sin(ang), pos, rms, 1e-3, inter)
    for _ in range(20):
        at = tuple(rng.integers(0, n) for n in x.shape)
        e = np.zeros_like(x)
        e[at] = 1e-6
        assert abs(((z(x + e, w) - z(x - e, w)) * dz).sum() / 2e-6 - dx[at]) < 1e-7
        c = rng.integers(0, 10)
        f = np.zeros(10)
        f[c] = 1e-6
        assert abs(((z(x, w + f) - z(x, w - f)) * dz).sum() / 2e-6 - dw[c]) < 1e-7
    # turning keeps lengths: an l2-normed row without weights has length 1
    if not rms:
        y = od.qk_fwd(x, None, np.cos(ang), np.sin(ang), pos, rms, 0.0, inter)
        assert np.allclose((y * y).sum(-1), 1)
