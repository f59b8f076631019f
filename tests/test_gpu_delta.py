"""The gated delta rule on the GPU against the fp64 oracle.

Tolerances (relL2 per output, against the unrounded oracle on the values the
GPU saw):
* fp32 inputs 1e-5, the bar of the other fp32 paths of this library;
* bf16 inputs: an output rounded to bf16 is off by at most 2^-9 of each
  element, and the tensor-core kernels round operands to 11 bits (2^-12 each,
  a handful in sequence): 2^-9 + 1e-3 in all, 2.95e-3;
* fp32 states from bf16 inputs 1e-5: they are carried with operands of 22 bits
  where they are asked for; dinit, a gradient that leaves unrounded, 1e-3 (the
  operands' rounding alone);
* dg is a sum of P x N terms of both signs: besides its own relative bar, a
  thousandth of that bar times the sum of the terms' magnitudes.
"""
import numpy as np
import pytest
import torch

import deterministic_mamba2_ssd_gb300 as ssd
import oracle.delta as od
from _helpers import relerr
from deterministic_mamba2_ssd_gb300.inputs import make_delta_inputs

pytestmark = pytest.mark.gpu

TOL = {torch.float32: 1e-5, torch.bfloat16: 2.0 ** -9 + 1e-3}
STATE_TOL = 1e-5
NAMES = ("q", "k", "v", "g", "beta")


def _dev(d):
    return {k: (None if x is None else x.cuda()) for k, x in d.items()}


def _off(got, want, tol, extra=0.0):
    got = got.detach().cpu().double().numpy()
    err, norm = np.linalg.norm(got - want), np.linalg.norm(want)
    assert np.isfinite(got).all()
    return err / max(tol * norm + extra, 1e-30)


def _check(d, scale=None, wide=False):
    """Forward and backward against the oracle; the worst error as a share of its bar."""
    g = _dev(d)
    dt = d["q"].dtype
    sc = d["q"].shape[-1] ** -0.5 if scale is None else scale
    if wide:   # q, k, v as slices of one projection's rows
        rows = torch.cat([g[n].flatten(2) for n in "qkv"], 2)
        at, parts = 0, {}
        for n in "qkv":
            w = g[n].shape[2] * g[n].shape[3]
            parts[n] = rows[:, :, at:at + w].unflatten(2, tuple(g[n].shape[2:]))
            at += w
        g.update(parts)
    o, saved = ssd.delta_fwd(*(g[n] for n in NAMES), scale=scale, init_states=g["init"], cu_seqlens=g["cu"],
                             want_final=True)
    r = ssd.delta_bwd(saved, g["dout"], dfinal=g["dfinal"], want_dinit=True)
    torch.cuda.synchronize()
    ref = od.bwd(*(d[n] for n in NAMES), sc, d["dout"], d["init"], d["cu"], d["dfinal"])
    tol = TOL[dt]
    share = {"o": _off(o, ref["o"], tol), "final": _off(saved.final, ref["final"], STATE_TOL),
             "dinit": _off(r["dinit"], ref["dinit"], STATE_TOL if dt == torch.float32 else 1e-3)}
    for n in ("dq", "dk", "dv", "dbeta"):
        share[n] = _off(r[n], ref[n], tol)
        assert r[n].dtype == dt
    share["dg"] = _off(r["dg"], ref["dg"], tol, 1e-3 * tol * np.linalg.norm(ref["dg_abs"]))
    bad = {k: v for k, v in share.items() if not v < 1}
    assert not bad, (bad, share)
    return share


CASES = [
    dict(b=1, T=1, H=2, P=16, G=1, N=64),
    dict(b=2, T=63, H=4, P=32, G=2, N=64),
    dict(b=1, T=64, H=2, P=64, G=2, N=128),
    dict(b=2, T=65, H=6, P=64, G=2, N=128, with_init=True, with_dfinal=True),
    dict(b=1, T=300, H=4, P=128, G=4, N=128, with_init=True),
    dict(b=3, T=129, H=3, P=48, G=1, N=64, with_dfinal=True),
    dict(b=1, T=200, H=4, P=192, G=2, N=128),
    dict(b=1, T=130, H=2, P=40, G=1, N=72, with_init=True, with_dfinal=True),    # no tile's sizes
    dict(b=2, T=70, H=3, P=7, G=3, N=5, with_init=True),
    dict(b=1, T=67, H=2, P=1, G=1, N=1),
    dict(b=1, T=90, H=1, P=20, G=1, N=256),
    dict(b=1, T=333, H=4, P=64, G=2, N=128, seq_lens=(64, 1, 0, 128, 77, 63), with_init=True, with_dfinal=True),
    dict(b=1, T=140, H=2, P=24, G=1, N=40, seq_lens=(0, 65, 0, 75), with_init=True, with_dfinal=True),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_delta_matches_oracle(case, dtype):
    d = make_delta_inputs(dtype=dtype, seed=case["T"], **case)
    print(ssd.delta_path_name(ssd.make_delta_dims(case["b"], case["T"], case["H"], case["P"], case["G"], case["N"],
                                                  dtype=dtype)), {k: "%.2f" % v for k, v in _check(d).items()})


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("P,N", [(64, 128), (9, 33)])
def test_delta_strided_rows_and_scale(dtype, P, N):
    d = make_delta_inputs(2, 100, 4, P, 2, N, dtype=dtype, seed=3, with_init=True)
    _check(d, scale=0.25, wide=True)
    _check(d, scale=-1.5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N", [128, 24])
def test_delta_extreme_gates(dtype, N):
    """Full forgetting (g = -inf and the type's lowest value), no decay, no and full writing, a zero key."""
    d = make_delta_inputs(1, 150, 4, 32, 2, N, dtype=dtype, seed=8, with_init=True, with_dfinal=True)
    d["g"][0, 20, 0] = -np.inf
    d["g"][0, 70:73, 1] = torch.finfo(torch.float32).min
    d["g"][0, :, 2] = 0
    d["beta"][0, 30:90, 0] = 0
    d["beta"][0, :, 3] = 1
    d["k"][0, 10] = 0
    d["k"][0, 100] = d["k"][0, 99]     # the same key twice
    share = _check(d)
    print({k: "%.2f" % v for k, v in share.items()})


@pytest.mark.parametrize("vscale,dscale", [(1e5, 1e-6), (1e-6, 1e5), (1e10, 1e-12)])
def test_delta_magnitudes(vscale, dscale):
    """Values and output gradients far from 1 (a loss scale, a badly scaled layer)."""
    d = make_delta_inputs(1, 200, 4, 64, 2, 128, dtype=torch.bfloat16, seed=9, with_init=True)
    d["v"], d["init"], d["dout"] = d["v"] * vscale, d["init"] * vscale, d["dout"] * dscale
    _check(d)


def test_delta_correlated_keys():
    """Keys that hardly differ: the triangular system is far from the identity."""
    d = make_delta_inputs(1, 260, 4, 64, 2, 128, dtype=torch.bfloat16, seed=10)
    base = torch.randn(1, 1, 2, 128, generator=torch.Generator().manual_seed(1))
    k = base + 0.3 * d["k"].float() * 128 ** 0.5
    d["k"] = (k / k.norm(dim=-1, keepdim=True)).to(torch.bfloat16)
    d["g"] = d["g"] * 0.01
    _check(d)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_delta_gradient_by_differences(dtype):
    """The backward against central differences of the GPU's own forward, along random directions."""
    d = _dev(make_delta_inputs(1, 80, 2, 32, 1, 64, dtype=dtype, seed=11, with_init=True))
    o, saved = ssd.delta_fwd(*(d[n] for n in NAMES), init_states=d["init"])
    r = ssd.delta_bwd(saved, d["dout"])
    gen = torch.Generator(device="cuda").manual_seed(2)

    def loss(x):
        out, _ = ssd.delta_fwd(*(x[n] for n in NAMES), init_states=x["init"])
        return (out.double() * d["dout"].double()).sum()

    for n in ("v", "g", "beta", "init"):
        h = 2.0 ** -4 if n in ("v", "init") else 2.0 ** -6
        move = torch.randn(d[n].shape, generator=gen, device="cuda")
        up, dn = dict(d), dict(d)
        up[n], dn[n] = (d[n].float() + h * move).to(d[n].dtype), (d[n].float() - h * move).to(d[n].dtype)
        step = (up[n].double() - dn[n].double())
        diff = (loss(up) - loss(dn)).item()
        want = (r["d" + n].double() * step).sum().item()
        # the loss is linear in v and init; in g and beta the h^2 term is about h^2 of the value.  Rounding: each o
        # carries 2^-9 (bf16) or 2^-22 of itself, summed over independent elements
        size = (o.double() * d["dout"].double()).square().sum().sqrt().item()
        bar = (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -20) * 2 * size + 3 * TOL[dtype] * abs(want) + \
            (0.02 * (r["d" + n].double() * step).square().sum().sqrt().item() if n in ("g", "beta") else 0.0)
        assert abs(diff - want) < 3 * bar, (n, diff, want, bar)


def test_delta_empty_row_and_length_zero():
    d = _dev(make_delta_inputs(2, 0, 2, 16, 1, 64, with_init=True))
    o, fin = ssd.delta_prefill(*(d[n] for n in NAMES), init_states=d["init"])
    assert o.numel() == 0 and torch.equal(fin, d["init"])
    o, saved = ssd.delta_fwd(*(d[n] for n in NAMES), init_states=d["init"], want_final=True)
    dfin = torch.randn_like(fin)
    r = ssd.delta_bwd(saved, d["dout"], dfinal=dfin)
    assert torch.equal(r["dinit"], dfin) and r["dq"].numel() == 0


@pytest.mark.parametrize("dtype,P,N", [(torch.bfloat16, 64, 128), (torch.float32, 24, 40)])
def test_delta_bitwise_repeat_and_streams(dtype, P, N):
    """The same bits on every run, on another stream, and with sequences packed or as rows."""
    d = _dev(make_delta_inputs(3, 190, 4, P, 2, N, dtype=dtype, seed=4, with_init=True, with_dfinal=True))

    def go(stream=None, packed=False):
        x = dict(d)
        if packed:
            x.update({n: d[n].flatten(0, 1)[None] for n in NAMES + ("dout",)})
            x["cu"] = torch.tensor([0, 190, 380, 570], dtype=torch.int32, device="cuda")
        o, saved = ssd.delta_fwd(*(x[n] for n in NAMES), init_states=x["init"], cu_seqlens=x["cu"], want_final=True,
                                 stream=stream)
        r = ssd.delta_bwd(saved, x["dout"], dfinal=x["dfinal"], stream=stream)
        torch.cuda.synchronize()
        return [o.flatten(), saved.final.flatten()] + [r[n].flatten() for n in sorted(r)]

    ref = go()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(ref, go()))
    assert all(torch.equal(a, b) for a, b in zip(ref, go(stream=torch.cuda.Stream())))
    assert all(torch.equal(a, b) for a, b in zip(ref, go(packed=True)))


@pytest.mark.parametrize("dtype,P,N,tokens", [(torch.bfloat16, 128, 128, 1), (torch.bfloat16, 64, 128, 4),
                                              (torch.float32, 10, 7, 3), (torch.float32, 33, 200, 1),
                                              (torch.bfloat16, 64, 64, 17)])
def test_delta_step(dtype, P, N, tokens):
    """In place on a pool, rows out of order, idle rows between them, untouched states left as they are."""
    d = make_delta_inputs(6, tokens, 4, P, 2, N, dtype=dtype, seed=tokens)
    slots = torch.tensor([7, -1, 0, 3, 9, 2], dtype=torch.int32)   # -1 and 9 are idle
    pool = torch.randn(9, 4, P, N, generator=torch.Generator().manual_seed(1))
    live = [0, 2, 3, 5]
    g = _dev(d)
    states = pool.cuda()
    o = ssd.delta_step(*(g[n] for n in NAMES), states, slots=slots.cuda())
    torch.cuda.synchronize()
    init = pool[slots[live].long()]
    want_o, want_s = od.fwd(*(d[n][live] for n in NAMES), N ** -0.5, init)
    # fp32 arithmetic on every path of this form
    tol = 1e-5 if dtype == torch.float32 else 2.0 ** -9 + 1e-5
    assert relerr(o[live], want_o) < tol
    assert relerr(states.cpu()[slots[live].long()], want_s) < 1e-5
    assert (o[[1, 4]] == 0).all()
    rest = [i for i in range(9) if i not in slots[live].tolist()]
    assert torch.equal(states.cpu()[rest], pool[rest])


def test_delta_step_continues_a_prefill():
    d = _dev(make_delta_inputs(2, 133, 4, 64, 2, 128, seed=6))
    o, fin = ssd.delta_prefill(*(d[n] for n in NAMES))
    part = {n: d[n][:, :130].contiguous() for n in NAMES}
    _, states = ssd.delta_prefill(*(part[n] for n in NAMES))
    for t in range(130, 133):
        ot = ssd.delta_step(*(d[n][:, t:t + 1].contiguous() for n in NAMES), states)
        assert relerr(ot, o[:, t:t + 1].double().cpu().numpy()) < 2 * TOL[torch.bfloat16]
    assert relerr(states, fin.double().cpu().numpy()) < 2 * STATE_TOL


def test_delta_autograd():
    d = _dev(make_delta_inputs(1, 100, 4, 64, 2, 128, seed=7, with_init=True, with_dfinal=True))
    leaves = {n: d[n].clone().requires_grad_(True) for n in NAMES + ("init",)}
    o, fin = ssd.delta(*(leaves[n] for n in NAMES), init_states=leaves["init"])
    torch.autograd.backward([o, fin], [d["dout"], d["dfinal"]])
    _, saved = ssd.delta_fwd(*(d[n] for n in NAMES), init_states=d["init"], want_final=True)
    r = ssd.delta_bwd(saved, d["dout"], dfinal=d["dfinal"])
    for n in leaves:
        assert torch.equal(leaves[n].grad, r["d" + n].to(leaves[n].dtype)), n


def test_delta_nan_and_inf_reach_only_their_own():
    """A NaN value stays in its head, row and later tokens; other heads and rows are as without it."""
    d = _dev(make_delta_inputs(1, 100, 4, 64, 2, 128, seed=12))
    ref, _ = ssd.delta_prefill(*(d[n] for n in NAMES))
    for bad in (float("nan"), float("inf")):
        v = d["v"].clone()
        v[0, 50, 1, 3] = bad
        o, _ = ssd.delta_prefill(d["q"], d["k"], v, d["g"], d["beta"])
        assert not torch.isfinite(o[0, 50, 1, 3])
        keep = torch.ones_like(o, dtype=torch.bool)
        keep[0, 50:, 1, 3] = False
        chunk = torch.zeros_like(keep)
        chunk[0, :, 1, 3] = True      # earlier tokens of that row may share the chunk's products
        assert torch.equal(o[keep & ~chunk], ref[keep & ~chunk])
