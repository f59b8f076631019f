"""The query/key norm with rotation on the GPU against the fp64 oracle.
Tolerances: fp32 arithmetic throughout, so 1e-5 for fp32 outputs (weight
gradients too: sums of up to thousands of terms in fp32, 2^-24 sqrt(n) each),
and one rounding, 2^-9, on top for bf16 ones."""
import pytest
import torch

import deterministic_mamba2_ssd_gb300 as ssd
import oracle.delta as od
from _helpers import relerr

pytestmark = pytest.mark.gpu

TOL = {torch.float32: 1e-5, torch.bfloat16: 2.0 ** -9 + 1e-5}


def _inputs(b, T, hq, hk, D, R, dtype, weights, seed=0, sliced=False):
    gen = torch.Generator().manual_seed(seed)
    rows = torch.randn(b, T, (hq + hk) * D + 8, generator=gen).to(dtype)
    q, k = rows[..., :hq * D].unflatten(2, (hq, D)), rows[..., hq * D:(hq + hk) * D].unflatten(2, (hk, D))
    if not sliced:
        q, k = q.contiguous(), k.contiguous()
    d = dict(q=q, k=k, wq=None, wk=None, cos=None, sin=None, positions=None)
    if weights:
        d["wq"], d["wk"] = 1 + 0.2 * torch.randn(D, generator=gen), 1 + 0.2 * torch.randn(D, generator=gen)
    if R:
        ang = 3 * torch.randn(50, R // 2, generator=gen)
        d["cos"], d["sin"] = ang.cos(), ang.sin()
        d["positions"] = torch.randint(0, 50, (b, T), generator=gen, dtype=torch.int32)
    d["dyq"], d["dyk"] = (torch.randn(x.shape, generator=gen).to(dtype) for x in (q, k))
    return d


def _dev(d):
    rows = {}

    def move(x):   # keep slices slices: both views share one storage on the device too
        if x is None:
            return None
        base = x._base
        if base is None or base.numel() == x.numel():
            return x.cuda()
        if id(base) not in rows:
            rows[id(base)] = base.cuda()
        return rows[id(base)].as_strided(x.shape, x.stride(), x.storage_offset())
    return {n: move(x) for n, x in d.items()}


CASES = [
    (1, 1, 1, 1, 128, 128), (2, 65, 16, 8, 128, 64), (1, 300, 4, 4, 64, 64), (3, 33, 5, 3, 256, 32),
    (1, 100, 6, 2, 32, 0), (1, 77, 3, 1, 72, 36), (2, 20, 2, 2, 1, 0), (1, 50, 2, 3, 7, 6), (1, 40, 2, 1, 130, 130),
    (1, 9, 2, 2, 512, 100), (2, 31, 4, 2, 128, 24), (1, 5000, 2, 1, 128, 128),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("case", CASES, ids=[str(c) for c in CASES])
def test_qk_matches_oracle(case, inter, norm, dtype):
    b, T, hq, hk, D, R = case
    weights, sliced = (T + inter) % 2 == 0, norm == "rms"
    d = _inputs(b, T, hq, hk, D, R, dtype, weights, seed=D + R, sliced=sliced)
    g = _dev(d)
    how = dict(norm=norm, eps=1e-5, interleaved=inter)
    put = {n: g[n] for n in ("wq", "wk", "cos", "sin", "positions")}
    yq, yk = ssd.qk_fwd(g["q"], g["k"], **put, **how)
    r = ssd.qk_bwd(g["q"], g["k"], g["dyq"], g["dyk"], **put, **how)
    torch.cuda.synchronize()
    for n, y in (("q", yq), ("k", yk)):
        rest = (d["cos"], d["sin"], d["positions"], norm == "rms", 1e-5, inter)
        assert relerr(y, od.qk_fwd(d[n], d["w" + n], *rest)) < TOL[dtype]
        dx, dw = od.qk_bwd(d[n], d["dy" + n], d["w" + n], *rest)
        # dx is u minus its part along h: where they nearly cancel (one element a row) only the scale of u counts
        u = od.qk_bwd(d[n] * 0 + 1, d["dy" + n], d["w" + n], *rest)[0] if D == 1 else dx
        if D > 1:
            assert relerr(r["d" + n], dx) < TOL[dtype]
        else:
            assert abs(r["d" + n].double().cpu().numpy() - dx).max() < TOL[dtype] * 1e3 * max(1.0, abs(u).max())
        assert r["d" + n].dtype == dtype
        if weights:
            assert relerr(r["dw" + n], dw) < 1e-5
        else:
            assert "dw" + n not in r


def test_qk_wide_and_narrow_kernels_agree():
    """The same rows off a 16-byte boundary take the narrow kernel."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    flat = torch.randn(2, 50 * 4 * 128 + 1, generator=gen, device="cuda").to(torch.bfloat16)
    q, k = (flat[i, :-1].view(1, 50, 4, 128) for i in range(2))
    q1, k1 = (torch.empty_like(flat[i])[1:].view(1, 50, 4, 128) for i in range(2))
    q1.copy_(q), k1.copy_(k)
    assert q1.data_ptr() % 16 or k1.data_ptr() % 16
    a, b = ssd.qk_fwd(q.contiguous(), k.contiguous()), ssd.qk_fwd(q1, k1)
    for x, y in zip(a, b):
        assert relerr(x, y.double().cpu().numpy()) < 2.0 ** -8


def test_qk_zero_rows_and_bad_positions():
    d = _dev(_inputs(1, 8, 2, 2, 64, 64, torch.float32, True))
    d["q"][0, 3] = 0
    d["positions"][0, 5] = 50          # past the table
    d["positions"][0, 6] = -1
    put = {n: d[n] for n in ("wq", "wk", "cos", "sin", "positions")}
    yq, yk = ssd.qk_fwd(d["q"], d["k"], **put)
    assert (yq[0, 3] == 0).all()
    for y in (yq, yk):
        assert y[0, 5:7].isnan().all() and torch.isfinite(y[0, :5]).all() and torch.isfinite(y[0, 7]).all()


def test_qk_repeat_streams_autograd_and_no_tokens():
    d = _dev(_inputs(2, 700, 4, 2, 128, 64, torch.bfloat16, True))
    put = {n: d[n] for n in ("wq", "wk", "cos", "sin", "positions")}
    ref = ssd.qk_bwd(d["q"], d["k"], d["dyq"], d["dyk"], **put)
    for s in (None, None, torch.cuda.Stream()):
        torch.cuda.synchronize()
        r = ssd.qk_bwd(d["q"], d["k"], d["dyq"], d["dyk"], **put, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(ref[n], r[n]) for n in ref)
    leaves = {n: d[n].clone().requires_grad_(True) for n in ("q", "k", "wq", "wk")}
    y = ssd.qk_norm(leaves["q"], leaves["k"], leaves["wq"], leaves["wk"], d["cos"], d["sin"], d["positions"])
    torch.autograd.backward(y, [d["dyq"], d["dyk"]])
    assert all(torch.equal(leaves[n].grad, ref["d" + n]) for n in leaves)
    e = {n: d[n][:, :0].contiguous() for n in ("q", "k", "dyq", "dyk", "positions")}
    put["positions"] = e["positions"]
    yq, _ = ssd.qk_fwd(e["q"], e["k"], **put)
    r = ssd.qk_bwd(e["q"], e["k"], e["dyq"], e["dyk"], **put)
    assert yq.numel() == 0 and (r["dwq"] == 0).all() and (r["dwk"] == 0).all()
