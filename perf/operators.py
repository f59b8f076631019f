"""Cases of the gated delta rule and of the query/key norm with rotation.

Three operators are measured here, each on inputs of the kind its path meets:

* ``qk``    -- norm of queries and keys for each head, with the position
  rotation in the same pass; forward, or forward and backward;
* ``delta`` -- the gated delta rule over whole sequences; forward with the
  final state (prefill), or forward and backward (a training step);
* ``step``  -- the gated delta rule's recurrent form for single tokens (or a
  few drafted ones), updating a pool of states in place.

With S a (headdim, dstate) state per head, and per token a log decay g <= 0,
a step size beta, key k, query q and value v:

    S <- exp(g) S;  e = v - S k;  S <- S + beta e k^T;  o = scale S q
"""
import math

import numpy as np
import torch

own = False

CHUNK = 64
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---- cases -----------------------------------------------------------------

def listed():
    return [
        # one token of each of 32 running sequences: the norm before a decode step, a few microseconds
        dict(name="qk_decode", op="qk", grad=False, dtype="bf16", tokens=32, qheads=16, kheads=16, dim=128, rotary=128,
             norm="l2", weights=False, interleaved=False),
        # odd head size, partial and interleaved rotation, fp32, ragged token count
        dict(name="qk_odd_fp32", op="qk", grad=True, dtype="fp32", tokens=1111, qheads=6, kheads=3, dim=72, rotary=36,
             norm="rms", weights=True, interleaved=True),
        # a training step at the sequence length of the packed batch, weights with their gradient
        dict(name="qk_train_32k", op="qk", grad=True, dtype="bf16", tokens=32768, qheads=32, kheads=16, dim=128,
             rotary=64, norm="rms", weights=True, interleaved=False),
        # one sequence answering: latency alone counts
        dict(name="step_one", op="step", dtype="bf16", seqs=1, tokens=1, heads=32, groups=16, headdim=128, dstate=128),
        # a serving batch with idle slots between the running ones
        dict(name="step_serve", op="step", dtype="bf16", seqs=192, tokens=1, heads=32, groups=16, headdim=128,
             dstate=128),
        # four drafted tokens a sequence, the smaller head of this library's own models
        dict(name="step_draft", op="step", dtype="bf16", seqs=48, tokens=4, heads=64, groups=8, headdim=64, dstate=128),
        # a short prompt of odd length, one sequence
        dict(name="prefill_short", op="delta", grad=False, dtype="bf16", batch=1, seqlen=333, packed=False, heads=32,
             groups=16, headdim=128, dstate=128),
        # prompts of many lengths packed into one row, one of a single token
        dict(name="prefill_packed", op="delta", grad=False, dtype="bf16", batch=9, seqlen=1821, packed=True, heads=32,
             groups=16, headdim=128, dstate=128),
        # one long prompt
        dict(name="prefill_16k", op="delta", grad=False, dtype="bf16", batch=1, seqlen=16384, packed=False, heads=32,
             groups=16, headdim=128, dstate=128),
        # training on rows of the shorter benchmark length
        dict(name="train_2k", op="delta", grad=True, dtype="bf16", batch=4, seqlen=2048, packed=False, heads=32,
             groups=16, headdim=128, dstate=128),
        # training on one long row, this library's own head sizes and many heads on a group
        dict(name="train_16k", op="delta", grad=True, dtype="bf16", batch=1, seqlen=16384, packed=False, heads=64,
             groups=8, headdim=64, dstate=128),
        # fp32 all through, head sizes that fill no tile
        dict(name="train_odd_fp32", op="delta", grad=True, dtype="fp32", batch=2, seqlen=517, packed=False, heads=6,
             groups=2, headdim=40, dstate=72),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk", "step", "delta", "delta"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "qk":
        dim = rng.choice([64, 128, 128, 2 * rng.randint(8, 128)])
        kheads = rng.choice([1, 2, 3, 4, 8, 16])
        qheads = kheads * rng.choice([1, 1, 2])
        return dict(op="qk", grad=rng.random() < 0.6, dtype=dtype, tokens=_log(rng, 1, 20000), qheads=qheads,
                    kheads=kheads, dim=dim, rotary=2 * rng.randint(0, dim // 2), norm=rng.choice(["l2", "rms"]),
                    weights=rng.random() < 0.5, interleaved=rng.random() < 0.5)
    # bf16 and the sizes of whole tiles are the ordinary case; the rest are any sizes
    if rng.random() < 0.65:
        headdim, dstate = rng.choice([64, 128, 64, 128, 32, 48, 96, 192]), rng.choice([64, 128, 128])
    else:
        headdim, dstate = rng.randint(1, 136), rng.randint(1, 136)
    groups = rng.choice([1, 2, 4, 8, 16])
    heads = groups * rng.choice([1, 1, 2, 3, 4])
    if op == "step":
        return dict(op="step", dtype=dtype, seqs=_log(rng, 1, 128), tokens=rng.choice([1, 1, 1, 2, 3, 5, 8]),
                    heads=min(heads, 32) // groups * groups or groups, groups=groups, headdim=headdim, dstate=dstate)
    grad = rng.random() < 0.6
    top = 12000 if dtype == "bf16" and heads <= 16 else 3000
    total = _log(rng, 1, top)
    batch = min(total, rng.choice([1, 1, 2, 3, 5, 8]))
    return dict(op="delta", grad=grad, dtype=dtype, batch=batch, seqlen=max(1, total // batch),
                packed=rng.random() < 0.4, heads=heads, groups=groups, headdim=headdim, dstate=dstate)


# ---- inputs ----------------------------------------------------------------

def _gen(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed))
    return g


def _lengths(case):
    """Token counts of the sequences: equal rows, or a packed row of unequal ones (the last of one token)."""
    b, t = case["batch"], case["seqlen"]
    if not case["packed"] or b * t < 2 * b:
        return [t] * b
    total = b * t
    w = [(3 * i + 2) % 7 + 0.37 for i in range(b)]
    lens = [max(1, int(total * x / sum(w))) for x in w]
    if b > 1:
        lens[-1] = 1
    lens[0] += total - sum(lens)
    return lens


def _rates(shape, heads, gen, dev):
    """Log decays and step sizes as a layer makes them: g = A softplus(.), A = -exp(U(log 1, log 16)), beta a sigmoid."""
    A = -torch.exp(torch.rand(heads, generator=gen, device=dev) * math.log(16.0))
    g = A * torch.nn.functional.softplus(torch.randn(shape, generator=gen, device=dev) - 4.0)
    return g, torch.sigmoid(torch.randn(shape, generator=gen, device=dev))


def _keys(shape, gen, dev, dt):
    x = torch.randn(shape, generator=gen, device=dev)
    return (x / x.square().sum(-1, keepdim=True).add(1e-6).sqrt()).to(dt)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen, dt = _gen(seed, dev), TYPES[case["dtype"]]
    s = dict(case=case)
    if case["op"] == "qk":
        n, hq, hk, d, r = (case[k] for k in ("tokens", "qheads", "kheads", "dim", "rotary"))
        # queries and keys lie side by side in the rows of one projection, values after them
        pad = 8 * ((d + 7) // 8)
        rows = torch.randn((n, (hq + hk) * d + pad), generator=gen, device=dev).to(dt)
        s["q"] = rows[:, :hq * d].unflatten(1, (hq, d)).unsqueeze(0)
        s["k"] = rows[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d)).unsqueeze(0)
        s["wq"] = s["wk"] = None
        if case["weights"]:
            s["wq"] = 1 + 0.1 * torch.randn(d, generator=gen, device=dev)
            s["wk"] = 1 + 0.1 * torch.randn(d, generator=gen, device=dev)
        s["cos"] = s["sin"] = s["pos"] = None
        if r:
            top = 32768
            ang = torch.arange(top, device=dev, dtype=torch.float64)[:, None] * \
                10000.0 ** (-torch.arange(0, r, 2, device=dev, dtype=torch.float64) / r)
            s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
            s["pos"] = torch.randint(0, top, (1, n), generator=gen, device=dev, dtype=torch.int32) if n < 256 else \
                torch.arange(n, device=dev, dtype=torch.int32)[None]
        if case["grad"]:
            s["dyq"] = torch.randn((1, n, hq, d), generator=gen, device=dev).to(dt)
            s["dyk"] = torch.randn((1, n, hk, d), generator=gen, device=dev).to(dt)
        return s
    H, G, P, N = (case[k] for k in ("heads", "groups", "headdim", "dstate"))
    s["scale"] = N ** -0.5
    if case["op"] == "step":
        b, t = case["seqs"], case["tokens"]
        slots = b + b // 4 + 1   # the pool has idle states too
        s["states"] = torch.randn((slots, H, P, N), generator=gen, device=dev) * 0.1
        s["slots"] = torch.randperm(slots, generator=gen, device=dev)[:b].to(torch.int32)
    else:
        lens = _lengths(case)
        s["lens"] = lens
        b, t = (1, sum(lens)) if case["packed"] else (case["batch"], case["seqlen"])
        s["cu"] = None
        if case["packed"]:
            s["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=dev)
    s["q"], s["k"] = _keys((b, t, G, N), gen, dev, dt), _keys((b, t, G, N), gen, dev, dt)
    # values are the tail of the projection's rows, whose head the norm has read
    wide = torch.randn((b, t, 8 * G + H * P), generator=gen, device=dev).to(dt)
    s["v"] = wide[..., 8 * G:].unflatten(2, (H, P))
    s["g"], s["beta"] = _rates((b, t, H), H, gen, dev)
    if case.get("grad"):
        s["do"] = torch.randn((b, t, H, P), generator=gen, device=dev).to(dt)
    return s


# ---- the calls -------------------------------------------------------------

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import deterministic_mamba2_ssd_gb300 as ssd
    c = s["case"]
    if c["op"] == "qk":
        kw = dict(wq=s["wq"], wk=s["wk"], cos=s["cos"], sin=s["sin"], positions=s["pos"], norm=c["norm"], eps=1e-6,
                  interleaved=c["interleaved"])
        yq, yk = ssd.qk_fwd(s["q"], s["k"], **kw)
        out = dict(yq=yq, yk=yk)
        if c["grad"]:
            out.update(ssd.qk_bwd(s["q"], s["k"], s["dyq"], s["dyk"], **kw))
        return out
    if c["op"] == "step":
        o = ssd.delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["states"], slots=s["slots"], scale=s["scale"])
        return dict(o=o, states=s["states"])
    if not c["grad"]:
        o, final = ssd.delta_prefill(s["q"], s["k"], s["v"], s["g"], s["beta"], scale=s["scale"], cu_seqlens=s["cu"])
        return dict(o=o, final=final)
    o, saved = ssd.delta_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], scale=s["scale"], cu_seqlens=s["cu"])
    return dict(o=o, **ssd.delta_bwd(saved, s["do"]))


# ---- plain forms -----------------------------------------------------------

def _run_plain(s):
    c = s["case"]
    if c["op"] == "qk":
        return _plain_qk(s)
    if c["op"] == "step":
        return _plain_step(s)
    return _plain_delta(s)


def _rotate(y, cs, sn, inter):
    """The first 2 * cs.shape[-1] elements of y turned by the angles of (cos, sin)."""
    r = 2 * cs.shape[-1]
    x, rest = y[..., :r], y[..., r:]
    a, b = (x[..., 0::2], x[..., 1::2]) if inter else (x[..., :r // 2], x[..., r // 2:])
    u, v = a * cs - b * sn, a * sn + b * cs
    z = torch.stack([u, v], -1).flatten(-2) if inter else torch.cat([u, v], -1)
    return torch.cat([z, rest], -1)


def _plain_qk(s):
    c, out = s["case"], {}
    cs = sn = None
    if s["cos"] is not None:
        cs, sn = s["cos"][s["pos"].long()][:, :, None], s["sin"][s["pos"].long()][:, :, None]
    over = c["dim"] if c["norm"] == "rms" else 1
    for n in "qk":
        x, w = s[n].float(), s["w" + n]
        r = torch.rsqrt(x.square().sum(-1, keepdim=True) / over + 1e-6)
        xh = x * r
        y = xh if w is None else xh * w
        out["y" + n] = (y if cs is None else _rotate(y, cs, sn, c["interleaved"])).to(s[n].dtype)
        if c["grad"]:
            dy = s["dy" + n].float()
            dy = dy if cs is None else _rotate(dy, cs, -sn, c["interleaved"])
            if w is not None:
                out["dw" + n] = (dy * xh).sum((0, 1, 2))
                dy = dy * w
            out["d" + n] = (r * (dy - xh * ((dy * xh).sum(-1, keepdim=True) / over))).to(s[n].dtype)
    return out


def _plain_step(s):
    c, at = s["case"], s["slots"].long()
    H, rep = c["heads"], c["heads"] // c["groups"]
    q, k = (s[n].float().repeat_interleave(rep, 2) for n in "qk")
    v, dec = s["v"].float(), s["g"].exp()
    S, o = s["states"][at], []
    for t in range(c["tokens"]):
        S = S * dec[:, t, :, None, None]
        e = v[:, t] - (S * k[:, t, :, None, :]).sum(-1)
        S = S + (s["beta"][:, t, :, None] * e)[..., None] * k[:, t, :, None, :]
        o.append(s["scale"] * (S * q[:, t, :, None, :]).sum(-1))
    s["states"][at] = S
    return dict(o=torch.stack(o, 1).to(s["v"].dtype), states=s["states"])


def _rows(s, names):
    """The named tensors as fp32 (sequence, token, ...), each sequence padded with zeros to whole chunks, and the way back."""
    lens, dev = s["lens"], s["v"].device
    top = CHUNK * ((max(lens) + CHUNK - 1) // CHUNK)
    at = torch.arange(top, device=dev)[None] < torch.tensor(lens, device=dev)[:, None]
    out = {}
    for n in names:
        x = s[n].float().flatten(0, 1)
        y = torch.zeros((len(lens), top) + x.shape[1:], device=dev)
        y[at] = x
        out[n] = y

    def back(y, like):
        return y[at].reshape(like.shape[:2] + y.shape[2:])
    return out, back


def _chunks(x):
    """(B, T, H, d) as (B, H, chunk, token, d)."""
    b, t = x.shape[:2]
    return x.reshape(b, t // CHUNK, CHUNK, *x.shape[2:]).movedim(3, 1)


def _tokens(x):
    """(B, H, chunk, token, d) as (B, T, H, d)."""
    return x.movedim(1, 3).flatten(1, 2)


def _plain_delta(s):
    """Chunks of 64 tokens: inside a chunk the rule is a unit triangular system, between chunks a recurrence on S."""
    c, dt = s["case"], s["v"].dtype
    rep, scale = c["heads"] // c["groups"], s["scale"]
    x, back = _rows(s, ["q", "k", "v", "g", "beta"] + (["do"] if c["grad"] else []))
    q, k = (_chunks(x[n].repeat_interleave(rep, 2)) for n in "qk")
    v, G = _chunks(x["v"]), _chunks(x["g"][..., None]).cumsum(3)
    beta = _chunks(x["beta"][..., None])
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=v.device).tril()
    dec = torch.exp((G - G.mT).masked_fill(~low, -math.inf))        # exp(G_t - G_s), s <= t
    kk = (k @ k.mT) * dec * low.tril(-1)
    att = (q @ k.mT) * dec
    # (I + L diag(beta))^-1 of a nilpotent L: the product of I + (-L diag(beta))^(2^i)
    pw = -kk * beta.mT
    inv = pw + torch.eye(CHUNK, device=v.device)
    for _ in range(5):
        pw = pw @ pw
        inv = inv + pw @ inv
    del pw
    eG, last = G.exp(), G[..., -1:, :]
    tail = torch.exp(last - G)
    B, H, nc = v.shape[:3]
    S = torch.zeros((B, H, v.shape[-1], k.shape[-1]), device=v.device)
    Ss, es = [], []
    for i in range(nc):
        Ss.append(S)
        es.append(inv[:, :, i] @ (v[:, :, i] - eG[:, :, i] * (k[:, :, i] @ S.mT)))
        S = last[:, :, i].exp() * S + (tail[:, :, i] * beta[:, :, i] * es[-1]).mT @ k[:, :, i]
    e, Sc = torch.stack(es, 2), torch.stack(Ss, 2)
    o = scale * (eG * (q @ Sc.mT) + att @ (beta * e))
    res = dict(o=back(_tokens(o), s["v"]).to(dt))
    if not c["grad"]:
        return dict(res, final=S)
    do = _chunks(x["do"])
    attdo = scale * (att.mT @ do)
    dS = torch.zeros_like(S)
    dSs, dus, drs = [None] * nc, [None] * nc, [None] * nc
    for i in range(nc - 1, -1, -1):
        dSs[i] = dS
        dus[i] = attdo[:, :, i] + tail[:, :, i] * (k[:, :, i] @ dS.mT)
        drs[i] = inv[:, :, i].mT @ (beta[:, :, i] * dus[i])
        dS = last[:, :, i].exp() * dS + (scale * eG[:, :, i] * do[:, :, i]).mT @ q[:, :, i] \
            - (eG[:, :, i] * drs[i]).mT @ k[:, :, i]
    du, dr, dSc = torch.stack(dus, 2), torch.stack(drs, 2), torch.stack(dSs, 2)
    n1, n2 = dr @ e.mT, scale * (do @ e.mT)
    m1, m2 = -n1 * dec * low.tril(-1) * beta.mT, n2 * dec * beta.mT
    dbeta = (du * e).sum(-1, keepdim=True) - (n1 * kk).sum(-2)[..., None]
    dq = scale * eG * (do @ Sc) + m2 @ k
    up = m1 @ k - eG * (dr @ Sc)
    state = tail * beta * (e @ dSc)
    down = m1.mT @ k + m2.mT @ q + state
    dG = ((q * dq).sum(-1) + (k * up).sum(-1) - (k * down).sum(-1))
    dG[..., -1] += last[..., 0, 0].exp() * (Sc * dSc).sum((-1, -2)) + (k * state).sum((-1, -2))
    dg = dG.flip(-1).cumsum(-1).flip(-1)[..., None]

    def shared(y):
        return back(_tokens(y).unflatten(2, (c["groups"], rep)).sum(3), s["q"]).to(dt)
    return dict(res, dq=shared(dq), dk=shared(up + down), dv=back(_tokens(dr), s["v"]).to(dt),
                dg=back(_tokens(dg)[..., 0], s["g"]).to(dt), dbeta=back(_tokens(dbeta)[..., 0], s["g"]).to(dt))


# ---- the definition in 64 bits ----------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "qk":
        return _exact_qk(s)
    if case["op"] == "step":
        return _exact_step(s)
    return _exact_delta(s)


def _exact_qk(s):
    """One 2 x 2 turn at a time; the gradients by the quotient rule of x / sqrt(m(x))."""
    c, out = s["case"], {}
    d, r = c["dim"], c["rotary"]
    over = d if c["norm"] == "rms" else 1
    first = list(range(0, r, 2)) if c["interleaved"] else list(range(r // 2))
    second = list(range(1, r, 2)) if c["interleaved"] else list(range(r // 2, r))
    cs = sn = None
    if r:
        cs = s["cos"].double()[s["pos"][0].long()][:, None]
        sn = s["sin"].double()[s["pos"][0].long()][:, None]
    for n in "qk":
        x = s[n][0].double()
        w = torch.ones(d, dtype=torch.float64, device=x.device) if s["w" + n] is None else s["w" + n].double()
        root = ((x * x).sum(-1) / over + 1e-6).sqrt()[..., None]
        y = x * w / root
        if r:
            t = y.clone()
            t[..., first] = y[..., first] * cs - y[..., second] * sn
            t[..., second] = y[..., first] * sn + y[..., second] * cs
            y = t
        out["y" + n] = y[None]
        if c["grad"]:
            g = s["dy" + n][0].double()
            if r:
                t = g.clone()
                t[..., first] = g[..., first] * cs + g[..., second] * sn
                t[..., second] = g[..., second] * cs - g[..., first] * sn
                g = t
            out["d" + n] = (g * w / root - x * (g * w * x).sum(-1)[..., None] / (over * root ** 3))[None]
            if s["w" + n] is not None:
                out["dw" + n] = (g * x / root).sum((0, 1))
    return out


def _exact_step(s):
    c, rep = s["case"], s["case"]["heads"] // s["case"]["groups"]
    pool = s["states"].double()
    o = torch.zeros(s["v"].shape, dtype=torch.float64, device=pool.device)
    for i, at in enumerate(s["slots"].tolist()):
        S = pool[at]
        for t in range(c["tokens"]):
            k, q = (s[n][i, t].double().repeat_interleave(rep, 0) for n in "kq")
            S = S * s["g"][i, t].double().exp()[:, None, None]
            e = s["v"][i, t].double() - torch.einsum("hpn,hn->hp", S, k)
            S = S + torch.einsum("hp,hn->hpn", s["beta"][i, t].double()[:, None] * e, k)
            o[i, t] = s["scale"] * torch.einsum("hpn,hn->hp", S, q)
        pool[at] = S
    return dict(o=o, states=pool)


def _exact_delta(s):
    """Token by token, and back again from states kept every 64 tokens; tokens past a row's end change nothing."""
    c = s["case"]
    rep, scale, lens, dev = c["heads"] // c["groups"], s["scale"], s["lens"], s["v"].device
    top, nb = max(lens), len(lens)
    start = np.concatenate([[0], np.cumsum(lens)[:-1]])
    idx = torch.from_numpy(np.minimum(start[:, None] + np.arange(top)[None], sum(lens) - 1)).to(dev)
    live = (torch.arange(top, device=dev)[None] < torch.tensor(lens, device=dev)[:, None]).double()
    flat = {n: s[n].flatten(0, 1) for n in ("q", "k", "v", "g", "beta") + (("do",) if c["grad"] else ())}

    def token(t):
        on = live[:, t, None]
        q, k = (flat[n][idx[:, t]].double().repeat_interleave(rep, 1)[..., None, :] for n in "qk")
        v = flat["v"][idx[:, t]].double()[..., None]
        return q, k, v, (flat["g"][idx[:, t]].double() * on)[..., None, None], (flat["beta"][idx[:, t]].double() * on)

    H, P, N = c["heads"], c["headdim"], c["dstate"]
    total = sum(lens)
    out = {n: torch.zeros((total,) + shape, dtype=torch.float64, device=dev) for n, shape in
           [("o", (H, P))] + ([("dq", (H, N)), ("dk", (H, N)), ("dv", (H, P)), ("dg", (H,)), ("dbeta", (H,))]
                              if c["grad"] else [])}

    def put(name, t, val):
        on = live[:, t] > 0
        out[name][idx[on, t]] = val[on]

    S = torch.zeros((nb, H, P, N), dtype=torch.float64, device=dev)
    kept = []
    for t in range(top):
        if c["grad"] and t % 64 == 0:
            kept.append(S)
        q, k, v, g, beta = token(t)
        S = S * g.exp()
        e = v - S @ k.mT
        S = S + (beta[..., None, None] * e) @ k
        put("o", t, scale * (S @ q.mT)[..., 0])
    if not c["grad"]:
        return dict(o=out["o"].reshape(s["v"].shape), final=S)
    dS = torch.zeros_like(S)
    for b0 in range((top - 1) // 64 * 64, -1, -64):
        S, mids = kept[b0 // 64], []
        for t in range(b0, min(b0 + 64, top)):
            q, k, v, g, beta = token(t)
            Sd = S * g.exp()
            e = v - Sd @ k.mT
            S = Sd + (beta[..., None, None] * e) @ k
            mids.append((Sd, e, S))
        for t in range(min(b0 + 64, top) - 1, b0 - 1, -1):
            q, k, v, g, beta = token(t)
            Sd, e, S1 = mids[t - b0]
            do = flat["do"][idx[:, t]].double()[..., None] * live[:, t, None, None, None]
            put("dq", t, scale * (S1.mT @ do)[..., 0])
            dS = dS + scale * do @ q
            du = dS @ k.mT
            put("dbeta", t, (du * e)[..., 0].sum(-1))
            de = beta[..., None, None] * du
            put("dv", t, de[..., 0])
            put("dk", t, (dS.mT @ (beta[..., None, None] * e) - Sd.mT @ de)[..., 0])
            dS = dS - de @ k
            put("dg", t, (dS * Sd).sum((-1, -2)))
            dS = dS * g.exp()

    def shared(x):
        return x.unflatten(1, (c["groups"], rep)).sum(2).reshape(s["q"].shape)
    return dict(o=out["o"].reshape(s["v"].shape), dq=shared(out["dq"]), dk=shared(out["dk"]),
                dv=out["dv"].reshape(s["v"].shape), dg=out["dg"].reshape(s["g"].shape),
                dbeta=out["dbeta"].reshape(s["g"].shape))


# ---- work ------------------------------------------------------------------

def work(case):
    """Bytes: each input read once, each output written once.  Operations: the products of the definition."""
    el = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "qk":
        n, d = case["tokens"] * (case["qheads"] + case["kheads"]), case["dim"]
        angles = case["tokens"] * (4 + 4 * case["rotary"]) if case["rotary"] else 0
        passes = 4 if case["grad"] else 2     # x, y and, with gradients, dy, dx
        return dict(bytes=passes * n * d * el + angles, flops=n * d * (6 + (12 if case["grad"] else 0)))
    H, G, P, N = (case[k] for k in ("heads", "groups", "headdim", "dstate"))
    if case["op"] == "step":
        tok = case["seqs"] * case["tokens"]
        return dict(bytes=2 * case["seqs"] * H * P * N * 4 + tok * (2 * G * N * el + 2 * H * P * el + 8 * H),
                    flops=tok * H * 7 * N * P)
    tok = case["batch"] * case["seqlen"]
    once = tok * (2 * G * N * el + 2 * H * P * el + 8 * H)
    if not case["grad"]:
        return dict(bytes=once + case["batch"] * H * P * N * 4, flops=tok * H * 6 * N * P)
    # q, k, v, g, beta, do in; o, dq, dk, dv, dg, dbeta out
    return dict(bytes=once + tok * (2 * G * N * el + 2 * H * P * el + 2 * H * el), flops=tok * H * 20 * N * P)
