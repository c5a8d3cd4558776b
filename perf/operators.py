"""Cases and plain forms of the operators that stand before and beside the
sparse attention layer: rotary positions over (time, height, width), the norm of
queries and keys for each head with the rotation in the same pass, and dense
attention over packed sequences with grouped heads.

Sizes are those of the synthetic layers (tiny, small, Wan and HunyuanVideo
grids) or generic.  ``own`` selects between elementary torch operations and the
library's calls.
"""
from __future__ import annotations

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
THETA = 10000.0


def _lens(text):
    return [int(x) for x in text.split(",")]


# ------------------------------------------------------------------- cases
def _rope_case(name, **kw):
    c = dict(op="rope", dtype="bf16", B=1, H=24, T=1, Hg=1, W=1, text=0, D=128, half=False, packed="", inverse=False)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def _norm_case(name, **kw):
    c = dict(op="norm", dtype="bf16", B=1, H=24, Hk=24, T=1, Hg=1, W=1, text=0, D=128, half=False, train=False)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def _attn_case(name, **kw):
    c = dict(op="attn", dtype="bf16", H=8, Hk=8, D=128, lq="256", lk="256", causal=False, packed=True, token_major=False,
             train=False)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # the smallest call: one head of a 256-token clip in float32, where only latency counts
        _rope_case("rope_tiny_f32", dtype="f32", H=1, T=4, Hg=8, W=8, D=64),
        # a training batch that packs clips and single images of different sizes in one row of tokens, each
        # token with its own (t, y, w); the gradient's direction, in the layout with pairs D/2 apart
        _rope_case("rope_packed_grad_bf16", packed="9x30x53,1x45x80,13x45x79,1x17x17,3x31x41", T=33, Hg=45, W=80,
                   text=77, half=True, inverse=True),
        # the small layer before its attention, read from a fused projection
        _norm_case("norm_rope_small_bf16", H=8, Hk=8, T=8, Hg=16, W=16),
        # the HunyuanVideo-shaped layer before its attention, with its text tokens
        _norm_case("norm_rope_hunyuan_bf16", T=33, Hg=45, W=80, text=256),
        # a training step of the Wan-shaped layer's norms: outputs and all gradients
        _norm_case("norm_rope_wan_train_bf16", H=40, Hk=40, T=21, Hg=45, W=80, train=True),
        # odd sizes in float32: batch, grouped heads, a head width that fills no power of two
        _norm_case("norm_rope_odd_train_f32", dtype="f32", B=3, H=10, Hk=5, T=7, Hg=19, W=23, text=13, D=96, train=True),
        # the smallest attention call: the tiny layer
        _attn_case("attn_tiny_f32", dtype="f32", H=1, Hk=1, D=64, lq="256", lk="256", packed=False),
        # one new row for each of four clips that are at different points: every key is read for one query
        _attn_case("attn_single_rows_bf16", H=24, Hk=8, lq="1,1,1,1", lk="119056,75600,40001,3601", causal=True),
        # clips of different lengths packed in one batch, causal, grouped heads, straight from the projection's layout
        _attn_case("attn_packed_causal_bf16", H=24, Hk=8, lq="18000,1,3600,129,7777,0,10823",
                   lk="18000,1,3600,129,7777,0,10823", causal=True, token_major=True),
        # the dense layer that warm-up steps run, HunyuanVideo length, a quarter of its heads
        _attn_case("attn_hunyuan_bf16", H=6, Hk=6, lq="119056", lk="119056", packed=False),
        # a training step on a packed batch of shorter clips, causal, grouped heads, D = 64
        _attn_case("attn_train_packed_bf16", H=16, Hk=4, D=64, lq="3600,1,7219,511,2048,64,5001",
                   lk="3600,1,7219,511,2048,64,5001", causal=True, train=True),
        # a training step of the Wan-shaped dense layer, four of its heads
        _attn_case("attn_train_wan_bf16", H=4, Hk=4, lq="75600", lk="75600", packed=False, train=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _grid(rng, most):
    while True:
        g = (_log_int(rng, 1, 33), _log_int(rng, 1, 60), _log_int(rng, 1, 90))
        if g[0] * g[1] * g[2] <= most:
            return g


def draw(rng):
    kind = rng.choice(["rope", "norm", "norm", "attn", "attn", "attn"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    D = rng.choice([32, 64, 96, 128, 128])
    text = rng.choice([0, _log_int(rng, 1, 512)])
    if kind == "rope":
        packed = ""
        T, Hg, W = _grid(rng, 75600)
        if rng.random() < 0.5:
            packed = ",".join("x".join(str(rng.randint(1, e)) for e in (T, Hg, W)) for _ in range(rng.randint(1, 6)))
        return _rope_case("", dtype=dtype, B=rng.choice([1, 1, 2, 3]), H=rng.randint(1, 40), T=T, Hg=Hg, W=W, text=text,
                          D=D, half=rng.random() < 0.5, packed=packed, inverse=rng.random() < 0.5)
    if kind == "norm":
        T, Hg, W = _grid(rng, 75600)
        Hk, g = rng.randint(1, 20), rng.choice([1, 1, 2])
        return _norm_case("", dtype=dtype, B=rng.choice([1, 1, 2]), H=Hk * g, Hk=Hk, T=T, Hg=Hg, W=W, text=text, D=D,
                          half=rng.random() < 0.5, train=rng.random() < 0.5)
    train = rng.random() < 0.4
    Hk, g = rng.randint(1, 8), rng.choice([1, 1, 2, 3, 4])
    causal = rng.random() < 0.5
    shape = rng.choice(["same", "same", "cross", "rows"])
    if shape == "rows":     # few query rows over long key sequences
        n = rng.randint(1, 6)
        lk = [_log_int(rng, 1, 100000) for _ in range(n)]
        lq = [rng.randint(1, 4) for _ in range(n)]
        train = False
    elif shape == "cross":  # video rows over text keys
        n = rng.randint(1, 4)
        lk = [_log_int(rng, 1, 600) for _ in range(n)]
        lq = [_log_int(rng, 1, 12000) for _ in range(n)]
    else:
        n = rng.randint(1, 6)
        lk = [_log_int(rng, 1, 6000) for _ in range(n)]
        lq = lk
    packed = n > 1 or rng.random() < 0.5
    return _attn_case("", dtype=dtype, H=Hk * g, Hk=Hk, D=D, lq=",".join(map(str, lq)), lk=",".join(map(str, lk)),
                      causal=causal, packed=packed, token_major=rng.random() < 0.5, train=train)


# ------------------------------------------------------------------- work
def _tokens(case):
    if case.get("op") == "rope" and case["packed"]:
        n = sum(math.prod(int(x) for x in g.split("x")) for g in case["packed"].split(","))
    else:
        n = case["T"] * case["Hg"] * case["W"]
    return n + case["text"]


def _visible(nq, nk, causal):
    """Number of (query, key) pairs that the mask leaves."""
    if not causal:
        return nq * nk
    off = nk - nq                              # row i sees keys 0 .. i + off
    first = max(0, -off)                       # first row that sees a key
    rows = nq - first
    return rows * (first + off + 1) + rows * (rows - 1) // 2 if rows > 0 else 0


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    D = case["D"]
    if case["op"] == "rope":
        rows = case["B"] * case["H"] * _tokens(case)
        pos = 12 * _tokens(case) if case["packed"] else 0
        return {"bytes": 2 * rows * D * e + pos, "flops": 3 * rows * D}
    if case["op"] == "norm":
        rows = case["B"] * (case["H"] + case["Hk"]) * _tokens(case)
        if case["train"]:   # x, dy in; y, dx out (weights and their gradients are a few hundred bytes)
            return {"bytes": 4 * rows * D * e, "flops": 20 * rows * D}
        return {"bytes": 2 * rows * D * e, "flops": 7 * rows * D}
    lq, lk = _lens(case["lq"]), _lens(case["lk"])
    pairs = case["H"] * sum(_visible(a, b, case["causal"]) for a, b in zip(lq, lk))
    qb, kb = case["H"] * sum(lq) * D * e, case["Hk"] * sum(lk) * D * e
    if case["train"]:       # forward 2 products, backward 5 (the scores are formed again); q, do, k, v in; o, dq, dk, dv out
        return {"bytes": 4 * qb + 4 * kb, "flops": 14 * D * pairs}
    return {"bytes": 2 * qb + 2 * kb, "flops": 4 * D * pairs}


# ------------------------------------------------------------------- inputs
def _positions(case, dev):
    """int32 [N, 3] of a packed row of clips and images; text tokens get -1."""
    parts = []
    for g in case["packed"].split(","):
        t, y, w = (int(x) for x in g.split("x"))
        parts.append(torch.stack(torch.meshgrid(torch.arange(t), torch.arange(y), torch.arange(w), indexing="ij"),
                                 -1).reshape(-1, 3))
    parts.append(torch.full((case["text"], 3), -1))
    return torch.cat(parts).to(torch.int32).to(dev)


def _rand(gen, shape, dt):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dt)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(1000003 * seed + 17)
    dt, D = _DT[case["dtype"]], case["D"]
    st = {"case": case}
    if case["op"] in ("rope", "norm"):
        N = _tokens(case)
        st["N"] = N
        st["positions"] = _positions(case, dev) if case.get("packed") else None
        if own:
            import block_sparse_attention_means_b200 as park
            st["rope"] = park.rope_table((case["T"], case["Hg"], case["W"]), D, half=case["half"], device=dev)
        else:
            st["table"] = _table(case, dev, torch.float64)
    if case["op"] == "rope":
        # queries as the projection leaves them: [B, N, H, D]
        st["x"] = _rand(gen, (case["B"], N, case["H"], D), dt).transpose(1, 2)
        return st
    if case["op"] == "norm":
        H, Hk = case["H"], case["Hk"]
        gain = 1.0 + 0.5 * torch.randn(H + Hk, 1, generator=gen, device=dev)  # heads differ in scale
        # q, k and v of a fused projection, one row of (H + 2 Hk) heads for each token
        qkv = torch.empty(case["B"], N, H + 2 * Hk, D, device=dev, dtype=dt)
        for b in range(case["B"]):
            qkv[b, :, :H + Hk] = (_rand(gen, (N, H + Hk, D), torch.float32) * gain).to(dt)
        st["q"], st["k"] = qkv[:, :, :H].transpose(1, 2), qkv[:, :, H:H + Hk].transpose(1, 2)
        st["wq"] = (1.0 + 0.1 * torch.randn(D, generator=gen, device=dev)).to(dt)
        st["wk"] = (1.0 + 0.1 * torch.randn(D, generator=gen, device=dev)).to(dt)
        if case["train"]:
            st["dq"] = _rand(gen, (case["B"], H, N, D), dt)
            st["dk"] = _rand(gen, (case["B"], Hk, N, D), dt)
        return st
    lq, lk = _lens(case["lq"]), _lens(case["lk"])
    H, Hk, Nq, Nk = case["H"], case["Hk"], sum(lq), sum(lk)

    def tensor(h, n, mix):
        shape = (1, n, h, D) if case["token_major"] else (1, h, n, D)
        x = _rand(gen, shape, torch.float32)
        if mix is not None:  # a direction that queries and keys share: scores with some structure, not only noise
            a = torch.randn((1, n, 1, 1) if case["token_major"] else (1, 1, n, 1), generator=gen, device=dev)
            x += 0.5 * a * mix
        x = x.to(dt)
        return x.transpose(1, 2) if case["token_major"] else x

    mix = torch.randn(D, generator=gen, device=dev)
    st["q"], st["k"], st["v"] = tensor(H, Nq, mix), tensor(Hk, Nk, mix), tensor(Hk, Nk, None)
    if case["train"]:
        st["do"] = tensor(H, Nq, None)
    if case["packed"]:
        cu = lambda l: torch.tensor([0] + l, dtype=torch.int32).cumsum(0).to(torch.int32).to(dev)  # noqa: E731
        st["cu_q"], st["cu_k"] = cu(lq), cu(lk)
    else:
        st["cu_q"] = st["cu_k"] = None
    return st


# ------------------------------------------------------------------- plain forms
def _pairs(D):
    n = D // 2
    return n - 2 * (n // 3), n // 3, n // 3


def _table(case, dev, dt):
    """cos and sin of the angles of every position on each axis, in float64 (far positions)."""
    out = []
    for extent, n in zip((case["T"], case["Hg"], case["W"]), _pairs(case["D"])):
        freq = THETA ** (-torch.arange(n, device=dev, dtype=torch.float64) / max(n, 1))
        a = torch.arange(extent, device=dev, dtype=torch.float64)[:, None] * freq
        out.append((a.cos().to(dt), a.sin().to(dt)))
    return out


def _token_angles(st, dt):
    """cos and sin [N, D/2] of each token; text tokens get angle 0."""
    case, table = st["case"], st["table"]
    dev = table[0][0].device
    if st["positions"] is not None:
        pos = st["positions"].long()
    else:
        t, y, w = case["T"], case["Hg"], case["W"]
        n = torch.arange(t * y * w, device=dev)
        pos = torch.stack([n // (y * w), n // w % y, n % w], -1)
        pos = torch.cat([pos, torch.full((case["text"], 3), -1, device=dev)])
    text = (pos[:, :1] < 0)
    pos = pos.clamp_min(0)
    c = torch.cat([table[a][0][pos[:, a]] for a in range(3)], 1).to(dt)
    s = torch.cat([table[a][1][pos[:, a]] for a in range(3)], 1).to(dt)
    return torch.where(text, torch.ones_like(c), c), torch.where(text, torch.zeros_like(s), s)


def _rotate(x, c, s, half):
    if half:
        h = x.shape[-1] // 2
        a, b = x[..., :h], x[..., h:]
        return torch.cat([a * c - b * s, a * s + b * c], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)


def _plain_norm(x, w, c, s, half, dt):
    out = torch.empty(x.shape, device=x.device, dtype=dt)
    for b in range(x.shape[0]):
        f = x[b].float()
        f = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * w.float()
        out[b] = _rotate(f, c, s, half).to(dt)
    return out


def _plain_norm_grad(dy, x, w, c, s, half, dt):
    dx = torch.empty(x.shape, device=x.device, dtype=dt)
    dw = torch.zeros(x.shape[-1], device=x.device)
    for b in range(x.shape[0]):
        f = x[b].float()
        r = torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)
        f = f * r
        g = _rotate(dy[b].float(), c, -s, half)
        dw += (g * f).sum((0, 1))
        g = g * w.float()
        dx[b] = ((g - f * (g * f).mean(-1, keepdim=True)) * r).to(dt)
    return dx, dw


def _sequences(case):
    q0 = k0 = 0
    for nq, nk in zip(_lens(case["lq"]), _lens(case["lk"])):
        yield q0, nq, k0, nk
        q0 += nq
        k0 += nk


def _row_step(case, nk, budget):
    return max(1, budget // max(1, case["H"] * nk))


def _mask(i0, i1, nq, nk, dev):
    """True where row i does not see key j (causal, rows aligned with the last keys)."""
    i = torch.arange(i0, i1, device=dev)[:, None]
    return torch.arange(nk, device=dev)[None] > i + (nk - nq)


def _probabilities(q, k, scale, case, i0, i1, nq, nk, G):
    """Softmax of the scores [Hk, G, rows, keys]; rows without a key are 0."""
    Hk, n, D = k.shape[0], i1 - i0, q.shape[-1]
    s = torch.matmul(q.reshape(Hk, G * n, D), k.transpose(1, 2)).view(Hk, G, n, nk) * scale
    if case["causal"]:
        s.masked_fill_(_mask(i0, i1, nq, nk, q.device), -math.inf)
    m = s.amax(-1, keepdim=True)
    s.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    l = s.sum(-1, keepdim=True)
    return s.div_(torch.where(l == 0, torch.ones_like(l), l))


def _plain_attention(st, dt):
    case = st["case"]
    q, k, v = st["q"][0], st["k"][0], st["v"][0]
    H, Hk, D = case["H"], case["Hk"], case["D"]
    G, scale = H // Hk, D ** -0.5
    o = torch.zeros(1, *q.shape, device=q.device, dtype=dt)
    grads = None
    if case["train"]:
        do = st["do"][0]
        grads = [torch.zeros(1, *q.shape, device=q.device, dtype=dt), torch.zeros(1, *k.shape, device=q.device, dtype=dt),
                 torch.zeros(1, *v.shape, device=q.device, dtype=dt)]
    for q0, nq, k0, nk in _sequences(case):
        if nq == 0 or nk == 0:
            continue
        kf, vf = k[:, k0:k0 + nk].float(), v[:, k0:k0 + nk].float()
        if case["train"]:
            dk, dv = torch.zeros_like(kf), torch.zeros_like(vf)
        step = _row_step(case, nk, 1 << 29)
        for i0 in range(0, nq, step):
            i1 = min(nq, i0 + step)
            n = i1 - i0
            qf = q[:, q0 + i0:q0 + i1].float().reshape(Hk, G, n, D)
            p = _probabilities(qf, kf, scale, case, i0, i1, nq, nk, G).view(Hk, G * n, nk)
            o[0, :, q0 + i0:q0 + i1] = torch.matmul(p, vf).view(H, n, D).to(dt)
            if case["train"]:
                dof = do[:, q0 + i0:q0 + i1].float().reshape(Hk, G * n, D)
                dv += torch.matmul(p.transpose(1, 2), dof)
                ds = torch.matmul(dof, vf.transpose(1, 2))
                ds.sub_((ds * p).sum(-1, keepdim=True)).mul_(p).mul_(scale)
                grads[0][0, :, q0 + i0:q0 + i1] = torch.matmul(ds, kf).view(H, n, D).to(dt)
                dk += torch.matmul(ds.transpose(1, 2), qf.reshape(Hk, G * n, D))
                del ds
            del p
        if case["train"]:
            grads[1][0, :, k0:k0 + nk] = dk.to(dt)
            grads[2][0, :, k0:k0 + nk] = dv.to(dt)
    return (o, *grads) if case["train"] else o


def _run_plain(st):
    case = st["case"]
    dt = _DT[case["dtype"]]
    if case["op"] == "attn":
        return _plain_attention(st, dt)
    c, s = _token_angles(st, torch.float32)
    if case["op"] == "rope":
        return _rotate(st["x"].float(), c, -s if case["inverse"] else s, case["half"]).to(dt)
    q = _plain_norm(st["q"], st["wq"], c, s, case["half"], dt)
    k = _plain_norm(st["k"], st["wk"], c, s, case["half"], dt)
    if not case["train"]:
        return q, k
    dq, dwq = _plain_norm_grad(st["dq"], st["q"], st["wq"], c, s, case["half"], dt)
    dk, dwk = _plain_norm_grad(st["dk"], st["k"], st["wk"], c, s, case["half"], dt)
    return q, k, dq, dk, dwq, dwk


def _run_own(st):
    import block_sparse_attention_means_b200 as park
    case = st["case"]
    if case["op"] == "rope":
        return park.rope(st["x"], st["rope"], positions=st["positions"], inverse=case["inverse"])
    if case["op"] == "norm":
        q, k = park.qk_norm_rope(st["q"], st["k"], st["wq"], st["wk"], rope=st["rope"], eps=EPS)
        if not case["train"]:
            return q, k
        return (q, k, *park.qk_norm_rope_bwd(st["dq"], st["dk"], st["q"], st["k"], st["wq"], st["wk"], rope=st["rope"],
                                             eps=EPS))
    kw = dict(causal=case["causal"], cu_q=st["cu_q"], cu_k=st["cu_k"])
    if not case["train"]:
        return park.attention(st["q"], st["k"], st["v"], **kw)
    o, lse = park.attention(st["q"], st["k"], st["v"], return_lse=True, **kw)
    return (o, *park.attention_bwd(st["do"], st["q"], st["k"], st["v"], o, lse, **kw))


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------- exact values
def _exact_rotation(st, dev):
    """Unit complex numbers [N, D/2], complex128, from the definition for each token."""
    case = st["case"]
    if st["positions"] is not None:
        pos = st["positions"].double()
    else:
        g = [torch.arange(e, device=dev, dtype=torch.float64) for e in (case["T"], case["Hg"], case["W"])]
        pos = torch.cartesian_prod(*g).reshape(-1, 3)
        pos = torch.cat([pos, torch.zeros(case["text"], 3, device=dev, dtype=torch.float64)])
    pos = torch.where(pos < 0, torch.zeros_like(pos), pos)
    ang = [pos[:, a:a + 1] * torch.pow(torch.tensor(THETA, device=dev, dtype=torch.float64),
                                       -torch.arange(n, device=dev).double() / max(n, 1))
           for a, n in enumerate(_pairs(case["D"]))]
    ang = torch.cat(ang, 1)
    return torch.polar(torch.ones_like(ang), ang)


def _exact_turn(x, z, half):
    """x float64 [..., N, D] as complex pairs times z [N, D/2]."""
    D = x.shape[-1]
    pairs = x.reshape(*x.shape[:-1], 2, D // 2).transpose(-1, -2) if half else x.reshape(*x.shape[:-1], D // 2, 2)
    y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
    return (y.transpose(-1, -2) if half else y).reshape(x.shape)


def _exact_norm(x, w, dy, z, half):
    """Output, and with dy the gradients, head by head in float64."""
    y = torch.empty(x.shape, device=x.device, dtype=torch.float64)
    dx = torch.empty_like(y) if dy is not None else None
    dw = torch.zeros(x.shape[-1], device=x.device, dtype=torch.float64)
    w = w.double()
    D = x.shape[-1]
    for b in range(x.shape[0]):
        for h in range(x.shape[1]):
            v = x[b, h].double()
            ms = torch.einsum("nd,nd->n", v, v) / D + EPS
            y[b, h] = _exact_turn(v * w / ms.sqrt()[:, None], z, half)
            if dy is not None:
                g = _exact_turn(dy[b, h].double(), z.conj(), half)
                dw += torch.einsum("nd,nd,n->d", g, v, ms.rsqrt())
                gw = g * w
                t = torch.einsum("nd,nd->n", gw, v) / D
                dx[b, h] = gw / ms.sqrt()[:, None] - v * (t / ms ** 1.5)[:, None]
    return y, dx, dw


def _exact_attention(st):
    case = st["case"]
    H, Hk, D = case["H"], case["Hk"], case["D"]
    dev = st["q"].device
    f64 = dict(device=dev, dtype=torch.float64)
    o = torch.zeros(st["q"].shape, **f64)
    if case["train"]:
        dq, dk, dv = torch.zeros(st["q"].shape, **f64), torch.zeros(st["k"].shape, **f64), torch.zeros(st["v"].shape, **f64)
    for q0, nq, k0, nk in _sequences(case):
        if nq == 0 or nk == 0:
            continue
        step = max(1, (1 << 28) // nk)
        last = torch.arange(nq, device=dev) + (nk - nq if case["causal"] else nk)  # last visible key of each row
        for h in range(H):
            kh = h // (H // Hk)
            K, V = st["k"][0, kh, k0:k0 + nk].double(), st["v"][0, kh, k0:k0 + nk].double()
            for i0 in range(0, nq, step):
                rows = slice(q0 + i0, q0 + min(nq, i0 + step))
                Q = st["q"][0, h, rows].double()
                see = torch.arange(nk, device=dev)[None] <= last[i0:i0 + step, None]
                z = torch.where(see, Q @ K.T / math.sqrt(D), -math.inf)
                z = torch.where(see, torch.exp(z - torch.logsumexp(z, 1, keepdim=True)), 0.0)
                o[0, h, rows] = z @ V
                if case["train"]:
                    dO = st["do"][0, h, rows].double()
                    dv[0, kh, k0:k0 + nk] += z.T @ dO
                    z = z * (dO @ V.T - (dO * o[0, h, rows]).sum(1, keepdim=True)) / math.sqrt(D)
                    dq[0, h, rows] = z @ K
                    dk[0, kh, k0:k0 + nk] += z.T @ Q
    return (o, dq, dk, dv) if case["train"] else o


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "attn":
        pairs = case["H"] * sum(_visible(a, b, False) for a, b in zip(_lens(case["lq"]), _lens(case["lk"])))
        return None if pairs * (2.5 if case["train"] else 1.0) > 1.5e11 else _exact_attention(st)
    z = _exact_rotation(st, st["x"].device if case["op"] == "rope" else st["q"].device)
    if case["op"] == "rope":
        out = torch.empty(st["x"].shape, device=st["x"].device, dtype=torch.float64)
        for b in range(case["B"]):
            for h in range(case["H"]):
                out[b, h] = _exact_turn(st["x"][b, h].double(), z.conj() if case["inverse"] else z, case["half"])
        return out
    q, dq, dwq = _exact_norm(st["q"], st["wq"], st.get("dq"), z, case["half"])
    k, dk, dwk = _exact_norm(st["k"], st["wk"], st.get("dk"), z, case["half"])
    return (q, k, dq, dk, dwq, dwk) if case["train"] else (q, k)
