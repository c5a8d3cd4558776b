"""Rotary positions, the norm of queries and keys with the rotation, and dense
attention against plain float64 forms, with bounds derived from the roundings.

Roundings, relative to the value rounded: u = finfo(type).eps / 2 for each result
stored in the tensors' type (bf16 2^-8, float32 2^-24), E = 2^-24 for each float32
operation inside.  Each bound below counts them element by element.
"""
import math

import numpy as np
import pytest
import torch

import block_sparse_attention_means_b200 as park
from block_sparse_attention_means_b200 import _lib

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
E = 2.0 ** -24
TINY = 2.0 ** -126   # probabilities below the smallest normal number are flushed to 0
U = {BF: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(autouse=True)
def clean_status():
    park.status_word().zero_()
    yield
    torch.cuda.synchronize()
    assert park.status_word().item() == 0
    park.status_word().zero_()


def rand(seed, *shape, dt=F32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dt).cuda()


def layout(x, kind):
    """The same values in another memory layout of [B, H, N, D]."""
    if kind == "heads":
        return x.contiguous()
    if kind == "tokens":                          # [B, N, H, D]
        return x.transpose(1, 2).contiguous().transpose(1, 2)
    if kind == "fused":                           # one part of [B, N, 3, H, D]
        b, h, n, d = x.shape
        buf = torch.full((b, n, 3, h, d), float("nan"), dtype=x.dtype, device=x.device)
        buf[:, :, 1] = x.transpose(1, 2)
        return buf[:, :, 1].transpose(1, 2)
    raise ValueError(kind)


def within(got, want, tol, what=""):
    got = got.double()
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} outside, worst {((got - want).abs() / tol.clamp_min(1e-300)).max().item():.3g} of the bound"


# ------------------------------------------------------------------ rotary positions
def angles(extent, pairs, theta, scale, pos):
    """cos, sin [N, sum(pairs)] for positions [N, 3] (negative: text)."""
    out = []
    text = (pos < 0).any(-1, keepdim=True)
    for a in range(3):
        f = theta ** (-torch.arange(pairs[a], dtype=torch.float64) / max(1, pairs[a]))
        out.append(torch.where(text, 0.0, scale[a] * pos[:, a:a + 1].double() * f))
    ang = torch.cat(out, -1)
    return ang.cos().cuda(), ang.sin().cuda()


def grid_positions(extent, n):
    t, y, w = extent
    i = torch.arange(n)
    pos = torch.stack([i // (y * w), i // w % y, i % w], -1)
    pos[i >= t * y * w] = -1
    return pos


def plain_rotate(x, c, s, half):
    """x float64 [..., N, D]; c, s [N, P] or [B, 1, N, P] for the first P pairs."""
    D, P = x.shape[-1], c.shape[-1]
    ia = torch.arange(P, device=x.device) * (1 if half else 2)
    ib = ia + (D // 2 if half else 1)
    y = x.clone()
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ia] * s + x[..., ib] * c
    return y


def pair_mass(x, half):
    """|a| + |b| of each element's pair."""
    D = x.shape[-1]
    if half:
        m = x[..., :D // 2].abs() + x[..., D // 2:].abs()
        return torch.cat([m, m], -1)
    m = x[..., 0::2].abs() + x[..., 1::2].abs()
    return m.repeat_interleave(2, -1)




ROPE = [
    # B, H, extent, text, D, half, dtype, layout
    (1, 1, (4, 8, 8), 0, 64, False, F32, "heads"),
    (2, 3, (3, 5, 7), 4, 128, False, BF, "fused"),
    (2, 3, (3, 5, 7), 4, 128, True, BF, "tokens"),
    (1, 5, (1, 1, 1), 0, 32, True, F32, "heads"),
    (3, 2, (2, 3, 1), 1, 96, False, BF, "tokens"),
    (1, 7, (2, 9, 5), 0, 96, True, F32, "fused"),
    (1, 40, (1, 3, 3), 2, 64, True, BF, "heads"),
]


@pytest.mark.parametrize("B,H,extent,text,D,half,dt,kind", ROPE)
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_grid(B, H, extent, text, D, half, dt, kind, inverse):
    n = math.prod(extent) + text
    x = layout(rand(1, B, H, n, D, dt=dt), kind)
    r = park.rope_table(extent, D, half=half)
    y = park.rope(x, r, inverse=inverse)
    c, s = angles(extent, r.pairs, 10000.0, (1, 1, 1), grid_positions(extent, n))
    want = plain_rotate(x.double(), c, -s if inverse else s, half)
    within(y, want, U[dt] * want.abs() + 4 * E * pair_mass(x.double(), half))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("per_batch", [False, True])
def test_rope_positions(dt, per_batch):
    B, H, n, D, extent = 2, 3, 77, 128, (9, 6, 11)
    g = torch.Generator().manual_seed(3)
    pos = torch.stack([torch.randint(0, e, (B, n), generator=g) for e in extent], -1)
    pos[:, 5] = -1
    pos[1, 70:, 1] = -7                            # any negative coordinate is text
    if not per_batch:
        pos[:] = pos[1].clone()
    x = rand(4, B, H, n, D, dt=dt)
    scale = (0.5, 1.0, 2.25)
    r = park.rope_table(extent, D, pairs=(20, 10, 30), theta=500.0, scale=scale)
    p = (pos if per_batch else pos[0]).to(torch.int32).contiguous().cuda()
    y = park.rope(x, r, positions=p)
    for b in range(B):
        c, s = angles(extent, (20, 10, 30), 500.0, scale, pos[b])
        want = plain_rotate(x[b].double(), c, s, False)
        within(y[b], want, U[dt] * want.abs() + 4 * E * pair_mass(x[b].double(), False))
    assert torch.equal(y[..., 120:], x[..., 120:])  # the last four pairs are not rotated
    assert torch.equal(y[:, :, 5], x[:, :, 5])


def test_rope_far_positions():
    """Angles of positions near 2^20 keep float32's accuracy of their cosine."""
    D, far = 64, 1 << 20
    r = park.rope_table((far, 1, 1), D, pairs=(32, 0, 0))
    pos = torch.zeros(50, 3, dtype=torch.int32)
    pos[:, 0] = torch.arange(far - 50, far)
    x = rand(5, 1, 2, 50, D)
    y = park.rope(x, r, positions=pos.cuda())
    c, s = angles((far, 1, 1), (32, 0, 0), 10000.0, (1, 1, 1), pos.long())
    want = plain_rotate(x.double(), c, s, False)
    # the angle itself, below 2^20, carries float64 roundings (2^-53 each, a few): 2^-30
    within(y, want, U[F32] * want.abs() + (4 * E + 2.0 ** -30) * pair_mass(x.double(), False))


def test_rope_in_place_and_back():
    x = rand(6, 2, 3, 40, 128)
    r = park.rope_table((2, 4, 5), 128)
    keep = x.clone()
    y = park.rope(x, r)
    assert park.rope(x, r, out=x) is x and torch.equal(x, y)
    back = park.rope(x, r, inverse=True)
    within(back, keep.double(), 16 * E * pair_mass(keep.double(), False))


def test_rope_position_out_of_range_is_reported():
    x = rand(7, 1, 2, 6, 64)
    r = park.rope_table((2, 3, 4), 64)
    pos = torch.zeros(6, 3, dtype=torch.int32)
    pos[2] = torch.tensor([1, 3, 0])
    pos[4] = torch.tensor([0, 0, 2 ** 31 - 1])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = park.rope(x, r, positions=pos.cuda(), status=status)
    assert status.item() == _lib.PARK_ERR_INDEX
    assert torch.equal(y[:, :, [0, 1, 2, 3, 4, 5]], x)  # position 0 and the refused ones do not turn
    with pytest.raises(ValueError):
        park.rope(x, r, positions=pos.cuda().long())
    with pytest.raises(ValueError):
        park.rope(x, r, positions=pos.cuda()[:5])
    with pytest.raises(ValueError):
        park.rope(x, park.rope_table((2, 3, 4), 128))


# ------------------------------------------------------------------ norm + rotation
NORM = [
    # B, H, Hk, extent, text, D, half, dtype, weights, layout
    (1, 8, 8, (2, 5, 9), 3, 128, False, BF, BF, "fused"),
    (2, 6, 2, (1, 7, 3), 0, 96, True, F32, F32, "tokens"),
    (1, 1, 1, (1, 1, 1), 0, 64, False, BF, F32, "heads"),
    (3, 4, 1, (2, 2, 2), 5, 32, False, F32, None, "heads"),
    (1, 24, 24, (1, 2, 3), 1, 128, True, BF, None, "fused"),
    (1, 3, 5, (4, 11, 13), 0, 64, True, BF, BF, "tokens"),
]


def plain_norm(x, w, c, s, half, eps):
    f = x / ((x * x).mean(-1, keepdim=True) + eps).sqrt() * w
    return plain_rotate(f, c, s, half), f


def norm_inputs(B, H, Hk, extent, text, D, half, dt, wdt, kind):
    n = math.prod(extent) + text
    q, k = layout(rand(10, B, H, n, D, dt=dt), kind), layout(rand(11, B, Hk, n, D, dt=dt) * 3, kind)
    w = [None, None] if wdt is None else [(1 + 0.3 * rand(12 + i, D)).to(wdt) for i in range(2)]
    r = park.rope_table(extent, D, half=half)
    c, s = angles(extent, r.pairs, 10000.0, (1, 1, 1), grid_positions(extent, n))
    return n, q, k, w, r, c, s


@pytest.mark.parametrize("B,H,Hk,extent,text,D,half,dt,wdt,kind", NORM)
def test_norm_rope(B, H, Hk, extent, text, D, half, dt, wdt, kind):
    n, q, k, w, r, c, s = norm_inputs(B, H, Hk, extent, text, D, half, dt, wdt, kind)
    eps = 1e-6
    out = park.qk_norm_rope(q, k, w[0], w[1], rope=r, eps=eps)
    for got, x, wt in zip(out, (q, k), w):
        assert got.is_contiguous()
        wd = torch.ones(D, device="cuda", dtype=torch.float64) if wt is None else wt.double()
        want, f = plain_norm(x.double(), wd, c, s, half, eps)
        # the mean of squares: products, sums of 8 and log2(16) levels, 1/D, eps: 16 E, half of
        # that in the root, 2 ulp (4 E) of rsqrt, two products: 16 E; the rotation 4 E
        within(got, want, U[dt] * want.abs() + 20 * E * pair_mass(f, half))
    plain = park.qk_norm_rope(q, k, w[0], w[1], eps=eps)   # no rotation
    for got, x, wt in zip(plain, (q, k), w):
        wd = torch.ones(D, device="cuda", dtype=torch.float64) if wt is None else wt.double()
        f = x.double() / ((x.double() ** 2).mean(-1, keepdim=True) + eps).sqrt() * wd
        within(got, f, (U[dt] + 16 * E) * f.abs())


@pytest.mark.parametrize("B,H,Hk,extent,text,D,half,dt,wdt,kind", NORM)
def test_norm_rope_backward(B, H, Hk, extent, text, D, half, dt, wdt, kind):
    n, q, k, w, r, c, s = norm_inputs(B, H, Hk, extent, text, D, half, dt, wdt, kind)
    eps = 1e-5
    gq, gk = layout(rand(20, B, H, n, D, dt=dt), kind), rand(21, B, Hk, n, D, dt=dt)
    dq, dk, dwq, dwk = park.qk_norm_rope_bwd(gq, gk, q, k, w[0], w[1], rope=r, eps=eps)
    for got, dw, x, wt, gy in ((dq, dwq, q, w[0], gq), (dk, dwk, k, w[1], gk)):
        wd = torch.ones(D, device="cuda", dtype=torch.float64) if wt is None else wt.double()
        x64 = x.double()
        rr = ((x64 ** 2).mean(-1, keepdim=True) + eps).rsqrt()
        g = plain_rotate(gy.double(), c, -s, half)
        h, xh = g * wd, x64 * rr
        want = rr * (h - xh * (h * xh).mean(-1, keepdim=True))
        # g: 4 E of its pair; r: 12 E; the mean of h xh: those, its products and sums (12 E)
        # of the terms' magnitudes; the outer products and the difference 4 E
        pm = pair_mass(gy.double(), half) * wd.abs()
        mean_abs = (pm * xh.abs()).mean(-1, keepdim=True)
        tol = U[dt] * want.abs() + rr * E * (24 * pm + 48 * xh.abs() * mean_abs)
        within(got, want, tol, "dx")
        if wt is None:
            assert dw is None
            continue
        want_w = (g * xh).sum((0, 1, 2))
        rows = B * x.shape[1] * n
        # each term 18 E; a thread's chain of sums is at most all rows long, then 5 + 8 + 9 + 75 levels
        tol_w = (min(rows, 700) + 18 + 100) * E * (pair_mass(gy.double(), half) * xh.abs()).sum((0, 1, 2))
        within(dw, want_w, tol_w, "dw")


def test_norm_rope_gradient_against_differences():
    """Float32 gradients against central differences of the float64 form along directions."""
    B, H, Hk, n, D = 1, 2, 1, 6, 64
    q, k, wq, wk = rand(30, B, H, n, D), rand(31, B, Hk, n, D), 1 + 0.2 * rand(32, D), 1 + 0.2 * rand(33, D)
    r = park.rope_table((1, 2, 3), D)
    c, s = angles((1, 2, 3), r.pairs, 10000.0, (1, 1, 1), grid_positions((1, 2, 3), n))
    gq, gk = rand(34, B, H, n, D), rand(35, B, Hk, n, D)
    grads = park.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, rope=r, eps=1e-6)

    def loss(args):
        a, b, u, v = args
        return (plain_norm(a, u, c, s, False, 1e-6)[0] * gq.double()).sum() + \
            (plain_norm(b, v, c, s, False, 1e-6)[0] * gk.double()).sum()
    base = [t.double() for t in (q, k, wq, wk)]
    for i in range(4):
        d = rand(40 + i, *base[i].shape).double()
        step = 1e-5
        up = [b + step * d if j == i else b for j, b in enumerate(base)]
        dn = [b - step * d if j == i else b for j, b in enumerate(base)]
        slope = (loss(up) - loss(dn)) / (2 * step)
        got = (grads[i].double() * d).sum()
        # third derivatives of order one times step^2 and float64 noise / step: far below 1e-5 of the terms
        assert abs(got - slope) <= 1e-5 * (grads[i].double() * d).abs().sum()


@pytest.mark.parametrize("size,eps", [(1e17, 1e-6), (1e14, 1e-6), (1e-14, 1e-24), (0.0, 1e-24)])
def test_norm_rope_rows_of_any_size(size, eps):
    """Rows whose 1/rms has a cube, or a square times the sums, out of float32's range; bounds as above."""
    D = 64
    q, k = rand(62, 1, 3, 9, D) * size, rand(63, 1, 1, 9, D) * size
    gq, gk, w = rand(64, 1, 3, 9, D), rand(65, 1, 1, 9, D), 1 + 0.3 * rand(66, D)
    out = park.qk_norm_rope(q, k, w, w, eps=eps)
    dq, dk, dwq, dwk = park.qk_norm_rope_bwd(gq, gk, q, k, w, w, eps=eps)
    for y, got, dw, x, gy in ((out[0], dq, dwq, q, gq), (out[1], dk, dwk, k, gk)):
        x64, wd, g = x.double(), w.double(), gy.double()
        rr = ((x64 ** 2).mean(-1, keepdim=True) + eps).rsqrt()
        within(y, x64 * rr * wd, (U[F32] + 16 * E) * (x64 * rr * wd).abs())
        h, xh = g * wd, x64 * rr
        want = rr * (h - xh * (h * xh).mean(-1, keepdim=True))
        mean_abs = (h * xh).abs().mean(-1, keepdim=True)
        within(got, want, U[F32] * want.abs() + rr * E * (24 * h.abs() + 48 * xh.abs() * mean_abs))
        within(dw, (g * xh).sum((0, 1, 2)), (27 + 118) * E * (g * xh).abs().sum((0, 1, 2)))


def test_norm_rope_same_bits_and_in_place():
    n, q, k, w, r, c, s = norm_inputs(2, 5, 3, (3, 7, 5), 2, 128, False, BF, BF, "heads")
    g = rand(50, *q.shape, dt=BF), rand(51, *k.shape, dt=BF)
    first = park.qk_norm_rope_bwd(*g, q, k, *w, rope=r)
    for _ in range(3):
        for a, b in zip(first, park.qk_norm_rope_bwd(*g, q, k, *w, rope=r)):
            assert torch.equal(a, b)
    inplace = park.qk_norm_rope_bwd(g[0].clone(), g[1].clone(), q, k, *w, rope=r)
    h = [t.clone() for t in g]
    park.qk_norm_rope_bwd(h[0], h[1], q, k, *w, rope=r, dq=h[0], dk=h[1])
    assert torch.equal(h[0], inplace[0]) and torch.equal(h[1], inplace[1])
    y = park.qk_norm_rope(q, k, *w, rope=r)
    park.qk_norm_rope(q, k, *w, rope=r, q_out=q, k_out=k)
    assert torch.equal(q, y[0]) and torch.equal(k, y[1])


def test_norm_rope_zero_rows_and_no_rows():
    q = rand(60, 1, 2, 5, 64)
    q[:, :, 2] = 0
    y, _ = park.qk_norm_rope(q, q.clone())
    assert torch.equal(y[:, :, 2], torch.zeros_like(y[:, :, 2])) and y.isfinite().all()
    g = rand(61, 1, 2, 5, 64)
    dq, _, _, _ = park.qk_norm_rope_bwd(g, g, q, q)
    assert dq.isfinite().all()
    e = torch.empty(1, 2, 0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    assert park.qk_norm_rope(e, e)[0].shape == e.shape
    out = park.qk_norm_rope_bwd(e, e, e, e, w, w)
    assert torch.equal(out[2], torch.zeros(64, device="cuda")) and torch.equal(out[3], out[2])
    assert park.rope(e, park.rope_table((1, 1, 1), 64)).shape == e.shape


# ------------------------------------------------------------------ dense attention
def plain_attention(q, k, v, scale, causal, do=None):
    """One sequence, one head, float64: values and the magnitudes that the bounds need."""
    nq, nk = q.shape[0], k.shape[0]
    see = torch.ones(nq, nk, dtype=torch.bool, device=q.device)
    if causal:
        see = torch.arange(nk, device=q.device)[None] <= torch.arange(nq, device=q.device)[:, None] + (nk - nq)
    s = torch.where(see, q @ k.T * scale, -math.inf)
    lse = torch.logsumexp(s, 1) if nk else torch.full((nq,), -math.inf, device=q.device, dtype=torch.float64)
    p = torch.where(see, torch.exp(s - torch.where(lse.isinf(), 0.0, lse)[:, None]), 0.0)
    return see, p, lse, p @ v


def attn_check(q, k, v, got, lse, causal, scale, dt, do=None, grads=None, cu=None):
    """Compares every sequence and head of packed or batched tensors with the bounds.

    Scores: D products and sums in float32, ds = (D + 4) E scale |q|.|k| (the tensor
    cores' sums included), so p is off by 2 ds relative (numerator and sum) + 8 E for the
    exponential and the sum.  bf16: p rounds once before its product with v (U of each
    term), and its exponential is a polynomial good to 2^-18.5 < 48 E (far below the 2^-8
    that follows), in numerator and sum: 96 E in the place of 8."""
    ex = 96 if dt == BF else 8
    B, Hq, Hk = q.shape[0], q.shape[1], k.shape[1]
    u, up = U[dt], (U[BF] if dt == BF else 0.0)
    D = q.shape[-1]
    seqs = [(b, slice(None), slice(None)) for b in range(B)] if cu is None else \
        [(0, slice(a, b), slice(c, d)) for a, b, c, d in zip(cu[0][:-1], cu[0][1:], cu[1][:-1], cu[1][1:])]
    for b, rq, rk in seqs:
        for hk in range(Hk):
            kk, vv = k[b, hk, rk].double(), v[b, hk, rk].double()
            dk, dv, tk, tv = (torch.zeros_like(kk) for _ in range(4))
            for h in range(hk * (Hq // Hk), (hk + 1) * (Hq // Hk)):
                qq = q[b, h, rq].double()
                see, p, want_lse, o = plain_attention(qq, kk, vv, scale, causal)
                if qq.shape[0] == 0:
                    continue
                es = (D + 4) * E * abs(scale) * (qq.abs() @ kk.abs().T)
                rel = 2 * torch.where(see, es, 0.0).amax(1, keepdim=True) if kk.shape[0] else torch.zeros_like(qq[:, :1])
                rel = rel + (ex + math.log2(max(2, kk.shape[0]))) * E + kk.shape[0] * E
                ov = p @ vv.abs()
                tol_o = u * o.abs() + (up + rel) * ov + 1e-37
                within(got[b, h, rq], o, tol_o, f"o {b} {h} {rq}")
                if lse is not None:
                    dead = want_lse.isinf()
                    assert torch.equal(lse[b, h, rq][dead].double(), want_lse[dead])
                    within(lse[b, h, rq][~dead], want_lse[~dead], (rel[:, 0] + 4 * E * (1 + want_lse.abs()))[~dead], "lse")
                if do is None:
                    continue
                g = do[b, h, rq].double()
                dp = g @ vv.T
                delta = (g * o).sum(1, keepdim=True)
                ds = p * (dp - delta)
                # p from the stored lse: the score's error, lse's (rel + 4 E (1 + |lse|))
                lz = torch.where(want_lse.isinf(), 0.0, want_lse)[:, None]
                rp = torch.where(see, es, 0.0) + rel + 4 * E * (1 + lz.abs()) + ex * E
                # dp: D products and sums; delta: from the stored o (its bound), D products and sums
                edp = (D + 4) * E * (g.abs() @ vv.abs().T)
                edel = (g.abs() * tol_o).sum(1, keepdim=True) + (D + 4) * E * (g * o).abs().sum(1, keepdim=True)
                eds = rp * ds.abs() + p * (1 + rp) * (edp + edel) + (up + 4 * E) * ds.abs()
                eds = eds + up * p * (edp + edel)
                # a p below 2^-126 becomes 0, in either type's exponent range: off by less than 2^-126 for each
                # pair, which the relative terms above do not count (they scale with p)
                eds = eds + torch.where(see, TINY * (dp.abs() + delta.abs()), 0.0)
                dq = scale * ds @ kk
                n_k = kk.shape[0]
                tol = u * dq.abs() + abs(scale) * (eds @ kk.abs() + (n_k + 4) * E * (ds.abs() @ kk.abs())) + 1e-37
                within(grads[0][b, h, rq], dq, tol, f"dq {b} {h} {rq}")
                dk += scale * ds.T @ qq
                dv += p.T @ g
                n_q = qq.shape[0] * (Hq // Hk)
                tk += abs(scale) * (eds.T @ qq.abs() + (n_q + 4) * E * (ds.abs().T @ qq.abs()))
                tv += ((rp + up) * p + TINY * see).T @ g.abs() + (n_q + 4) * E * (p.T @ g.abs())
            if do is not None:
                within(grads[1][b, hk, rk], dk, u * dk.abs() + tk + 1e-37, f"dk {b} {hk} {rk}")
                within(grads[2][b, hk, rk], dv, u * dv.abs() + tv + 1e-37, f"dv {b} {hk} {rk}")


def cu_of(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()


BATCHED = [
    # B, Hq, Hk, Nq, Nk, D, causal, dtype, layout
    (1, 1, 1, 1, 1, 64, False, BF, "heads"),
    (1, 1, 1, 256, 256, 64, False, F32, "heads"),
    (2, 4, 2, 130, 130, 128, True, BF, "tokens"),
    (2, 6, 2, 61, 190, 96, True, F32, "fused"),
    (1, 3, 1, 257, 129, 128, True, BF, "fused"),      # 128 rows see no key
    (1, 2, 2, 300, 77, 32, False, BF, "heads"),
    (2, 2, 1, 1, 515, 128, True, BF, "tokens"),       # single rows over many keys
    (1, 8, 2, 3, 1000, 96, False, BF, "tokens"),
    (1, 4, 4, 384, 640, 128, False, BF, "heads"),
    (1, 2, 1, 513, 513, 64, True, BF, "heads"),
    (1, 2, 1, 100, 40, 64, True, F32, "tokens"),      # 60 rows see no key
    (3, 1, 1, 200, 1, 128, False, BF, "heads"),
    (1, 5, 1, 700, 700, 96, True, BF, "tokens"),
]


def attn_inputs(B, Hq, Hk, Nq, Nk, D, dt, kind, seed=100):
    q, k, v, do = (layout(rand(seed + i, B, h, n, D, dt=dt), kind)
                   for i, (h, n) in enumerate(((Hq, Nq), (Hk, Nk), (Hk, Nk), (Hq, Nq))))
    return q, k, v, do


@pytest.mark.parametrize("B,Hq,Hk,Nq,Nk,D,causal,dt,kind", BATCHED)
def test_attention_batched(B, Hq, Hk, Nq, Nk, D, causal, dt, kind):
    q, k, v, do = attn_inputs(B, Hq, Hk, Nq, Nk, D, dt, kind)
    o, lse = park.attention(q, k, v, causal=causal, return_lse=True)
    attn_check(q, k, v, o, lse, causal, D ** -0.5, dt)
    assert torch.equal(o, park.attention(q, k, v, causal=causal))
    grads = park.attention_bwd(do, q, k, v, o, lse, causal=causal)
    attn_check(q, k, v, o, lse, causal, D ** -0.5, dt, do, grads)


PACKED = [
    (4, 2, [1500, 3, 700], [77, 200, 1], 128, False, BF, "tokens"),       # many rows over few keys: split over the rows
    (2, 1, [1500, 0, 900, 130], [60, 10, 1000, 0], 64, True, BF, "heads"),
    (4, 2, [900, 3, 400], [77, 100, 1], 96, False, F32, "tokens"),
    (2, 1, [5, 1, 40, 2], [900, 300, 1, 0], 128, True, F32, "heads"),     # few rows over many keys in float32
    # Hq, Hk, lq, lk, D, causal, dtype, layout
    (4, 2, [5, 0, 131, 1, 64, 300], [5, 0, 131, 1, 64, 300], 128, True, BF, "tokens"),
    (2, 1, [17, 3, 0, 200], [0, 140, 9, 33], 64, True, BF, "heads"),      # no keys, no queries, more queries than keys
    (2, 2, [128, 128, 256], [128, 128, 256], 128, False, BF, "fused"),
    (6, 2, [1, 1, 2, 1], [700, 3, 129, 1], 96, True, BF, "tokens"),
    (3, 3, [40, 1, 90], [40, 1, 90], 96, True, F32, "tokens"),
    (2, 1, [0, 7, 65], [12, 0, 130], 32, False, F32, "heads"),
    (2, 1, [1, 0, 2] * 100, [2, 5, 1] * 100, 64, True, BF, "heads"),
    (2, 1, [3] * 33, [1] * 33, 32, True, F32, "heads"),
    (2, 1, [3] * 70, [4] * 70, 64, True, BF, "heads"),                    # more sequences than a warp scans at once
]


@pytest.mark.parametrize("Hq,Hk,lq,lk,D,causal,dt,kind", PACKED)
def test_attention_packed(Hq, Hk, lq, lk, D, causal, dt, kind):
    tail = 9                                        # rows behind the last sequence
    nq, nk = sum(lq) + tail, sum(lk) + tail
    q, k, v, do = attn_inputs(1, Hq, Hk, nq, nk, D, dt, kind)
    for t, n in ((q, nq), (k, nk), (v, nk), (do, nq)):
        t[:, :, n - tail:] = float("nan")           # and they hold anything
    cu_q, cu_k = cu_of(lq), cu_of(lk)
    kw = dict(causal=causal, scale=0.3, cu_q=cu_q, cu_k=cu_k)
    O = torch.full_like(q, 7.0)
    L = torch.full(q.shape[:3], 7.0, device="cuda")
    o, lse = park.attention(q, k, v, O=O, lse=L, return_lse=True, **kw)
    assert o is O and lse is L
    assert (O[:, :, nq - tail:] == 7).all() and (L[:, :, nq - tail:] == 7).all()
    outs = [torch.full_like(t, 7.0) for t in (q, k, v)]
    grads = park.attention_bwd(do, q, k, v, o, lse, dQ=outs[0], dK=outs[1], dV=outs[2], **kw)
    for t, n in zip(grads, (nq, nk, nk)):
        assert (t[:, :, n - tail:] == 7).all()
    attn_check(q, k, v, o, lse, causal, 0.3, dt, do, grads, (cu_q.tolist(), cu_k.tolist()))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_hidden_keys_and_values_do_not_reach_a_row(dt, bad):
    """A key row, a value row and (for dk, dv) query and gradient rows behind the mask hold NaN or infinities."""
    n, D, at = 300, 128, 205
    q, k, v, do = attn_inputs(1, 2, 1, n, n, D, dt, "tokens")
    good, glse = park.attention(q, k, v, causal=True, return_lse=True)
    ggrads = park.attention_bwd(do, q, k, v, good, glse, causal=True)
    k2, v2 = k.clone(), v.clone()
    v2[:, :, at, 3:9] = bad                          # rows before `at` do not see it
    k2[:, :, at] = bad
    o, lse = park.attention(q, k2, v2, causal=True, return_lse=True)
    assert torch.equal(o[:, :, :at], good[:, :, :at]) and torch.equal(lse[:, :, :at], glse[:, :, :at])
    grads = park.attention_bwd(do, q, k2, v2, o, lse, causal=True)
    assert torch.equal(grads[0][:, :, :at], ggrads[0][:, :, :at])
    # with only a value row bad, the rows that see it hold it in those columns alone
    o, _ = park.attention(q, k, v2, causal=True, return_lse=True)
    assert torch.equal(o[:, :, :at], good[:, :, :at])
    assert not o[:, :, at:, 3:9].isfinite().any()
    assert torch.equal(o[:, :, at:, 9:], good[:, :, at:, 9:]) and torch.equal(o[:, :, at:, :3], good[:, :, at:, :3])
    # a query row and its gradient: keys behind it do not see it
    q2, do2 = q.clone(), do.clone()
    q2[:, :, at - 100] = bad
    do2[:, :, at - 100, 5] = bad
    o, lse = park.attention(q2, k, v, causal=True, return_lse=True)
    grads = park.attention_bwd(do2, q2, k, v, o, lse, causal=True)
    hidden = slice(at - 99, n)
    assert torch.equal(grads[1][:, :, hidden], ggrads[1][:, :, hidden])
    assert torch.equal(grads[2][:, :, hidden], ggrads[2][:, :, hidden])


def test_gradient_of_a_dominant_key():
    """Every row gives one key a p halfway between two bf16 numbers: rounded to bf16 it would be 2^-8 off in every term of
    dv, in the same direction.  A key like that gets 16 bits from its third step of 128 rows on, so the sum over 4,096 rows is
    off by 256 / 4096 of 2^-8, 2^-16 for the second rounding, p's own error and the sum's: the result is the rounding of
    a number within that of the value."""
    n, D, at = 4096, 128, 77
    scale = float(np.float32(math.log(0.501953125 / 0.498046875 * (n - 1)) / 8))
    q, k, v = torch.zeros(1, 1, n, D), torch.zeros(1, 1, n, D), rand(330, 1, 1, n, D, dt=BF)
    q[..., 0], k[0, 0, at, 0] = 1, 8
    q, k = q.to(BF).cuda(), k.to(BF).cuda()
    do = rand(331, 1, 1, 1, D, dt=BF).expand(1, 1, n, D).contiguous()
    o, lse = park.attention(q, k, v, scale=scale, return_lse=True)
    dv = park.attention_bwd(do, q, k, v, o, lse, scale=scale)[2][0, 0, at].double()
    t = 8 * scale
    p = 1 / (1 + (n - 1) * math.exp(-t))
    want = n * p * do[0, 0, 0].double()
    es = (D + 4) * E * t
    rp = es + 2 * es + (96 + math.log2(n)) * E + n * E + 4 * E * (1 + t) + 96 * E
    e = (256 / n * U[BF] + 2 ** -16 + rp + (n + 4) * E) * want.abs()
    low, high = (want - e).to(BF).double(), (want + e).to(BF).double()
    assert ((dv >= low) & (dv <= high)).all()
    # the bound tells the difference: most columns would be outside with p rounded once
    once = (want * (0.5 / p)).to(BF).double()
    assert ((once < low) | (once > high)).float().mean() > 0.5


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_dominant_keys_in_every_place(causal, D):
    """Keys that draw most of the attention in whole and in cut tiles, for heads that share them, packed."""
    lens = [2300, 40, 1000]
    N = sum(lens)
    q, k, v, do = (rand(340 + i, 1, h, N, D, dt=BF) for i, h in enumerate((4, 2, 2, 4)))
    u = rand(345, D)
    q = (q + 0.7 * u).to(BF)
    for key in (0, 130, 2299, 2320, 2340, 2700):
        k[0, :, key] = (u * (5 + key % 3)).to(BF)
    cu = cu_of(lens)
    o, lse = park.attention(q, k, v, causal=causal, cu_q=cu, cu_k=cu, return_lse=True)
    grads = park.attention_bwd(do, q, k, v, o, lse, causal=causal, cu_q=cu, cu_k=cu)
    bounds = cu.tolist()
    attn_check(q, k, v, o, lse, causal, 1 / math.sqrt(D), BF, do, grads, (bounds, bounds))
    again = park.attention_bwd(do, q, k, v, o, lse, causal=causal, cu_q=cu, cu_k=cu)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


def test_attention_scores_of_large_range():
    """Scores over hundreds of log2 units: the running maximum moves by far more than a tile's spread."""
    n, D = 600, 128
    q, k, v, do = attn_inputs(1, 1, 1, n, n, D, BF, "heads")
    ramp = torch.linspace(-6, 6, n, device="cuda")
    k = (k * 0.1 + (ramp[:, None] * torch.sign(rand(3, D)))[None, None]).to(BF)
    q = (torch.sign(rand(3, D)) + 0.1 * q.float()).to(BF)
    o, lse = park.attention(q, k, v, return_lse=True)
    attn_check(q, k, v, o, lse, False, D ** -0.5, BF)
    kr = k.flip(2).contiguous()
    o, lse = park.attention(q, kr, v, return_lse=True)
    grads = park.attention_bwd(do, q, kr, v, o, lse)
    attn_check(q, kr, v, o, lse, False, D ** -0.5, BF, do, grads)


def test_attention_gradient_against_differences():
    n, D, scale = 33, 32, 0.2
    q, k, v, do = attn_inputs(1, 2, 1, n, n + 4, D, F32, "heads")
    do = do[:, :, :n]
    o, lse = park.attention(q, k, v, causal=True, scale=scale, return_lse=True)
    grads = park.attention_bwd(do, q, k, v, o, lse, causal=True, scale=scale)
    base = [t.double() for t in (q, k, v)]

    def loss(a, b, c):
        return sum((plain_attention(a[0, h], b[0, 0], c[0, 0], scale, True)[3] * do[0, h].double()).sum() for h in range(2))
    for i in range(3):
        d = rand(70 + i, *base[i].shape).double()
        step = 1e-5
        up = loss(*[b + step * d if j == i else b for j, b in enumerate(base)])
        dn = loss(*[b - step * d if j == i else b for j, b in enumerate(base)])
        got = (grads[i].double() * d).sum()
        assert abs(got - (up - dn) / (2 * step)) <= 1e-5 * (grads[i].double() * d).abs().sum()


def test_attention_same_bits():
    q, k, v, do = attn_inputs(1, 6, 2, 500, 500, 128, BF, "heads")
    o, lse = park.attention(q, k, v, causal=True, return_lse=True)
    g = park.attention_bwd(do, q, k, v, o, lse, causal=True)
    for _ in range(3):
        o2, lse2 = park.attention(q, k, v, causal=True, return_lse=True)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        for a, b in zip(g, park.attention_bwd(do, q, k, v, o, lse, causal=True)):
            assert torch.equal(a, b)


def test_attention_bad_bounds_are_reported():
    """Sequences whose bounds fall, or leave the tensors, are skipped; the others are right."""
    q, k, v, do = attn_inputs(1, 2, 2, 100, 100, 64, BF, "heads")
    cu_q = torch.tensor([0, 40, 30, 30, 101], dtype=torch.int32).cuda()
    cu_k = torch.tensor([0, 40, 50, 60, 100], dtype=torch.int32).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    O = torch.full_like(q, 7.0)
    o, lse = park.attention(q, k, v, cu_q=cu_q, cu_k=cu_k, O=O, return_lse=True, status=status)
    assert status.item() == _lib.PARK_ERR_INDEX
    assert (O[:, :, 40:] == 7).all()
    attn_check(q[:, :, :40], k[:, :, :40], v[:, :, :40], O[:, :, :40], lse[:, :, :40], False, 0.125, BF)
    status.zero_()
    park.attention_bwd(do, q, k, v, o, lse, cu_q=cu_q, cu_k=cu_k, status=status)
    assert status.item() == _lib.PARK_ERR_INDEX


def test_attention_refuses():
    q, k, v, do = attn_inputs(1, 4, 2, 32, 32, 64, BF, "heads")
    with pytest.raises(ValueError):
        park.attention(q, k[:, :1].expand(1, 2, 32, 64), v)
    with pytest.raises(ValueError):
        park.attention(q[:, :3], k, v)
    with pytest.raises(TypeError):
        park.attention(q, k.float(), v)
    with pytest.raises(ValueError):
        park.attention(q, k, v[:, :, :31])
    with pytest.raises(ValueError):
        park.attention(q, k, v, cu_q=cu_of([32]))
    with pytest.raises(ValueError):
        park.attention(q, k, v, cu_q=cu_of([32])[:1], cu_k=cu_of([32])[:1])
    with pytest.raises(ValueError):
        park.attention(q, k, v, cu_q=cu_of([32]).long(), cu_k=cu_of([32]).long())
    with pytest.raises(ValueError):
        park.attention(torch.cat([q, q]), torch.cat([k, k]), torch.cat([v, v]), cu_q=cu_of([32]), cu_k=cu_of([32]))
    with pytest.raises(ValueError):
        park.attention(q[..., 1:33], k[..., 1:33], v[..., 1:33])
    with pytest.raises(ValueError):
        park.attention(q, k, v, O=torch.empty(1, 4, 1, 64, dtype=BF, device="cuda").expand(1, 4, 32, 64))
    with pytest.raises(_lib.ParkError):
        park.attention(q, k, v, scale=float("nan"))


def test_empty_sides():
    e = torch.empty(1, 2, 0, 64, dtype=BF, device="cuda")
    x, do = rand(1, 1, 2, 5, 64, dt=BF), rand(2, 1, 2, 5, 64, dt=BF)
    assert park.attention(e, x, x).shape == e.shape
    o, lse = park.attention(x, e, e, return_lse=True)
    assert torch.equal(o, torch.zeros_like(o)) and (lse == -math.inf).all()
    dq, dk, dv = park.attention_bwd(do, x, e, e, o, lse)
    assert torch.equal(dq, torch.zeros_like(dq)) and dk.shape == e.shape
    oe, le = park.attention(e, x, x, return_lse=True)
    dq, dk, dv = park.attention_bwd(e, e, x, x, oe, le)
    assert torch.equal(dk, torch.zeros_like(dk)) and torch.equal(dv, torch.zeros_like(dv))


# ------------------------------------------------------------------ streams, graphs, sizes
def test_other_stream_and_two_calls_at_once():
    q, k, v, do = attn_inputs(1, 4, 4, 700, 700, 128, BF, "heads")
    want = park.attention(q, k, v)
    w = torch.ones(128, device="cuda")
    r = park.rope_table((7, 10, 10), 128)
    want_n = park.qk_norm_rope(q, k, w, w, rope=r)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [(park.attention(q, k, v, stream=s), park.qk_norm_rope(q, k, w, w, rope=r, stream=s)) for s in streams]
    torch.cuda.synchronize()
    for o, n in got:
        assert torch.equal(o, want) and torch.equal(n[0], want_n[0]) and torch.equal(n[1], want_n[1])


def test_captured_and_replayed():
    """A whole training step of norm, rotation and attention in a graph, replayed on new inputs."""
    B, H, n, D = 1, 4, 333, 128
    r = park.rope_table((3, 10, 11), D)
    w = torch.ones(D, device="cuda", dtype=BF)
    x = [rand(200 + i, B, H, n, D, dt=BF) for i in range(4)]

    def step(q, k, v, do):
        a, b = park.qk_norm_rope(q, k, w, w, rope=r)
        o, lse = park.attention(a, b, v, causal=True, return_lse=True)
        da, db, dv = park.attention_bwd(do, a, b, v, o, lse, causal=True)
        return (o, dv, *park.qk_norm_rope_bwd(da, db, q, k, w, w, rope=r))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(*x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*x)
    for seed in (300, 400):
        for i, t in enumerate(x):
            t.copy_(rand(seed + i, B, H, n, D, dt=BF))
        want = step(*x)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)


def test_offsets_beyond_32_bits():
    """Heads more than 2^31 elements apart."""
    n, D, gap = 130, 128, (1 << 31) + 4096
    buf = torch.empty(gap + n * D, dtype=BF, device="cuda")
    far = torch.as_strided(buf, (1, 2, n, D), (2 * gap, gap, D, 1))
    q, k, v, do = attn_inputs(1, 2, 2, n, n, D, BF, "heads")
    r = park.rope_table((1, 13, 10), D)
    want = park.attention(q, k, v, causal=True, return_lse=True)
    grads = park.attention_bwd(do, q, k, v, *want, causal=True)
    turned, normed = park.rope(q, r), park.qk_norm_rope(q, k, rope=r)
    far.copy_(q)
    assert torch.equal(park.rope(far, r), turned)
    assert torch.equal(park.qk_norm_rope(far, k, rope=r)[0], normed[0])
    assert torch.equal(park.attention(far, k, v, causal=True), want[0])
    assert torch.equal(park.attention_bwd(do, far, k, v, *want, causal=True)[1], grads[1])
    far.copy_(k)
    assert torch.equal(park.attention(q, far, v, causal=True), want[0])
    O = far
    park.attention(q, k, v, causal=True, O=O)
    assert torch.equal(O, want[0])
    park.attention_bwd(do, q, k, v, *want, causal=True, dQ=O)
    assert torch.equal(O, grads[0])


@pytest.mark.parametrize("nq,nk", [(600, 900), (40000, 300)])   # one and two row tiles in a block
def test_waits_that_run_out_are_reported(nq, nk):
    """With the wait limit at 1 ns the tensor-core kernels report the timeout and end; the next call is right."""
    q, k, v, do = attn_inputs(1, 2, 2, nq, nk, 128, BF, "heads")
    want, lse = park.attention(q, k, v, return_lse=True)
    grads = park.attention_bwd(do, q, k, v, want, lse)
    torch.cuda.synchronize()
    for call in (lambda s: park.attention(q, k, v, status=s),
                 lambda s: park.attention_bwd(do, q, k, v, want, lse, status=s)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        park.set_wait_limit_ns(1)
        try:
            call(status)
            torch.cuda.synchronize()
        finally:
            park.set_wait_limit_ns(0)
        assert status.item() == _lib.PARK_ERR_TIMEOUT
        assert torch.equal(park.attention(q, k, v), want)
        for a, b in zip(park.attention_bwd(do, q, k, v, want, lse), grads):
            assert torch.equal(a, b)


# ------------------------------------------------------------------ together
def test_layer_with_norm_and_rotation():
    """layer(pre=...) from a fused projection equals the steps taken one by one."""
    B, H, T, Hg, W, text, D = 1, 2, 4, 8, 8, 16, 128
    shape = park.Shape(B, H, T, Hg, W, text, D)
    qkv = rand(500, B, shape.N, 3, H, D, dt=BF)
    q, k = (qkv[:, :, i].transpose(1, 2) for i in range(2))
    v = qkv[:, :, 2].transpose(1, 2).contiguous()
    w = [(1 + 0.1 * rand(501 + i, D)).to(BF) for i in range(2)]
    r = park.rope_table((T, Hg, W), D)
    a, b = park.qk_norm_rope(q, k, *w, rope=r)
    want, rw = park.layer(a, b, v, shape, 8, 8, 0.9, 3)
    got, rg = park.layer(q, k, v, shape, 8, 8, 0.9, 3, pre=park.NormRope(*w, rope=r))
    torch.cuda.synchronize()
    assert rw.status_code() == 0 and rg.status_code() == 0
    assert torch.equal(got, want) and torch.equal(rw.mask, rg.mask)
    only, _ = park.layer(q, k, v, shape, 8, 8, 0.9, 3, pre=park.NormRope(rope=r, norm=False))
    a, b = park.rope(q, r).contiguous(), park.rope(k, r).contiguous()
    want, _ = park.layer(a, b, v, shape, 8, 8, 0.9, 3)
    assert torch.equal(only, want)


def test_dense_attention_equals_the_sparse_layer_with_every_block_kept():
    """p = 1 keeps every block: both are softmax attention over all keys of the same rows."""
    B, H, T, Hg, W, text, D = 1, 3, 4, 8, 8, 19, 128
    shape = park.Shape(B, H, T, Hg, W, text, D)
    q, k, v = (rand(510 + i, B, H, shape.N, D, dt=BF) for i in range(3))
    sparse, r = park.layer(q, k, v, shape, 8, 8, 1.0, 2)
    dense = park.attention(q, k, v)
    torch.cuda.synchronize()
    assert r.status_code() == 0
    # each within its own roundings of the exact value: p and o once each, twice over
    for h in range(H):
        _, p, _, o = plain_attention(q[0, h].double(), k[0, h].double(), v[0, h].double(), D ** -0.5, False)
        tol = 2 * U[BF] * (o.abs() + p @ v[0, h].double().abs()) * 1.05
        assert ((sparse[0, h].double() - dense[0, h].double()).abs() <= tol).all()


@pytest.mark.parametrize("G", [1, 3])
def test_single_rows_over_long_keys(G):
    """The split over the keys at its usual lengths, first call on new memory and again."""
    lk = [30000, 1, 17777, 257, 4096]
    q, k, v, _ = attn_inputs(1, 4 * G, 4, len(lk), sum(lk), 128, BF, "tokens", seed=600)
    kw = dict(cu_q=cu_of([1] * len(lk)), cu_k=cu_of(lk), causal=True)
    first, lse = park.attention(q, k, v, return_lse=True, **kw)
    attn_check(q, k, v, first, lse, True, 128 ** -0.5, BF, cu=(kw["cu_q"].tolist(), kw["cu_k"].tolist()))
    for _ in range(20):
        k = k.clone()
        assert torch.equal(park.attention(q, k, v, **kw), first)
