"""The operators at the sizes where a real layer's instances of the kernels run: warps that walk many heads of a token,
rings that wrap, blocks of 256 query rows with both halves live, groups of heads.  Same float64 forms and bounds as
test_gpu_ops.py, whose cases are small."""
import pytest
import torch

import block_sparse_attention_means_b200 as park
import test_gpu_ops as base
from test_gpu_ops import BF, F32, attn_check, attn_inputs, clean_status, cu_of, layout, rand  # noqa: F401

pytestmark = pytest.mark.gpu

# From 32 x 148 = 4,736 tokens on a warp walks all heads of a token; a few hundred tokens give it some of them.  A step
# of a warp is 32 / (lanes of a row) heads (8, 4, 2, 2 at D = 32, 64, 96, 128), 4 steps are in flight in bf16 and 2 in
# float32: head counts that are no multiple of either, with more than one turn of the loop.
GRID, TEXT = (9, 12, 22), 24                      # 2,400 tokens
LONG = [
    # B, H, Hk, extent, text, D, half, dtype, weights, layout
    (2, 11, 5, GRID, TEXT, 128, False, BF, BF, "fused"),
    (2, 11, 5, GRID, TEXT, 128, True, F32, F32, "tokens"),
    (2, 19, 5, GRID, TEXT, 64, True, BF, F32, "heads"),
    (2, 19, 7, GRID, TEXT, 64, False, F32, None, "fused"),
    (2, 11, 3, GRID, TEXT, 96, True, BF, BF, "tokens"),
    (2, 11, 5, GRID, TEXT, 96, False, F32, F32, "heads"),
    (2, 37, 9, GRID, TEXT, 32, False, BF, None, "tokens"),
    (2, 37, 9, GRID, TEXT, 32, True, F32, BF, "fused"),
    (1, 40, 8, (5, 8, 14), 40, 128, True, BF, BF, "fused"),      # 600 tokens: 6 heads a warp
    (1, 40, 40, (5, 20, 19), 100, 96, False, F32, F32, "heads"),  # 2,000 tokens: 14 heads a warp
]


@pytest.mark.parametrize("B,H,Hk,extent,text,D,half,dt,wdt,kind", LONG)
def test_rope_many_heads(B, H, Hk, extent, text, D, half, dt, wdt, kind):
    for inverse in (False, True):
        base.test_rope_grid(B, H, extent, text, D, half, dt, kind, inverse)
    x = rand(1, B, H, 2 * 3 * 5, D, dt=dt)
    r = park.rope_table((2, 3, 5), D, half=half)
    y = park.rope(x, r)
    assert torch.equal(park.rope(x, r, out=x), y)


@pytest.mark.parametrize("B,H,Hk,extent,text,D,half,dt,wdt,kind", LONG)
def test_norm_rope_many_heads(B, H, Hk, extent, text, D, half, dt, wdt, kind):
    base.test_norm_rope(B, H, Hk, extent, text, D, half, dt, wdt, kind)


@pytest.mark.parametrize("B,H,Hk,extent,text,D,half,dt,wdt,kind", LONG)
def test_norm_rope_backward_many_heads(B, H, Hk, extent, text, D, half, dt, wdt, kind):
    base.test_norm_rope_backward(B, H, Hk, extent, text, D, half, dt, wdt, kind)


@pytest.mark.parametrize("B,H,Hk,extent,text,D,half,dt,wdt,kind", LONG)
def test_in_place_many_heads(B, H, Hk, extent, text, D, half, dt, wdt, kind):
    """Rows are read ahead of those that are written: onto the inputs the same bits come out."""
    n, q, k, w, r, c, s = base.norm_inputs(B, H, Hk, extent, text, D, half, dt, wdt, kind)
    gq, gk = layout(rand(20, B, H, n, D, dt=dt), kind), layout(rand(21, B, Hk, n, D, dt=dt), kind)
    turned = park.rope(q, r)
    y = park.qk_norm_rope(q, k, *w, rope=r)
    grads = park.qk_norm_rope_bwd(gq, gk, q, k, *w, rope=r)
    again = park.qk_norm_rope_bwd(gq, gk, q, k, *w, rope=r, dq=gq, dk=gk)
    assert all(a is None and b is None or torch.equal(a, b) for a, b in zip(grads, again))
    keep = q.clone()
    assert torch.equal(park.rope(q, r, out=q), turned)
    q.copy_(keep)
    park.qk_norm_rope(q, k, *w, rope=r, q_out=q, k_out=k)
    assert torch.equal(q, y[0]) and torch.equal(k, y[1])


# ------------------------------------------------------------------ dense attention
def check_attention(want, q, k, v, do, dt, **kw):
    """Forward and backward within the bounds, through the forward instance of `want` rows."""
    D = q.shape[-1]
    park.profile_enable(True)
    try:
        o, lse = park.attention(q, k, v, return_lse=True, **kw)
        torch.cuda.synchronize()
        ran = [n for n in park.profile_collect() if n.startswith("k_dense_fwd")]
    finally:
        park.profile_enable(False)
    assert ran == [("k_dense_fwd_tc, " if dt == BF else "k_dense_fwd_simt, ") + f"{want} rows"]
    grads = park.attention_bwd(do, q, k, v, o, lse, **kw)
    cu = None if kw.get("cu_q") is None else (kw["cu_q"].tolist(), kw["cu_k"].tolist())
    attn_check(q, k, v, o, lse, kw.get("causal", False), D ** -0.5, dt, do, grads, cu)


BATCHED = [
    # rows of a block, B, Hq, Hk, Nq, Nk, D, causal, dtype, layout
    (256, 1, 40, 40, 600, 600, 128, False, BF, "heads"),
    (256, 1, 40, 40, 600, 600, 128, True, BF, "fused"),
    (256, 1, 40, 40, 600, 600, 64, False, BF, "tokens"),
    (256, 1, 40, 40, 600, 600, 64, True, BF, "heads"),
    (256, 1, 48, 16, 600, 1100, 128, True, BF, "tokens"),     # three heads side by side, 5 to 9 key tiles
    (256, 1, 48, 16, 600, 700, 64, True, BF, "fused"),
    (256, 2, 26, 13, 700, 520, 96, False, BF, "tokens"),
    (256, 1, 40, 40, 700, 300, 128, True, BF, "heads"),       # 400 rows see no key: whole first halves without work
    (256, 3, 16, 16, 401, 129, 32, True, BF, "heads"),
    (256, 1, 2, 2, 40000, 300, 128, False, BF, "heads"),
    (128, 1, 40, 40, 500, 500, 128, True, F32, "fused"),
    (128, 1, 40, 40, 500, 500, 128, False, F32, "heads"),
    (128, 1, 40, 40, 500, 700, 96, True, F32, "tokens"),
    (128, 1, 40, 40, 600, 250, 64, True, F32, "heads"),       # 350 rows see no key
    (128, 2, 48, 16, 300, 333, 64, False, F32, "fused"),
    (128, 1, 40, 40, 500, 500, 32, True, F32, "tokens"),
    (64, 1, 2, 2, 700, 700, 128, True, F32, "heads"),         # with split keys
    (64, 1, 2, 1, 700, 650, 64, True, F32, "tokens"),
    (64, 1, 2, 2, 700, 700, 32, False, F32, "fused"),
    (64, 1, 20, 20, 500, 450, 128, False, F32, "tokens"),     # without
    (64, 1, 20, 20, 500, 500, 64, True, F32, "heads"),
    (64, 1, 20, 20, 500, 500, 32, True, F32, "heads"),
]


@pytest.mark.parametrize("rows,B,Hq,Hk,Nq,Nk,D,causal,dt,kind", BATCHED)
def test_attention_large(rows, B, Hq, Hk, Nq, Nk, D, causal, dt, kind):
    check_attention(rows, *attn_inputs(B, Hq, Hk, Nq, Nk, D, dt, kind), dt, causal=causal)


PACKED = [
    # rows, Hq, Hk, lq, lk, D, causal, dtype, layout
    (256, 16, 16, [700, 500, 0, 611, 1, 450], [700, 500, 0, 611, 1, 450], 128, True, BF, "tokens"),
    (256, 24, 12, [600, 1, 900, 300], [420, 700, 1300, 0], 64, True, BF, "heads"),
    (256, 16, 16, [450, 30] * 17, [450, 70] * 17, 96, False, BF, "fused"),           # more sequences than a warp ranks
    (128, 24, 24, [700, 500, 0, 611, 1, 450], [700, 500, 0, 611, 1, 450], 128, True, F32, "tokens"),
    (128, 40, 20, [500, 130, 257], [77, 600, 257], 64, False, F32, "heads"),
    (64, 4, 2, [300, 70, 128], [300, 900, 128], 96, True, F32, "tokens"),
    # keys of all heads beyond 128 MB: more than one group of heads in the order of blocks
    (256, 40, 40, [6500, 300], [6500, 300], 128, True, BF, "heads"),
    (128, 40, 40, [3300, 101], [3300, 101], 128, True, F32, "tokens"),
]


@pytest.mark.parametrize("rows,Hq,Hk,lq,lk,D,causal,dt,kind", PACKED)
def test_attention_packed_large(rows, Hq, Hk, lq, lk, D, causal, dt, kind):
    check_attention(rows, *attn_inputs(1, Hq, Hk, sum(lq), sum(lk), D, dt, kind), dt, causal=causal, cu_q=cu_of(lq),
                    cu_k=cu_of(lk))


@pytest.mark.parametrize("D", [32, 64, 96, 128])
@pytest.mark.parametrize("G", [1, 3])
def test_float32_single_rows_over_long_keys(G, D):
    lk = [20000, 1, 7777, 257]
    q, k, v, do = attn_inputs(1, 2 * G, 2, len(lk), sum(lk), D, F32, "tokens", seed=600)
    check_attention(16, q, k, v, do, F32, causal=True, cu_q=cu_of([1] * len(lk)), cu_k=cu_of(lk))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_hidden_rows_in_large_blocks(dt, bad, D):
    """Keys, values, queries and gradients behind the mask hold NaN or infinities (blocks of 256 rows, 128 in float32)."""
    n, at, H, Hk = 600, 405, 40, 20
    q, k, v, do = attn_inputs(1, H, Hk, n, n, D, dt, "tokens")
    good, glse = park.attention(q, k, v, causal=True, return_lse=True)
    ggrads = park.attention_bwd(do, q, k, v, good, glse, causal=True)
    k2, v2 = k.clone(), v.clone()
    v2[:, :, at, 3:9] = bad                          # rows before `at` do not see it
    k2[:, :, at] = bad
    o, lse = park.attention(q, k2, v2, causal=True, return_lse=True)
    assert torch.equal(o[:, :, :at], good[:, :, :at]) and torch.equal(lse[:, :, :at], glse[:, :, :at])
    grads = park.attention_bwd(do, q, k2, v2, o, lse, causal=True)
    assert torch.equal(grads[0][:, :, :at], ggrads[0][:, :, :at])
    o, _ = park.attention(q, k, v2, causal=True, return_lse=True)
    assert torch.equal(o[:, :, :at], good[:, :, :at]) and not o[:, :, at:, 3:9].isfinite().any()
    assert torch.equal(o[:, :, at:, 9:], good[:, :, at:, 9:]) and torch.equal(o[:, :, at:, :3], good[:, :, at:, :3])
    q2, do2 = q.clone(), do.clone()
    q2[:, :, at - 200] = bad
    do2[:, :, at - 200, 5] = bad
    o, lse = park.attention(q2, k, v, causal=True, return_lse=True)
    grads = park.attention_bwd(do2, q2, k, v, o, lse, causal=True)
    for i in (1, 2):
        assert torch.equal(grads[i][:, :, at - 199:], ggrads[i][:, :, at - 199:])
