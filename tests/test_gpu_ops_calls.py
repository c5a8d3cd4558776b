"""Calls of the operators and of layer(pre=...) beyond the plain one: rows of NaN where the keys are split, conditions
that reach the result's status, objects made on one stream and used on another."""
import math

import pytest
import torch

import block_sparse_attention_means_b200 as park
from block_sparse_attention_means_b200 import _lib
from test_gpu_ops import BF, F32, angles, attn_inputs, clean_status, grid_positions, pair_mass, plain_rotate, rand, within  # noqa: F401
from test_gpu_ops import E, U

pytestmark = pytest.mark.gpu


# 3 to 4 parts (joined by one warp a row) and more than 4 (by eight); 300 x 300 x 30 is not split
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("H,nq,nk", [(1, 2, 1000), (1, 2, 6000), (30, 300, 300)])
def test_a_query_row_of_nan(dt, H, nq, nk):
    """Its o and lse are NaN however the keys are split; the other rows keep their bits."""
    q, k, v, _ = attn_inputs(1, H, H, nq, nk, 64, dt, "heads")
    good, glse = park.attention(q, k, v, return_lse=True)
    q[0, 0, 1] = float("nan")
    o, lse = park.attention(q, k, v, return_lse=True)
    assert o[0, 0, 1].isnan().all() and lse[0, 0, 1].isnan()
    keep = torch.ones(1, H, nq, dtype=torch.bool, device="cuda")
    keep[0, 0, 1] = False
    assert torch.equal(o[keep], good[keep]) and torch.equal(lse[keep], glse[keep])


@pytest.mark.parametrize("norm", [True, False])
def test_layer_reports_what_pre_meets(norm):
    """A position out of range leaves its token unrotated: the layer's own result says so, the next one is good again."""
    B, H, T, Hg, W, text, D = 1, 2, 4, 8, 8, 16, 128
    shape = park.Shape(B, H, T, Hg, W, text, D)
    q, k, v = (rand(700 + i, B, H, shape.N, D, dt=BF) for i in range(3))
    pos = grid_positions((T, Hg, W), shape.N).to(torch.int32).contiguous()
    bad = pos.clone()
    bad[9] = torch.tensor([0, Hg, 0])
    r = park.rope_table((T, Hg, W), D)
    args = (q, k, v, shape, 8, 8, 0.9, 3)
    out = None
    for p, code in ((bad, _lib.PARK_ERR_INDEX), (pos, _lib.PARK_OK), (bad, _lib.PARK_ERR_INDEX)):
        pre = park.NormRope(rope=r, positions=p.cuda(), norm=norm)
        _, out = park.layer(*args, out=out, pre=pre)
        assert out.status_code() == code
    # what the layer itself meets comes first
    v[0, 0, 3, 3] = float("nan")
    _, out = park.layer(*args, out=out, pre=pre)
    assert out.status_code() == _lib.PARK_ERR_RANGE


def test_rope_table_used_at_once_on_another_stream():
    """A table made on a stream that is still busy is whole when the call that made it returns."""
    D, extent = 64, (40, 30, 20)
    x = rand(710, 1, 2, math.prod(extent), D)
    c, s = angles(extent, (12, 10, 10), 10000.0, (1, 1, 1), grid_positions(extent, x.shape[2]))
    want = plain_rotate(x.double(), c, s, False)
    park.rope(x, park.rope_table(extent, D))    # (the kernels are loaded: loading one may wait for the device)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.full((2 * (40 * 12 + 30 * 10 + 20 * 10),), 3.0, device="cuda")  # what the table's memory holds before
        torch.cuda._sleep(400_000_000)                                       # about 0.2 s
    r = park.rope_table(extent, D, stream=side)
    y = park.rope(x, r)
    within(y, want, U[F32] * want.abs() + 4 * E * pair_mass(x.double(), False))


def test_rope_table_in_a_capture():
    """Inside a capture nothing waits: the graph fills the table."""
    x = rand(711, 1, 2, 24, 64)
    want = park.rope(x, park.rope_table((2, 3, 4), 64))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = park.rope(x, park.rope_table((2, 3, 4), 64))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_the_layer_on_a_busy_stream():
    """What the call allocates and drops (workspace, normed queries and keys) is not handed out to others before it has
    run: the current stream allocates and fills as much while the call waits behind other work."""
    B, H, T, Hg, W, text, D = 1, 2, 4, 8, 8, 16, 128
    shape = park.Shape(B, H, T, Hg, W, text, D)
    q, k, v = (rand(720 + i, B, H, shape.N, D, dt=BF) for i in range(3))
    pre = park.NormRope(rope=park.rope_table((T, Hg, W), D))
    a, b = pre(q, k)
    want, r = park.layer(a, b, v, shape, 8, 8, 0.9, 3)
    size = park.workspace_size(shape, 8, 8)
    side = torch.cuda.Stream()
    calls = (lambda: park.layer(q, k, v, shape, 8, 8, 0.9, 3, stream=side, pre=pre)[0],
             lambda: park.layer(a, b, v, shape, 8, 8, 0.9, 3, stream=side)[0],
             lambda: park.sparse_attn(a, b, v, shape, 8, 8, r, stream=side),
             lambda: park.retrieve(a, b, shape, 8, 8, 0.9, 3, stream=side).mask)
    for call, res in zip(calls, (want, want, want, r.mask)):
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        with torch.cuda.stream(side):
            torch.cuda._sleep(800_000_000)               # about 0.4 s
        got = call()
        over = [torch.full((size,), 0x55, dtype=torch.uint8, device="cuda") for _ in range(3)]
        over += [torch.full_like(t, 7.0) for t in (q, k, q, k)]
        assert not side.query()
        torch.cuda.synchronize()
        assert torch.equal(got, res)


def test_captured_layer_reports_each_replay():
    """A captured layer(pre=...) clears and reports its status with every replay, without the default status word."""
    B, H, T, Hg, W, text, D = 1, 2, 4, 8, 8, 16, 128
    shape = park.Shape(B, H, T, Hg, W, text, D)
    q, k, v = (rand(730 + i, B, H, shape.N, D, dt=BF) for i in range(3))
    good = grid_positions((T, Hg, W), shape.N).to(torch.int32).contiguous().cuda()
    bad = good.clone()
    bad[70, 2] = W
    pos = good.clone()
    pre = park.NormRope(rope=park.rope_table((T, Hg, W), D), positions=pos)
    want, _ = park.layer(q, k, v, shape, 8, 8, 0.9, 3, pre=pre)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, r = park.layer(q, k, v, shape, 8, 8, 0.9, 3, pre=pre)
    for p, code in ((good, _lib.PARK_OK), (bad, _lib.PARK_ERR_INDEX), (good, _lib.PARK_OK)):
        pos.copy_(p)
        graph.replay()
        assert r.status_code() == code
    assert torch.equal(got, want)


def test_training_steps_and_layers_at_once():
    """Steps in both types, graphs of them and a layer on streams of their own: the bits of each alone."""
    n, D = 1100, 128
    r = park.rope_table((11, 10, 10), D)
    shape = park.Shape(1, 4, 11, 10, 10, 0, D)
    w = torch.ones(D, device="cuda")

    def step(x):
        a, b = park.qk_norm_rope(x[0], x[1], w, w, rope=r)
        o, lse = park.attention(a, b, x[2], causal=True, return_lse=True)
        da, db, dv = park.attention_bwd(x[3], a, b, x[2], o, lse, causal=True)
        return (o, dv, *park.qk_norm_rope_bwd(da, db, x[0], x[1], w, w, rope=r))
    jobs = []
    for i, (dt, hq, hk) in enumerate(((BF, 4, 4), (F32, 6, 2), (BF, 20, 20), (BF, 8, 1))):
        x = attn_inputs(1, hq, hk, n, n, D, dt, "tokens", seed=740 + 10 * i)
        jobs.append(lambda x=x: step(x))
    x = attn_inputs(1, 4, 4, n, n, D, BF, "heads", seed=780)[:3]
    jobs.append(lambda: (park.layer(*x, shape, 12, 12, 0.9, 3, pre=park.NormRope(rope=r))[0],))
    want = [[t.clone() for t in job()] for job in jobs]
    graphs = []
    for job in jobs[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = job()
        graphs.append((g, out))
    streams = [torch.cuda.Stream() for _ in range(len(jobs) + len(graphs))]
    for _ in range(4):
        torch.cuda.synchronize()
        got = []
        for job, s in zip(jobs, streams):
            with torch.cuda.stream(s):
                got.append(job())
        for (g, _), s in zip(graphs, streams[len(jobs):]):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got + [out for _, out in graphs], want + want[:2]):
            assert all(torch.equal(u, t) for u, t in zip(a, b))
