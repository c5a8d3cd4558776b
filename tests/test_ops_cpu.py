"""Refusals of the operators before and beside the layer, without a GPU: every bad
argument is answered on the host, before anything is enqueued."""
import copy
import ctypes
import pickle
import types

import pytest
import torch

import block_sparse_attention_means_b200 as park
from block_sparse_attention_means_b200 import _lib

FAKE = 0x1000   # an aligned address that no refused call touches
B, H, N, D = 2, 4, 40, 64


def operand(ptr=FAKE, heads=H, sb=H * N * D, sh=N * D, sn=D):
    return _lib.ParkOperand(ptr, heads, sb, sh, sn)


def axes(extent=(2, 4, 5), pairs=(12, 10, 10), half=0, table=FAKE):
    return _lib.ParkRopeAxes((ctypes.c_int * 3)(*extent), (ctypes.c_int * 3)(*pairs), half, table)


@pytest.fixture(autouse=True)
def nothing_enqueued():
    before = park.launch_count()
    yield
    assert park.launch_count() == before


def rope(x=None, y=None, b=B, n=N, d=D, dt=_lib.PARK_BF16, ax=None, pos=0, sb=0, status=FAKE):
    x, y, ax = x or operand(), y or operand(0x100000), ax or axes()
    return _lib.load().park_rope(x, y, b, n, d, dt, ctypes.byref(ax), pos, sb, 0, status, None)


@pytest.mark.parametrize("kw, code", [
    (dict(x=operand(0)), _lib.PARK_ERR_INVALID_ARG),
    (dict(x=operand(FAKE + 8)), _lib.PARK_ERR_INVALID_ARG),                  # 16-byte alignment
    (dict(x=operand(sn=D + 4)), _lib.PARK_ERR_INVALID_ARG),                  # rows not on 16 bytes
    (dict(x=operand(sh=0)), _lib.PARK_ERR_INVALID_ARG),                      # broadcast axis
    (dict(x=operand(sb=-H * N * D)), _lib.PARK_ERR_INVALID_ARG),
    (dict(y=operand(0x100000, sn=D // 2)), _lib.PARK_ERR_INVALID_ARG),       # overlapping output rows
    (dict(y=operand(0x100000, sh=(N - 1) * D)), _lib.PARK_ERR_INVALID_ARG),
    (dict(y=operand(0x100000, heads=H + 1)), _lib.PARK_ERR_INVALID_ARG),
    (dict(x=operand(heads=0)), _lib.PARK_ERR_INVALID_ARG),
    (dict(d=48), _lib.PARK_ERR_UNSUPPORTED),
    (dict(d=160), _lib.PARK_ERR_UNSUPPORTED),
    (dict(d=0), _lib.PARK_ERR_INVALID_ARG),
    (dict(dt=2), _lib.PARK_ERR_INVALID_ARG),
    (dict(b=0), _lib.PARK_ERR_INVALID_ARG),
    (dict(n=-1), _lib.PARK_ERR_INVALID_ARG),
    (dict(n=1 << 31), _lib.PARK_ERR_UNSUPPORTED),
    (dict(status=0), _lib.PARK_ERR_INVALID_ARG),
    (dict(ax=axes(table=0)), _lib.PARK_ERR_INVALID_ARG),
    (dict(ax=axes(extent=(0, 4, 5))), _lib.PARK_ERR_INVALID_ARG),
    (dict(ax=axes(pairs=(12, 11, 10))), _lib.PARK_ERR_INVALID_ARG),          # 33 pairs of 32
    (dict(ax=axes(pairs=(-1, 11, 10))), _lib.PARK_ERR_INVALID_ARG),
    (dict(pos=FAKE, sb=-3), _lib.PARK_ERR_INVALID_ARG),
    (dict(pos=FAKE + 2), _lib.PARK_ERR_INVALID_ARG),
])
def test_rope_refuses(kw, code):
    assert rope(**kw) == code


def test_empty_rope_call_is_good():
    assert rope(n=0) == _lib.PARK_OK
    assert rope(x=operand(0), y=operand(0), n=0) == _lib.PARK_OK


def test_rope_table_refuses():
    lib, one = _lib.load(), (ctypes.c_double * 3)(1, 1, 1)
    assert lib.park_rope_table_floats(axes()) == 2 * (2 * 12 + 4 * 10 + 5 * 10)
    assert lib.park_rope_table_floats(axes(extent=(0, 1, 1))) == 0
    assert lib.park_rope_table(axes(table=0), 1e4, one, None) == _lib.PARK_ERR_INVALID_ARG
    assert lib.park_rope_table(axes(), 0.0, one, None) == _lib.PARK_ERR_INVALID_ARG
    assert lib.park_rope_table(axes(), float("inf"), one, None) == _lib.PARK_ERR_INVALID_ARG
    assert lib.park_rope_table(axes(), 1e4, (ctypes.c_double * 3)(1, float("nan"), 1), None) == \
        _lib.PARK_ERR_INVALID_ARG
    assert lib.park_rope_table(axes(), 1e4, None, None) == _lib.PARK_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        park.rope_table((2, 4), 64)
    with pytest.raises(ValueError):
        park.rope_table((2, 4, 5), 64, pairs=(32, 1, 0))
    with pytest.raises(ValueError):
        park.rope_table((2, 0, 5), 64)


def norm(q=None, k=None, wq=FAKE, wk=FAKE, wdt=_lib.PARK_BF16, eps=1e-6, ax=None, pos=0, qo=None, ko=None, status=FAKE):
    q, k = q or operand(), k or operand(0x100000, heads=2)
    qo, ko = qo or operand(0x200000), ko or operand(0x300000, heads=2)
    return _lib.load().park_qk_norm_rope(q, k, wq, wk, wdt, eps, ctypes.byref(ax) if ax else None, pos, 0, qo, ko, B, N,
                                         D, _lib.PARK_BF16, status, None)


@pytest.mark.parametrize("kw", [
    dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(wdt=3), dict(wq=FAKE + 1),
    dict(pos=FAKE), dict(status=0), dict(qo=operand(0x200000, heads=3)), dict(ko=operand(0x300000, heads=4)),
    dict(q=operand(0)), dict(k=operand(0x100000, heads=2, sn=D + 1)), dict(ax=axes(pairs=(33, 0, 0))),
])
def test_norm_refuses(kw):
    assert norm(**kw) == _lib.PARK_ERR_INVALID_ARG


def test_norm_backward_refuses():
    lib, need = _lib.load(), ctypes.c_size_t(0)
    assert lib.park_qk_norm_rope_bwd_workspace(B, N, 48, need) == _lib.PARK_ERR_UNSUPPORTED
    assert lib.park_qk_norm_rope_bwd_workspace(0, N, D, need) == _lib.PARK_ERR_INVALID_ARG
    assert lib.park_qk_norm_rope_bwd_workspace(B, N, D, None) == _lib.PARK_ERR_INVALID_ARG
    assert lib.park_qk_norm_rope_bwd_workspace(B, N, D, need) == _lib.PARK_OK and need.value > 0

    def call(ws=FAKE, size=need.value, eps=1e-6, heads=H):
        o = [operand(0x100000 * i, heads=H if i != 6 else heads) for i in range(1, 7)]
        return lib.park_qk_norm_rope_bwd(o[0], o[1], o[2], o[3], FAKE, FAKE, _lib.PARK_F32, eps, None, 0, 0, o[4], o[5],
                                         FAKE, FAKE, B, N, D, _lib.PARK_BF16, ws, size, FAKE, None)
    assert call(size=need.value - 1) == _lib.PARK_ERR_WORKSPACE
    assert call(ws=0) == _lib.PARK_ERR_INVALID_ARG
    assert call(ws=FAKE + 8) == _lib.PARK_ERR_INVALID_ARG
    assert call(eps=0.0) == _lib.PARK_ERR_INVALID_ARG
    assert call(eps=2.0 ** -81) == _lib.PARK_ERR_INVALID_ARG and norm(eps=2.0 ** -81) == _lib.PARK_ERR_INVALID_ARG
    assert call(heads=H + 1) == _lib.PARK_ERR_INVALID_ARG


def shape(b=B, d=D, dt=_lib.PARK_BF16, nq=N, nk=N, n_seq=0, cu_q=0, cu_k=0, causal=0, scale=0.125):
    return _lib.ParkAttnShape(b, d, dt, nq, nk, n_seq, cu_q, cu_k, causal, scale)


def attention(s=None, q=None, k=None, v=None, o=None, status=FAKE):
    s = s or shape()
    return _lib.load().park_attention(s, q or operand(), k or operand(0x100000), v or operand(0x200000),
                                      o or operand(0x300000), None, FAKE, 1 << 40, status, None)


@pytest.mark.parametrize("kw, code", [
    (dict(s=shape(b=0)), _lib.PARK_ERR_INVALID_ARG),
    (dict(s=shape(nq=-1)), _lib.PARK_ERR_INVALID_ARG),
    (dict(s=shape(nk=-1)), _lib.PARK_ERR_INVALID_ARG),
    (dict(s=shape(d=48)), _lib.PARK_ERR_UNSUPPORTED),
    (dict(s=shape(dt=5)), _lib.PARK_ERR_INVALID_ARG),
    (dict(s=shape(scale=float("nan"))), _lib.PARK_ERR_INVALID_ARG),
    (dict(s=shape(scale=float("inf"))), _lib.PARK_ERR_INVALID_ARG),
    (dict(s=shape(scale=0.0)), _lib.PARK_ERR_INVALID_ARG),
    (dict(s=shape(scale=-0.1)), _lib.PARK_ERR_INVALID_ARG),
    (dict(s=shape(n_seq=-1)), _lib.PARK_ERR_INVALID_ARG),
    (dict(s=shape(n_seq=2, cu_q=FAKE, cu_k=FAKE)), _lib.PARK_ERR_INVALID_ARG),       # packed with B = 2
    (dict(s=shape(b=1, n_seq=2, cu_q=FAKE)), _lib.PARK_ERR_INVALID_ARG),
    (dict(s=shape(nk=1 << 31)), _lib.PARK_ERR_UNSUPPORTED),
    (dict(s=shape(nq=1 << 31)), _lib.PARK_ERR_UNSUPPORTED),
    (dict(s=shape(nq=1 << 62), k=operand(0x100000, heads=1), v=operand(0x200000, heads=1)), _lib.PARK_ERR_UNSUPPORTED),
    (dict(s=shape(b=4, nq=1 << 62)), _lib.PARK_ERR_UNSUPPORTED),
    (dict(s=shape(b=4, nk=1 << 62)), _lib.PARK_ERR_UNSUPPORTED),
    (dict(k=operand(0x100000, heads=3), v=operand(0x200000, heads=3)), _lib.PARK_ERR_INVALID_ARG),
    (dict(v=operand(0x200000, heads=2)), _lib.PARK_ERR_INVALID_ARG),
    (dict(o=operand(0x300000, heads=2)), _lib.PARK_ERR_INVALID_ARG),
    (dict(o=operand(0x300000, sn=D - 8)), _lib.PARK_ERR_INVALID_ARG),
    (dict(q=operand(FAKE + 2)), _lib.PARK_ERR_INVALID_ARG),
    (dict(v=operand(0)), _lib.PARK_ERR_INVALID_ARG),
    (dict(status=0), _lib.PARK_ERR_INVALID_ARG),
])
def test_attention_refuses(kw, code):
    assert attention(**kw) == code


def test_attention_without_queries_is_good():
    assert attention(s=shape(nq=0), q=operand(0), o=operand(0)) == _lib.PARK_OK


def test_attention_backward_refuses():
    lib, need, s = _lib.load(), ctypes.c_size_t(0), shape()
    assert lib.park_attention_workspace(s, H, H, 1, need) == _lib.PARK_OK and need.value >= B * H * N * 4
    assert lib.park_attention_workspace(s, H, 3, 1, need) == _lib.PARK_ERR_INVALID_ARG
    assert lib.park_attention_workspace(s, H, H, 1, None) == _lib.PARK_ERR_INVALID_ARG
    lib.park_attention_workspace(s, H, H, 1, need)

    def call(lse=FAKE, size=need.value, ws=FAKE, bad=None, op=None):
        o = [operand(0x100000 * i) for i in range(1, 9)]
        if bad is not None:
            o[bad] = op
        return lib.park_attention_bwd(s, o[0], o[1], o[2], o[3], o[4], lse, o[5], o[6], o[7], ws, size, FAKE, None)
    assert call(size=need.value - 1) == _lib.PARK_ERR_WORKSPACE
    assert call(ws=0) == _lib.PARK_ERR_INVALID_ARG
    assert call(lse=0) == _lib.PARK_ERR_INVALID_ARG
    for i in range(8):
        assert call(bad=i, op=operand(0)) == _lib.PARK_ERR_INVALID_ARG
        if i != 1 and i != 2:
            assert call(bad=i, op=operand(0x900000, heads=2)) == _lib.PARK_ERR_INVALID_ARG
    for i in (5, 6, 7):
        assert call(bad=i, op=operand(0x900000, sh=D)) == _lib.PARK_ERR_INVALID_ARG


@pytest.mark.parametrize("dt", [_lib.PARK_BF16, _lib.PARK_F32])
@pytest.mark.parametrize("backward", [0, 1])
def test_attention_workspace_stays_small(dt, backward):
    """Besides delta (4 bytes a row) the parts of a split take 256 MB and a little at most, whatever the sequences."""
    lib, need = _lib.load(), ctypes.c_size_t(0)
    for n_seq in (0, 1, 2, 31, 70, 500, 5000):
        for nq in (1, 70, 2300, 9400, 32000, 200000):
            for nk in (1, 70, 3000, 32000, 130000, 2000000):
                for hq, hk in ((1, 1), (8, 1), (32, 1), (24, 8), (40, 40)):
                    s = shape(b=1, d=128, dt=dt, nq=nq, nk=nk, n_seq=n_seq, cu_q=FAKE, cu_k=FAKE)
                    assert lib.park_attention_workspace(s, hq, hk, backward, need) == _lib.PARK_OK
                    parts = need.value - backward * 4 * hq * nq
                    assert parts <= (256 << 20) + 4096, (n_seq, nq, nk, hq, hk, parts)
                    if n_seq == 0:
                        assert parts <= 80 << 20, (nq, nk, hq, hk, parts)


@pytest.mark.parametrize("where", ["cpu", torch.device("cpu")])
def test_host_devices_are_refused(where):
    with pytest.raises(ValueError):
        park.rope_table((2, 4, 5), 64, device=where)
    with pytest.raises(ValueError):
        park.status_word(where)


def test_python_refuses_host_tensors():
    x = torch.zeros(1, 1, 4, 64)
    r = park.Rope((1, 1, 4), (10, 10, 10), False, torch.zeros(600))
    with pytest.raises(ValueError):
        park.rope(x, r)
    with pytest.raises(ValueError):
        park.qk_norm_rope(x, x)
    with pytest.raises(ValueError):
        park.attention(x, x, x)
    with pytest.raises(ValueError):
        park.attention_bwd(x, x, x, x, x, x)


@pytest.mark.parametrize("table", [
    torch.zeros(127), torch.zeros(0), torch.zeros(128, dtype=torch.float64), torch.zeros(256)[::2],
])
def test_a_rope_whose_table_does_not_fit_its_axes_is_refused(table):
    """The kernels index the table by the axes: 4 positions of 16 pairs are 128 values."""
    with pytest.raises(ValueError):
        park.Rope((4, 1, 1), (16, 0, 0), False, table).c()
    good = park.Rope((4, 1, 1), (16, 0, 0), False, torch.zeros(128))
    assert good.c() is good.c()
    good.extent = (5, 1, 1)
    with pytest.raises(ValueError):
        good.c()
    good.extent, good.table = (4, 1, 1), table
    with pytest.raises(ValueError):
        good.c()
    with pytest.raises(ValueError):
        park.Rope((4, 1), (16, 0), False, torch.zeros(128)).c()


def test_a_narrower_view_of_the_table_is_refused():
    r = park.Rope((4, 1, 1), (16, 0, 0), False, torch.zeros(128))
    r.c()
    r.table = r.table[:64]
    with pytest.raises(ValueError):
        r.c()


@pytest.mark.parametrize("again", [copy.copy, copy.deepcopy, lambda r: pickle.loads(pickle.dumps(r))])
def test_a_rope_in_use_can_be_copied(again):
    r = park.Rope((4, 1, 1), (16, 0, 0), True, torch.arange(128.0))
    r.c()
    s = again(r)
    assert (s.extent, s.pairs, s.half) == (r.extent, r.pairs, r.half) and torch.equal(s.table, r.table)
    assert s.c().table == s.table.data_ptr() and r.c().table == r.table.data_ptr()
    n = again(park.NormRope(torch.ones(64), None, rope=r, eps=1e-5))
    assert n.eps == 1e-5 and torch.equal(n.q_weight, torch.ones(64)) and torch.equal(n.rope.table, r.table)


@pytest.mark.parametrize("dt, waves", [(_lib.PARK_BF16, 2), (_lib.PARK_F32, 4)])
@pytest.mark.parametrize("hq, hk", [(24, 8), (8, 8), (5, 5)])
@pytest.mark.parametrize("nk", [20000, 60000, 100000, 200000, 400000, 1000000])
def test_single_rows_split_their_keys_into_whole_waves(dt, waves, hq, hk, nk):
    """One row over many keys: about `waves` blocks for each SM at every length (bf16: no more, they run at once), read off
    the parts' workspace."""
    lib, need, d = _lib.load(), ctypes.c_size_t(0), 128
    s = shape(b=1, d=d, dt=dt, nq=1, nk=nk)
    assert lib.park_attention_workspace(s, hq, hk, 0, need) == _lib.PARK_OK
    parts = need.value // (hq * (d + 1) * 4)
    tile = 128 if dt == _lib.PARK_BF16 else 64
    least = min(waves * 148, (nk + tile - 1) // tile * hk / 4)   # (parts of a few tiles at least)
    assert least / 1.5 - hk <= parts * hk <= waves * 148 + (hk if dt == _lib.PARK_F32 else 0)


def stand_in(index, shape=(1, 2, 40, 64), dtype=torch.bfloat16):
    """What the layer's calls look at of a tensor on another device."""
    return types.SimpleNamespace(shape=shape, dtype=dtype, is_contiguous=lambda: True, is_cuda=True,
                                 device=torch.device("cuda", index), get_device=lambda: index, data_ptr=lambda: FAKE,
                                 numel=lambda: 1 << 30)


def test_the_layer_runs_on_its_tensors_device_and_stream(monkeypatch):
    from block_sparse_attention_means_b200 import ops
    seen, here = [], [0]

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            here.append(self.index)

        def __exit__(self, *exc):
            here.pop()
    lib = types.SimpleNamespace(**{n: lambda *a, n=n: seen.append((n, here[-1], a[-1].value)) or 0
                                   for n in ("park_retrieve", "park_sparse_attn", "park_layer")})
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: here[-1])
    monkeypatch.setattr(ops, "_raw_stream", lambda index: 1000 * index)
    monkeypatch.setattr(_lib, "load", lambda: lib)
    shape = park.Shape(1, 2, 2, 4, 5, 0, 64)
    r = types.SimpleNamespace(status=stand_in(1), c=_lib.ParkRetrieval)
    q, ws = stand_in(1), stand_in(1)
    park.retrieve(q, q, shape, 4, 4, 0.9, 3, out=r, ws=ws)
    park.sparse_attn(q, q, q, shape, 4, 4, r, O=stand_in(1), ws=ws)
    park.layer(q, q, q, shape, 4, 4, 0.9, 3, O=stand_in(1), out=r, ws=ws)
    assert seen == [(n, 1, 1000) for n in ("park_retrieve", "park_sparse_attn", "park_layer")] and here == [0]
    # tensors, results or a stream of different devices
    host = stand_in(0)
    host.device = torch.device("cpu")
    with pytest.raises(ValueError):
        park.retrieve(q, stand_in(0), shape, 4, 4, 0.9, 3, out=r, ws=ws)
    with pytest.raises(ValueError):
        park.layer(q, q, q, shape, 4, 4, 0.9, 3, O=stand_in(0), out=r, ws=ws)
    with pytest.raises(ValueError):
        park.layer(q, q, q, shape, 4, 4, 0.9, 3, O=stand_in(1, (1, 2, 39, 64)), out=r, ws=ws)
    with pytest.raises(ValueError):
        park.layer(q, q, q, shape, 4, 4, 0.9, 3, O=stand_in(1), out=r, ws=host)
    with pytest.raises(ValueError):
        park.layer(q, q, q, shape, 4, 4, 0.9, 3, O=stand_in(1), out=types.SimpleNamespace(status=stand_in(0)), ws=ws)
    with pytest.raises(ValueError):
        park.retrieve(q, q, shape, 4, 4, 0.9, 3, out=r, ws=ws, stream=types.SimpleNamespace(device=stand_in(0).device))
    assert len(seen) == 3
