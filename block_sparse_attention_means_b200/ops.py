"""Operators before and beside the layer: rotary positions over (time, height,
width), the RMS norm of queries and keys for each head with the rotation in the
same pass, and dense attention over whole prompts, each with its gradient.

Thin binding like park.py: torch supplies device memory and streams, every step
runs in the library's CUDA kernels.  Nothing here is recorded by autograd: results
carry no graph, also from inputs that require gradients, which come from the
..._bwd calls (in a torch.autograd.Function, say).  Tensors are [B, H, N, D] on one CUDA device
in torch.bfloat16 or torch.float32, D a multiple of 32 up to 128, the last axis
contiguous; the other strides are free as long as rows start on 16 bytes, so the
parts of a fused projection [B, N, 3, H, D] are passed as views.

Temporary memory and outputs that the caller does not pass come from the stream
that the call runs on.  Conditions that only the device can see (a position or a
sequence bound out of range, a bounded wait that ran out) go to a status word,
``status`` or else ``status_word(device)``, which is written on an error and
never cleared by a call; 0 means that all calls so far were good.
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
import math

import torch

from . import _lib

_DT = {torch.bfloat16: _lib.PARK_BF16, torch.float32: _lib.PARK_F32}
_status_words: dict[int, torch.Tensor] = {}


def _device_index(device) -> int:
    dev = torch.device("cuda" if device is None else device)  # (a number: that CUDA device)
    if dev.type != "cuda":
        raise ValueError(f"device {dev}: expected a CUDA device")
    return torch.cuda.current_device() if dev.index is None else dev.index


def status_word(device=None) -> torch.Tensor:
    """The device's default status word, int32 [1] (see include/park.h for the codes).
    Read it with ``.item()`` and clear it with ``.zero_()``."""
    index = _device_index(device)
    if index not in _status_words:
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("the device has no status word yet: call status_word(device) before the capture, or "
                               "pass status=")
        with torch.cuda.device(index):
            word = torch.zeros(1, dtype=torch.int32, device="cuda")
            torch.cuda.current_stream().synchronize()  # once: any stream may use it from here on
        _status_words.setdefault(index, word)  # (another thread may have been first)
    return _status_words[index]


def _check(name: str, t, shape=None, dtype=None, device=None, output=False) -> None:
    """Says in words what is wrong with a tensor (the library checks the same, as codes)."""
    if not isinstance(t, torch.Tensor) or t.dim() != 4 or not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor [B, H, N, D]")
    if t.dtype not in _DT or (dtype is not None and t.dtype != dtype):
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype or 'torch.bfloat16 or torch.float32'}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    D = t.shape[3]
    if D % 32 != 0 or not 32 <= D <= 128:
        raise ValueError(f"{name}: head dimension {D} is not a multiple of 32 up to 128")
    if t.numel() == 0:
        return
    unit = 16 // t.element_size()
    rows = [s for s, n in zip(t.stride()[:3], t.shape[:3]) if n > 1]
    if t.stride(3) != 1 or t.data_ptr() % 16 != 0 or any(s <= 0 or s % unit for s in rows):
        raise ValueError(f"{name}: rows must be contiguous and start on 16 bytes (strides {tuple(t.stride())}); "
                         f"expanded axes are not taken: give shared heads as fewer heads")
    if output:
        reach = D - 1
        for s, n in sorted((s, n) for s, n in zip(t.stride()[:3], t.shape[:3]) if n > 1):
            if s <= reach:
                raise ValueError(f"{name}: an output's elements must not overlap (strides {tuple(t.stride())})")
            reach += s * (n - 1)


def _same(x, *others) -> bool:
    """All on one CUDA device, in one dtype that the library takes, with four axes."""
    dev, dt = x.get_device(), x.dtype
    if dev < 0 or dt not in _DT or x.dim() != 4:
        return False
    for t in others:
        if t.get_device() != dev or t.dtype is not dt or t.dim() != 4:
            return False
    return True


def _op(name: str, t: torch.Tensor) -> _lib.ParkOperand:
    """The tensor as the library takes it (which checks the pointer and the outer strides)."""
    shape, st = t.shape, t.stride()
    if st[3] != 1:
        _check(name, t)
    return _lib.ParkOperand(t.data_ptr(), shape[1], st[0], st[1], st[2])


def _done(rc: int, what: str, inputs=(), outputs=()) -> None:
    """Raises for a refused call: in words where a tensor is the cause, else the library's code."""
    if rc != _lib.PARK_OK:
        for name, t in inputs:
            _check(name, t)
        for name, t in outputs:
            _check(name, t, output=True)
        _lib.check(rc, what)


def _ptr(t):
    return None if t is None else t.data_ptr()


# the current stream's handle; the raw query costs 0.2 us of a call's 10 to 20, the Stream object 3
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


class _On:
    """Runs a call on the tensors' device and the given (or current) stream, so that
    memory allocated inside belongs to that stream; yields the stream's handle."""
    __slots__ = ("index", "dev", "ctx")

    def __init__(self, index: int, stream):
        self.index, self.dev, self.ctx = index, None, None
        if stream is not None:
            if stream.device.index != index:
                raise ValueError(f"stream on {stream.device}, tensors on cuda:{index}")
            self.ctx = torch.cuda.stream(stream)
        if torch.cuda.current_device() != index:
            self.dev = torch.cuda.device(index)

    def __enter__(self):
        if self.dev is not None:
            self.dev.__enter__()
        if self.ctx is not None:
            self.ctx.__enter__()
        return _raw_stream(self.index)

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)
        if self.dev is not None:
            self.dev.__exit__(*exc)


def _status(status, index: int) -> int:
    if status is None:
        word = _status_words.get(index)
        return (status_word(index) if word is None else word).data_ptr()
    if status.dtype != torch.int32 or status.numel() != 1 or status.get_device() != index:
        raise ValueError("status must be int32 [1] on the tensors' device")
    return status.data_ptr()


def _workspace(ws, need: int, like):
    """(tensor that keeps it alive, pointer, bytes)"""
    if ws is None:
        if need == 0:
            return None, None, 0
        ws = torch.empty(need, dtype=torch.uint8, device=like.device)
    elif not ws.is_contiguous() or ws.get_device() != like.get_device():
        raise ValueError("ws must be contiguous on the tensors' device")
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


# ------------------------------------------------------------------ rotary positions
@dataclasses.dataclass
class Rope:
    """Rotary axes and their table (see park_rope_axes in include/park.h)."""
    extent: tuple            # (frames, rows, columns)
    pairs: tuple             # rotated pairs of each axis
    half: bool               # False: pairs (2j, 2j+1); True: (j, j + D/2)
    table: torch.Tensor      # float32, (cos, sin) of every position of every axis

    def c(self) -> _lib.ParkRopeAxes:
        t = self.table
        key = (self.extent, self.pairs, self.half, t.data_ptr(), t.numel(), t.dtype)
        made = self.__dict__.get("_c")
        if made is None or made[0] != key:
            axes = _axes(self.extent, self.pairs, self.half, key[3])
            need = _lib.load().park_rope_table_floats(axes)
            if t.dtype != torch.float32 or not t.is_contiguous() or t.numel() < need:
                raise ValueError(f"rope table: expected {need} contiguous float32 values for extents {self.extent} and "
                                 f"pairs {self.pairs}, got {t.numel()} of {t.dtype}")
            made = self.__dict__["_c"] = (key, axes)
        return made[1]

    def __getstate__(self):  # copies and pickles make their own C struct
        return {k: v for k, v in self.__dict__.items() if k != "_c"}


def _axes(extent, pairs, half, table) -> _lib.ParkRopeAxes:
    if len(extent) != 3 or len(pairs) != 3:
        raise ValueError("extent and pairs have one entry for each of the three axes")
    i3 = ctypes.c_int * 3
    return _lib.ParkRopeAxes(i3(*extent), i3(*pairs), bool(half), table)


def rope_table(extent, D: int, pairs=None, theta: float = 10000.0, scale=(1.0, 1.0, 1.0), half: bool = False,
               device=None, stream=None) -> Rope:
    """Table of the angles (scale_a pos) theta^(-j / pairs_a) of each axis, made once
    and kept.  extent = (frames, rows, columns); pairs defaults to the split of D/2
    that the synthetic layers use: a third each for rows and columns, the rest for
    time (22/21/21 at D = 128).  For plain 1-D positions pass extent (n, 1, 1) and
    pairs (D/2, 0, 0).  The call returns when the table is filled, so that any stream may
    use it at once; inside a capture it does not wait, and the graph fills the table."""
    if pairs is None:
        third = D // 2 // 3
        pairs = (D // 2 - 2 * third, third, third)
    extent, pairs = tuple(int(x) for x in extent), tuple(int(x) for x in pairs)
    if len(extent) != 3 or len(pairs) != 3 or len(scale) != 3:
        raise ValueError("extent, pairs and scale have one entry for each of the three axes")
    if min(extent) < 1 or min(pairs) < 0 or sum(pairs) > D // 2:
        raise ValueError(f"extents {extent} must be positive and pairs {pairs} sum to at most D/2 = {D // 2}")
    dev = torch.device("cuda", _device_index(device))
    with _On(dev.index, stream) as st:
        n = _lib.load().park_rope_table_floats(_axes(extent, pairs, half, None))
        r = Rope(extent, pairs, bool(half), torch.empty(max(2, n), dtype=torch.float32, device=dev))
        rc = _lib.load().park_rope_table(r.c(), float(theta),
                                         (ctypes.c_double * 3)(*[float(x) for x in scale]), st)
        _lib.check(rc, "park_rope_table")
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream().synchronize()  # once: any stream may use it from here on
    return r


def _rope_args(rope, positions, B: int, N: int, D: int, index: int):
    if rope is None:
        if positions is not None:
            raise ValueError("positions without rope")
        return None, None, 0
    if rope.table.get_device() != index:
        raise ValueError(f"rope table on {rope.table.device}, tensors on cuda:{index}")
    if sum(rope.pairs) > D // 2:
        raise ValueError(f"rope rotates {sum(rope.pairs)} pairs, the head has {D // 2}")
    if positions is None:
        return rope.c(), None, 0
    if (positions.dtype != torch.int32 or positions.get_device() != index or not positions.is_contiguous()
            or tuple(positions.shape) not in ((N, 3), (B, N, 3))):
        raise ValueError(f"positions must be contiguous int32 [N, 3] or [B, N, 3] with N = {N} on cuda:{index}")
    return rope.c(), positions.data_ptr(), 3 * N if positions.dim() == 3 else 0


def _output(name: str, out, like):
    if not _same(like, out) or out.shape != like.shape:
        _check(name, out, like.shape, like.dtype, like.device, output=True)
    return out


def rope(x, rope: Rope, positions=None, inverse: bool = False, out=None, status=None, stream=None) -> torch.Tensor:
    """x rotated by its tokens' positions; ``inverse`` rotates back, which is also the
    gradient (dx from dy).  positions: int32 [N, 3] or [B, N, 3] with (t, y, w) of each
    token, negative for text (not rotated); None: the grid order of Shape, tokens behind
    the grid not rotated.  ``out`` may be x."""
    if not isinstance(x, torch.Tensor) or not _same(x):
        _check("x", x)
    if rope is None:
        raise ValueError("rope is missing")
    (B, H, N, D), index = x.shape, x.get_device()
    with _On(index, stream) as st:
        out = torch.empty_like(x) if out is None else _output("out", out, x)
        axes, pos, sb = _rope_args(rope, positions, B, N, D, index)
        if B * H == 0:
            return out
        rc = _lib.load().park_rope(_op("x", x), _op("out", out), B, N, D, _DT[x.dtype], axes, pos, sb, inverse,
                                   _status(status, index), st)
    if rc:
        _done(rc, "park_rope", (("x", x),), (("out", out),))
    return out


# ------------------------------------------------------------------ norm + rotation
def _pair_check(q, k, more=()):
    if not isinstance(q, torch.Tensor) or not isinstance(k, torch.Tensor) or not _same(q, k):
        _check("q", q)
        _check("k", k, None, q.dtype, q.device)
    B, H, N, D = q.shape
    ks = k.shape
    if ks[0] != B or ks[2] != N or ks[3] != D:
        _check("k", k, (B, ks[1], N, D))
    if min(B, H, ks[1]) < 1:
        raise ValueError("q and k need at least one batch entry and one head")
    for name, t, like in more:
        if not _same(like, t) or t.shape != like.shape:
            _check(name, t, like.shape, q.dtype, q.device)
    return B, N, D, q.get_device()


def _weights(q_weight, k_weight, D: int, index: int):
    if q_weight is None and k_weight is None:
        return None, None, _lib.PARK_F32
    a, b = (q_weight if q_weight is not None else k_weight), (k_weight if k_weight is not None else q_weight)
    want = (D,)
    for name, w in (("q_weight", a), ("k_weight", b)):
        if w.shape != want or w.dtype not in _DT or w.stride(0) != 1 or w.get_device() != index:
            raise ValueError(f"{name} must be contiguous [D] in bfloat16 or float32 on cuda:{index}")
    if a.dtype is not b.dtype:
        raise TypeError("q_weight and k_weight have different dtypes")
    return _ptr(q_weight), _ptr(k_weight), _DT[a.dtype]


def _contiguous_like(t):
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def qk_norm_rope(q, k, q_weight=None, k_weight=None, rope: Rope | None = None, positions=None, eps: float = 1e-6,
                 q_out=None, k_out=None, status=None, stream=None):
    """(q', k'): each head row divided by its root mean square (with eps, at least 2^-80), times the
    weight [D] (None: ones), rotated as by ``rope`` (None: not), in one pass, float32
    inside and rounded once.  q has H heads, k may have fewer.  New outputs are
    contiguous [B, H, N, D], the layout that layer() takes; q_out may be q, k_out k."""
    B, N, D, index = _pair_check(q, k)
    with _On(index, stream) as st:
        q_out = _contiguous_like(q) if q_out is None else _output("q_out", q_out, q)
        k_out = _contiguous_like(k) if k_out is None else _output("k_out", k_out, k)
        axes, pos, sb = _rope_args(rope, positions, B, N, D, index)
        wq, wk, wdt = _weights(q_weight, k_weight, D, index)
        rc = _lib.load().park_qk_norm_rope(_op("q", q), _op("k", k), wq, wk, wdt, eps, axes, pos, sb,
                                           _op("q_out", q_out), _op("k_out", k_out), B, N, D, _DT[q.dtype],
                                           _status(status, index), st)
    if rc:
        _done(rc, "park_qk_norm_rope", (("q", q), ("k", k)), (("q_out", q_out), ("k_out", k_out)))
    return q_out, k_out


@functools.lru_cache(maxsize=1024)
def _norm_bwd_workspace(B: int, N: int, D: int) -> int:
    need = ctypes.c_size_t(0)
    _lib.check(_lib.load().park_qk_norm_rope_bwd_workspace(B, N, D, ctypes.byref(need)),
               "park_qk_norm_rope_bwd_workspace")
    return need.value


def qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight=None, k_weight=None, rope: Rope | None = None, positions=None,
                     eps: float = 1e-6, dq=None, dk=None, ws=None, status=None, stream=None):
    """(dq, dk, dq_weight, dk_weight) from the gradients of qk_norm_rope's outputs and its
    own inputs.  dq, dk in the inputs' type; the weights' gradients float32 [D], None
    where there is no weight."""
    B, N, D, index = _pair_check(q, k, (("dq_out", dq_out, q), ("dk_out", dk_out, k)))
    with _On(index, stream) as st:
        dq = _contiguous_like(q) if dq is None else _output("dq", dq, q)
        dk = _contiguous_like(k) if dk is None else _output("dk", dk, k)
        axes, pos, sb = _rope_args(rope, positions, B, N, D, index)
        wq, wk, wdt = _weights(q_weight, k_weight, D, index)
        ws, wp, wn = _workspace(ws, _norm_bwd_workspace(B, N, D), q)
        dw = [torch.empty(D, dtype=torch.float32, device=q.device) if w is not None else None
              for w in (q_weight, k_weight)]
        rc = _lib.load().park_qk_norm_rope_bwd(
            _op("dq_out", dq_out), _op("dk_out", dk_out), _op("q", q), _op("k", k), wq, wk, wdt, eps, axes, pos, sb,
            _op("dq", dq), _op("dk", dk), _ptr(dw[0]), _ptr(dw[1]), B, N, D, _DT[q.dtype], wp, wn,
            _status(status, index), st)
    if rc:
        _done(rc, "park_qk_norm_rope_bwd", (("dq_out", dq_out), ("dk_out", dk_out), ("q", q), ("k", k)),
              (("dq", dq), ("dk", dk)))
    return dq, dk, dw[0], dw[1]


@dataclasses.dataclass
class NormRope:
    """What layer(pre=...) does to raw queries and keys first: the norm for each head
    (norm=False: none) and the rotation (rope=None: none)."""
    q_weight: torch.Tensor | None = None
    k_weight: torch.Tensor | None = None
    rope: Rope | None = None
    positions: torch.Tensor | None = None
    eps: float = 1e-6
    norm: bool = True

    def __call__(self, q, k, status=None, stream=None):
        if self.norm:
            return qk_norm_rope(q, k, self.q_weight, self.k_weight, self.rope, self.positions, self.eps, status=status,
                                stream=stream)
        if self.rope is None:
            raise ValueError("NormRope with neither norm nor rope")
        _pair_check(q, k)
        with _On(q.get_device(), stream):
            outs = [_contiguous_like(t) for t in (q, k)]
        return tuple(rope(t, self.rope, self.positions, out=o, status=status, stream=stream)
                     for t, o in zip((q, k), outs))


# ------------------------------------------------------------------ dense attention
def _attn_shape(q, k, causal, scale, cu_q, cu_k) -> _lib.ParkAttnShape:
    B, _, Nq, D = q.shape
    n_seq = 0
    if (cu_q is None) != (cu_k is None):
        raise ValueError("cu_q and cu_k go together")
    if cu_q is not None:
        for name, cu in (("cu_q", cu_q), ("cu_k", cu_k)):
            if (cu.dtype != torch.int32 or cu.dim() != 1 or not cu.is_contiguous()
                    or cu.get_device() != q.get_device()):
                raise ValueError(f"{name} must be a contiguous int32 vector on {q.device}")
        if cu_q.numel() != cu_k.numel() or cu_q.numel() < 2:
            raise ValueError("cu_q and cu_k hold the sequences' bounds: n_seq + 1 entries each")
        if B != 1:
            raise ValueError("packed sequences need B = 1")
        n_seq = cu_q.numel() - 1
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    return _lib.ParkAttnShape(B, D, _DT[q.dtype], Nq, k.shape[2], n_seq, _ptr(cu_q), _ptr(cu_k), bool(causal), scale)


def _attn_check(Q, K, V) -> int:
    if (not all(isinstance(t, torch.Tensor) for t in (Q, K, V)) or not _same(Q, K, V) or K.shape != V.shape
            or K.shape[0] != Q.shape[0] or K.shape[3] != Q.shape[3]):
        _check("Q", Q)
        _check("K", K, None, Q.dtype, Q.device)
        _check("K", K, (Q.shape[0], K.shape[1], K.shape[2], Q.shape[3]))
        _check("V", V, K.shape, Q.dtype, Q.device)
    B, H, hk = Q.shape[0], Q.shape[1], K.shape[1]
    if B < 1 or H < 1 or hk < 1 or H % hk:
        raise ValueError(f"{hk} key heads do not divide {H} query heads (batch {B})")
    return Q.get_device()


def _lse(lse, Q):
    if lse.shape != Q.shape[:3] or lse.dtype != torch.float32 or not lse.is_contiguous() or lse.device != Q.device:
        raise ValueError(f"lse must be contiguous float32 {tuple(Q.shape[:3])} on {Q.device}")
    return lse


@functools.lru_cache(maxsize=1024)
def _attn_workspace(B: int, Hq: int, Hk: int, Nq: int, Nk: int, D: int, dtype: int, n_seq: int, backward: int) -> int:
    # the bounds' addresses only have to be there
    s, n = _lib.ParkAttnShape(B, D, dtype, Nq, Nk, n_seq, 1, 1, 0, 1.0), ctypes.c_size_t(0)
    _lib.check(_lib.load().park_attention_workspace(ctypes.byref(s), Hq, Hk, backward, ctypes.byref(n)),
               "park_attention_workspace")
    return n.value


def _attn_need(Q, K, s, backward: int) -> int:
    return _attn_workspace(s.B, Q.shape[1], K.shape[1], s.Nq, s.Nk, s.D, s.dtype, s.n_seq, backward)


def attention_workspace_size(Q, K, cu_q=None, cu_k=None, backward: bool = False) -> int:
    """Bytes of device workspace that attention (or attention_bwd) takes for these tensors."""
    return _attn_need(Q, K, _attn_shape(Q, K, False, None, cu_q, cu_k), int(backward))


def attention(Q, K, V, causal: bool = False, scale: float | None = None, cu_q=None, cu_k=None, O=None,
              return_lse: bool = False, lse=None, ws=None, status=None, stream=None):
    """Dense attention: O, or (O, lse) with return_lse.

    Q [B, Hq, Nq, D], K and V [B, Hk, Nk, D], Hk dividing Hq (query head h reads key head
    h // (Hq // Hk)).  cu_q, cu_k (int32 [n_seq + 1] on the device, B = 1) pack sequences
    of different, possibly zero, lengths; rows outside them are not written (in a new O
    they are undefined).  causal: row i sees keys j <= i + n_k - n_q.  Rows without a key
    give 0 and lse = -inf.  scale > 0 defaults to 1/sqrt(D)."""
    index = _attn_check(Q, K, V)
    with _On(index, stream) as st:
        O = torch.empty_like(Q) if O is None else _output("O", O, Q)
        if lse is not None:
            _lse(lse, Q)
        elif return_lse:
            lse = torch.empty(Q.shape[:3], dtype=torch.float32, device=Q.device)
        s = _attn_shape(Q, K, causal, scale, cu_q, cu_k)
        ws, wp, wn = _workspace(ws, _attn_need(Q, K, s, 0), Q)
        rc = _lib.load().park_attention(s, _op("Q", Q), _op("K", K), _op("V", V), _op("O", O), _ptr(lse), wp, wn,
                                        _status(status, index), st)
    if rc:
        _done(rc, "park_attention", (("Q", Q), ("K", K), ("V", V)), (("O", O),))
    return (O, lse) if return_lse else O


def attention_bwd(dO, Q, K, V, O, lse, causal: bool = False, scale: float | None = None, cu_q=None, cu_k=None, dQ=None,
                  dK=None, dV=None, ws=None, status=None, stream=None):
    """(dQ, dK, dV) from dO and from attention's inputs and results, O and lse of one call
    over all of a row's keys (not joined from calls over parts of them); dK and dV are sums
    over the query heads that share a key head.  Rows outside the packed sequences are
    not written (in new tensors they are undefined)."""
    index = _attn_check(Q, K, V)
    for name, t in (("O", O), ("dO", dO)):
        if not isinstance(t, torch.Tensor) or not _same(Q, t) or t.shape != Q.shape:
            _check(name, t, Q.shape, Q.dtype, Q.device)
    _lse(lse, Q)
    with _On(index, stream) as st:
        outs = [torch.empty_like(like) if t is None else _output(name, t, like)
                for name, t, like in (("dQ", dQ, Q), ("dK", dK, K), ("dV", dV, V))]
        s = _attn_shape(Q, K, causal, scale, cu_q, cu_k)
        ws, wp, wn = _workspace(ws, _attn_need(Q, K, s, 1), Q)
        rc = _lib.load().park_attention_bwd(s, _op("dO", dO), _op("Q", Q), _op("K", K), _op("V", V), _op("O", O),
                                            _ptr(lse), _op("dQ", outs[0]), _op("dK", outs[1]), _op("dV", outs[2]), wp,
                                            wn, _status(status, index), st)
    if rc:
        _done(rc, "park_attention_bwd", (("dO", dO), ("Q", Q), ("K", K), ("V", V), ("O", O)),
              tuple(zip(("dQ", "dK", "dV"), outs)))
    return tuple(outs)
