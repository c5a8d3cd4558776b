"""Operators before and beside the layer: rotary positions over (time, height,
width), the RMS norm of queries and keys for each head with the rotation in the
same pass, and dense attention over whole prompts, each with its gradient.

Thin binding like park.py: torch supplies device memory and streams, every step
runs in the library's CUDA kernels.  Tensors are [B, H, N, D] on one CUDA device
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
import math

import torch

from . import _lib

_DT = {torch.bfloat16: _lib.PARK_BF16, torch.float32: _lib.PARK_F32}
_status_words: dict[int, torch.Tensor] = {}


def status_word(device=None) -> torch.Tensor:
    """The device's default status word, int32 [1] (see include/park.h for the codes).
    Read it with ``.item()`` and clear it with ``.zero_()``."""
    dev = torch.device("cuda" if device is None else device)
    index = torch.cuda.current_device() if dev.index is None else dev.index
    if index not in _status_words:
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("the device has no status word yet: call status_word(device) before the capture, or "
                               "pass status=")
        with torch.cuda.device(index):
            word = torch.zeros(1, dtype=torch.int32, device="cuda")
            torch.cuda.current_stream().synchronize()  # once: any stream may use it from here on
        _status_words[index] = word
    return _status_words[index]


def _check(name: str, t: torch.Tensor, shape=None, dtype=None, device=None, output=False) -> None:
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


def _op(t: torch.Tensor) -> _lib.ParkOperand:
    st = [s if n > 1 else 0 for s, n in zip(t.stride()[:3], t.shape[:3])]
    return _lib.ParkOperand(t.data_ptr(), t.shape[1], st[0], st[1], st[2])


def _ptr(t) -> ctypes.c_void_p:
    return ctypes.c_void_p(t.data_ptr() if t is not None else 0)


class _On:
    """Runs a call on the tensors' device and the given (or current) stream, so that
    memory allocated inside belongs to that stream."""

    def __init__(self, device, stream):
        if stream is not None and stream.device != device:
            raise ValueError(f"stream on {stream.device}, tensors on {device}")
        self.dev, self.stream = torch.cuda.device(device), stream

    def __enter__(self):
        self.dev.__enter__()
        self.ctx = torch.cuda.stream(self.stream) if self.stream is not None else None
        if self.ctx is not None:
            self.ctx.__enter__()
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)
        self.dev.__exit__(*exc)


def _status(status, device) -> torch.Tensor:
    if status is None:
        return status_word(device)
    if status.dtype != torch.int32 or status.numel() != 1 or status.device != device:
        raise ValueError("status must be int32 [1] on the tensors' device")
    return status


def _workspace(ws, need: int, device) -> torch.Tensor:
    if ws is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    if not ws.is_contiguous() or ws.device != device:
        raise ValueError("ws must be contiguous on the tensors' device")
    return ws


# ------------------------------------------------------------------ rotary positions
@dataclasses.dataclass
class Rope:
    """Rotary axes and their table (see park_rope_axes in include/park.h)."""
    extent: tuple            # (frames, rows, columns)
    pairs: tuple             # rotated pairs of each axis
    half: bool               # False: pairs (2j, 2j+1); True: (j, j + D/2)
    table: torch.Tensor      # float32, (cos, sin) of every position of every axis

    def c(self) -> _lib.ParkRopeAxes:
        i3 = ctypes.c_int * 3
        return _lib.ParkRopeAxes(i3(*self.extent), i3(*self.pairs), int(self.half),
                                 ctypes.c_void_p(self.table.data_ptr()))


def rope_table(extent, D: int, pairs=None, theta: float = 10000.0, scale=(1.0, 1.0, 1.0), half: bool = False,
               device=None, stream=None) -> Rope:
    """Table of the angles (scale_a pos) theta^(-j / pairs_a) of each axis, made once
    and kept.  extent = (frames, rows, columns); pairs defaults to the split of D/2
    that the synthetic layers use: a third each for rows and columns, the rest for
    time (22/21/21 at D = 128).  For plain 1-D positions pass extent (n, 1, 1) and
    pairs (D/2, 0, 0)."""
    if pairs is None:
        third = D // 2 // 3
        pairs = (D // 2 - 2 * third, third, third)
    extent, pairs = tuple(int(x) for x in extent), tuple(int(x) for x in pairs)
    if len(extent) != 3 or len(pairs) != 3 or len(scale) != 3:
        raise ValueError("extent, pairs and scale have one entry for each of the three axes")
    if min(extent) < 1 or min(pairs) < 0 or sum(pairs) > D // 2:
        raise ValueError(f"extents {extent} must be positive and pairs {pairs} sum to at most D/2 = {D // 2}")
    dev = torch.device("cuda" if device is None else device)
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    with _On(dev, stream) as st:
        r = Rope(extent, pairs, bool(half), torch.empty(0, dtype=torch.float32, device=dev))
        n = _lib.load().park_rope_table_floats(ctypes.byref(r.c()))
        r.table = torch.empty(max(2, n), dtype=torch.float32, device=dev)
        rc = _lib.load().park_rope_table(ctypes.byref(r.c()), float(theta),
                                         (ctypes.c_double * 3)(*[float(x) for x in scale]), st)
    _lib.check(rc, "park_rope_table")
    return r


def _rope_args(rope, positions, B: int, N: int, D: int, device):
    if rope is None:
        if positions is not None:
            raise ValueError("positions without rope")
        return None, ctypes.c_void_p(0), 0
    if rope.table.device != device:
        raise ValueError(f"rope table on {rope.table.device}, tensors on {device}")
    if sum(rope.pairs) > D // 2:
        raise ValueError(f"rope rotates {sum(rope.pairs)} pairs, the head has {D // 2}")
    if positions is None:
        return ctypes.byref(rope.c()), ctypes.c_void_p(0), 0
    if (positions.dtype != torch.int32 or positions.device != device or not positions.is_contiguous()
            or tuple(positions.shape) not in ((N, 3), (B, N, 3))):
        raise ValueError(f"positions must be contiguous int32 [N, 3] or [B, N, 3] with N = {N} on {device}")
    return ctypes.byref(rope.c()), _ptr(positions), 3 * N if positions.dim() == 3 else 0


def rope(x, rope: Rope, positions=None, inverse: bool = False, out=None, status=None, stream=None) -> torch.Tensor:
    """x rotated by its tokens' positions; ``inverse`` rotates back, which is also the
    gradient (dx from dy).  positions: int32 [N, 3] or [B, N, 3] with (t, y, w) of each
    token, negative for text (not rotated); None: the grid order of Shape, tokens behind
    the grid not rotated.  ``out`` may be x."""
    _check("x", x)
    B, H, N, D = x.shape
    with _On(x.device, stream) as st:
        out = torch.empty_like(x) if out is None else out
        _check("out", out, x.shape, x.dtype, x.device, output=True)
        axes, pos, sb = _rope_args(rope, positions, B, N, D, x.device)
        if axes is None:
            raise ValueError("rope is missing")
        rc = _lib.load().park_rope(_op(x), _op(out), B, N, D, _DT[x.dtype], axes, pos, sb, int(inverse),
                                   _ptr(_status(status, x.device)), st) if B * H else 0
    _lib.check(rc, "park_rope")
    return out


# ------------------------------------------------------------------ norm + rotation
def _pair_check(q, k, more=()):
    _check("q", q)
    B, _, N, D = q.shape
    _check("k", k, (B, k.shape[1] if k.dim() == 4 else 0, N, D), q.dtype, q.device)
    if min(B, q.shape[1], k.shape[1]) < 1:
        raise ValueError("q and k need at least one batch entry and one head")
    for name, t, like in more:
        _check(name, t, like.shape, q.dtype, q.device)
    return B, N, D


def _weights(q_weight, k_weight, D: int, device):
    dt = None
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is None:
            continue
        if tuple(w.shape) != (D,) or w.dtype not in _DT or not w.is_contiguous() or w.device != device:
            raise ValueError(f"{name} must be contiguous [D] in bfloat16 or float32 on {device}")
        if dt is not None and w.dtype != dt:
            raise TypeError("q_weight and k_weight have different dtypes")
        dt = w.dtype
    return _ptr(q_weight), _ptr(k_weight), _DT[dt or torch.float32]


def qk_norm_rope(q, k, q_weight=None, k_weight=None, rope: Rope | None = None, positions=None, eps: float = 1e-6,
                 q_out=None, k_out=None, status=None, stream=None):
    """(q', k'): each head row divided by its root mean square (with eps > 0), times the
    weight [D] (None: ones), rotated as by ``rope`` (None: not), in one pass, float32
    inside and rounded once.  q has H heads, k may have fewer.  New outputs are
    contiguous [B, H, N, D], the layout that layer() takes; q_out may be q, k_out k."""
    B, N, D = _pair_check(q, k)
    with _On(q.device, stream) as st:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device) if q_out is None else q_out
        k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device) if k_out is None else k_out
        _check("q_out", q_out, q.shape, q.dtype, q.device, output=True)
        _check("k_out", k_out, k.shape, k.dtype, k.device, output=True)
        axes, pos, sb = _rope_args(rope, positions, B, N, D, q.device)
        wq, wk, wdt = _weights(q_weight, k_weight, D, q.device)
        rc = _lib.load().park_qk_norm_rope(_op(q), _op(k), wq, wk, wdt, float(eps), axes, pos, sb, _op(q_out),
                                           _op(k_out), B, N, D, _DT[q.dtype], _ptr(_status(status, q.device)), st)
    _lib.check(rc, "park_qk_norm_rope")
    return q_out, k_out


def qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight=None, k_weight=None, rope: Rope | None = None, positions=None,
                     eps: float = 1e-6, dq=None, dk=None, ws=None, status=None, stream=None):
    """(dq, dk, dq_weight, dk_weight) from the gradients of qk_norm_rope's outputs and its
    own inputs.  dq, dk in the inputs' type; the weights' gradients float32 [D], None
    where there is no weight."""
    B, N, D = _pair_check(q, k, (("dq_out", dq_out, q), ("dk_out", dk_out, k)))
    lib = _lib.load()
    with _On(q.device, stream) as st:
        dq = torch.empty(q.shape, dtype=q.dtype, device=q.device) if dq is None else dq
        dk = torch.empty(k.shape, dtype=k.dtype, device=k.device) if dk is None else dk
        _check("dq", dq, q.shape, q.dtype, q.device, output=True)
        _check("dk", dk, k.shape, k.dtype, k.device, output=True)
        axes, pos, sb = _rope_args(rope, positions, B, N, D, q.device)
        wq, wk, wdt = _weights(q_weight, k_weight, D, q.device)
        need = ctypes.c_size_t(0)
        _lib.check(lib.park_qk_norm_rope_bwd_workspace(B, N, D, ctypes.byref(need)), "park_qk_norm_rope_bwd_workspace")
        ws = _workspace(ws, need.value, q.device)
        dw = [torch.empty(D, dtype=torch.float32, device=q.device) if w is not None else None
              for w in (q_weight, k_weight)]
        rc = lib.park_qk_norm_rope_bwd(_op(dq_out), _op(dk_out), _op(q), _op(k), wq, wk, wdt, float(eps), axes, pos, sb,
                                       _op(dq), _op(dk), _ptr(dw[0]), _ptr(dw[1]), B, N, D, _DT[q.dtype], _ptr(ws),
                                       ws.numel() * ws.element_size(), _ptr(_status(status, q.device)), st)
    _lib.check(rc, "park_qk_norm_rope_bwd")
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
        with _On(q.device, stream):
            outs = [torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k)]
        return tuple(rope(t, self.rope, self.positions, out=o, status=status, stream=stream)
                     for t, o in zip((q, k), outs))


# ------------------------------------------------------------------ dense attention
def _attn_shape(q, k, causal, scale, cu_q, cu_k) -> _lib.ParkAttnShape:
    B, _, Nq, D = q.shape
    Nk, n_seq = k.shape[2], 0
    if (cu_q is None) != (cu_k is None):
        raise ValueError("cu_q and cu_k go together")
    if cu_q is not None:
        for name, cu in (("cu_q", cu_q), ("cu_k", cu_k)):
            if cu.dtype != torch.int32 or cu.dim() != 1 or not cu.is_contiguous() or cu.device != q.device:
                raise ValueError(f"{name} must be a contiguous int32 vector on {q.device}")
        if cu_q.numel() != cu_k.numel() or cu_q.numel() < 2:
            raise ValueError("cu_q and cu_k hold the sequences' bounds: n_seq + 1 entries each")
        if B != 1:
            raise ValueError("packed sequences need B = 1")
        n_seq = cu_q.numel() - 1
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    return _lib.ParkAttnShape(B, D, _DT[q.dtype], Nq, Nk, n_seq, _ptr(cu_q), _ptr(cu_k), int(bool(causal)), scale)


def _attn_check(Q, K, V):
    _check("Q", Q)
    if K.dim() != 4 or V.dim() != 4:
        raise ValueError("K, V: expected CUDA tensors [B, H, N, D]")
    B, H, _, D = Q.shape
    _check("K", K, (B, K.shape[1], K.shape[2], D), Q.dtype, Q.device)
    _check("V", V, K.shape, Q.dtype, Q.device)
    if min(B, H, K.shape[1]) < 1 or H % K.shape[1]:
        raise ValueError(f"{K.shape[1]} key heads do not divide {H} query heads")


def _lse(lse, Q):
    want = tuple(Q.shape[:3])
    if tuple(lse.shape) != want or lse.dtype != torch.float32 or not lse.is_contiguous() or lse.device != Q.device:
        raise ValueError(f"lse must be contiguous float32 {want} on {Q.device}")
    return lse


def attention_workspace_size(Q, K, causal: bool = False, cu_q=None, cu_k=None, backward: bool = False) -> int:
    """Bytes of device workspace that attention (or attention_bwd) takes for these tensors."""
    s, n = _attn_shape(Q, K, causal, None, cu_q, cu_k), ctypes.c_size_t(0)
    _lib.check(_lib.load().park_attention_workspace(ctypes.byref(s), Q.shape[1], K.shape[1], int(backward),
                                                    ctypes.byref(n)), "park_attention_workspace")
    return int(n.value)


def attention(Q, K, V, causal: bool = False, scale: float | None = None, cu_q=None, cu_k=None, O=None,
              return_lse: bool = False, lse=None, ws=None, status=None, stream=None):
    """Dense attention: O, or (O, lse) with return_lse.

    Q [B, Hq, Nq, D], K and V [B, Hk, Nk, D], Hk dividing Hq (query head h reads key head
    h // (Hq // Hk)).  cu_q, cu_k (int32 [n_seq + 1] on the device, B = 1) pack sequences
    of different, possibly zero, lengths; rows outside them are not written (in a new O
    they are undefined).  causal: row i sees keys j <= i + n_k - n_q.  Rows without a key
    give 0 and lse = -inf.  scale defaults to 1/sqrt(D)."""
    _attn_check(Q, K, V)
    lib = _lib.load()
    with _On(Q.device, stream) as st:
        O = torch.empty_like(Q) if O is None else O
        _check("O", O, Q.shape, Q.dtype, Q.device, output=True)
        if lse is None:
            lse = torch.empty(Q.shape[:3], dtype=torch.float32, device=Q.device) if return_lse else None
        else:
            _lse(lse, Q)
        s, need = _attn_shape(Q, K, causal, scale, cu_q, cu_k), ctypes.c_size_t(0)
        _lib.check(lib.park_attention_workspace(ctypes.byref(s), Q.shape[1], K.shape[1], 0, ctypes.byref(need)),
                   "park_attention_workspace")
        ws = _workspace(ws, need.value, Q.device)
        rc = lib.park_attention(ctypes.byref(s), _op(Q), _op(K), _op(V), _op(O), _ptr(lse), _ptr(ws),
                                ws.numel() * ws.element_size(), _ptr(_status(status, Q.device)), st)
    _lib.check(rc, "park_attention")
    return (O, lse) if return_lse else O


def attention_bwd(dO, Q, K, V, O, lse, causal: bool = False, scale: float | None = None, cu_q=None, cu_k=None, dQ=None,
                  dK=None, dV=None, ws=None, status=None, stream=None):
    """(dQ, dK, dV) from dO and from attention's inputs and results; dK and dV are sums
    over the query heads that share a key head.  Rows outside the packed sequences are
    not written (in new tensors they are undefined)."""
    _attn_check(Q, K, V)
    _check("O", O, Q.shape, Q.dtype, Q.device)
    _check("dO", dO, Q.shape, Q.dtype, Q.device)
    _lse(lse, Q)
    lib = _lib.load()
    with _On(Q.device, stream) as st:
        outs = []
        for name, t, like in (("dQ", dQ, Q), ("dK", dK, K), ("dV", dV, V)):
            t = torch.empty_like(like) if t is None else t
            _check(name, t, like.shape, Q.dtype, Q.device, output=True)
            outs.append(t)
        s, need = _attn_shape(Q, K, causal, scale, cu_q, cu_k), ctypes.c_size_t(0)
        _lib.check(lib.park_attention_workspace(ctypes.byref(s), Q.shape[1], K.shape[1], 1, ctypes.byref(need)),
                   "park_attention_workspace")
        ws = _workspace(ws, need.value, Q.device)
        rc = lib.park_attention_bwd(ctypes.byref(s), _op(dO), _op(Q), _op(K), _op(V), _op(O), _ptr(lse), _op(outs[0]),
                                    _op(outs[1]), _op(outs[2]), _ptr(ws), ws.numel() * ws.element_size(),
                                    _ptr(_status(status, Q.device)), st)
    _lib.check(rc, "park_attention_bwd")
    return tuple(outs)
