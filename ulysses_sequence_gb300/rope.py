"""Torch helpers of the rotary calls (include/ulysses.h, "Rotary positions of queries and keys"); the package offers
them under its own name.

``Rope`` holds the frequencies; ``qk_rope_fwd`` and ``qk_rope_bwd`` turn (and norm) the queries and keys of a sharded
layout between ``qkv_proj`` and ``attn_fwd``, and their gradients behind ``attn_bwd``; ``qk_rope_rows`` does
the packed rows of a serving step, in front of ``kv_append`` and ``paged_attn_fwd``.

Tensors must be on the current device; a call runs on the current stream or on the one given, and what it
allocates belongs to that stream. Wrong types, shapes, strides or devices raise ValueError before anything
is launched, what the library refuses raises UlyssesError.
"""

from __future__ import annotations

import ctypes
import math
from fractions import Fraction
from typing import Optional

import torch

import ulysses_sequence_gb300 as U
from .paged import _BF16, _F32, _I32, _INT_MAX, _new, _refuse, _row_stride, _stream_of

# 2 pi to 60 digits: a frequency of 64 bits in turns needs some 40
_TWO_PI = Fraction(6283185307179586476925286766559005768394338798750211641949889, 10 ** 60)


def rope_frequencies(rot: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                     trained: int = 4096, low: float = 1.0, high: float = 32.0):
    """(frequencies, amplitude): radians a token of the rot / 2 pairs, base^(-2 e / rot), for contexts `factor` times as long
    as the `trained` one:
      None      as they are;
      "linear"  all divided by factor (positions interpolated);
      "ntk"     base grown by factor^(rot / (rot - 2)): the slowest pair is stretched by factor, the fastest not at all;
      "yarn"    by parts: with the turns r that a pair makes over `trained` tokens, frequencies of r >= high stay, those of
                r <= low are divided by factor, linearly in r between; the amplitude is 0.1 ln(factor) + 1. This is the formula
                as published. Models have also been released with the ramp taken over the pair's number e between rounded
                ends, which gives other frequencies: those go to Rope(frequencies=, amplitude=)."""
    if rot < 0 or rot % 2 != 0:
        raise ValueError(f"rope_frequencies: rot must be even and not negative, got {rot}")
    if not (base > 0 and factor >= 1 and trained > 0):
        raise ValueError(f"rope_frequencies: base and trained must be positive, factor at least 1, got {base}, {trained}, {factor}")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"rope_frequencies: scaling must be None, 'linear', 'ntk' or 'yarn', got {scaling!r}")
    if scaling == "yarn" and not high > low:
        raise ValueError(f"rope_frequencies: high must be above low, got {low}, {high}")
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = [base ** (-2.0 * e / rot) for e in range(rot // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling != "yarn":
        return f, 1.0
    out = []
    for x in f:
        keep = min(1.0, max(0.0, (trained * x / (2 * math.pi) - low) / (high - low)))
        out.append(x * keep + x / factor * (1 - keep))
    return out, 0.1 * math.log(factor) + 1.0


class Rope:
    """The rotation of heads of d elements, the first `rot` of which (all by default) are turned: the frequencies on the
    device, the pairs' layout (halves, or neighbours when interleaved) and the amplitude. `frequencies` (radians a
    token, rot / 2 of them) may be given instead of base and scaling; amplitude overrides that of the scaling."""

    def __init__(self, d: int, rot: Optional[int] = None, base: float = 10000.0, interleaved: bool = False,
                 scaling: Optional[str] = None, factor: float = 1.0, trained: int = 4096, low: float = 1.0, high: float = 32.0,
                 frequencies=None, amplitude: Optional[float] = None, device="cuda"):
        rot = d if rot is None else rot
        if rot < 0 or rot > d or rot % 16 != 0:
            raise ValueError(f"Rope: rot must be a multiple of 16 from 0 to {d}, got {rot}")
        own = 1.0
        if frequencies is None:
            frequencies, own = rope_frequencies(rot, base, scaling, factor, trained, low, high)
        frequencies = [float(f) for f in frequencies]
        if len(frequencies) != rot // 2 or not all(math.isfinite(f) for f in frequencies):
            raise ValueError(f"Rope: frequencies must be {rot // 2} finite numbers, got {len(frequencies)}")
        self.d, self.rot, self.interleaved, self.frequencies = d, rot, bool(interleaved), frequencies
        self.amplitude = own if amplitude is None else float(amplitude)
        turns = [round(Fraction(f) / _TWO_PI * 2 ** 64) % 2 ** 64 for f in frequencies]
        self.turns = torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in turns], dtype=torch.int64, device=device)
        if not self.turns.is_cuda:
            raise ValueError(f"Rope: the frequencies must be on a CUDA device, got {self.turns.device}")
        self.device = self.turns.get_device()
        self.struct = U.RopeStruct(self.turns.data_ptr(), rot, int(self.interleaved), self.amplitude)
        self.ref = ctypes.byref(self.struct)


def _weights(w_q, w_k, d: int, device: int, where: str):
    """(pointer, pointer, whether they are fp32) of the norms' weights."""
    if w_q is None or w_k is None:
        if w_q is not w_k:
            raise ValueError(f"{where}: w_q and w_k must be given together")
        return None, None, 0
    dtype, shape = w_q.dtype, (d,)
    if dtype is not _BF16 and dtype is not _F32:
        _refuse(w_q, "w_q", shape, "bf16 or fp32", device, where)
    if not (w_q.shape == shape and w_q.get_device() == device and w_q.is_contiguous()):
        _refuse(w_q, "w_q", shape, dtype, device, where)
    if not (w_k.shape == shape and w_k.dtype is dtype and w_k.get_device() == device and w_k.is_contiguous()):
        _refuse(w_k, "w_k", shape, dtype, device, where)
    return w_q.data_ptr(), w_k.data_ptr(), int(dtype is _F32)


def _rows(x, T: int, heads: int, d: int, device: int, name: str, where: str) -> int:
    """_row_stride, with a short way for contiguous rows."""
    if x.is_contiguous() and x.shape == (T, heads, d) and x.dtype is _BF16 and x.get_device() == device:
        return heads * d
    return _row_stride(x, T, heads, d, device, name, where)


def _like(x, device: int, stream):
    """An output of x's shape and type, for the stream of the call."""
    return torch.empty_like(x) if stream is None else _new(x.shape, _BF16, device, stream)


def _same(x, name: str, shape, device: int, where: str) -> None:
    if not (x.shape == shape and x.dtype is _BF16 and x.get_device() == device and x.is_contiguous()):
        _refuse(x, name, shape, _BF16, device, where)


def _sharded(q, k, P: int, rope: Rope, layout: int, kv_heads: int, where: str) -> "U.Shape":
    """Shape of the sharded tensors of a call, checked."""
    if layout not in (U.LAYOUT_TOKEN_SHARDED, U.LAYOUT_HEAD_SHARDED):
        raise ValueError(f"{where}: layout must be LAYOUT_TOKEN_SHARDED or LAYOUT_HEAD_SHARDED, got {layout}")
    if q.dim() != 5 or k.dim() != 5:
        raise ValueError(f"{where}: q and k must be [{P}][B][tokens][heads][{rope.d}], got {tuple(q.shape)} and {tuple(k.shape)}")
    groups, B, tokens, heads, d = q.shape
    k_groups, k_B, k_tokens, kh, k_d = k.shape
    if groups != P or d != rope.d or k_groups != P or k_B != B or k_tokens != tokens or k_d != d:
        raise ValueError(f"{where}: q and k must be [{P}][B][tokens][heads][{rope.d}], got {tuple(q.shape)} and {tuple(k.shape)}")
    dev = rope.device
    if not (q.dtype is _BF16 and q.get_device() == dev and q.is_contiguous()):
        _refuse(q, "q", q.shape, _BF16, dev, where)
    if not (k.dtype is _BF16 and k.get_device() == dev and k.is_contiguous()):
        _refuse(k, "k", k.shape, _BF16, dev, where)
    if layout == U.LAYOUT_TOKEN_SHARDED:
        if kv_heads not in (0, kh):
            raise ValueError(f"{where}: kv_heads is {kv_heads}, k has {kh}")
        sizes = (B, tokens * P, heads, d, P, kh)
    else:
        H_kv = kv_heads or kh * P
        if kh != U.kv_heads_per_group(H_kv, P):
            raise ValueError(f"{where}: {H_kv} key/value heads over {P} groups do not give {kh} each")
        sizes = (B, tokens, heads * P, d, P, H_kv)
    if max(sizes) > _INT_MAX:
        raise ValueError(f"{where}: sizes must fit 32 bits, got {sizes}")
    return U.Shape(*sizes)


def _pos0(pos0: int, where: str) -> None:
    if not -2 ** 62 <= pos0 <= 2 ** 62:
        raise ValueError(f"{where}: pos0 must fit 62 bits, got {pos0}")


def qk_rope_fwd(q, k, P: int, rope: Rope, w_q=None, w_k=None, eps: float = 1e-6, layout: int = U.LAYOUT_TOKEN_SHARDED,
                pos0: int = 0, q_out=None, k_out=None, stream=None, kv_heads: int = 0):
    """Queries q and keys k of a sharded layout (as attn_fwd takes them, bf16), each head normed with w_q and w_k [d] (bf16
    or fp32) when they are given, then turned by its token's position, pos0 + the global token. Returns (q_out, k_out), new
    tensors unless given; q_out may be q and k_out may be k. kv_heads names H_kv when the head layout replicates key
    heads."""
    where, dev = "qk_rope_fwd", rope.device
    shape = _sharded(q, k, P, rope, layout, kv_heads, where)
    _pos0(pos0, where)
    wq, wk, wide = _weights(w_q, w_k, rope.d, dev, where)
    st = _stream_of(dev, stream, where)
    if q_out is None:
        q_out = _like(q, dev, stream)
    else:
        _same(q_out, "q_out", q.shape, dev, where)
    if k_out is None:
        k_out = _like(k, dev, stream)
    else:
        _same(k_out, "k_out", k.shape, dev, where)
    rc = U.load().ulysses_qk_rope_fwd(shape, layout, rope.ref, pos0, q.data_ptr(), k.data_ptr(), wq, wk, wide, eps,
                                      q_out.data_ptr(), k_out.data_ptr(), st)
    if rc:
        U.check(rc, where)
    return q_out, k_out


def qk_rope_bwd(dq_out, dk_out, P: int, rope: Rope, q=None, k=None, w_q=None, w_k=None, eps: float = 1e-6,
                layout: int = U.LAYOUT_TOKEN_SHARDED, pos0: int = 0, dq=None, dk=None, dw_q=None, dw_k=None, workspace=None,
                stream=None, kv_heads: int = 0):
    """Gradient of qk_rope_fwd from those of its outputs. Without weights returns (dq, dk); with them q and k are the
    forward's inputs, and (dq, dk, dw_q, dw_k) come back, the weights' gradients in fp32. dq may be dq_out or q, dk may be
    dk_out or k."""
    where, dev = "qk_rope_bwd", rope.device
    shape = _sharded(dq_out, dk_out, P, rope, layout, kv_heads, where)
    _pos0(pos0, where)
    wq, wk, wide = _weights(w_q, w_k, rope.d, dev, where)
    st = _stream_of(dev, stream, where)
    if dq is None:
        dq = _like(dq_out, dev, stream)
    else:
        _same(dq, "dq", dq_out.shape, dev, where)
    if dk is None:
        dk = _like(dk_out, dev, stream)
    else:
        _same(dk, "dk", dk_out.shape, dev, where)
    if wq is None:
        rc = U.load().ulysses_qk_rope_bwd(shape, layout, rope.ref, pos0, dq_out.data_ptr(), dk_out.data_ptr(), None, None, None,
                                          None, 0, 0.0, dq.data_ptr(), dk.data_ptr(), None, None, None, 0, st)
        if rc:
            U.check(rc, where)
        return dq, dk
    if q is None or k is None:
        raise ValueError(f"{where}: with weights, the forward's q and k are needed")
    _same(q, "q", dq_out.shape, dev, where)
    _same(k, "k", dk_out.shape, dev, where)
    if dw_q is None:
        dw_q = _new((rope.d,), _F32, dev, stream)
    elif not (dw_q.shape == (rope.d,) and dw_q.dtype is _F32 and dw_q.get_device() == dev and dw_q.is_contiguous()):
        _refuse(dw_q, "dw_q", (rope.d,), _F32, dev, where)
    if dw_k is None:
        dw_k = _new((rope.d,), _F32, dev, stream)
    elif not (dw_k.shape == (rope.d,) and dw_k.dtype is _F32 and dw_k.get_device() == dev and dw_k.is_contiguous()):
        _refuse(dw_k, "dw_k", (rope.d,), _F32, dev, where)
    if workspace is None:
        workspace = _new((max(U.ulysses_qk_rope_bwd_workspace_size(shape), 256),), torch.uint8, dev, stream)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"{where}: workspace must be contiguous on device {dev}")
    rc = U.load().ulysses_qk_rope_bwd(shape, layout, rope.ref, pos0, dq_out.data_ptr(), dk_out.data_ptr(), q.data_ptr(),
                                      k.data_ptr(), wq, wk, wide, eps, dq.data_ptr(), dk.data_ptr(), dw_q.data_ptr(),
                                      dw_k.data_ptr(), workspace.data_ptr(), workspace.nbytes, st)
    if rc:
        U.check(rc, where)
    return dq, dk, dw_q, dw_k


def qk_rope_rows(q, k, rope: Rope, positions=None, cu_q=None, kv_lens=None, w_q=None, w_k=None, eps: float = 1e-6, q_out=None,
                 k_out=None, stream=None):
    """qk_rope_fwd over the packed rows of a serving step, q [T][H][d] and k [T][H_kv][d] bf16 (rows may be strided, as in
    slices of a fused QKV product). Positions are given (int32 [T]), or those of paged_attn_fwd from cu_q [B+1] and
    kv_lens [B]: row t of request i stands at kv_lens[i] - cu_q[i+1] + t, and rows behind the last request are left as they
    were in q_out and k_out. q_out may be q and k_out may be k. Returns (q_out, k_out)."""
    where, dev = "qk_rope_rows", rope.device
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError(f"{where}: q and k must be [T][heads][{rope.d}], got {tuple(q.shape)} and {tuple(k.shape)}")
    T, H, d = q.shape
    H_kv = k.shape[1]
    if T > _INT_MAX or H > _INT_MAX or H_kv > _INT_MAX:
        raise ValueError(f"{where}: rows and heads must fit 32 bits, got {T}, {H}, {H_kv}")
    if d != rope.d:
        raise ValueError(f"{where}: q must be bf16 [{T}][{H}][{rope.d}], got {tuple(q.shape)}")
    q_stride = _rows(q, T, H, d, dev, "q", where)
    k_stride = _rows(k, T, H_kv, d, dev, "k", where)
    B = at = ends = lens = None
    if positions is not None:
        if cu_q is not None or kv_lens is not None:
            raise ValueError(f"{where}: positions, or cu_q and kv_lens, not both")
        if not (positions.shape == (T,) and positions.dtype is _I32 and positions.get_device() == dev and positions.is_contiguous()):
            _refuse(positions, "positions", (T,), _I32, dev, where)
        B, at = 0, positions.data_ptr()
    elif cu_q is None or kv_lens is None:
        raise ValueError(f"{where}: positions, or cu_q and kv_lens, must be given")
    else:
        B = kv_lens.shape[0] if kv_lens.dim() else 0
        if B > _INT_MAX:
            raise ValueError(f"{where}: requests must fit 32 bits, got {B}")
        if not (kv_lens.shape == (B,) and kv_lens.dtype is _I32 and kv_lens.get_device() == dev and kv_lens.is_contiguous()):
            _refuse(kv_lens, "kv_lens", (B,), _I32, dev, where)
        if not (cu_q.shape == (B + 1,) and cu_q.dtype is _I32 and cu_q.get_device() == dev and cu_q.is_contiguous()):
            _refuse(cu_q, "cu_q", (B + 1,), _I32, dev, where)
        ends, lens = cu_q.data_ptr(), kv_lens.data_ptr()
    wq, wk, wide = _weights(w_q, w_k, d, dev, where)
    st = _stream_of(dev, stream, where)
    q_out_stride, k_out_stride = H * d, H_kv * d
    if q_out is None:
        q_out = _new((T, H, d), _BF16, dev, stream)
    else:
        q_out_stride = q_stride if q_out is q else _rows(q_out, T, H, d, dev, "q_out", where)
    if k_out is None:
        k_out = _new((T, H_kv, d), _BF16, dev, stream)
    else:
        k_out_stride = k_stride if k_out is k else _rows(k_out, T, H_kv, d, dev, "k_out", where)
    rc = U.load().ulysses_qk_rope_rows(T, H, H_kv, d, rope.ref, q.data_ptr(), q_stride, k.data_ptr(), k_stride, at, B, ends, lens,
                                       wq, wk, wide, eps, q_out.data_ptr(), q_out_stride, k_out.data_ptr(), k_out_stride, st)
    if rc:
        U.check(rc, where)
    return q_out, k_out
