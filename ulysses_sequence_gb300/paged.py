"""Torch helpers of the paged key/value cache calls (include/ulysses.h, "Serving from a paged key/value
cache"); the package offers them under its own name.

One serving step is ``page_plan`` (block tables and slots from request lengths), ``kv_append`` (the new
tokens' keys and values to their slots) and ``paged_attn_fwd`` (attention over the pages). Every length
stays on the device, so a step can be captured into a CUDA graph and replayed while requests grow.

Tensors must be on the current device; a call runs on the current stream or on the one given, and what it
allocates belongs to that stream. Wrong types, shapes, strides or devices raise ValueError before anything
is launched, what the library refuses raises UlyssesError.

The calls are small enough for the host's work to show, so the checks are plain conditions in line, and a
message is put together only when one fails.
"""

from __future__ import annotations

import ctypes
from typing import Optional

import torch

import ulysses_sequence_gb300 as U

_I32, _BF16, _F32 = torch.int32, torch.bfloat16, torch.float32
_E4M3, _E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
_INT_MAX = 2 ** 31 - 1  # of the C ABI's int arguments, which ctypes would wrap
# The short cuts behind torch.cuda.current_device() and current_stream().cuda_stream (an append of 64 rows takes the
# host 4.6 us with them and 6.1 us without), where this build of torch has them.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda device: torch.cuda.current_stream(device).cuda_stream)


def _refuse(x, name: str, shape, dtype, device: int, where: str):
    raise ValueError(f"{where}: {name} must be contiguous {dtype} {tuple(shape)} on device {device}, got {x.dtype} "
                     f"{tuple(x.shape)} with strides {x.stride()} on {x.device}")


def _stream_of(device: int, stream, where: str) -> int:
    """The CUDA stream of a call on this device, which must be the current one."""
    if device < 0:
        raise ValueError(f"{where}: tensors must be on a CUDA device")
    if device != _current_device():
        raise ValueError(f"{where}: the tensors are on device {device}, the current device is {_current_device()}")
    if stream is None:
        return _raw_stream(device)
    if stream.device.index != device:
        raise ValueError(f"{where}: the stream is on {stream.device}, the tensors on device {device}")
    return stream.cuda_stream


def _new(shape, dtype, device: int, stream):
    """An output allocated for the stream of the call, so that its memory is not reused before the call has run."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _no_table(x, where: str):
    raise ValueError(f"{where}: block_table must be int32 [B][max_pages], got {x.dtype} {tuple(x.shape)}")


def _table_stride(x, B: int, device: int, where: str) -> int:
    """Row stride of an int32 block table [B][max_pages] with contiguous rows on this device."""
    if x.dtype is _I32 and x.dim() == 2 and x.shape[0] == B and x.get_device() == device:
        row, one = x.stride()
        if one == 1 or x.shape[1] < 2 or B == 0:
            return row if B > 1 else x.shape[1]
    raise ValueError(f"{where}: block_table must be int32 [{B}][max_pages] with contiguous rows on device {device}, "
                     f"got {x.dtype} {tuple(x.shape)} with strides {x.stride()} on {x.device}")


def _row_stride(x, T: int, heads: int, d: int, device: int, name: str, where: str) -> int:
    """Row stride of bf16 token rows [T][heads][d] whose rows are contiguous, on this device."""
    if x.shape == (T, heads, d) and x.dtype is _BF16 and x.get_device() == device:
        row, head, one = x.stride()
        if T == 0:
            return heads * d
        if one == 1 and (heads == 1 or head == d):
            return row if T > 1 else heads * d
    raise ValueError(f"{where}: {name} must be bf16 [{T}][{heads}][{d}] with contiguous rows on device {device}, got "
                     f"{x.dtype} {tuple(x.shape)} with strides {x.stride()} on {x.device}")


class PagedCache:
    """A pool of key/value pages for the C ABI: k and v bf16 [num_pages][page_size][H_kv][d] with equal
    strides and contiguous heads (any order of the first three dimensions in memory)."""

    codes = False

    def __init__(self, k, v):
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride():
            raise ValueError("PagedCache: k and v must have the same shape [num_pages][page_size][H_kv][d] and strides")
        if k.dtype != _BF16 or v.dtype != _BF16 or k.stride(3) != 1:
            raise ValueError("PagedCache: k and v must be bf16 with contiguous heads")
        if max(k.shape) > _INT_MAX:
            raise ValueError(f"PagedCache: sizes must fit 32 bits, got {tuple(k.shape)}")
        if not k.is_cuda or k.device != v.device:
            raise ValueError("PagedCache: k and v must be on one CUDA device")
        self.k, self.v, self.device = k, v, k.get_device()
        self.num_pages, self.page_size, self.H_kv, self.d = k.shape
        self.struct = U.KVCacheStruct(k.data_ptr(), v.data_ptr(), *k.shape, k.stride(0), k.stride(1), k.stride(2))
        self.ref = ctypes.byref(self.struct)

    @staticmethod
    def empty(num_pages: int, page_size: int, H_kv: int, d: int, device="cuda") -> "PagedCache":
        """A pool in the token layout, its contents undefined (unwritten entries are never used)."""
        return PagedCache(*(torch.empty((num_pages, page_size, H_kv, d), dtype=_BF16, device=device) for _ in range(2)))


class PagedCache8:
    """A pool of key/value pages in 8 bits for the C ABI: k and v float8_e4m3fn [num_pages][page_size][H_kv][d], strided like
    PagedCache's, and k_scale and v_scale float8_e8m0fnu [num_pages][page_size / block][H_kv] contiguous, one power of
    two for each `block` tokens of a page and head: key = k * k_scale. Scales lie in [2^-117, 2^119]."""

    codes = True

    def __init__(self, k, v, k_scale, v_scale):
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride():
            raise ValueError("PagedCache8: k and v must have the same shape [num_pages][page_size][H_kv][d] and strides")
        if k.dtype != _E4M3 or v.dtype != _E4M3 or k.stride(3) != 1:
            raise ValueError("PagedCache8: k and v must be float8_e4m3fn with contiguous heads")
        if max(k.shape) > _INT_MAX:
            raise ValueError(f"PagedCache8: sizes must fit 32 bits, got {tuple(k.shape)}")
        pages, page, H_kv, _ = k.shape
        blocks = k_scale.shape[1] if k_scale.dim() == 3 else 0
        for name, x in (("k_scale", k_scale), ("v_scale", v_scale)):
            if x.dtype != _E8M0 or blocks < 1 or x.shape != (pages, blocks, H_kv) or page % blocks or not x.is_contiguous():
                raise ValueError(f"PagedCache8: {name} must be contiguous float8_e8m0fnu [{pages}][blocks that divide {page}][{H_kv}], got "
                                 f"{x.dtype} {tuple(x.shape)} with strides {x.stride()}")
        if not k.is_cuda or any(x.device != k.device for x in (v, k_scale, v_scale)):
            raise ValueError("PagedCache8: k, v and their scales must be on one CUDA device")
        self.k, self.v, self.k_scale, self.v_scale, self.device = k, v, k_scale, v_scale, k.get_device()
        self.num_pages, self.page_size, self.H_kv, self.d = k.shape
        self.block = page // blocks
        self.struct = U.KVCache8Struct(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), *k.shape, k.stride(0),
                                       k.stride(1), k.stride(2), self.block)
        self.ref = ctypes.byref(self.struct)

    @staticmethod
    def empty(num_pages: int, page_size: int, H_kv: int, d: int, block: Optional[int] = None, device="cuda") -> "PagedCache8":
        """A pool in the token layout, its codes undefined (unwritten entries are never used), its scales the smallest; one
        scale a page and head unless `block` says how many tokens share one."""
        block = page_size if block is None else block
        if block < 1 or page_size % block:
            raise ValueError(f"PagedCache8: block must divide page_size {page_size}, got {block}")
        kv = (torch.empty((num_pages, page_size, H_kv, d), dtype=torch.uint8, device=device).view(_E4M3) for _ in range(2))
        scales = (torch.full((num_pages, page_size // block, H_kv), 10, dtype=torch.uint8, device=device).view(_E8M0) for _ in range(2))
        return PagedCache8(*kv, *scales)


def page_plan(cached_lens, new_lens, free_pages, n_free, block_table, page_size: int, num_pages: int, T: int, cu_q=None,
              kv_lens=None, slot_map=None, info=None, stream=None):
    """Block tables and slot maps of one step from request lengths, on the GPU (all int32): B requests hold
    cached_lens[B] tokens and add new_lens[B]; new pages come from the end of free_pages[: n_free[0]] and
    are written into block_table [B][max_pages] in place. Returns (cu_q [B+1], kv_lens [B], slot_map [T],
    info [4] = rows planned, pages taken, pages missing, tokens dropped). The list is not changed:
    ``n_free -= info[1:2]`` keeps the pages."""
    where = "page_plan"
    if not (0 <= T <= _INT_MAX and -1 <= num_pages <= _INT_MAX and -1 <= page_size <= _INT_MAX):
        raise ValueError(f"{where}: T, num_pages and page_size must fit 32 bits, got {T}, {num_pages}, {page_size}")
    B, width = block_table.shape if block_table.dim() == 2 else _no_table(block_table, where)
    capacity = free_pages.numel()
    if B > _INT_MAX or width > _INT_MAX or capacity > _INT_MAX:
        raise ValueError(f"{where}: requests, pages of a request and free pages must fit 32 bits, got {B}, {width}, {capacity}")
    dev = block_table.get_device()
    table_stride = _table_stride(block_table, B, dev, where)
    one, many = (B,), (B + 1,)
    if not (cached_lens.shape == one and cached_lens.dtype is _I32 and cached_lens.get_device() == dev
            and cached_lens.is_contiguous()):
        _refuse(cached_lens, "cached_lens", one, _I32, dev, where)
    if not (new_lens.shape == one and new_lens.dtype is _I32 and new_lens.get_device() == dev and new_lens.is_contiguous()):
        _refuse(new_lens, "new_lens", one, _I32, dev, where)
    if not (n_free.shape == (1,) and n_free.dtype is _I32 and n_free.get_device() == dev):
        _refuse(n_free, "n_free", (1,), _I32, dev, where)
    if not (free_pages.dim() == 1 and free_pages.dtype is _I32 and free_pages.get_device() == dev
            and free_pages.is_contiguous()):
        _refuse(free_pages, "free_pages", (capacity,), _I32, dev, where)
    st = _stream_of(dev, stream, where)
    if cu_q is None:
        cu_q = _new(many, _I32, dev, stream)
    elif not (cu_q.shape == many and cu_q.dtype is _I32 and cu_q.get_device() == dev and cu_q.is_contiguous()):
        _refuse(cu_q, "cu_q", many, _I32, dev, where)
    if kv_lens is None:
        kv_lens = _new(one, _I32, dev, stream)
    elif not (kv_lens.shape == one and kv_lens.dtype is _I32 and kv_lens.get_device() == dev and kv_lens.is_contiguous()):
        _refuse(kv_lens, "kv_lens", one, _I32, dev, where)
    if slot_map is None:
        slot_map = _new((T,), _I32, dev, stream)
    elif not (slot_map.shape == (T,) and slot_map.dtype is _I32 and slot_map.get_device() == dev
              and slot_map.is_contiguous()):
        _refuse(slot_map, "slot_map", (T,), _I32, dev, where)
    if info is None:
        info = _new((4,), _I32, dev, stream)
    elif not (info.shape == (4,) and info.dtype is _I32 and info.get_device() == dev and info.is_contiguous()):
        _refuse(info, "info", (4,), _I32, dev, where)
    rc = U.load().ulysses_page_plan(B, T, page_size, width, table_stride, num_pages, cached_lens.data_ptr(),
                                    new_lens.data_ptr(), free_pages.data_ptr(), capacity, n_free.data_ptr(),
                                    block_table.data_ptr(), cu_q.data_ptr(), kv_lens.data_ptr(), slot_map.data_ptr(),
                                    info.data_ptr(), st)
    if rc:
        U.check(rc, where)
    return cu_q, kv_lens, slot_map, info


def kv_append(k, v, cache, slot_map, stream=None) -> None:
    """Writes the keys and values of new tokens, k, v bf16 [T][H_kv][d] (rows may be strided, as in a slice of a
    fused QKV product), to the slots slot_map[T] of the cache. Tokens with a slot outside the pool are skipped.
    Into a PagedCache8 they are rounded to codes, and the scales of their blocks are set (a block that begins with one
    of them) or grown, its older tokens rounded again; rows of one block must then follow one another, without
    skipped ones between them, as page_plan places them."""
    where, dev = "kv_append", cache.device
    T = k.shape[0] if k.dim() else 0
    if T > _INT_MAX:
        raise ValueError(f"{where}: tokens must fit 32 bits, got {T}")
    k_stride = _row_stride(k, T, cache.H_kv, cache.d, dev, "k", where)
    v_stride = _row_stride(v, T, cache.H_kv, cache.d, dev, "v", where)
    if not (slot_map.shape == (T,) and slot_map.dtype is _I32 and slot_map.get_device() == dev
            and slot_map.is_contiguous()):
        _refuse(slot_map, "slot_map", (T,), _I32, dev, where)
    lib = U.load()
    append = lib.ulysses_kv_append8 if cache.codes else lib.ulysses_kv_append
    rc = append(cache.ref, T, k.data_ptr(), k_stride, v.data_ptr(), v_stride, slot_map.data_ptr(), _stream_of(dev, stream, where))
    if rc:
        U.check(rc, where)


def paged_attn_workspace(q, cache, max_q: int = 0):
    """Workspace of paged_attn_fwd for q [T][H][d]; its size depends on H, d and max_q alone, so one serves every
    step of a program. Calls that may overlap on the GPU need one each."""
    if not -1 <= max_q <= _INT_MAX:
        raise ValueError(f"paged_attn_workspace: max_q must fit 32 bits, got {max_q}")
    if q.dim() != 3:
        raise ValueError(f"paged_attn_workspace: q must be [T][H][d], got {tuple(q.shape)}")
    n = U.ulysses_paged_attn_workspace_size(q.shape[1], cache.H_kv, cache.d, max_q)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)


def paged_attn_fwd(q, cache, cu_q, kv_lens, block_table, max_q: int = 0, mask: Optional["U.Mask"] = None,
                   window: int = 0, scale: float = 0.0, o=None, lse=None, workspace=None, stream=None):
    """Attention of packed new tokens q bf16 [T][H][d] (request i owns rows cu_q[i] .. cu_q[i+1]) over the pages that
    block_table [B][max_pages] of a PagedCache or PagedCache8 names, kv_lens[B] keys each, the new tokens last. mask: Mask.causal() (the default)
    by position, with an optional sliding window, or Mask.none(). max_q bounds the new tokens of a request where
    known (1 when decoding; 0: unknown). Returns (o bf16 [T][H][d], lse fp32 [H][T]); rows behind the last
    request are left as they were."""
    where, dev = "paged_attn_fwd", cache.device
    if not (-1 <= window <= _INT_MAX and -1 <= max_q <= _INT_MAX):
        raise ValueError(f"{where}: window and max_q must fit 32 bits, got {window}, {max_q}")
    if q.dim() != 3:
        raise ValueError(f"{where}: q must be [T][H][d], got {tuple(q.shape)}")
    T, H, d = shape = q.shape
    B, width = block_table.shape if block_table.dim() == 2 else _no_table(block_table, where)
    if T > _INT_MAX or B > _INT_MAX or width > _INT_MAX:
        raise ValueError(f"{where}: rows, requests and pages of a request must fit 32 bits, got {T}, {B}, {width}")
    q_stride = _row_stride(q, T, H, cache.d, dev, "q", where)
    table_stride = _table_stride(block_table, B, dev, where)
    if not (cu_q.shape == (B + 1,) and cu_q.dtype is _I32 and cu_q.get_device() == dev and cu_q.is_contiguous()):
        _refuse(cu_q, "cu_q", (B + 1,), _I32, dev, where)
    if not (kv_lens.shape == (B,) and kv_lens.dtype is _I32 and kv_lens.get_device() == dev and kv_lens.is_contiguous()):
        _refuse(kv_lens, "kv_lens", (B,), _I32, dev, where)
    st = _stream_of(dev, stream, where)
    if o is None:
        o = _new(shape, _BF16, dev, stream)
    elif not (o.shape == shape and o.dtype is _BF16 and o.get_device() == dev and o.is_contiguous()):
        _refuse(o, "o", shape, _BF16, dev, where)
    if lse is None:
        lse = _new((H, T), _F32, dev, stream)
    elif not (lse.shape == (H, T) and lse.dtype is _F32 and lse.get_device() == dev and lse.is_contiguous()):
        _refuse(lse, "lse", (H, T), _F32, dev, where)
    if workspace is None:
        n = U.ulysses_paged_attn_workspace_size(H, cache.H_kv, d, max_q)
        workspace = _new((max(n, 256),), torch.uint8, dev, stream)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"{where}: workspace must be contiguous on device {dev}")
    lib = U.load()
    attn = lib.ulysses_paged_attn8_fwd if cache.codes else lib.ulysses_paged_attn_fwd
    rc = attn(cache.ref, B, T, H, max_q, U.MASK_CAUSAL if mask is None else mask.kind, window, scale, q.data_ptr(), q_stride,
              cu_q.data_ptr(), kv_lens.data_ptr(), block_table.data_ptr(), table_stride, width, o.data_ptr(), lse.data_ptr(),
              workspace.data_ptr(), workspace.nbytes, st)
    if rc:
        U.check(rc, where)
    return o, lse
