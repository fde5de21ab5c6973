"""Paged caches: step planning, encode, decode and attention over pages of int4 / int8 codes.

torch-facing wrappers over the paged entry points of the C ABI (argument checks and
marshalling only). A page holds ``P`` tokens (16, 32, 64 or 128) of every KV head:

  codes   uint8 [num_pages, Hkv, P, head_dim * bits / 8]
  scales  fp16  [num_pages, Hkv, P, head_dim / group]

and a token's place is its slot, ``page * P + offset``. The calls run on the device of
their tensors (all on one device, the plans' own) on its current stream, or on ``stream``.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import NamedTuple

import torch

from ._lib import PagedEncodeJob, check, lib
from .api import Plan, _ptr, _same_dim

PAGE_SIZES = (16, 32, 64, 128)


def _check(t, name: str, dtype, device, shape=None, contiguous: bool = True):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _plans_on(device, *plans) -> None:
    for pl in plans:
        if pl.device_index != device.index:
            raise ValueError(f"the plan was made on cuda:{pl.device_index}, the tensors are on {device}")


@contextlib.contextmanager
def _on(device, stream):
    """The tensors' device current, and the stream handle for the call."""
    if torch.cuda.current_device() == device.index:
        yield ctypes.c_void_p((stream or torch.cuda.current_stream(device)).cuda_stream)
    else:
        with torch.cuda.device(device):
            yield ctypes.c_void_p((stream or torch.cuda.current_stream(device)).cuda_stream)


def _new(make, shape, dtype, device, stream):
    """A tensor that belongs to the call's stream (so that its memory is not reused while the call
    still runs there): the current one, or ``stream``."""
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=device)


def _pages(codes, scales, plan: Plan, name: str, device=None):
    """Checks one pair of page buffers; returns (num_pages, Hkv, page size)."""
    if not isinstance(codes, torch.Tensor) or codes.dim() != 4:
        raise ValueError(f"{name}_codes must be a tensor [num_pages, Hkv, page_size, code bytes]")
    n, H, P, _ = codes.shape
    if P not in PAGE_SIZES:
        raise ValueError(f"page size must be one of {PAGE_SIZES}, got {P}")
    _check(codes, f"{name}_codes", torch.uint8, device, (n, H, P, plan.code_row_bytes))
    _check(scales, f"{name}_scales", torch.float16, codes.device, (n, H, P, plan.head_dim // plan.group))
    return n, H, P


class PagePlan(NamedTuple):
    """What :func:`page_plan` writes. ``slots`` and ``positions`` int32 [n]: the new tokens, packed
    request after request (-1 behind the last, slots -1 for refused requests); ``q_starts`` int32
    [B + 1]; ``kv_lens`` int32 [B]: lengths after the step; ``info`` int32 [4]: new tokens, pages
    taken, requests refused, pages wanted."""
    slots: torch.Tensor
    positions: torch.Tensor
    q_starts: torch.Tensor
    kv_lens: torch.Tensor
    info: torch.Tensor

    @classmethod
    def empty(cls, B: int, n_tokens: int, device, stream=None) -> "PagePlan":
        def new(n):
            return _new(torch.empty, n, torch.int32, device, stream)
        return cls(new(n_tokens), new(n_tokens), new(B + 1), new(B), new(4))


def page_plan(kv_lens, q_lens, block_table, free_pages, free_head, page_size: int, n_tokens: int = None,
              out: PagePlan = None, free_head_out=None, stream=None) -> PagePlan:
    """One serving step's block tables and slot maps, built on the GPU (see kvq_page_plan).

    kv_lens, q_lens int32 [B]: cached and new tokens; block_table int32 [B, max_pages] (rows may be
    strided) gets the new pages; free_pages int32 [F]; free_head int32 [1] counts the entries taken
    and is moved on in place unless ``free_head_out`` is given. ``n_tokens``: length of the slot map
    (at least the number of new tokens), or pass ``out``; ``out.kv_lens`` may be ``kv_lens``."""
    if not isinstance(kv_lens, torch.Tensor) or kv_lens.dim() != 1:
        raise ValueError("kv_lens must be a 1-D tensor")
    dev, B = kv_lens.device, kv_lens.shape[0]
    _check(kv_lens, "kv_lens", torch.int32, None)
    _check(q_lens, "q_lens", torch.int32, dev, (B,))
    _check(block_table, "block_table", torch.int32, dev, contiguous=False)
    if block_table.dim() != 2 or block_table.shape[0] != B or (block_table.numel() > 1 and block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError("block_table must be [B, max_pages] with contiguous rows")
    _check(free_pages, "free_pages", torch.int32, dev)
    _check(free_head, "free_head", torch.int32, dev, (1,))
    if free_head_out is None:
        free_head_out = free_head
    _check(free_head_out, "free_head_out", torch.int32, dev, (1,))
    if out is None:
        if n_tokens is None:
            raise ValueError("page_plan needs n_tokens or out")
        out = PagePlan.empty(B, int(n_tokens), dev, stream)
    n = out.slots.shape[0]
    _check(out.slots, "out.slots", torch.int32, dev, (n,))
    _check(out.positions, "out.positions", torch.int32, dev, (n,))
    _check(out.q_starts, "out.q_starts", torch.int32, dev, (B + 1,))
    _check(out.kv_lens, "out.kv_lens", torch.int32, dev, (B,))
    _check(out.info, "out.info", torch.int32, dev, (4,))
    M = block_table.shape[1]
    stride = block_table.stride(0) if B > 1 else M
    with _on(dev, stream) as s:
        check(lib.kvq_page_plan(_ptr(kv_lens), _ptr(q_lens), B, _ptr(block_table), M, stride, _ptr(free_pages),
                                free_pages.numel(), _ptr(free_head), _ptr(free_head_out), int(page_size),
                                _ptr(out.slots), _ptr(out.positions), n, _ptr(out.q_starts), _ptr(out.kv_lens),
                                _ptr(out.info), s), "kvq_page_plan")
    return out


def page_release(done, kv_lens, block_table, free_pages, free_head, page_size: int, stream=None) -> None:
    """Rows with ``done`` (bool or uint8 [B]) give their pages back to the free list and get length 0
    (see kvq_page_release); kv_lens, free_pages and free_head are changed in place."""
    if not isinstance(kv_lens, torch.Tensor) or kv_lens.dim() != 1:
        raise ValueError("kv_lens must be a 1-D tensor")
    dev, B = kv_lens.device, kv_lens.shape[0]
    _check(kv_lens, "kv_lens", torch.int32, None)
    if not isinstance(done, torch.Tensor) or done.dtype not in (torch.bool, torch.uint8):
        raise ValueError("done must be a bool or uint8 tensor")
    _check(done, "done", done.dtype, dev, (B,))
    _check(block_table, "block_table", torch.int32, dev, contiguous=False)
    if block_table.dim() != 2 or block_table.shape[0] != B or (block_table.numel() > 1 and block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError("block_table must be [B, max_pages] with contiguous rows")
    _check(free_pages, "free_pages", torch.int32, dev)
    _check(free_head, "free_head", torch.int32, dev, (1,))
    M = block_table.shape[1]
    with _on(dev, stream) as s:
        check(lib.kvq_page_release(_ptr(done), _ptr(kv_lens), _ptr(block_table), block_table.stride(0) if B > 1 else M,
                                   B, M, int(page_size), _ptr(free_pages), free_pages.numel(), _ptr(free_head), s),
              "kvq_page_release")


def encode_paged(jobs, slots, stream=None) -> None:
    """Encode tokens into pages: ``jobs`` is a sequence of (plan, x, codes, scales), x fp16
    [n, Hkv, D] (any token and head strides that are multiples of 8, e.g. a slice of a fused
    projection), ``slots`` int32 [n] shared by all jobs; a slot outside the pages (-1) skips its
    token. Two jobs (K and V) share a launch. See kvq_encode_paged."""
    if not jobs:
        return
    dev = slots.device if isinstance(slots, torch.Tensor) else None
    arr = (PagedEncodeJob * len(jobs))()
    geometry = None
    for i, (plan, x, codes, scales) in enumerate(jobs):
        _check(x, f"jobs[{i}].x", torch.float16, None, contiguous=False)
        if x.dim() != 3 or (x.shape[2] > 1 and x.stride(2) != 1):
            raise ValueError(f"jobs[{i}].x must be [n, Hkv, head_dim] with contiguous rows")
        n, H, D = x.shape
        _same_dim(D, plan)
        pages, Hc, P = _pages(codes, scales, plan, f"jobs[{i}]", x.device)
        if Hc != H:
            raise ValueError(f"jobs[{i}]: x has {H} heads, the pages {Hc}")
        _check(slots, "slots", torch.int32, x.device, (n,))
        _plans_on(x.device, plan)
        if geometry is not None and geometry != (n, H, P, pages):
            raise ValueError(f"jobs[{i}] has other sizes than jobs[0]")
        geometry = (n, H, P, pages)
        arr[i] = PagedEncodeJob(plan.handle.value, x.data_ptr(), codes.data_ptr(), scales.data_ptr(), x.stride(0),
                                x.stride(1))
    n, H, P, pages = geometry
    if n == 0 or H == 0:
        return
    with _on(dev, stream) as s:
        check(lib.kvq_encode_paged(arr, len(jobs), n, H, P, pages, _ptr(slots), s), "kvq_encode_paged")


def decode_paged(plan: Plan, codes, scales, slots, out=None, stream=None) -> torch.Tensor:
    """The rows at ``slots`` (int32 [n], any order) decoded to fp16 [n, Hkv, D]; a slot outside the
    pages gives zeros. See kvq_decode_paged."""
    pages, H, P = _pages(codes, scales, plan, "decode_paged")
    dev = codes.device
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        raise ValueError("slots must be a 1-D tensor")
    n, D = slots.shape[0], plan.head_dim
    _check(slots, "slots", torch.int32, dev)
    _plans_on(dev, plan)
    if out is None:
        out = _new(torch.empty, (n, H, D), torch.float16, dev, stream)
    _check(out, "out", torch.float16, dev, (n, H, D))
    if n == 0 or H == 0:
        return out
    with _on(dev, stream) as s:
        check(lib.kvq_decode_paged(plan.handle, _ptr(codes), _ptr(scales), pages, P, H, _ptr(slots), n, _ptr(out), s),
              "kvq_decode_paged")
    return out


def paged_workspace_size(B: int, Hq: int, Hkv: int, head_dim: int, n_tokens: int, max_q_len: int) -> int:
    return int(lib.kvq_paged_workspace_size(B, Hq, Hkv, head_dim, n_tokens, max_q_len))


def make_paged_workspace(B: int, Hq: int, Hkv: int, head_dim: int, n_tokens: int = None, max_q_len: int = 1,
                         device=None, stream=None) -> torch.Tensor:
    """A zero-initialised workspace for :func:`attend_paged` with up to ``B`` requests, ``n_tokens``
    query tokens and ``max_q_len`` of one request. Calls that may overlap need one each."""
    n = max(16, paged_workspace_size(B, Hq, Hkv, head_dim, B if n_tokens is None else n_tokens, max_q_len))
    return _new(torch.zeros, n, torch.uint8, device or torch.device("cuda"), stream)


def attend_paged(pk: Plan, pv: Plan, q, k_codes, k_scales, v_codes, v_scales, block_table, kv_lens, q_starts=None,
                 max_q_len: int = None, max_kv_len: int = None, window: int = 0, softmax_scale: float = 0.0, out=None,
                 workspace=None, stream=None) -> torch.Tensor:
    """Causal attention of ragged queries over paged caches (see kvq_attend_paged).

    q fp16 [n, Hq, D] (token and head strides multiples of 8); block_table int32 [B, max_pages];
    kv_lens int32 [B], the new tokens included; q_starts int32 [B + 1] or None for one query token
    per request (n == B). ``max_q_len`` / ``max_kv_len`` bound the lengths, which the host cannot
    see (defaults: n and the table's capacity); a tight ``max_q_len`` picks the right kernel.
    ``window`` > 0: each token attends the last ``window`` tokens up to itself. Returns fp16
    [n, Hq, D]; rows of ``out`` that belong to no request are left as they were."""
    _check(q, "q", torch.float16, None, contiguous=False)
    if q.dim() != 3 or (q.shape[2] > 1 and q.stride(2) != 1):
        raise ValueError("q must be [n, Hq, head_dim] with contiguous rows")
    n, Hq, D = q.shape
    dev = q.device
    _same_dim(D, pk, pv)
    _plans_on(dev, pk, pv)
    pages, Hkv, P = _pages(k_codes, k_scales, pk, "k", dev)
    if _pages(v_codes, v_scales, pv, "v", dev) != (pages, Hkv, P):
        raise ValueError("K and V pages differ in size")
    _check(kv_lens, "kv_lens", torch.int32, dev)
    if kv_lens.dim() != 1:
        raise ValueError("kv_lens must be 1-D")
    B = kv_lens.shape[0]
    _check(block_table, "block_table", torch.int32, dev, contiguous=False)
    if block_table.dim() != 2 or block_table.shape[0] != B or (block_table.numel() > 1 and block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError("block_table must be [B, max_pages] with contiguous rows")
    M = block_table.shape[1]
    if q_starts is not None:
        _check(q_starts, "q_starts", torch.int32, dev, (B + 1,))
    elif n != B:
        raise ValueError(f"without q_starts every request has one query token: q has {n}, kv_lens {B}")
    if max_q_len is None:
        max_q_len = 1 if q_starts is None else max(1, n)
    if max_kv_len is None:
        max_kv_len = min(M * P, 0x7fffffff - 256)
    if out is None:
        out = _new(torch.empty, (n, Hq, D), torch.float16, dev, stream)
    _check(out, "out", torch.float16, dev, (n, Hq, D))
    if workspace is None:
        workspace = make_paged_workspace(max(B, 1), Hq, max(Hkv, 1), D, n, max(1, int(max_q_len)), dev, stream)
    _check(workspace, "workspace", torch.uint8, dev)
    with _on(dev, stream) as s:
        check(lib.kvq_attend_paged(pk.handle, pv.handle, _ptr(q), q.stride(0), q.stride(1), _ptr(k_codes),
                                   _ptr(k_scales), _ptr(v_codes), _ptr(v_scales), pages, P, _ptr(block_table), M,
                                   block_table.stride(0) if B > 1 else M, _ptr(kv_lens), _ptr(q_starts), B, n, Hq,
                                   Hkv, int(max_q_len), int(max_kv_len), int(window), float(softmax_scale), _ptr(out),
                                   _ptr(workspace), workspace.numel(), s), "kvq_attend_paged")
    return out
