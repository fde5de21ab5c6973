"""Paged caches: step planning, encode, decode and attention over pages of int4 / int8 codes.

torch-facing entry points over the paged calls of the C ABI; arguments are checked and passed on
by the compiled binding (csrc/paged_binding.cpp). A page holds ``P`` tokens (16, 32, 64 or 128) of every KV head:

  codes   uint8 [num_pages, Hkv, P, head_dim * bits / 8]
  scales  fp16  [num_pages, Hkv, P, head_dim / group]

and a token's place is its slot, ``page * P + offset``. The calls run on the device of
their tensors (all on one device, the plans' own) on its current stream, or on ``stream``.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from ._lib import check, lib
from .api import Plan


class _Binding:
    """Stands for the compiled binding until a call needs it (the dense calls never do)."""

    def __getattr__(self, name):
        global _paged
        try:
            from . import _paged as binding
        except ImportError as e:
            raise ImportError(f"the paged calls' compiled binding does not load ({e}): build it with "
                              "`python rotated_int4_kv_b200/build.py` (g++, for the installed torch)") from e
        binding.set_check(check)
        _paged = binding
        return getattr(binding, name)


_paged = _Binding()
PAGE_SIZES = (16, 32, 64, 128)
ATTEND_PAGED_PATHS = {"auto": 0, "few": 1, "prompt": 2}


def _new(make, shape, dtype, device, stream):
    """A tensor that belongs to the call's stream (so that its memory is not reused while the call
    still runs there): the current one, or ``stream``."""
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=device)


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
    made = _paged.page_plan(kv_lens, q_lens, block_table, free_pages, free_head, page_size, n_tokens, out, free_head_out,
                            None if stream is None else stream.cuda_stream)
    return out if made is None else PagePlan(*made)


def page_release(done, kv_lens, block_table, free_pages, free_head, page_size: int, stream=None) -> None:
    """Rows with ``done`` (bool or uint8 [B]) give their pages back to the free list and get length 0
    (see kvq_page_release); kv_lens, free_pages and free_head are changed in place."""
    _paged.page_release(done, kv_lens, block_table, free_pages, free_head, page_size,
                        None if stream is None else stream.cuda_stream)


def encode_paged(jobs, slots, stream=None) -> None:
    """Encode tokens into pages: ``jobs`` is a sequence of (plan, x, codes, scales), x fp16
    [n, Hkv, D] (any token and head strides from D on that are multiples of 8, e.g. a slice of a fused
    projection), ``slots`` int32 [n] shared by all jobs; a slot outside the pages (-1) skips its
    token. Two jobs (K and V) share a launch. See kvq_encode_paged."""
    _paged.encode_paged(jobs, slots, None if stream is None else stream.cuda_stream)


def decode_paged(plan: Plan, codes, scales, slots, out=None, stream=None) -> torch.Tensor:
    """The rows at ``slots`` (int32 [n], any order) decoded to fp16 [n, Hkv, D]; a slot outside the
    pages gives zeros. See kvq_decode_paged."""
    return _paged.decode_paged(plan, codes, scales, slots, out, None if stream is None else stream.cuda_stream)


def paged_workspace_size(B: int, Hq: int, Hkv: int, head_dim: int, n_tokens: int, max_q_len: int) -> int:
    return int(lib.kvq_paged_workspace_size(B, Hq, Hkv, head_dim, n_tokens, max_q_len))


def make_paged_workspace(B: int, Hq: int, Hkv: int, head_dim: int, n_tokens: int = None, max_q_len: int = 1,
                         device=None, stream=None) -> torch.Tensor:
    """A workspace for :func:`attend_paged` with up to ``B`` requests, ``n_tokens``
    query tokens and ``max_q_len`` of one request. Calls that may overlap need one each."""
    n = max(16, paged_workspace_size(B, Hq, Hkv, head_dim, B if n_tokens is None else n_tokens, max_q_len))
    return _new(torch.empty, n, torch.uint8, device or torch.device("cuda"), stream)


def set_attend_paged_path(path: str) -> None:
    """Select the kernel of :func:`attend_paged`: "auto" (by sizes and bounds), "few" (few query rows per
    request) or "prompt" (many). Workspaces are sized for the setting."""
    check(lib.kvq_set_attend_paged_path(ATTEND_PAGED_PATHS[path]), "kvq_set_attend_paged_path")


def get_attend_paged_path() -> str:
    v = int(lib.kvq_get_attend_paged_path())
    return {n: k for k, n in ATTEND_PAGED_PATHS.items()}[v]


def attend_paged(pk: Plan, pv: Plan, q, k_codes, k_scales, v_codes, v_scales, block_table, kv_lens, q_starts=None,
                 max_q_len: int = None, max_kv_len: int = None, window: int = 0, softmax_scale: float = 0.0, out=None,
                 workspace=None, stream=None) -> torch.Tensor:
    """Causal attention of ragged queries over paged caches (see kvq_attend_paged).

    q fp16 [n, Hq, D] (token and head strides multiples of 8); block_table int32 [B, max_pages];
    kv_lens int32 [B], the new tokens included; q_starts int32 [B + 1] or None for one query token
    per request (n == B). ``max_q_len`` / ``max_kv_len`` bound the lengths, which the host cannot
    see (defaults: n and the table's capacity); tight bounds choose the kernel best and save a few
    microseconds.
    ``window`` > 0: each token attends the last ``window`` tokens up to itself. Returns fp16
    [n, Hq, D]; rows of ``out`` that belong to no request are left as they were (without ``out``:
    with any contents)."""
    return _paged.attend_paged(pk, pv, q, k_codes, k_scales, v_codes, v_scales, block_table, kv_lens, q_starts, max_q_len,
                               max_kv_len, window, softmax_scale, out, workspace,
                               None if stream is None else stream.cuda_stream)
