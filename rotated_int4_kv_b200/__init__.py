"""B200-native SRFT-int4 KV-cache compression and decode attention.

The compute path lives in ``libkvq.so`` (hand-written CUDA for sm_100a, C ABI in
``include/kvq.h``); this package only marshals torch tensors into it.
"""
from ._lib import LIB_PATH, KvqError, lib  # noqa: F401
from .cache import Int4KVCache, PagedInt4KVCache  # noqa: F401
from .api import (Plan, attend_combine, attend_decode, attend_decode_append, attend_decode_batch,  # noqa: F401
                  attend_decode_context_parallel, attend_decode_noalloc, attend_decode_partial, attend_decode_ref,
                  attend_split_info, debug_wait_timeout, gather_partials,
                  decode, encode, encode_batch, get_decode_path, get_encode_path, make_workspace, poll_device_errors,
                  set_decode_path, set_encode_path, workspace_size)
from .paged import (PagePlan, attend_paged, decode_paged, encode_paged, get_attend_paged_path,  # noqa: F401
                    make_paged_workspace, page_plan, page_release, paged_workspace_size, set_attend_paged_path)

__all__ = ["Plan", "Int4KVCache", "attend_decode_partial", "attend_combine", "gather_partials",
           "attend_decode_context_parallel", "encode", "encode_batch", "decode", "attend_decode", "attend_decode_append", "attend_decode_batch",
           "attend_decode_noalloc", "attend_decode_ref", "attend_split_info", "debug_wait_timeout", "workspace_size", "make_workspace", "poll_device_errors",
           "set_encode_path", "get_encode_path", "set_decode_path", "get_decode_path",
           "PagedInt4KVCache", "PagePlan", "page_plan", "page_release", "encode_paged", "decode_paged", "attend_paged",
           "paged_workspace_size", "make_paged_workspace", "set_attend_paged_path", "get_attend_paged_path",
           "KvqError", "LIB_PATH", "lib"]
