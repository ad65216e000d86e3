"""GB300-native paged decode attention: Python binding of libpagedkv.so.

Functions carry the names of the C ABI in include/pagedkv.h and only marshal
arguments (torch tensors -> device pointers and sizes, current stream); every step
of the computation runs in the library's CUDA kernels.  There is no CPU path:
calls on tensors that are not CUDA tensors raise.

    pa_decode               paged single-query attention (partition + merge kernels)
    pa_decode_append        the newest tokens' append fused with the decode
    pa_decode_plan /        the balanced split's CTA starts computed on the host, and
      pa_decode_planned       the decode (and append) that starts from them
    pa_decode_shared        decode reading each shared prefix block once per group
    pa_attend               several query tokens a sequence: prompts' chunks, cross attention
    pa_reshape_and_cache    write new tokens' K/V rows through a slot mapping
    pa_copy_blocks          copy-on-write block copies
    pa_swap_blocks          block moves between the device pool and pinned host memory
    pa_gather_blocks /      pack blocks into a contiguous staging buffer and back
      pa_scatter_blocks       (the local halves of a KV transfer)
    pa_q8_append /          the same cache in 8 bits (e4m3 codes, a scale per block and
      pa_q8_decode            kv head): quantising append, and decode attention over it
    pa_build_tables         block tables, lengths and slot maps grown and released on the GPU
    pa_fork_tables          the next batch's tables from rows of this one's, on the GPU (samples,
                              beams), with reference counts and copies of half-filled blocks
    pa_rope /               rotary positions of queries and keys, and the same with the append
      pa_rope_append          of keys and values
    BlockAllocator          host ref-counted block allocator (pa_alloc_*)
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
from typing import List, Optional, Sequence, Tuple

from ._lib import load as _load, library_path  # noqa: F401

PA_OK, PA_ERR_INVALID, PA_ERR_UNSUPPORTED, PA_ERR_CUDA, PA_ERR_OOM, PA_ERR_TIMEOUT = range(6)
PA_F32, PA_F16, PA_BF16 = 0, 1, 2


class PagedKVError(RuntimeError):
    def __init__(self, status: int, where: str):
        lib = _load()
        msg = lib.pa_status_string(status).decode()
        if status == PA_ERR_CUDA:
            msg += f" (cudaError {lib.pa_last_cuda_error()})"
        super().__init__(f"{where}: {msg}")
        self.status = status


class OutOfBlocks(PagedKVError, MemoryError):
    pass


def _check(status: int, where: str) -> None:
    if status == PA_ERR_OOM:
        raise OutOfBlocks(status, where)
    if status != PA_OK:
        raise PagedKVError(status, where)


def _dtype_code(t) -> int:
    import torch
    codes = {torch.float32: PA_F32, torch.float16: PA_F16, torch.bfloat16: PA_BF16}
    if t.dtype not in codes:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return codes[t.dtype]


def _cuda(t, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _dev_ptr(t, name: str):
    """Pointer of a CUDA tensor or of a pinned host tensor (device-accessible)."""
    if not (t.is_cuda or t.is_pinned()):
        raise ValueError(f"{name} must be a CUDA tensor or pinned host memory")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _stream(stream) -> int:
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream if hasattr(s, "cuda_stream") else int(s)


def _torch_stream(stream, device):
    """`stream` (None: torch's current stream; a torch stream; or a raw cudaStream_t)
    as a torch stream object."""
    import torch
    if stream is None:
        return torch.cuda.current_stream(device)
    if hasattr(stream, "cuda_stream"):
        return stream
    return torch.cuda.ExternalStream(int(stream), device=device)


def _launch_scratch(nbytes: int, device, stream):
    """A uint8 workspace for a launch on `stream`, taken from torch's caching
    allocator on that stream.  The tensor is dropped when the call returns, while
    the launch may still be running; allocated on the launch's own stream, its
    block is handed out again only to later work on that stream, which runs after
    the launch."""
    import torch
    with torch.cuda.stream(_torch_stream(stream, device)):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


# ----------------------------------------------------------------------------
# decode
# ----------------------------------------------------------------------------
def pa_decode_partition_size(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                             max_blocks_per_seq, partition_size=0) -> int:
    return _load().pa_decode_partition_size(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                            max_blocks_per_seq, partition_size)


def pa_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                             max_blocks_per_seq, partition_size=0) -> int:
    n = _load().pa_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                         max_blocks_per_seq, partition_size)
    if n == ctypes.c_size_t(-1).value:
        raise PagedKVError(PA_ERR_INVALID, "pa_decode_workspace_size")
    return n


def alloc_workspace(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq,
                    partition_size=0, device="cuda", stream=None):
    """A caller-owned workspace tensor of the size pa_decode needs (None if 0),
    allocated on `stream` (default: torch's current stream)."""
    n = pa_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                 max_blocks_per_seq, partition_size)
    return _launch_scratch(n, device, stream) if n > 0 else None


def pa_decode(out, q, k_cache, v_cache, block_tables, context_lens, scale: float,
              num_q_heads: int, num_kv_heads: int, head_dim: int, block_size: int,
              partition_size: int = 0, workspace=None, stream=None):
    """out[S, Hq, d] <- paged decode attention (see pa_decode in include/pagedkv.h).

    q/out [S, Hq, d]; caches [num_blocks, B, Hkv, d]; block_tables int32 [S, W];
    context_lens int32 [S]; workspace: uint8 CUDA tensor or None (allocated here)."""
    import torch
    S = q.shape[0]
    W = block_tables.shape[1]
    if workspace is None:
        workspace = alloc_workspace(S, num_q_heads, num_kv_heads, head_dim, block_size, W,
                                    partition_size, q.device, stream)
    ws_ptr = _cuda(workspace, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise TypeError("block_tables and context_lens must be int32")
    st = _load().pa_decode(_cuda(out, "out"), _cuda(q, "q"), _cuda(k_cache, "k_cache"),
                           _cuda(v_cache, "v_cache"), _cuda(block_tables, "block_tables"), W,
                           _cuda(context_lens, "context_lens"), S, k_cache.shape[0], float(scale),
                           num_q_heads, num_kv_heads, head_dim, block_size, _dtype_code(q),
                           partition_size, ws_ptr, ws_bytes, _stream(stream))
    _check(st, "pa_decode")
    return out


def pa_decode_append(out, q, k_cache, v_cache, k_new, v_new, block_tables, context_lens,
                     scale: float, num_q_heads: int, num_kv_heads: int, head_dim: int,
                     block_size: int, partition_size: int = 0, workspace=None, stream=None):
    """Append each sequence's newest token (k_new/v_new [S, Hkv, d], position
    context_lens[s] - 1) to the caches and decode, in one launch; the same result as
    pa_reshape_and_cache followed by pa_decode."""
    import torch
    S = q.shape[0]
    W = block_tables.shape[1]
    if workspace is None:
        workspace = alloc_workspace(S, num_q_heads, num_kv_heads, head_dim, block_size, W,
                                    partition_size, q.device, stream)
    ws_ptr = _cuda(workspace, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise TypeError("block_tables and context_lens must be int32")
    st = _load().pa_decode_append(_cuda(out, "out"), _cuda(q, "q"), _cuda(k_cache, "k_cache"),
                                  _cuda(v_cache, "v_cache"), _cuda(k_new, "k_new"),
                                  _cuda(v_new, "v_new"), _cuda(block_tables, "block_tables"), W,
                                  _cuda(context_lens, "context_lens"), S, k_cache.shape[0],
                                  float(scale), num_q_heads, num_kv_heads, head_dim, block_size,
                                  _dtype_code(q), partition_size, ws_ptr, ws_bytes, _stream(stream))
    _check(st, "pa_decode_append")
    return out


_DTYPE_NAMES = {"f32": PA_F32, "f16": PA_F16, "bf16": PA_BF16}


def _dtype_arg(dtype) -> int:
    """A pa_dtype code from a code, a name ('f32', 'f16', 'bf16') or a torch dtype."""
    if isinstance(dtype, int):
        return dtype
    if isinstance(dtype, str):
        return _DTYPE_NAMES[dtype]
    import torch
    return {torch.float32: PA_F32, torch.float16: PA_F16, torch.bfloat16: PA_BF16}[dtype]


def pa_decode_plan_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq,
                         dtype) -> int:
    """Size of a pa_decode_plan for these arguments on the current device."""
    n = _load().pa_decode_plan_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                     max_blocks_per_seq, _dtype_arg(dtype))
    if n == ctypes.c_size_t(-1).value:
        raise PagedKVError(PA_ERR_INVALID, "pa_decode_plan_bytes")
    return n


def pa_decode_plan(block_tables, context_lens, num_q_heads: int, num_kv_heads: int, head_dim: int,
                   block_size: int, dtype, plan_bytes: Optional[int] = None):
    """Host-side schedule of the balanced-split decode (see pa_decode_plan in
    include/pagedkv.h): int32 numpy array of plan_bytes / 4 entries, from HOST block
    tables [S, W] and context lengths [S] (numpy arrays or CPU tensors).  plan_bytes
    defaults to pa_decode_plan_bytes(...) on the current device."""
    import numpy as np
    bt = np.ascontiguousarray(np.asarray(block_tables, dtype=np.int32))
    cl = np.ascontiguousarray(np.asarray(context_lens, dtype=np.int32))
    S = cl.shape[0]
    W = bt.shape[1] if bt.ndim == 2 else 1
    if plan_bytes is None:
        plan_bytes = pa_decode_plan_bytes(S, num_q_heads, num_kv_heads, head_dim, block_size, W, dtype)
    plan = np.empty(plan_bytes // 4, dtype=np.int32)
    st = _load().pa_decode_plan(plan.ctypes.data, plan_bytes, bt.ctypes.data if S else None, W,
                                cl.ctypes.data if S else None, S, num_q_heads, num_kv_heads, head_dim,
                                block_size, _dtype_arg(dtype))
    _check(st, "pa_decode_plan")
    return plan


def pa_decode_planned(out, q, k_cache, v_cache, block_tables, context_lens, plan, scale: float,
                      num_q_heads: int, num_kv_heads: int, head_dim: int, block_size: int,
                      k_new=None, v_new=None, workspace=None, stream=None):
    """pa_decode (balanced split), or with k_new/v_new pa_decode_append, whose CTAs
    start where `plan` (a CUDA int32 copy of pa_decode_plan's output for the same
    lengths and tables) says; bit-identical to the unplanned call."""
    import torch
    S = q.shape[0]
    W = block_tables.shape[1]
    if workspace is None:
        workspace = alloc_workspace(S, num_q_heads, num_kv_heads, head_dim, block_size, W, 0, q.device,
                                    stream)
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32 or plan.dtype != torch.int32:
        raise TypeError("block_tables, context_lens and plan must be int32")
    st = _load().pa_decode_planned(_cuda(out, "out"), _cuda(q, "q"), _cuda(k_cache, "k_cache"),
                                   _cuda(v_cache, "v_cache"),
                                   _cuda(k_new, "k_new") if k_new is not None else None,
                                   _cuda(v_new, "v_new") if v_new is not None else None,
                                   _cuda(block_tables, "block_tables"), W,
                                   _cuda(context_lens, "context_lens"), S, k_cache.shape[0], float(scale),
                                   num_q_heads, num_kv_heads, head_dim, block_size, _dtype_code(q),
                                   _cuda(plan, "plan"), plan.numel() * 4,
                                   _cuda(workspace, "workspace") if workspace is not None else None,
                                   workspace.numel() if workspace is not None else 0, _stream(stream))
    _check(st, "pa_decode_planned")
    return out


def pa_decode_shared_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                    max_blocks_per_seq) -> int:
    n = _load().pa_decode_shared_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                block_size, max_blocks_per_seq)
    if n == ctypes.c_size_t(-1).value:
        raise PagedKVError(PA_ERR_INVALID, "pa_decode_shared_workspace_size")
    return n


def pa_decode_shared(out, q, k_cache, v_cache, block_tables, context_lens, share, scale: float,
                     num_q_heads: int, num_kv_heads: int, head_dim: int, block_size: int,
                     k_new=None, v_new=None, workspace=None, stream=None):
    """Decode a batch whose sequence groups share leading blocks, reading each shared
    block once per group; share: int32 [S, 2] = (first member of the group or -1,
    shared leading blocks).  With k_new/v_new, also appends the newest tokens."""
    import torch
    S = q.shape[0]
    W = block_tables.shape[1]
    if workspace is None:
        n = pa_decode_shared_workspace_size(S, num_q_heads, num_kv_heads, head_dim, block_size, W)
        workspace = _launch_scratch(n, q.device, stream)
    if share.dtype != torch.int32 or block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise TypeError("share, block_tables and context_lens must be int32")
    st = _load().pa_decode_shared(_cuda(out, "out"), _cuda(q, "q"), _cuda(k_cache, "k_cache"),
                                  _cuda(v_cache, "v_cache"),
                                  _cuda(k_new, "k_new") if k_new is not None else None,
                                  _cuda(v_new, "v_new") if v_new is not None else None,
                                  _cuda(block_tables, "block_tables"), W,
                                  _cuda(context_lens, "context_lens"), _cuda(share, "share"), S,
                                  k_cache.shape[0], float(scale), num_q_heads, num_kv_heads, head_dim,
                                  block_size, _dtype_code(q), _cuda(workspace, "workspace"),
                                  workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "pa_decode_shared")
    return out


def pa_decode_shared_plan_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                max_blocks_per_seq, dtype) -> int:
    """Size of a pa_decode_shared_plan for these arguments on the current device."""
    n = _load().pa_decode_shared_plan_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                            max_blocks_per_seq, _dtype_arg(dtype))
    if n == ctypes.c_size_t(-1).value:
        raise PagedKVError(PA_ERR_INVALID, "pa_decode_shared_plan_bytes")
    return n


def pa_decode_shared_plan(block_tables, context_lens, share, num_q_heads: int, num_kv_heads: int,
                          head_dim: int, block_size: int, dtype, plan_bytes: Optional[int] = None):
    """Host-side schedule of both launches of the shared-prefix decode (see
    pa_decode_shared_plan in include/pagedkv.h): int32 numpy array, from HOST block
    tables [S, W], context lengths [S] and share entries [S, 2].  plan_bytes defaults
    to pa_decode_shared_plan_bytes(...) on the current device."""
    import numpy as np
    bt = np.ascontiguousarray(np.asarray(block_tables, dtype=np.int32))
    cl = np.ascontiguousarray(np.asarray(context_lens, dtype=np.int32))
    sh = np.ascontiguousarray(np.asarray(share, dtype=np.int32))
    S = cl.shape[0]
    W = bt.shape[1] if bt.ndim == 2 else 1
    if plan_bytes is None:
        plan_bytes = pa_decode_shared_plan_bytes(S, num_q_heads, num_kv_heads, head_dim, block_size, W,
                                                 dtype)
    plan = np.empty(plan_bytes // 4, dtype=np.int32)
    st = _load().pa_decode_shared_plan(plan.ctypes.data, plan_bytes, bt.ctypes.data if S else None, W,
                                       cl.ctypes.data if S else None, sh.ctypes.data if S else None, S,
                                       num_q_heads, num_kv_heads, head_dim, block_size, _dtype_arg(dtype))
    _check(st, "pa_decode_shared_plan")
    return plan


def pa_decode_shared_planned(out, q, k_cache, v_cache, block_tables, context_lens, share, plan,
                             scale: float, num_q_heads: int, num_kv_heads: int, head_dim: int,
                             block_size: int, k_new=None, v_new=None, workspace=None, stream=None):
    """pa_decode_shared whose CTAs, in both launches, start where `plan` (a CUDA int32
    copy of pa_decode_shared_plan's output for the same inputs) says; bit-identical
    to the unplanned call."""
    import torch
    S = q.shape[0]
    W = block_tables.shape[1]
    if workspace is None:
        n = pa_decode_shared_workspace_size(S, num_q_heads, num_kv_heads, head_dim, block_size, W)
        workspace = _launch_scratch(n, q.device, stream)
    if (share.dtype != torch.int32 or block_tables.dtype != torch.int32 or
            context_lens.dtype != torch.int32 or plan.dtype != torch.int32):
        raise TypeError("share, block_tables, context_lens and plan must be int32")
    st = _load().pa_decode_shared_planned(
        _cuda(out, "out"), _cuda(q, "q"), _cuda(k_cache, "k_cache"), _cuda(v_cache, "v_cache"),
        _cuda(k_new, "k_new") if k_new is not None else None,
        _cuda(v_new, "v_new") if v_new is not None else None,
        _cuda(block_tables, "block_tables"), W, _cuda(context_lens, "context_lens"), _cuda(share, "share"),
        S, k_cache.shape[0], float(scale), num_q_heads, num_kv_heads, head_dim, block_size, _dtype_code(q),
        _cuda(plan, "plan"), plan.numel() * 4, _cuda(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "pa_decode_shared_planned")
    return out


def share_groups(block_tables, context_lens, block_size: int, min_shared_blocks: int = 1):
    """share int32 [S, 2] for pa_decode_shared, from host block tables [S, W] and
    context lengths [S] (numpy or CPU tensors); see pa_share_groups."""
    import numpy as np
    bt = np.ascontiguousarray(np.asarray(block_tables, dtype=np.int32))
    cl = np.ascontiguousarray(np.asarray(context_lens, dtype=np.int32))
    S = cl.shape[0]
    share = np.empty((S, 2), dtype=np.int32)
    W = bt.shape[1] if bt.ndim == 2 else 0
    st = _load().pa_share_groups(bt.ctypes.data if S else None, S, W, cl.ctypes.data if S else None,
                                 block_size, min_shared_blocks, share.ctypes.data if S else None)
    _check(st, "pa_share_groups")
    return share


def share_saving(share, context_lens, block_size: int) -> float:
    """Fraction of the batch's block reads that pa_decode_shared saves over pa_decode:
    each group of m members sharing P blocks reads (m - 1) * P blocks fewer (when
    one item holds all m members' query rows)."""
    import numpy as np
    share = np.asarray(share)
    cl = np.asarray(context_lens).astype(np.int64)
    logical = int(((cl + block_size - 1) // block_size).sum())
    saved = 0
    for s in range(share.shape[0]):
        if share[s, 0] >= 0 and share[s, 0] != s:      # every member but the first
            saved += int(share[s, 1])
    return saved / logical if logical else 0.0


# pa_decode_shared pays for its second launch and its merges (a fixed ~10-15 us)
# once the groups save 10% of the block reads, or 256 MB of them (~37 us at
# 7 TB/s) on a large batch: the long multi-turn batch saves 2.7%, 580 MB, and
# decodes ~1% faster shared.
SHARE_MIN_SAVING = 0.10
SHARE_MIN_BYTES = 256 << 20


def share_pays(share, context_lens, block_size: int, block_bytes: int) -> bool:
    """Whether pa_decode_shared is expected to beat pa_decode on this batch.
    block_bytes: bytes of one block of K and V over all kv heads."""
    import numpy as np
    f = share_saving(share, context_lens, block_size)
    cl = np.asarray(context_lens).astype(np.int64)
    logical = int(((cl + block_size - 1) // block_size).sum()) * int(block_bytes)
    return f >= SHARE_MIN_SAVING or f * logical >= SHARE_MIN_BYTES


def pa_decode_noalloc(out, q, k_cache, v_cache, block_tables, context_lens, scale: float,
                      num_q_heads: int, num_kv_heads: int, head_dim: int, block_size: int,
                      partition_size: int = 0, stream=None):
    """pa_decode for callers that cannot allocate device memory: the split-KV
    scratch is the library's fixed device array (PA_DECODE_NOALLOC_SCRATCH_BYTES,
    shared by every call; calls overlapping on the GPU race).  Sizes needing more
    scratch raise PagedKVError (PA_ERR_UNSUPPORTED)."""
    import torch
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise TypeError("block_tables and context_lens must be int32")
    st = _load().pa_decode_noalloc(_cuda(out, "out"), _cuda(q, "q"), _cuda(k_cache, "k_cache"),
                                   _cuda(v_cache, "v_cache"), _cuda(block_tables, "block_tables"),
                                   block_tables.shape[1], _cuda(context_lens, "context_lens"),
                                   q.shape[0], k_cache.shape[0], float(scale), num_q_heads,
                                   num_kv_heads, head_dim, block_size, _dtype_code(q), partition_size,
                                   _stream(stream))
    _check(st, "pa_decode_noalloc")
    return out


# ----------------------------------------------------------------------------
# cache writes
# ----------------------------------------------------------------------------
def pa_reshape_and_cache(k, v, k_cache, v_cache, slot_mapping, stream=None):
    """k_cache[slot // B][slot % B] = k[t] (and v) for every token t with slot >= 0."""
    import torch
    if slot_mapping.dtype != torch.int64:
        raise TypeError("slot_mapping must be int64")
    n = slot_mapping.shape[0]
    if n == 0:
        return
    nb, B, hkv, d = k_cache.shape
    st = _load().pa_reshape_and_cache(_cuda(k, "k"), _cuda(v, "v"), _cuda(k_cache, "k_cache"),
                                      _cuda(v_cache, "v_cache"), _cuda(slot_mapping, "slot_mapping"),
                                      n, hkv, d, B, nb, _dtype_code(k_cache), _stream(stream))
    _check(st, "pa_reshape_and_cache")


def pa_copy_blocks(k_cache, v_cache, src_dst_pairs, stream=None):
    """k_cache[dst] = k_cache[src] (and v) for every (src, dst) row of the int32 [n, 2] pairs."""
    import torch
    if src_dst_pairs.dtype != torch.int32:
        raise TypeError("src_dst_pairs must be int32")
    n = src_dst_pairs.shape[0]
    if n == 0:
        return
    block_bytes = k_cache[0].numel() * k_cache.element_size()
    st = _load().pa_copy_blocks(_cuda(k_cache, "k_cache"), _cuda(v_cache, "v_cache"),
                                _cuda(src_dst_pairs, "src_dst_pairs"), n, k_cache.shape[0],
                                block_bytes, _stream(stream))
    _check(st, "pa_copy_blocks")


def pa_device_errors(stream=None) -> int:
    """The device-side error flags (PA_DEVERR_*) raised since the last read, after
    `stream` drains; reading clears them.  Set flags are returned, not raised (the
    C call's PA_ERR_TIMEOUT / PA_ERR_INVALID status); a CUDA failure raises."""
    flags = ctypes.c_uint(0)
    st = _load().pa_device_errors(ctypes.byref(flags), _stream(stream))
    if st not in (PA_ERR_TIMEOUT, PA_ERR_INVALID) or flags.value == 0:
        _check(st, "pa_device_errors")
    return flags.value


PA_DEVERR_TIMEOUT_FULL, PA_DEVERR_TIMEOUT_EMPTY, PA_DEVERR_SHARE, PA_DEVERR_PLAN = 1, 2, 4, 8
PLAN_BYTES_PER_CTA = 128
PA_WAIT_LIMIT_DEFAULT_NS = 2_000_000_000


def pa_set_wait_limit_ns(ns: int) -> int:
    """Limit (ns) of the device-side waits of decode launches enqueued from now on
    (0: the default, 2 s); returns the previous limit."""
    return int(_load().pa_set_wait_limit_ns(int(ns)))


def pa_status_string(status: int) -> str:
    return _load().pa_status_string(status).decode()


# ----------------------------------------------------------------------------
# host allocator
# ----------------------------------------------------------------------------
class BlockAllocator:
    """Ref-counted block allocator (pa_alloc_* of include/pagedkv.h); host only."""

    def __init__(self, num_blocks: int, block_size: int, free_order: Optional[Sequence[int]] = None):
        import numpy as np
        self._lib = _load()
        self._h = ctypes.c_void_p()
        self.num_blocks = num_blocks
        self.block_size = block_size
        ptr = None
        if free_order is not None:
            self._order = np.ascontiguousarray(free_order, dtype=np.int32)
            if self._order.shape != (num_blocks,):
                raise ValueError("free_order must have num_blocks entries")
            ptr = self._order.ctypes.data
        _check(self._lib.pa_alloc_create(ctypes.byref(self._h), num_blocks, block_size, ptr),
               "pa_alloc_create")

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            self._lib.pa_alloc_destroy(h)
            self._h = None

    def new_seq(self) -> int:
        sid = ctypes.c_int()
        _check(self._lib.pa_alloc_new_seq(self._h, ctypes.byref(sid)), "pa_alloc_new_seq")
        return sid.value

    def fork(self, parent: int) -> int:
        sid = ctypes.c_int()
        _check(self._lib.pa_alloc_fork(self._h, parent, ctypes.byref(sid)), "pa_alloc_fork")
        return sid.value

    def append(self, seq: int) -> Tuple[int, Optional[Tuple[int, int]]]:
        slot = ctypes.c_int64()
        src = ctypes.c_int32()
        dst = ctypes.c_int32()
        _check(self._lib.pa_alloc_append(self._h, seq, ctypes.byref(slot), ctypes.byref(src),
                                         ctypes.byref(dst)), "pa_alloc_append")
        return slot.value, ((src.value, dst.value) if src.value >= 0 else None)

    def append_n(self, seq: int, n: int):
        """n appends: (slots int64 [n], cow pairs int32 [k, 2])."""
        import numpy as np
        slots = np.empty(max(n, 1), dtype=np.int64)
        pairs = np.empty((max(n, 1), 2), dtype=np.int32)
        k = ctypes.c_int()
        _check(self._lib.pa_alloc_append_n(self._h, seq, n, slots.ctypes.data, pairs.ctypes.data,
                                           ctypes.byref(k), None), "pa_alloc_append_n")
        return slots[:n], pairs[:k.value]

    def free_seq(self, seq: int) -> None:
        _check(self._lib.pa_alloc_free_seq(self._h, seq), "pa_alloc_free_seq")

    def block_table(self, seq: int) -> List[int]:
        import numpy as np
        n = ctypes.c_int()
        _check(self._lib.pa_alloc_block_table(self._h, seq, None, 0, ctypes.byref(n)), "pa_alloc_block_table")
        out = np.empty(max(n.value, 1), dtype=np.int32)
        _check(self._lib.pa_alloc_block_table(self._h, seq, out.ctypes.data, n.value, ctypes.byref(n)),
               "pa_alloc_block_table")
        return out[:n.value].tolist()

    def seq_len(self, seq: int) -> int:
        n = ctypes.c_int()
        _check(self._lib.pa_alloc_seq_len(self._h, seq, ctypes.byref(n)), "pa_alloc_seq_len")
        return n.value

    def refcount(self, block: int) -> int:
        return self._lib.pa_alloc_refcount(self._h, block)

    def num_free(self) -> int:
        return self._lib.pa_alloc_num_free(self._h)

    def free_list(self) -> List[int]:
        import numpy as np
        n = ctypes.c_int()
        _check(self._lib.pa_alloc_free_list(self._h, None, 0, ctypes.byref(n)), "pa_alloc_free_list")
        out = np.empty(max(n.value, 1), dtype=np.int32)
        _check(self._lib.pa_alloc_free_list(self._h, out.ctypes.data, n.value, ctypes.byref(n)),
               "pa_alloc_free_list")
        return out[:n.value].tolist()

    def usage(self) -> dict:
        """Device-pool accounting (pa_alloc_usage_stats) plus the derived waste and
        sharing-saving fractions."""
        class _Usage(ctypes.Structure):
            _fields_ = [(n, ctypes.c_int64) for n in ("used_blocks", "logical_blocks", "token_slots",
                                                       "tokens", "resident_seqs", "swapped_seqs")]
        u = _Usage()
        _check(self._lib.pa_alloc_usage_stats(self._h, ctypes.byref(u)), "pa_alloc_usage_stats")
        d = {n: getattr(u, n) for n, _ in _Usage._fields_}
        d["waste"] = 1.0 - d["tokens"] / d["token_slots"] if d["token_slots"] else 0.0
        d["sharing_saving"] = 1.0 - d["used_blocks"] / d["logical_blocks"] if d["logical_blocks"] else 0.0
        return d

    # swap space in host memory -------------------------------------------------
    def set_host_pool(self, num_host_blocks: int) -> None:
        _check(self._lib.pa_alloc_set_host_pool(self._h, num_host_blocks), "pa_alloc_set_host_pool")
        self.num_host_blocks = num_host_blocks

    def _move(self, fn, name, seqs):
        import numpy as np
        ids = np.ascontiguousarray(list(seqs), dtype=np.int32).reshape(-1)
        n = ctypes.c_int()
        cap = max(1, sum(len(self.block_table(q)) for q in ids.tolist())) if ids.size else 1
        pairs = np.empty((cap, 2), dtype=np.int32)
        _check(fn(self._h, ids.ctypes.data if ids.size else None, int(ids.size), pairs.ctypes.data, cap,
                  ctypes.byref(n)), name)
        return pairs[:n.value]

    def swap_out(self, seqs) -> "object":
        """Move `seqs` to the host pool: int32 [k, 2] (device block, host block) pairs."""
        return self._move(self._lib.pa_alloc_swap_out, "pa_alloc_swap_out", seqs)

    def swap_in(self, seqs) -> "object":
        """Move `seqs` back to the device pool: int32 [k, 2] (host block, device block) pairs."""
        return self._move(self._lib.pa_alloc_swap_in, "pa_alloc_swap_in", seqs)

    def is_swapped(self, seq: int) -> bool:
        v = self._lib.pa_alloc_is_swapped(self._h, seq)
        if v < 0:
            raise PagedKVError(PA_ERR_INVALID, "pa_alloc_is_swapped")
        return bool(v)

    def host_refcount(self, block: int) -> int:
        return self._lib.pa_alloc_host_refcount(self._h, block)

    def num_free_host(self) -> int:
        return self._lib.pa_alloc_num_free_host(self._h)

    def host_free_list(self) -> List[int]:
        import numpy as np
        n = ctypes.c_int()
        _check(self._lib.pa_alloc_host_free_list(self._h, None, 0, ctypes.byref(n)), "pa_alloc_host_free_list")
        out = np.empty(max(n.value, 1), dtype=np.int32)
        _check(self._lib.pa_alloc_host_free_list(self._h, out.ctypes.data, n.value, ctypes.byref(n)),
               "pa_alloc_host_free_list")
        return out[:n.value].tolist()


def _block_bytes(cache) -> int:
    return cache[0].numel() * cache.element_size()


def pa_swap_blocks(src_k, src_v, dst_k, dst_v, src_dst_pairs, stream=None):
    """dst pool blocks <- src pool blocks for each (src, dst) pair; pools are [NB, ...]
    tensors on the device or in pinned host memory (pairs likewise)."""
    if src_dst_pairs.shape[0] == 0:
        return
    st = _load().pa_swap_blocks(_dev_ptr(src_k, "src_k"), _dev_ptr(src_v, "src_v"), _dev_ptr(dst_k, "dst_k"),
                                _dev_ptr(dst_v, "dst_v"), _dev_ptr(src_dst_pairs, "src_dst_pairs"),
                                int(src_dst_pairs.shape[0]), int(src_k.shape[0]), int(dst_k.shape[0]),
                                _block_bytes(src_k), _stream(stream))
    _check(st, "pa_swap_blocks")


def pa_gather_blocks(k_cache, v_cache, block_ids, staging_k, staging_v, stream=None):
    """staging[i] <- cache[block_ids[i]] (staging: [n, ...] device or pinned host tensors)."""
    if block_ids.shape[0] == 0:
        return
    st = _load().pa_gather_blocks(_dev_ptr(k_cache, "k_cache"), _dev_ptr(v_cache, "v_cache"),
                                  _dev_ptr(block_ids, "block_ids"), int(block_ids.shape[0]),
                                  int(k_cache.shape[0]), _dev_ptr(staging_k, "staging_k"),
                                  _dev_ptr(staging_v, "staging_v"), _block_bytes(k_cache), _stream(stream))
    _check(st, "pa_gather_blocks")


def pa_scatter_blocks(staging_k, staging_v, k_cache, v_cache, block_ids, stream=None):
    """cache[block_ids[i]] <- staging[i]."""
    if block_ids.shape[0] == 0:
        return
    st = _load().pa_scatter_blocks(_dev_ptr(staging_k, "staging_k"), _dev_ptr(staging_v, "staging_v"),
                                   _dev_ptr(k_cache, "k_cache"), _dev_ptr(v_cache, "v_cache"),
                                   _dev_ptr(block_ids, "block_ids"), int(block_ids.shape[0]),
                                   int(k_cache.shape[0]), _block_bytes(k_cache), _stream(stream))
    _check(st, "pa_scatter_blocks")


# ----------------------------------------------------------------------------
# the 8-bit cache, and tables built on the GPU
# ----------------------------------------------------------------------------
# (These calls take a few microseconds on the GPU for a small batch, so what the binding
# looks up per call is looked up once: library functions, torch's types and handles.)
@functools.lru_cache(maxsize=None)
def _fn(name: str):
    return getattr(_load(), name)


class _Torch:
    """torch's attributes that the calls below use."""

    def __init__(self):
        import torch
        self.int32, self.int64, self.uint8, self.float32 = torch.int32, torch.int64, torch.uint8, torch.float32
        self.codes = {torch.float32: PA_F32, torch.float16: PA_F16, torch.bfloat16: PA_BF16}
        self.device, self.empty = torch.cuda.device, torch.empty
        self.current_device = torch._C._cuda_getDevice
        self.current_stream = torch._C._cuda_getCurrentRawStream


@functools.lru_cache(maxsize=None)
def _torch() -> _Torch:
    return _Torch()


def _code(t) -> int:
    code = _torch().codes.get(t.dtype)
    return _dtype_code(t) if code is None else code


def _on_device(names, tensors):
    """Checks that the tensors are contiguous and on one CUDA device; returns (its index,
    None when it is the current device, else a context that makes it so)."""
    dev = tensors[0].get_device()          # -1: not a CUDA tensor
    for name, t in zip(names, tensors):
        if t.get_device() != dev or dev < 0 or not t.is_contiguous():
            _cuda(t, name)
            raise ValueError(f"{name} is on cuda:{t.get_device()}, {names[0]} on cuda:{dev}")
    T = _torch()
    return dev, None if dev == T.current_device() else T.device(dev)


def _raw_stream(stream, dev: int) -> int:
    """As _stream, on device `dev` (without building a stream object for the default)."""
    return _torch().current_stream(dev) if stream is None else _stream(stream)


def _call(name: str, device, *args) -> None:
    if device is None:
        st = _fn(name)(*args)
    else:
        with device:
            st = _fn(name)(*args)
    if st != PA_OK:
        _check(st, name)


def _want(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


@functools.lru_cache(maxsize=None)
def pa_q8_block_bytes(num_kv_heads: int, head_dim: int, block_size: int) -> int:
    """Bytes of one block of the 8-bit cache: codes of K and V, then the scales."""
    n = _load().pa_q8_block_bytes(num_kv_heads, head_dim, block_size)
    if n == ctypes.c_size_t(-1).value:
        raise PagedKVError(PA_ERR_UNSUPPORTED, "pa_q8_block_bytes")
    return n


def alloc_q8_cache(num_blocks: int, num_kv_heads: int, head_dim: int, block_size: int, device="cuda",
                   pin_memory: bool = False):
    """A zeroed 8-bit cache, uint8 [num_blocks, block bytes] (device="cpu" with
    pin_memory=True: a pool to swap to)."""
    import torch
    return torch.zeros(num_blocks, pa_q8_block_bytes(num_kv_heads, head_dim, block_size), dtype=torch.uint8,
                       device=device, pin_memory=pin_memory)


def q8_views(kv_cache, num_kv_heads: int, head_dim: int, block_size: int):
    """(codes, scales) of an 8-bit cache as views of its memory: float8_e4m3fn
    [num_blocks, Hkv, 2, B, d] and float32 [num_blocks, Hkv, 2], index 0 of the pair K
    and 1 V; a code stands for code * scale."""
    import torch
    if kv_cache.element_size() != 1:   # (the strides below count bytes)
        raise TypeError("kv_cache must be uint8")
    nb, size = kv_cache.shape
    _want(size == pa_q8_block_bytes(num_kv_heads, head_dim, block_size) and kv_cache.is_contiguous(),
          "kv_cache must be a contiguous [num_blocks, pa_q8_block_bytes(...)]")
    tile = block_size * head_dim
    at = kv_cache.storage_offset()
    codes = kv_cache.view(torch.float8_e4m3fn).as_strided(
        (nb, num_kv_heads, 2, block_size, head_dim), (size, 2 * tile, tile, head_dim, 1), at)
    scales = kv_cache.view(torch.float32).as_strided((nb, num_kv_heads, 2), (size // 4, 2, 1),
                                                     (at + num_kv_heads * 2 * tile) // 4)
    return codes, scales


def _check_counts(bits: int) -> None:
    """`bits`: sizes or-ed together (ctypes would pass on the low 32 bits of a larger one)."""
    _want(not bits >> 31, "tensors of 2^31 rows or columns and more are not taken")


def _check_batch(kv_cache, block_tables, context_lens, num_kv_heads, head_dim, block_size):
    T = _torch()
    if block_tables.dtype != T.int32 or context_lens.dtype != T.int32:
        raise TypeError("block_tables and context_lens must be int32")
    if kv_cache.dtype != T.uint8:
        raise TypeError("kv_cache must be uint8")
    if block_tables.dim() != 2 or context_lens.shape != block_tables.shape[:1]:
        raise ValueError("block_tables must be [S, W] and context_lens [S]")
    if kv_cache.dim() != 2 or kv_cache.shape[1] != pa_q8_block_bytes(num_kv_heads, head_dim, block_size):
        raise ValueError("kv_cache must be [num_blocks, pa_q8_block_bytes(...)]")


_APPEND_NAMES = ("k", "v", "kv_cache", "block_tables", "context_lens", "query_start")
_DECODE_NAMES = ("out", "q", "kv_cache", "block_tables", "context_lens")
_TABLE_NAMES = ("block_tables", "context_lens", "new_tokens", "free_list", "num_free", "query_start", "granted",
                "context_lens_out", "num_free_out", "slot_mapping")


def pa_q8_append(k, v, kv_cache, block_tables, context_lens, block_size: int, query_start=None, stream=None):
    """Write new K and V rows ([N, Hkv, d]) into the 8-bit cache at the ends of their
    sequences, raising a block's scale where a row needs it (see pa_q8_append in
    include/pagedkv.h).  query_start int32 [S + 1]: first row of each sequence; None:
    one row per sequence."""
    _want(k.dim() == 3 and k.shape == v.shape, "k and v must be [N, Hkv, d] and alike")
    if k.dtype != v.dtype:
        raise TypeError("k and v must have one dtype")
    n, hkv, d = k.shape
    S, W = block_tables.shape
    _check_batch(kv_cache, block_tables, context_lens, hkv, d, block_size)
    blocks = kv_cache.shape[0]
    _check_counts(n | S | W | blocks)
    tensors = (k, v, kv_cache, block_tables, context_lens)
    qs_ptr = None
    if query_start is not None:
        if query_start.dtype != _torch().int32:
            raise TypeError("query_start must be int32")
        _want(query_start.shape == (S + 1,), "query_start must be [S + 1]")
        tensors += (query_start,)
        qs_ptr = query_start.data_ptr()
    dev, device = _on_device(_APPEND_NAMES, tensors)
    _call("pa_q8_append", device, k.data_ptr(), v.data_ptr(), kv_cache.data_ptr(), block_tables.data_ptr(), W,
          context_lens.data_ptr(), qs_ptr, S, n, blocks, hkv, d, block_size, _code(k),
          _raw_stream(stream, dev))


def pa_q8_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                max_blocks_per_seq) -> int:
    n = _load().pa_q8_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                            max_blocks_per_seq)
    if n == ctypes.c_size_t(-1).value:
        raise PagedKVError(PA_ERR_INVALID, "pa_q8_decode_workspace_size")
    return n


def pa_q8_decode(out, q, kv_cache, block_tables, context_lens, scale: float, num_q_heads: int,
                 num_kv_heads: int, head_dim: int, block_size: int, workspace=None, stream=None):
    """out[S, Hq, d] <- decode attention over the 8-bit cache (see pa_q8_decode in
    include/pagedkv.h); workspace: uint8 CUDA tensor or None (allocated here)."""
    S, W = block_tables.shape
    _check_batch(kv_cache, block_tables, context_lens, num_kv_heads, head_dim, block_size)
    blocks = kv_cache.shape[0]
    _check_counts(S | W | blocks)
    _want(q.shape == (S, num_q_heads, head_dim) and out.shape == q.shape, "q and out must be [S, Hq, d]")
    if out.dtype != q.dtype:
        raise TypeError("q and out must have one dtype")
    dev, device = _on_device(_DECODE_NAMES, (out, q, kv_cache, block_tables, context_lens))
    if workspace is None:
        with device or contextlib.nullcontext():
            workspace = _launch_scratch(pa_q8_decode_workspace_size(S, num_q_heads, num_kv_heads, head_dim,
                                                                    block_size, W), q.device, stream)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on the device of q")
    _call("pa_q8_decode", device, out.data_ptr(), q.data_ptr(), kv_cache.data_ptr(), block_tables.data_ptr(), W,
          context_lens.data_ptr(), S, blocks, float(scale), num_q_heads, num_kv_heads, head_dim,
          block_size, _code(q), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
          _raw_stream(stream, dev))
    return out


def _check_pairs(pairs, *pools):
    T = _torch()
    if pairs.dtype != T.int32:
        raise TypeError("src_dst_pairs must be int32")
    _want(pairs.dim() == 2 and pairs.shape[1] == 2, "src_dst_pairs must be [n, 2]")
    for pool in pools:
        if pool.dtype != T.uint8:
            raise TypeError("the pools must be uint8")
        _want(pool.dim() == 2, "the pools must be [num_blocks, pa_q8_block_bytes(...)]")


def pa_q8_copy_blocks(kv_cache, src_dst_pairs, stream=None):
    """Block dst becomes a copy of block src, codes and scales, for every (src, dst) row of
    the int32 [n, 2] pairs."""
    _check_pairs(src_dst_pairs, kv_cache)
    n = src_dst_pairs.shape[0]
    if n == 0:
        return
    dev, device = _on_device(("kv_cache", "src_dst_pairs"), (kv_cache, src_dst_pairs))
    _call("pa_q8_copy_blocks", device, kv_cache.data_ptr(), src_dst_pairs.data_ptr(), n, kv_cache.shape[0],
          kv_cache.shape[1], _raw_stream(stream, dev))


def pa_q8_swap_blocks(src_cache, dst_cache, src_dst_pairs, stream=None):
    """dst pool blocks <- src pool blocks, codes and scales, for each (src, dst) pair; pools
    are 8-bit caches on the device or in pinned host memory (pairs likewise)."""
    _check_pairs(src_dst_pairs, src_cache, dst_cache)
    _want(src_cache.shape[1] == dst_cache.shape[1], "the pools have blocks of different sizes")
    if src_dst_pairs.shape[0] == 0:
        return
    src, dst = _dev_ptr(src_cache, "src_cache"), _dev_ptr(dst_cache, "dst_cache")
    pairs = _dev_ptr(src_dst_pairs, "src_dst_pairs")
    T = _torch()
    devs = {t.get_device() for t in (src_cache, dst_cache, src_dst_pairs)} - {-1}
    _want(len(devs) < 2, "the pools and pairs are on different devices")
    dev = devs.pop() if devs else T.current_device()
    _call("pa_q8_swap_blocks", None if dev == T.current_device() else T.device(dev), src, dst, pairs,
          src_dst_pairs.shape[0], src_cache.shape[0], dst_cache.shape[0], src_cache.shape[1],
          _raw_stream(stream, dev))


def pa_build_tables(block_tables, context_lens, new_tokens, free_list, num_free, block_size: int, slot_mapping,
                    query_start, granted, context_lens_out=None, num_free_out=None, stream=None):
    """One allocator step on the GPU (see pa_build_tables in include/pagedkv.h): releases
    the requests with new_tokens < 0, grows the others; all int32 CUDA tensors but
    slot_mapping (int64).  context_lens_out and num_free_out default to context_lens and
    num_free, updated in place."""
    if context_lens_out is None:
        context_lens_out = context_lens
    if num_free_out is None:
        num_free_out = num_free
    tensors = (block_tables, context_lens, new_tokens, free_list, num_free, query_start, granted, context_lens_out,
               num_free_out, slot_mapping)
    int32 = _torch().int32
    for name, t in zip(_TABLE_NAMES, tensors[:-1]):
        if t.dtype != int32:
            raise TypeError(f"{name} must be int32")
    if slot_mapping.dtype != _torch().int64:
        raise TypeError("slot_mapping must be int64")
    S, W = block_tables.shape
    one = (S,)
    _want(context_lens.shape == one and new_tokens.shape == one and granted.shape == one and
          context_lens_out.shape == one, "context_lens, new_tokens, granted and context_lens_out must be [S]")
    _want(query_start.shape == (S + 1,), "query_start must be [S + 1]")
    _want(num_free.numel() == 1 and num_free_out.numel() == 1, "num_free and num_free_out hold one number")
    _want(free_list.dim() == 1 and slot_mapping.dim() == 1, "free_list and slot_mapping must have one dimension")
    blocks, slots = free_list.shape[0], slot_mapping.shape[0]
    _check_counts(S | W | blocks | slots)
    dev, device = _on_device(_TABLE_NAMES, tensors)
    _call("pa_build_tables", device, block_tables.data_ptr(), W, context_lens_out.data_ptr(),
          context_lens.data_ptr(), new_tokens.data_ptr(), S, free_list.data_ptr(), blocks,
          num_free_out.data_ptr(), num_free.data_ptr(), block_size, granted.data_ptr(), query_start.data_ptr(),
          slot_mapping.data_ptr(), slots, _raw_stream(stream, dev))


_FORK_NAMES = ("block_tables", "context_lens", "parents", "extra_refs", "free_list", "num_free", "copy_pairs",
               "granted", "block_tables_out", "context_lens_out", "num_free_out")


def pa_fork_tables(block_tables_out, context_lens_out, block_tables, context_lens, parents, extra_refs, free_list,
                   num_free, block_size: int, copy_pairs, granted, num_free_out=None, stream=None):
    """New rows [C, W] that go on from old ones ([S, W]; parents int32 [C], outside [0, S):
    empty), sharing full blocks by extra_refs (int32 [num_blocks], references beyond the
    first), with copies for half-filled last blocks (copy_pairs int32 [C, 2]: run
    pa_copy_blocks) and the blocks that nobody holds any more back on the free list (see
    pa_fork_tables in include/pagedkv.h).  num_free_out defaults to num_free, in place."""
    if num_free_out is None:
        num_free_out = num_free
    tensors = (block_tables, context_lens, parents, extra_refs, free_list, num_free, copy_pairs, granted,
               block_tables_out, context_lens_out, num_free_out)
    int32 = _torch().int32
    for name, t in zip(_FORK_NAMES, tensors):
        if t.dtype != int32:
            raise TypeError(f"{name} must be int32")
    _want(block_tables.dim() == 2 and block_tables_out.dim() == 2, "block_tables must be [S, W]")
    S, W = block_tables.shape
    C = block_tables_out.shape[0]
    _want(block_tables_out.shape[1] == W, "block_tables_out must be [C, W]")
    _want(context_lens.shape == (S,) and context_lens_out.shape == (C,) and parents.shape == (C,) and
          granted.shape == (C,), "context_lens must be [S]; context_lens_out, parents and granted [C]")
    _want(copy_pairs.shape == (C, 2), "copy_pairs must be [C, 2]")
    _want(num_free.numel() == 1 and num_free_out.numel() == 1, "num_free and num_free_out hold one number")
    _want(free_list.dim() == 1 and extra_refs.shape == free_list.shape, "free_list and extra_refs must be [num_blocks]")
    blocks = free_list.shape[0]
    _check_counts(S | W | C | blocks)
    dev, device = _on_device(_FORK_NAMES, tensors)
    _call("pa_fork_tables", device, block_tables_out.data_ptr(), block_tables.data_ptr(), W,
          context_lens_out.data_ptr(), context_lens.data_ptr(), S, parents.data_ptr(), C, extra_refs.data_ptr(),
          free_list.data_ptr(), blocks, num_free_out.data_ptr(), num_free.data_ptr(), block_size,
          copy_pairs.data_ptr(), granted.data_ptr(), _raw_stream(stream, dev))


# ----------------------------------------------------------------------------
# attention of several query tokens per sequence
# ----------------------------------------------------------------------------
def pa_attend_workspace_size(num_q_heads: int, num_kv_heads: int, head_dim: int) -> int:
    """Bytes of workspace pa_attend needs on the current device, whatever the lengths."""
    n = _load().pa_attend_workspace_size(num_q_heads, num_kv_heads, head_dim)
    if n == ctypes.c_size_t(-1).value:
        raise PagedKVError(PA_ERR_INVALID, "pa_attend_workspace_size")
    return n


@functools.lru_cache(maxsize=None)
def _attend_workspace_bytes(dev: int, num_q_heads: int, num_kv_heads: int, head_dim: int) -> int:
    with _torch().device(dev):
        return pa_attend_workspace_size(num_q_heads, num_kv_heads, head_dim)


_ATTEND_NAMES = ("out", "k_cache", "v_cache", "block_tables", "context_lens", "query_start", "lse")


def pa_attend(out, q, k_cache, v_cache, block_tables, context_lens, query_start, scale: float, num_q_heads: int,
              num_kv_heads: int, head_dim: int, block_size: int, causal: bool = False, lse=None, workspace=None,
              stream=None):
    """out[N, Hq, d] <- attention of sequence s's query tokens, rows query_start[s] .. of q
    (query_start int32 [S + 1]), over its paged keys: all of them, or with `causal` those up
    to the token's own, the query tokens being the last of the context (see pa_attend in
    include/pagedkv.h).  q's rows may be strided; lse: float32 [N, Hq] for the rows'
    log-sum-exp, or None; workspace: uint8 CUDA tensor or None (allocated here)."""
    T = _torch()
    qshape = q.shape
    n = qshape[0] if qshape else 0
    _want(qshape == (n, num_q_heads, head_dim) and out.shape == qshape, "q and out must be [N, Hq, d]")
    q_stride = _row_stride(q, "q", n, num_q_heads * head_dim, head_dim)
    cache = k_cache.shape
    blocks = cache[0] if cache else 0
    _want(cache == (blocks, block_size, num_kv_heads, head_dim) and v_cache.shape == cache,
          "the caches must be [num_blocks, B, Hkv, d]")
    if not out.dtype is q.dtype is k_cache.dtype is v_cache.dtype:
        raise TypeError("out, q, k_cache and v_cache must have one dtype")
    if not block_tables.dtype is context_lens.dtype is query_start.dtype is T.int32:
        raise TypeError("block_tables, context_lens and query_start must be int32")
    _want(block_tables.dim() == 2, "block_tables must be [S, W]")
    S, W = block_tables.shape
    _want(context_lens.shape == (S,) and query_start.shape == (S + 1,),
          "context_lens must be [S] and query_start [S + 1]")
    _check_counts(n | S | W | blocks)
    tensors = (out, k_cache, v_cache, block_tables, context_lens, query_start)
    lse_ptr = None
    if lse is not None:
        if lse.dtype is not T.float32:
            raise TypeError("lse must be float32")
        _want(lse.shape == (n, num_q_heads), "lse must be [N, Hq]")
        tensors += (lse,)
        lse_ptr = lse.data_ptr()
    dev, device = _on_device(_ATTEND_NAMES, tensors)
    _want(q.get_device() == dev, "q must be on the device of out")
    if workspace is None:
        size = _attend_workspace_bytes(dev, num_q_heads, num_kv_heads, head_dim)
        workspace = T.empty(size, dtype=T.uint8, device=q.device) if stream is None else _launch_scratch(
            size, q.device, stream)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on the device of q")
    _call("pa_attend", device, out.data_ptr(), lse_ptr, q.data_ptr(), q_stride,
          k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(), W, context_lens.data_ptr(),
          query_start.data_ptr(), S, n, blocks, float(scale), int(causal), num_q_heads, num_kv_heads,
          head_dim, block_size, _code(q), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
          _raw_stream(stream, dev))
    return out


# ----------------------------------------------------------------------------
# rotary positions
# ----------------------------------------------------------------------------
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "bands": 3, "yarn": 4}


def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     original_len: float = 0.0, low: float = 1.0, high: float = 32.0):
    """(freqs int64 [rotary_dim / 2] on the host, amplitude) of pa_rope and pa_rope_append:
    turns per position in units of 2^-64, unscaled or scaled for long contexts ("linear",
    "ntk", "bands", "yarn"; see pa_rope_frequencies in include/pagedkv.h).  A program copies
    freqs to the device once."""
    import torch
    _want(scaling in ROPE_SCALINGS, f"scaling must be one of {sorted(ROPE_SCALINGS)}")
    _want(0 < rotary_dim <= 1 << 20 and rotary_dim % 2 == 0, "rotary_dim must be even and positive")
    freqs = torch.empty(rotary_dim // 2, dtype=torch.int64)
    amplitude = ctypes.c_float()
    _check(_load().pa_rope_frequencies(freqs.data_ptr(), ctypes.byref(amplitude), rotary_dim, base,
                                       ROPE_SCALINGS[scaling], factor, original_len, low, high),
           "pa_rope_frequencies")
    return freqs, amplitude.value


def _row_stride(t, name: str, n: int, dense: int, d: int) -> int:
    """Elements between the rows of a [n, H, d] tensor, whose rows (`dense` elements) have to be dense."""
    if t.is_contiguous():
        return dense
    row, head, one = t.stride()
    if one != 1 or (head != d and dense > d):
        raise ValueError(f"{name} must have dense [heads, head_dim] rows")
    return row if n > 1 else dense


def _rope_error(names, tensors, positions, freqs):
    """What is wrong with the types and places of a rotary call's tensors."""
    T = _torch()
    for name, t in zip(names, tensors):
        if t.dtype != tensors[0].dtype:
            raise TypeError(f"{name} and {names[0]} must have one dtype")
    if positions.dtype != T.int32 or freqs.dtype != T.int64:
        raise TypeError("positions must be int32 and freqs int64")
    dev = tensors[0].get_device()
    for name, t in zip(names + ("positions", "freqs"), tensors + (positions, freqs)):
        if t.get_device() != dev or dev < 0:
            raise ValueError(f"{name} must be a CUDA tensor on the device of {names[0]}")
    _on_device(("positions", "freqs"), (positions, freqs))
    raise ValueError("positions must be [N] and freqs [rotary_dim / 2]")


def pa_rope(q_out, q, k_out, k, positions, freqs, interleaved: bool = False, amplitude: float = 1.0, stream=None):
    """q_out, k_out [N, H, d] <- q, k turned by their positions (see pa_rope in
    include/pagedkv.h).  Rows may be strided (parts of a fused projection); q_out may be q
    and k_out k.  freqs int64 [rotary_dim / 2]: rope_frequencies's, on the device."""
    T = _torch()
    _want(q.dim() == 3 and k.dim() == 3, "q must be [N, Hq, d] and k [N, Hkv, d]")
    n, hq, d = q.shape
    kshape = k.shape
    hkv = kshape[1]
    _want(kshape == (n, hkv, d), "q must be [N, Hq, d] and k [N, Hkv, d]")
    _want(q_out.shape == (n, hq, d) and k_out.shape == kshape, "q_out must be as q and k_out as k")
    dtype, dev = q.dtype, q.get_device()
    for t in (q_out, k_out, k):
        if t.dtype is not dtype or t.get_device() != dev:
            _rope_error(("q", "q_out", "k_out", "k"), (q, q_out, k_out, k), positions, freqs)
    if (positions.dtype is not T.int32 or freqs.dtype is not T.int64 or positions.shape != (n,) or freqs.dim() != 1 or
            positions.get_device() != dev or freqs.get_device() != dev or dev < 0 or
            not positions.is_contiguous() or not freqs.is_contiguous()):
        _rope_error(("q",), (q,), positions, freqs)
    _check_counts(n)
    _call("pa_rope", None if dev == T.current_device() else T.device(dev), q_out.data_ptr(),
          _row_stride(q_out, "q_out", n, hq * d, d), q.data_ptr(), _row_stride(q, "q", n, hq * d, d), k_out.data_ptr(),
          _row_stride(k_out, "k_out", n, hkv * d, d), k.data_ptr(), _row_stride(k, "k", n, hkv * d, d),
          positions.data_ptr(), freqs.data_ptr(), n, hq, hkv, d, 2 * freqs.shape[0], int(interleaved), amplitude,
          _code(q), _raw_stream(stream, dev))


def pa_rope_append(q_out, q, k, v, k_cache, v_cache, positions, slot_mapping, freqs, interleaved: bool = False,
                   amplitude: float = 1.0, stream=None):
    """q_out [N, Hq, d] <- q turned by its positions; k turned likewise and v go through
    slot_mapping (int64 [N], negative: skipped) into the caches [num_blocks, B, Hkv, d] (see
    pa_rope_append in include/pagedkv.h).  q, k and v may be strided rows of one fused
    projection; q_out may be q."""
    T = _torch()
    _want(q.dim() == 3 and k_cache.dim() == 4, "q must be [N, Hq, d] and the caches [num_blocks, B, Hkv, d]")
    n, hq, d = q.shape
    cache = k_cache.shape
    blocks, size, hkv, _ = cache
    _want(cache == (blocks, size, hkv, d) and v_cache.shape == cache, "the caches must be [num_blocks, B, Hkv, d]")
    _want(k.shape == (n, hkv, d) and v.shape == (n, hkv, d), "k and v must be [N, Hkv, d]")
    _want(q_out.shape == (n, hq, d), "q_out must be as q")
    dtype, dev = q.dtype, q.get_device()
    for t in (q_out, k, v, k_cache, v_cache):
        if t.dtype is not dtype or t.get_device() != dev:
            _rope_error(("q", "q_out", "k", "v", "k_cache", "v_cache"), (q, q_out, k, v, k_cache, v_cache), positions,
                        freqs)
    if (positions.dtype is not T.int32 or freqs.dtype is not T.int64 or positions.shape != (n,) or freqs.dim() != 1 or
            positions.get_device() != dev or freqs.get_device() != dev or dev < 0 or
            not positions.is_contiguous() or not freqs.is_contiguous()):
        _rope_error(("q",), (q,), positions, freqs)
    if slot_mapping.dtype is not T.int64:
        raise TypeError("slot_mapping must be int64")
    _want(slot_mapping.shape == (n,), "slot_mapping must be [N]")
    for name, t in (("slot_mapping", slot_mapping), ("k_cache", k_cache), ("v_cache", v_cache)):
        if t.get_device() != dev or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous and on the device of q")
    _check_counts(n | blocks | size)
    _call("pa_rope_append", None if dev == T.current_device() else T.device(dev), q_out.data_ptr(),
          _row_stride(q_out, "q_out", n, hq * d, d), q.data_ptr(), _row_stride(q, "q", n, hq * d, d), k.data_ptr(),
          _row_stride(k, "k", n, hkv * d, d), v.data_ptr(), _row_stride(v, "v", n, hkv * d, d), k_cache.data_ptr(),
          v_cache.data_ptr(), positions.data_ptr(), slot_mapping.data_ptr(), freqs.data_ptr(), n, hq, hkv, d,
          2 * freqs.shape[0], int(interleaved), amplitude, size, blocks, _code(q), _raw_stream(stream, dev))


def pa_kv_transfer_worthwhile(reusable_tokens: int, threshold_tokens: int = 64) -> bool:
    """Fetch another engine's KV for a prefix (True) or recompute it (False)."""
    return bool(_load().pa_kv_transfer_worthwhile(int(reusable_tokens), int(threshold_tokens)))


__all__ = ["pa_decode", "pa_decode_append", "pa_decode_plan_bytes", "pa_decode_plan", "pa_decode_planned",
           "pa_decode_shared_plan_bytes", "pa_decode_shared_plan", "pa_decode_shared_planned",
           "PA_DEVERR_PLAN", "PLAN_BYTES_PER_CTA",
           "pa_decode_shared", "pa_decode_shared_workspace_size",
           "share_groups", "share_saving", "share_pays", "SHARE_MIN_SAVING", "SHARE_MIN_BYTES",
           "pa_decode_noalloc", "pa_decode_workspace_size", "pa_decode_partition_size", "alloc_workspace",
           "pa_reshape_and_cache", "pa_copy_blocks", "pa_swap_blocks", "pa_gather_blocks",
           "pa_scatter_blocks", "pa_q8_block_bytes", "alloc_q8_cache", "q8_views", "pa_q8_append", "pa_q8_decode",
           "pa_q8_decode_workspace_size", "pa_q8_copy_blocks", "pa_q8_swap_blocks", "pa_build_tables",
           "pa_attend", "pa_attend_workspace_size", "pa_fork_tables", "rope_frequencies", "ROPE_SCALINGS", "pa_rope", "pa_rope_append",
           "pa_kv_transfer_worthwhile", "pa_device_errors", "pa_set_wait_limit_ns",
           "PA_DEVERR_TIMEOUT_FULL", "PA_DEVERR_TIMEOUT_EMPTY", "PA_DEVERR_SHARE", "PA_WAIT_LIMIT_DEFAULT_NS", "pa_status_string",
           "BlockAllocator", "PagedKVError", "OutOfBlocks", "library_path"]
