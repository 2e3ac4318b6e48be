"""GB300 (sm_103a) document-masked causal attention over packed, chunked
micro-batches -- the local attention step of ByteScale's hybrid data
parallelism ("ByteScale: Communication-Efficient Scaling of LLM Training with
a 2048K Context Length on 16384 GPUs", research digest, sections 3.1-3.2).

The compute path is libhdpattn.so (include/hdpattn.h); this package is its
ctypes binding plus seeded workload generators.  Importing the package does
not load the library; the first call does, and fails loudly if it is absent.
"""
from __future__ import annotations

import contextlib
import math

from .binding import (  # noqa: F401
    EXPORTED,
    HDP_BALANCE_DP,
    HDP_BALANCE_PP,
    HDP_CACHE_BLOCK,
    HDP_CACHE_E4M3,
    HDP_CACHE_INT8,
    HDP_ERR_CUDA,
    HDP_ERR_DEVICE_TIMEOUT,
    HDP_ERR_INVALID_ARGUMENT,
    HDP_ERR_OUT_OF_MEMORY,
    HDP_ERR_UNSUPPORTED,
    HDP_MODE_FUSED,
    HDP_MODE_SPLIT,
    HDP_OK,
    HDP_PLAN_DEFAULT,
    HDP_PLAN_NO_SHARDS,
    HDP_PLAN_NO_SPLIT,
    HdpError,
    KVCache,
    OffloadModel,
    Plan,
    hdp_attention_bwd,
    hdp_attention_bwd_workspace_bytes,
    hdp_attention_fwd,
    hdp_attention_fwd_split_noalloc,
    hdp_balance_schedule,
    hdp_attention_workspace_bytes,
    hdp_cache_append,
    hdp_cache_attention,
    hdp_cache_attention_workspace_bytes,
    hdp_cache_read,
    hdp_cache_select,
    hdp_cache_select_workspace_bytes,
    hdp_device_status,
    hdp_fit_cost_model,
    hdp_flops_per_shard,
    hdp_kernel_launch_count,
    hdp_host_sync_count,
    hdp_set_wait_budget,
    hdp_last_error_message,
    hdp_lse_merge,
    hdp_lse_merge_rows,
    hdp_offload_ranks,
    hdp_plan_create,
    hdp_plan_create_ex,
    hdp_plan_destroy,
    hdp_plan_view,
    hdp_ring_attention_time,
    hdp_ring_step_compute,
    hdp_status_string,
    load,
)


def attention(q, k, v, d_lengths, capacity: int, mode: int = HDP_MODE_FUSED, scale: float | None = None,
              plan: Plan | None = None, stream=None):
    """Convenience wrapper: plan (unless given), attention, and (in SPLIT mode)
    the merge.  q [T][hq][d], k/v [T][hkv][d] bf16 CUDA tensors; returns
    (o bf16 [T][hq][d], lse fp32 [hq][T], plan)."""
    import torch

    T, hq, d = q.shape
    hkv = k.shape[1]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if plan is None:
        plan = hdp_plan_create(d_lengths, capacity, stream=stream)
    o = torch.empty_like(q)
    lse = torch.empty((hq, T), dtype=torch.float32, device=q.device)
    ws = None
    nbytes = hdp_attention_workspace_bytes(plan, hq, d, mode)
    if nbytes:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    hdp_attention_fwd(plan, q, k, v, hq, hkv, d, scale, mode, ws, o, lse, stream=stream)
    return o, lse, plan


def attention_backward(plan: Plan, q, k, v, o, lse, dout, scale: float | None = None, stream=None):
    """Gradients (dq, dk, dv) of sum(o * dout) for the forward that produced
    (o, lse) with this plan.  bf16 CUDA tensors in the forward's layouts."""
    import torch

    T, hq, d = q.shape
    hkv = k.shape[1]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    nbytes = hdp_attention_bwd_workspace_bytes(plan, hq, d)
    ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    hdp_attention_bwd(plan, q, k, v, o, lse, dout, hq, hkv, d, scale, ws, dq, dk, dv, stream=stream)
    return dq, dk, dv


_HERE = contextlib.nullcontext()


def _pool(stream, cache):
    """The stream whose memory pool a call's tensors come from: what is freed after the call is only given out again in
    that stream's order."""
    if stream is None:
        return _HERE
    import torch

    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=cache.device)
    return torch.cuda.stream(stream)


def _in_use(stream, cache, *inputs):
    """Inputs of a call on another torch stream: their memory, freed, is not given out before that stream has read it.
    (Nothing can be noted for a stream that torch does not own, which may be destroyed before the tensors are.)"""
    if stream is None or isinstance(stream, int):
        return
    import torch

    if isinstance(stream, torch.cuda.Stream) and not isinstance(stream, torch.cuda.ExternalStream):
        for t in (cache.k, cache.v, cache.scales, cache.bounds, *inputs):
            if t is not None:
                t.record_stream(stream)


# The calls below run on `stream`, or on the current one.  As everywhere in torch, a call on another stream than the one
# that made its inputs has to be ordered behind it (stream.wait_stream).  A torch stream keeps its inputs' memory until
# it has read them; with a raw handle or another's stream the caller keeps the inputs alive until the call has run.  What a call on
# another stream than the current one returns belongs to that stream.

def cache_append(cache: KVCache, page_table, lens, k, v, cu=None, stream=None):
    """Writes k, v [rows][hkv][d] bf16 into the cache: the newest tokens of each sequence, packed, with prefix sums cu
    (None: one row for each sequence).  lens counts them already."""
    hdp_cache_append(cache, page_table, lens, k, v, cu=cu, stream=stream)
    _in_use(stream, cache, page_table, lens, k, v, cu)


def cache_read(cache: KVCache, page_table, lens, rows: int, cu=None, stream=None):
    """The newest tokens of each sequence as (k, v) [rows][hkv][d] bf16: code * scale, exactly down to bf16's smallest number."""
    import torch

    s = cache._with(page_table, lens, cu, rows)
    with _pool(stream, cache):
        k = torch.empty((rows, cache.hkv, cache.d), dtype=torch.bfloat16, device=cache.device)
        v = torch.empty_like(k)
    cache._call("hdp_cache_read", stream, s, None if cu is None else cu.data_ptr(), rows, k.data_ptr(), v.data_ptr())
    _in_use(stream, cache, page_table, lens, cu)
    return k, v


def cache_select(cache: KVCache, page_table, lens, q, count: int, cu=None, keep_first: int = 1, keep_last: int = 1,
                 stream=None):
    """The `count` blocks of the cache with the highest upper bound of their scores, for each row of q [rows][hq][d]
    bf16 and kv head: int32 [rows][hkv][count], ascending, -1 behind the last."""
    import torch

    rows, hq = cache._rows_of(q, "q")
    s = cache._with(page_table, lens, cu, rows)
    nbytes = (rows * cache.hkv * page_table.shape[1] * 4 + 255) // 256 * 256  # hdp_cache_select_workspace_bytes
    with _pool(stream, cache):
        blocks = torch.empty((rows, cache.hkv, count), dtype=torch.int32, device=cache.device)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=cache.device)
    cache._call("hdp_cache_select", stream, s, None if cu is None else cu.data_ptr(), rows, q.data_ptr(), hq, count,
                keep_first, keep_last, ws.data_ptr(), nbytes, blocks.data_ptr())
    _in_use(stream, cache, page_table, lens, q, cu)
    return blocks


def cache_attention(cache: KVCache, page_table, lens, q, cu=None, blocks=None, scale: float | None = None,
                    stream=None):
    """Attention of q [rows][hq][d] bf16, the newest tokens of each sequence, over the cache, or over the chosen
    blocks only; returns (o bf16 [rows][hq][d], lse fp32 [hq][rows])."""
    import torch

    rows, hq = cache._rows_of(q, "q")
    s = cache._with(page_table, lens, cu, rows)
    count, list_ptr = cache._blocks_of(blocks, rows)
    if scale is None:
        scale = 1.0 / math.sqrt(cache.d)
    nbytes = cache._attention_bytes
    if nbytes is None:
        nbytes = cache._attention_bytes = hdp_cache_attention_workspace_bytes(cache, hq)
    with _pool(stream, cache):
        o = torch.empty_like(q)
        lse = torch.empty((hq, rows), dtype=torch.float32, device=cache.device)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=cache.device)
    cache._call("hdp_cache_attention", stream, s, None if cu is None else cu.data_ptr(), rows, q.data_ptr(), hq, scale,
                list_ptr, count, ws.data_ptr(), nbytes, o.data_ptr(), lse.data_ptr())
    _in_use(stream, cache, page_table, lens, q, cu, blocks)
    return o, lse
