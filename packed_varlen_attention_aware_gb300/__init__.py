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
    _cache_rows,
    _rotary,
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
    HDP_ROTARY_BACKWARD,
    HDP_ROTARY_NEIGHBOURS,
    HDP_TYPE_BF16,
    HDP_TYPE_FP16,
    HDP_TYPE_FP32,
    HdpError,
    KVCache,
    KVCache4,
    OffloadModel,
    PagePool,
    Plan,
    hdp_attention_bwd,
    hdp_attention_bwd_workspace_bytes,
    hdp_attention_fwd,
    hdp_attention_fwd_split_noalloc,
    hdp_balance_schedule,
    hdp_attention_workspace_bytes,
    hdp_cache_append,
    hdp_cache_assign,
    hdp_cache_attention,
    hdp_cache_attention_workspace_bytes,
    hdp_cache_read,
    hdp_cache_rows,
    hdp_cache_select,
    hdp_cache_select_workspace_bytes,
    hdp_device_status,
    hdp_fit_cost_model,
    hdp_flops_per_shard,
    hdp_fourbit_append,
    hdp_fourbit_attention,
    hdp_fourbit_attention_workspace_bytes,
    hdp_fourbit_read,
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
    hdp_rotary,
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


def _pool(stream, on):
    """The stream whose memory pool a call's tensors come from: what is freed after the call is only given out again in
    that stream's order.  `on`: a tensor or cache of the call's device."""
    if stream is None:
        return _HERE
    import torch

    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=on.device)
    return torch.cuda.stream(stream)


def _in_use(stream, cache, *inputs):
    """Inputs of a call on another torch stream: their memory, freed, is not given out before that stream has read it.
    (Nothing can be noted for a stream that torch does not own, which may be destroyed before the tensors are.)"""
    if stream is None or isinstance(stream, int):
        return
    import torch

    if isinstance(stream, torch.cuda.Stream) and not isinstance(stream, torch.cuda.ExternalStream):
        for t in (*(cache._buffers() if cache is not None else ()), *inputs):
            if t is not None:
                t.record_stream(stream)


# The calls below run on `stream`, or on the current one.  As everywhere in torch, a call on another stream than the one
# that made its inputs has to be ordered behind it (stream.wait_stream).  A torch stream keeps its inputs' memory until
# it has read them; with a raw handle or another's stream the caller keeps the inputs alive until the call has run.  What a call on
# another stream than the current one returns belongs to that stream.  A KVCache4 goes where a KVCache goes, but to
# cache_select and with lists of blocks.

def cache_append(cache: KVCache | KVCache4, page_table, lens, k, v, cu=None, stream=None):
    """Writes k, v [rows][hkv][d] bf16 into the cache: the newest tokens of each sequence, packed, with prefix sums cu
    (None: one row for each sequence).  lens counts them already."""
    hdp_cache_append(cache, page_table, lens, k, v, cu=cu, stream=stream)
    _in_use(stream, cache, page_table, lens, k, v, cu)


def cache_read(cache: KVCache | KVCache4, page_table, lens, rows: int, cu=None, stream=None):
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


def cache_attention(cache: KVCache | KVCache4, page_table, lens, q, cu=None, blocks=None, scale: float | None = None,
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
        ask = hdp_fourbit_attention_workspace_bytes if isinstance(cache, KVCache4) else hdp_cache_attention_workspace_bytes
        nbytes = cache._attention_bytes = ask(cache, hq)
    with _pool(stream, cache):
        o = torch.empty_like(q)
        lse = torch.empty((hq, rows), dtype=torch.float32, device=cache.device)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=cache.device)
    cache._call("hdp_cache_attention", stream, s, None if cu is None else cu.data_ptr(), rows, q.data_ptr(), hq, scale,
                list_ptr, count, ws.data_ptr(), nbytes, o.data_ptr(), lse.data_ptr())
    _in_use(stream, cache, page_table, lens, q, cu, blocks)
    return o, lse


def cache_assign(pool: PagePool, page_table, held, lens, stream=None):
    """Pages for sequences of these lengths: those that a sequence no longer needs go back to the pool, then each takes
    what it lacks; pool, page_table [sequences][columns] and held [sequences] int32 are updated in place.  Where pages run
    out, that sequence and the later ones keep what they hold, and hdp_device_status says so."""
    hdp_cache_assign(pool, page_table, held, lens, stream=stream)
    _in_use(stream, None, pool.free, pool.count, page_table, held, lens)


def cache_rows(lens, rows: int, cu=None, page_table=None, num_pages: int | None = None, stream=None):
    """(sequence, position, slot) of the rows of a call, the newest tokens of each sequence: int32, int32 and int64 = page
    * 64 + position % 64, -1 for rows of no sequence; slot is None without a page table.  With the lengths of packed
    documents as lens and their prefix sums as cu, position is each token's place in its document."""
    import torch

    with _pool(stream, lens):
        seq = lens.new_empty(rows, dtype=torch.int32)
        pos = lens.new_empty(rows, dtype=torch.int32)
        slot = None if page_table is None else lens.new_empty(rows, dtype=torch.int64)
    _cache_rows(lens, rows, seq, pos, slot, cu, page_table, num_pages, stream)
    _in_use(stream, None, lens, cu, page_table)
    return seq, pos, slot


def rotary_frequencies(rot: int, base: float = 10000.0, scaling: str | None = None, by: float = 1.0,
                       trained: int | None = None, fast: float = 32.0, slow: float = 1.0, device="cuda"):
    """(freqs float64 [rot / 2], factor) for rotary(): the angle of one position for each pair, base^(-2 i / rot).

    For contexts `by` times as long as the `trained` length:
      "linear"  every angle divided by `by`;
      "base"    the base times by^(rot / (rot - 2)): the slowest pair `by` times slower, the fastest as it was;
      "parts"   pairs with fewer than `slow` turns over the trained length `by` times slower, those with more than `fast`
                as they were, a linear ramp between; and q and k times 0.1 ln(by) + 1 (the factor)."""
    import torch

    if rot < 2 or rot % 2 or not base > 0:
        raise ValueError("rot must be even and at least 2, base positive")
    if scaling not in (None, "linear", "base", "parts") or not by > 0:
        raise ValueError('scaling must be None, "linear", "base" or "parts", and by positive')
    if scaling == "base":
        base = base * by ** (rot / (rot - 2)) if rot > 2 else base
    f = float(base) ** -(torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    factor = 1.0
    if scaling == "linear":
        f = f / by
    elif scaling == "parts":
        if trained is None or trained < 1 or not fast > slow:
            raise ValueError('"parts" needs the trained length and fast > slow')
        keep = ((trained * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
        f = f * (keep + (1 - keep) / by)
        factor = 0.1 * math.log(by) + 1 if by > 1 else 1.0
    return f.to(device), factor


def _turned(q, k, position, freqs, neighbours, backward, factor, inplace, stream):
    out = (q, k) if inplace else (None, None)
    with _pool(stream, q if q is not None else k):
        out = _rotary(q, k, position, freqs, *out, neighbours, backward, factor, stream)
    if inplace:
        import torch

        # a backward pass that has kept q or k from before refuses to use what is there now
        torch.autograd.graph.increment_version([x for x in (q, k) if x is not None])
    _in_use(stream, None, q, k, position, freqs)
    return out


def rotary(q, k, position, freqs, neighbours: bool = False, factor: float = 1.0, inplace: bool = False, stream=None):
    """Rotary positions of q [rows][hq][d] and k [rows][hkv][d] (either may be None; views of a fused projection are fine):
    pairs of the first 2 * len(freqs) channels of each head, channels i and i + len(freqs), or with neighbours 2 i and
    2 i + 1, are turned by position * freqs[i] and scaled by factor.  position int32 [rows] (cache_rows gives them), freqs
    float64 (rotary_frequencies).  Rows at a negative position are not written: in place they keep their values, in the new
    tensors that are returned otherwise those rows are not initialised.  In place, q and k must not share memory.  As
    everywhere in this package, gradients are not recorded: what is returned has no history, whatever q and k require, and
    rotary_backward is called for the gradients.  Returns the turned (q, k)."""
    return _turned(q, k, position, freqs, neighbours, False, factor, inplace, stream)


def rotary_backward(dq, dk, position, freqs, neighbours: bool = False, factor: float = 1.0, inplace: bool = False,
                    stream=None):
    """Gradients of the rows that went into rotary(), from those of the rows that came out of it."""
    return _turned(dq, dk, position, freqs, neighbours, True, factor, inplace, stream)
