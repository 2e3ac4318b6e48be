// Block tables and slot maps, made on the GPU from the requests' lengths.
//
// hdp_cache_assign.  A sequence of l tokens holds ceil(l / 64) pages.  With
// give_i and lack_i the pages that sequence i has too many and too few, and G_i,
// L_i their sums over the sequences before i, given pages go to the stack's places
//   top + sum give - 1 - (G_i + their rank in i's row)
// (the last sequence's last page first, so that giving back undoes taking), and
// a sequence takes the page at
//   top' - 1 - (L_i + rank),     top' = top + sum give,
// if all of its lack lies above the stack's bottom.  Every place follows from two
// prefix sums, so the moves are independent of each other.
//
// The work is a few bytes for each sequence and page moved; latency bounds it: a
// launch, the lengths, the scan, one or two rounds of dependent loads.  One CTA
// does it while the table is small; else a cluster of 8 shares the moves, each
// CTA scanning all sequences for itself (a scan of 2,048 takes less than handing
// its results on would).  Measured (one GB300, in a captured graph, by one CTA and
// by the cluster): 256 sequences, 4 pages taken 6.5 and 6.5 us; 64 sequences take
// 8,556 pages 13.5 and 8.0; one takes 32,768 16.7 and 6.9.
//
// hdp_cache_rows.  16 bytes written for each row: a warp has 128 consecutive
// rows, finds the first one's sequence together, and each lane walks on from it.
// 256 rows 3.3 us, 2M rows 9.4 (33.6 MB).
#include <cooperative_groups.h>

#include <string>

#include "kv_cache.cuh"

namespace hdp {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;              // 32 warps: scan() has a lane for each
constexpr int kEach = 2;                    // sequences of a thread
constexpr int kChunk = kThreads * kEach;    // sequences scanned at once
constexpr int kCtas = 8;                    // of a cluster

struct Assign {
  int32_t* free_pages;
  int32_t* free_count;
  int32_t* table;
  int32_t* held;
  const int32_t* lens;
  int num_pages, num_seqs, max_pages;
  unsigned int* err;
};

__device__ __forceinline__ void report(unsigned int* err, unsigned int code) {
  if (err) atomicCAS(err, 0u, code);
}

struct Need {
  int have, want;
};

__device__ __forceinline__ Need need_of(const Assign& p, int i) {
  long long l = __ldg(p.lens + i);
  int have = __ldcg(p.held + i);
  const long long top = static_cast<long long>(p.max_pages) * kBlock;
  if (l < 0 || l > top || have < 0 || have > p.max_pages) report(p.err, kErrCacheTable);
  l = min(max(l, 0LL), top);
  have = min(max(have, 0), p.max_pages);
  return {have, static_cast<int>((l + kBlock - 1) / kBlock)};
}

// Exclusive sums of x over the CTA's threads, in their order, and the total.
__device__ __forceinline__ long long scan(long long x, long long& total, long long* warp_sums) {
  static_assert(kThreads == 1024, "a lane for each warp");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long run = x;
#pragma unroll
  for (int s = 1; s < 32; s *= 2) {
    const long long up = __shfl_up_sync(0xffffffffu, run, s);
    if (lane >= s) run += up;
  }
  __syncthreads();  // the sums of the last call have been read
  if (lane == 31) warp_sums[warp] = run;
  __syncthreads();
  long long w = warp_sums[lane];
#pragma unroll
  for (int s = 1; s < 32; s *= 2) {
    const long long up = __shfl_up_sync(0xffffffffu, w, s);
    if (lane >= s) w += up;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const long long before = __shfl_sync(0xffffffffu, w, warp ? warp - 1 : 0);
  return run - x + (warp ? before : 0);
}

// Calls move(sequence of the chunk, rank in it, place in the flat order) for every
// page that a chunk moves: sums[i] is what lies before sequence i, `total` all of it.
template <class F>
__device__ __forceinline__ void each_move(const long long* sums, int n, long long total, int rank, int ctas, F move) {
  for (long long x = static_cast<long long>(rank) * kThreads + threadIdx.x; x < total; x += static_cast<long long>(ctas) * kThreads) {
    int lo = 0, hi = n;  // the last i with sums[i] <= x: it moves something
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (sums[mid] <= x) lo = mid;
      else hi = mid;
    }
    move(lo, static_cast<int>(x - sums[lo]), x);
  }
}

__global__ void __launch_bounds__(kThreads) k_cache_assign(const Assign p) {
  __shared__ long long s_sums[kChunk];
  __shared__ int s_from[kChunk];  // the first of the blocks that move
  __shared__ long long s_warp[32];
  __shared__ unsigned long long s_taken;
  const cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), ctas = cluster.num_blocks();
  const int first = threadIdx.x * kEach;

  // ---- how much there is to give and to take
  long long give = 0, lack = 0;
  for (int base = 0; base < p.num_seqs; base += kChunk)
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int i = base + k * kThreads + static_cast<int>(threadIdx.x);
      if (i >= p.num_seqs) continue;
      const Need d = need_of(p, i);
      give += max(d.have - d.want, 0);
      lack += max(d.want - d.have, 0);
    }
  int top = __ldcg(p.free_count);
  if (top < 0 || top > p.num_pages) report(p.err, kErrCacheTable);
  top = min(max(top, 0), p.num_pages);
  long long given, lacking;
  scan(give, given, s_warp);
  scan(lack, lacking, s_warp);
  if (threadIdx.x == 0) s_taken = 0;
  const long long end = top + given;
  if (end > p.num_pages) report(p.err, kErrCacheTable);  // some page was given twice
  cluster.sync();  // every CTA has read the counts that are written below

  // ---- pages given back (a sequence gives or takes: the rows do not meet)
  long long before = 0;
  for (int base = 0; given > 0 && base < p.num_seqs; base += kChunk) {
    const int n = min(kChunk, p.num_seqs - base);
    int count[kEach], sum = 0;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      count[k] = 0;
      if (first + k >= n) continue;
      const Need d = need_of(p, base + first + k);
      count[k] = max(d.have - d.want, 0);
      s_from[first + k] = d.want;
      sum += count[k];
    }
    long long total, at = scan(sum, total, s_warp);
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      s_sums[first + k] = at;
      at += count[k];
    }
    cluster.sync();  // the sums are there, and every CTA has read what this chunk holds
    each_move(s_sums, n, total, rank, ctas, [&](int i, int r, long long x) {
      const long long place = end - 1 - (before + x);
      if (place < p.num_pages)
        p.free_pages[place] = __ldcg(p.table + static_cast<long long>(base + i) * p.max_pages + s_from[i] + r);
    });
#pragma unroll
    for (int k = 0; k < kEach; ++k)
      if (rank == 0 && count[k] > 0) p.held[base + first + k] = s_from[first + k];
    before += total;
    __syncthreads();
  }
  if (given > 0) {
    __threadfence();
    cluster.sync();  // they can be taken
  }

  // ---- pages taken
  const long long stack = min(end, static_cast<long long>(p.num_pages));
  before = 0;
  for (int base = 0; lacking > 0 && base < p.num_seqs; base += kChunk) {
    const int n = min(kChunk, p.num_seqs - base);
    int count[kEach], sum = 0;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      count[k] = 0;
      if (first + k >= n) continue;
      const Need d = need_of(p, base + first + k);
      count[k] = max(d.want - d.have, 0);
      s_from[first + k] = d.have;
      sum += count[k];
    }
    long long total, at = scan(sum, total, s_warp);
    const long long mine = at;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      s_sums[first + k] = at;
      at += count[k];
    }
    cluster.sync();
    each_move(s_sums, n, total, rank, ctas, [&](int i, int r, long long x) {
      const long long next = i + 1 < n ? s_sums[i + 1] : total;
      if (before + next > stack) return;  // not enough for this sequence, nor for those behind it
      p.table[static_cast<long long>(base + i) * p.max_pages + s_from[i] + r] = __ldcg(p.free_pages + (stack - 1 - (before + x)));
    });
    at = before + mine;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      if (count[k] == 0) continue;
      at += count[k];
      if (at > stack) {
        report(p.err, kErrCachePool);
        continue;
      }
      if (rank == 0) p.held[base + first + k] = s_from[first + k] + count[k];
      atomicMax(&s_taken, static_cast<unsigned long long>(at));
    }
    before += total;
    __syncthreads();
  }
  if (rank == 0 && threadIdx.x == 0) *p.free_count = static_cast<int>(stack - static_cast<long long>(s_taken));
}

struct RowMap {
  const int32_t* table;  // null: no slots
  const int32_t* lens;
  const int32_t* cu;
  int num_seqs, max_pages, num_pages, rows;
  int32_t* seq;
  int32_t* pos;
  int64_t* slot;
  unsigned int* err;
};

constexpr int kMapThreads = 128;
constexpr int kMapRows = 4;  // of a lane

__global__ void __launch_bounds__(kMapThreads) k_cache_rows(const RowMap p) {
  const int lane = threadIdx.x & 31;
  const long long row0 = (static_cast<long long>(blockIdx.x) * (kMapThreads / 32) + (threadIdx.x >> 5)) * (32 * kMapRows);
  if (row0 >= p.rows) return;
  const long long longest = p.table ? static_cast<long long>(p.max_pages) * kBlock : 2147483647LL;
  int i = static_cast<int>(row0) + lane;
  if (p.cu) i = find_last(p.num_seqs, row0, [&](int s) { return static_cast<long long>(__ldg(p.cu + s)); });
#pragma unroll
  for (int k = 0; k < kMapRows; ++k) {
    const long long r = row0 + 32 * k + lane;
    if (r >= p.rows) return;
    int a, n;  // the sequence's first row and how many cu gives it
    if (!p.cu) {
      i = a = static_cast<int>(r);
      n = 1;
    } else {
      // the last sequence that begins at or before r: steps of 1, 2, 4, ... from the one before, then halved
      int step = 1;
      while (i + step < p.num_seqs && __ldg(p.cu + i + step) <= r) {
        i += step;
        step *= 2;
      }
      for (step /= 2; step; step /= 2)
        if (i + step < p.num_seqs && __ldg(p.cu + i + step) <= r) i += step;
      a = __ldg(p.cu + i);
      n = max(0, __ldg(p.cu + i + 1) - a);
    }
    const bool inside = a >= 0 && r >= a && r - a < n;
    int seq = -1, pos = -1;
    long long slot = -1;
    if (inside) {
      long long l = __ldg(p.lens + i);
      if (l < 0 || l > longest) report(p.err, kErrCacheTable);
      l = min(max(l, 0LL), longest);
      seq = i;
      const long long at = l - n + (r - a);
      pos = static_cast<int>(max(at, -2147483648LL));
      if (p.table && at >= 0) {
        const int page = __ldg(p.table + static_cast<long long>(i) * p.max_pages + at / kBlock);
        if (page >= 0 && page < p.num_pages) slot = static_cast<long long>(page) * kBlock + at % kBlock;
        else report(p.err, kErrCacheTable);
      }
    }
    if (p.seq) p.seq[r] = seq;
    if (p.pos) p.pos[r] = pos;
    if (p.slot) p.slot[r] = slot;
  }
}

}  // namespace
}  // namespace hdp

using namespace hdp;

extern "C" hdp_status_t hdp_cache_assign(int32_t* free_pages, int32_t* free_count, int32_t num_pages, int32_t* page_table,
                                         int32_t* held, const int32_t* lens, int32_t num_seqs, int32_t max_pages,
                                         void* stream) {
  if (!free_pages || !free_count || !page_table || !held || !lens)
    return fail(HDP_ERR_INVALID_ARGUMENT, "hdp_cache_assign: NULL argument");
  if (num_pages < 1 || num_seqs < 1 || max_pages < 1)
    return fail(HDP_ERR_INVALID_ARGUMENT, "hdp_cache_assign: num_pages, num_seqs and max_pages must be >= 1");
  if (num_seqs > (1 << 24)) return fail(HDP_ERR_UNSUPPORTED, "hdp_cache_assign: num_seqs must be at most 2^24");
  const Assign p = {free_pages, free_count, page_table, held, lens, num_pages, num_seqs, max_pages, device_error_word()};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<int64_t>(num_seqs) * max_pages <= kChunk ? 1 : kCtas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(attr.val.clusterDim.x);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  HDP_CUDA_TRY(cudaLaunchKernelEx(&cfg, k_cache_assign, p));
  note_launch();
  return HDP_OK;
}

extern "C" hdp_status_t hdp_cache_rows(const int32_t* page_table, const int32_t* lens, const int32_t* cu, int32_t num_seqs,
                                       int32_t max_pages, int32_t num_pages, int64_t rows, int32_t* sequence,
                                       int32_t* position, int64_t* slot, void* stream) {
  if (!lens) return fail(HDP_ERR_INVALID_ARGUMENT, "hdp_cache_rows: lens is NULL");
  if (num_seqs < 1) return fail(HDP_ERR_INVALID_ARGUMENT, "hdp_cache_rows: num_seqs must be >= 1");
  if (num_seqs > (1 << 24)) return fail(HDP_ERR_UNSUPPORTED, "hdp_cache_rows: num_seqs must be at most 2^24");
  if (rows < 0 || rows > 2147483647LL) return fail(HDP_ERR_INVALID_ARGUMENT, "hdp_cache_rows: rows must be 0 .. 2^31-1");
  if (!cu && rows != num_seqs) return fail(HDP_ERR_INVALID_ARGUMENT, "hdp_cache_rows: without cu, rows must equal num_seqs");
  if (slot && !page_table) return fail(HDP_ERR_INVALID_ARGUMENT, "hdp_cache_rows: slots need a page table");
  if (page_table && (max_pages < 1 || num_pages < 1))
    return fail(HDP_ERR_INVALID_ARGUMENT, "hdp_cache_rows: max_pages and num_pages must be >= 1");
  if (rows == 0) return HDP_OK;
  const RowMap p = {page_table, lens, cu, num_seqs, max_pages, num_pages, static_cast<int>(rows), sequence, position, slot,
                    device_error_word()};
  const int64_t per = kMapThreads * kMapRows;
  k_cache_rows<<<static_cast<unsigned>((rows + per - 1) / per), kMapThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  note_launch();
  HDP_CUDA_TRY(cudaGetLastError());
  return HDP_OK;
}
