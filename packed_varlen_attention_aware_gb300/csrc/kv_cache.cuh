// The 8-bit key/value cache as the kernels see it: where the rows of a call
// lie, the scale of a block, and the checks that every cache call shares.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"

namespace hdp {

constexpr int kBlock = HDP_CACHE_BLOCK;  // tokens of a page

// Device-side view of an hdp_cache_t.
struct CacheView {
  uint8_t* k;
  uint8_t* v;
  float* scales;
  int8_t* bounds;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* cu;  // null: one row for each sequence
  int num_pages, hkv, num_seqs, max_pages;
  int rows;
  unsigned int* err;
};

// Host: checks what every call needs and fills the view (kv_cache.cu).
hdp_status_t cache_view(const char* call, const hdp_cache_t* c, const int32_t* cu, int64_t rows, CacheView* out);

__device__ __forceinline__ void report_table(const CacheView& c) {
  if (c.err) atomicCAS(c.err, 0u, kErrCacheTable);
}

// Length of sequence i, inside its page table's columns.
__device__ __forceinline__ long long seq_len(const CacheView& c, int i) {
  const long long l = __ldg(c.lens + i), top = static_cast<long long>(c.max_pages) * kBlock;
  if (l < 0 || l > top) {
    report_table(c);
    return l < 0 ? 0 : top;
  }
  return l;
}

// First row and number of rows of sequence i in the call, inside [0, rows].
__device__ __forceinline__ void seq_rows(const CacheView& c, int i, int& row0, int& n) {
  if (!c.cu) {
    row0 = i;
    n = 1;
    return;
  }
  const int a = __ldg(c.cu + i), b = __ldg(c.cu + i + 1);
  row0 = a;
  n = a < 0 || a >= c.rows || b <= a ? 0 : min(b, c.rows) - a;
}

// Newest rows decide the positions: the row count that positions count from is
// the one cu states, even where `rows` cuts the last sequence short.
__device__ __forceinline__ long long first_position(const CacheView& c, int i, long long len) {
  if (!c.cu) return len - 1;
  return len - (static_cast<long long>(__ldg(c.cu + i + 1)) - __ldg(c.cu + i));
}

// Largest i in [0, n) with f(i) <= x, for an f that does not fall (0 if there
// is none).  All 32 lanes look at once: two dependent loads up to n = 1024,
// where a binary search would wait for ten.
template <class F>
__device__ __forceinline__ int find_last(int n, long long x, F f) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5;
    const int at = lo + lane * step;
    const unsigned ok = __ballot_sync(0xffffffffu, at < hi && f(at) <= x);
    const int last = ok ? 31 - __clz(ok) : 0;
    lo += last * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// The sequence that row t belongs to, or -1.
__device__ __forceinline__ int seq_of_row(const CacheView& c, int t) {
  if (!c.cu) return t;
  const int i = find_last(c.num_seqs, t, [&](int s) { return static_cast<long long>(__ldg(c.cu + s)); });
  int row0, n;
  seq_rows(c, i, row0, n);
  return t >= row0 && t - row0 < n ? i : -1;
}

// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// Page of block b of sequence i; -1 (and a report) if it lies outside the pool.
__device__ __forceinline__ int page_of(const CacheView& c, int i, int b) {
  const int p = __ldg(c.table + static_cast<long long>(i) * c.max_pages + b);
  if (p < 0 || p >= c.num_pages) {
    report_table(c);
    return -1;
  }
  return p;
}

// The block of a CTA: which sequence, block and rows `slot` stands for.
// Sequence i has the slots from cu[i] / 64 + 2 i on; n rows touch at most
// ceil((n + 62) / 64) + 1 <= cu[i+1] / 64 - cu[i] / 64 + 2 blocks.
struct Touched {
  int seq, block;
  int first, count;  // first token of the block that the call has, and how many
  long long row;     // row of that token
  bool fresh;        // the block's first token is among them
  long long row0, before;  // the slot also stands for `before` rows from row0 on, at negative positions
};

__device__ __forceinline__ bool touched_block(const CacheView& c, int slot, Touched& t) {
  const int i = c.cu ? find_last(c.num_seqs, slot,
                                 [&](int s) { return static_cast<long long>(__ldg(c.cu + s)) / kBlock + 2LL * s; })
                     : slot;
  int row0, n;
  seq_rows(c, i, row0, n);
  t.before = 0;
  if (n == 0) return false;
  const long long len = seq_len(c, i), p0 = first_position(c, i, len);
  const long long nth = c.cu ? slot - (row0 / kBlock + 2LL * i) : 0;
  if (nth == 0 && p0 < 0) {
    t.row0 = row0;
    t.before = min(static_cast<long long>(n), -p0);
  }
  const long long a0 = p0 > 0 ? p0 : 0;
  const long long b = a0 / kBlock + nth;
  const long long end = min(len, p0 + n);
  if (nth < 0 || b * kBlock >= end) return false;
  const long long a = max(a0, b * kBlock), z = min(end, (b + 1) * kBlock);
  if (z <= a) return false;
  t.seq = i;
  t.block = static_cast<int>(b);
  t.first = static_cast<int>(a - b * kBlock);
  t.count = static_cast<int>(z - a);
  t.row = row0 + (a - p0);
  t.fresh = t.first == 0;
  return true;
}

}  // namespace hdp
