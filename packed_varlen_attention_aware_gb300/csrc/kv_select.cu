// Choosing blocks of the 8-bit cache for each query by an upper bound of the
// scores of their keys.
//
// The bound of a block is sum_ch max(q_ch, 0) hi_ch + min(q_ch, 0) lo_ch with
// the channel-wise extremes lo, hi of its keys.  Everything in it is a whole
// number (8-bit extremes, query rows rounded to 8 bits, added up over the heads
// of the group to 16), so a block costs 2 d bytes and d two-way integer dot
// products whatever the group's size is, and the choice does not depend on the
// order of summation.  HBM bounds the scores (1/64 of the cache's bytes).
//
//   Up to 32,768 blocks (2M tokens) and a count of 512, one kernel scores and
//   chooses, a cluster of CTAs for each (row, kv head); beyond, the scores go
//   through memory.  The choice is a search over the key's value that counts the
//   keys above three cuts at a time (no atomics, so many equal keys cost
//   nothing); ballots then give each chosen block its place in ascending order.
#include <cooperative_groups.h>

#include <algorithm>
#include <string>

#include "kv_cache.cuh"

namespace hdp {
namespace {

constexpr int kScoreThreads = 256;
constexpr int kScoreBlocks = 256;  // blocks of a CTA: 32 a warp
constexpr int kTopThreads = 1024;
constexpr uint32_t kForced = 0xffffffffu, kNanKey = 0xfffffffeu;

struct SelectParams {
  CacheView c;
  const __nv_bfloat16* q;
  uint32_t* keys;  // [rows][hkv][max_pages]
  int32_t* out;
  int hq, g, count, first, last;
};

// Sequence, position and visible blocks of a row; false for a row of no sequence.
__device__ __forceinline__ bool row_place(const CacheView& c, int t, int& seq, int& have) {
  seq = seq_of_row(c, t);
  if (seq < 0) return false;
  const long long p = first_position(c, seq, seq_len(c, seq)) + (c.cu ? t - __ldg(c.cu + seq) : 0);
  have = p < 0 ? 0 : static_cast<int>(p / kBlock) + 1;
  return true;
}

// Keys in the order of the scores.
__device__ __forceinline__ uint32_t key_of(float score) {
  const uint32_t b = __float_as_uint(score);
  return b ^ (b & 0x80000000u ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ int dp2a_lo(int a, int b, int c) {
  int r;
  asm("dp2a.lo.s32.s32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ int dp2a_hi(int a, int b, int c) {
  int r;
  asm("dp2a.hi.s32.s32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// Scores of one (row, kv head) by a CTA of THREADS threads: a warp has 32 blocks
// at a time, a lane 16 channels of one extreme, so 16 (d = 128) or 8 lanes have
// a block.
template <int D, int THREADS>
struct Scorer {
  static constexpr int kLanes = D / 8;  // of a block: D / 16 for each extreme
  static constexpr int kAhead = 8;      // blocks of a group of lanes in flight
  struct Shared {
    int16_t __align__(16) q[2][D];  // sums over the group's heads of min(c, 0) and of max(c, 0)
    uint32_t top[THREADS / 32];
  };
  const SelectParams& p;
  int seq, have, head, lane, part;
  int qr[8];  // this lane's 16 channels of q
  uint4 x[kAhead];
  int page;

  __device__ __forceinline__ Scorer(const SelectParams& p, int seq, int have, int head)
      : p(p), seq(seq), have(have), head(head), lane(threadIdx.x & 31), part(lane % kLanes) {}
  // Page of block b0 + lane.
  __device__ __forceinline__ int page_at(int b0) const { return b0 + lane < have ? page_of(p.c, seq, b0 + lane) : -1; }
  // Asks for blocks first .. first + kAhead - 1 of each group of lanes.
  __device__ __forceinline__ void fetch(int first) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int pg = __shfl_sync(0xffffffffu, page, (lane & ~(kLanes - 1)) + first + i);
      x[i] = pg >= 0 ? __ldg(reinterpret_cast<const uint4*>(p.c.bounds + (static_cast<size_t>(pg) * p.c.hkv + head) * (2 * D)) + part)
                     : make_uint4(0, 0, 0, 0);
    }
  }
  // Rounds the group's query rows to whole numbers (all threads).
  __device__ __forceinline__ void query(Shared& sm, int row) {
    const __nv_bfloat16* q = p.q + (static_cast<size_t>(row) * p.hq + head * p.g) * D;
    uint32_t top = 0;
    for (int i = threadIdx.x; i < p.g * D / 8; i += THREADS) {
      const uint4 y = __ldg(reinterpret_cast<const uint4*>(q) + i);
      const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t lo = w[k] & 0x7fffu, hi = (w[k] >> 16) & 0x7fffu;
        top = max(top, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
      }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) sm.top[threadIdx.x >> 5] = top;
    __syncthreads();
    if (threadIdx.x < D) {
#pragma unroll
      for (int w = 0; w < THREADS / 32; ++w) top = max(top, sm.top[w]);
      // the smallest 2^e, e >= -126, with the largest magnitude at most 127 * 2^e (127 = 1.984375 * 2^6)
      const int e = max(static_cast<int>(top >> 7) - 127 - 6 + ((top & 0x7f) > 0x7e), -126);
      const float down = pow2i(-e);
      int neg = 0, pos = 0;
#pragma unroll 4
      for (int h = 0; h < p.g; ++h) {
        const float y = __bfloat162float(q[h * D + threadIdx.x]);
        const int c = (__float_as_uint(y) & 0x7fffffffu) < 0x7f800000u ? __float2int_rn(y * down) : 0;
        neg += min(c, 0);
        pos += max(c, 0);
      }
      sm.q[0][threadIdx.x] = static_cast<int16_t>(neg);
      sm.q[1][threadIdx.x] = static_cast<int16_t>(pos);
    }
    __syncthreads();
    const int4* src = reinterpret_cast<const int4*>(&sm.q[0][0] + part * 16);
    const int4 a = src[0], c = src[1];
    qr[0] = a.x;
    qr[1] = a.y;
    qr[2] = a.z;
    qr[3] = a.w;
    qr[4] = c.x;
    qr[5] = c.y;
    qr[6] = c.z;
    qr[7] = c.w;
  }
  // Key of block b0 + lane; its pages are in `page`, its first blocks asked for.
  __device__ __forceinline__ uint32_t key(int b0) {
    const float scale = page >= 0 ? __ldg(p.c.scales + 2 * (static_cast<size_t>(page) * p.c.hkv + head)) : 0.f;
    int mine = 0;
#pragma unroll
    for (int first = 0; first < kLanes; first += kAhead) {
      if (first) fetch(first);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {  // lane (group, first + i) keeps that block's sum
        int u = dp2a_lo(qr[0], x[i].x, 0);
        u = dp2a_hi(qr[1], x[i].x, u);
        u = dp2a_lo(qr[2], x[i].y, u);
        u = dp2a_hi(qr[3], x[i].y, u);
        u = dp2a_lo(qr[4], x[i].z, u);
        u = dp2a_hi(qr[5], x[i].z, u);
        u = dp2a_lo(qr[6], x[i].w, u);
        u = dp2a_hi(qr[7], x[i].w, u);
#pragma unroll
        for (int s = 1; s < kLanes; s *= 2) u += __shfl_xor_sync(0xffffffffu, u, s);
        if (part == first + i) mine = u;
      }
    }
    const int b = b0 + lane;
    if (b < p.first || b >= have - p.last) return kForced;
    if (page < 0) return 0;
    return scale == scale ? key_of(static_cast<float>(mine) * scale) : kNanKey;
  }
  // put(block, key) for this warp's blocks b0 .. b0 + 31, b0 + step .., below `to`.
  template <class P>
  __device__ __forceinline__ void all(Shared& sm, int row, int b0, int step, int to, P put) {
    if (b0 < to) {
      page = page_at(b0);
      fetch(0);  // its latency hides behind the query's work
    }
    query(sm, row);
    for (; b0 < to; b0 += step) {
      const bool more = to - b0 > step;
      const int next_page = more ? page_at(b0 + step) : -1;
      const uint32_t k = key(b0);
      if (b0 + lane < to) put(b0 + lane, k);
      page = next_page;
      if (more) fetch(0);
    }
  }
};

// Keys into memory: a CTA has 256 blocks of a (row, kv head).  Each warp's chain
// of waits (length, pages, bounds twice) bounds it, not their number: 32 warps an
// SM with 8 blocks of a lane group in flight took 16.5 us for 32,768 blocks of 8
// heads (67 MB), 20 warps with 16 blocks 17.8, loops over more blocks 18 to 40.
template <int D>
__global__ void __launch_bounds__(kScoreThreads, 4) k_cache_scores(const SelectParams p, int chunks) {
  using S = Scorer<D, kScoreThreads>;
  __shared__ typename S::Shared sm;
  const int unit = blockIdx.x / chunks, chunk = blockIdx.x - unit * chunks;
  const int row = unit / p.c.hkv, head = unit - row * p.c.hkv;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int seq, have;
  if (!row_place(p.c, row, seq, have)) return;
  if (have <= p.count || chunk * kScoreBlocks >= have) return;  // all are chosen, or none here
  S s(p, seq, have, head);
  const int b0 = chunk * kScoreBlocks + (threadIdx.x >> 5) * 32;
  s.page = s.page_at(b0);
  s.fetch(0);  // its latency hides behind the query's work
  s.query(sm, row);
  const uint32_t key = s.key(b0);
  if (b0 + s.lane < have) p.keys[(static_cast<size_t>(row) * p.c.hkv + head) * p.c.max_pages + b0 + s.lane] = key;
}

// Chooses the `count` largest of a CTA's keys, the earlier of equal ones, and
// calls emit(place, i) for each of a thread's that is chosen.  Item i of a
// thread comes after all items of the warps before its own, and after items of
// its warp with a smaller (i, lane).  key_at(i) is its key or 0, has(i) whether
// there is one; at least `count` of them are there.
// The first WARPS warps of the CTA take part (32,768 blocks, 8 heads: 31 us with
// 16 warps and 8 keys a thread, 32 with 32, 35 with 8).
struct TopShared {
  int4 count[2][32];
  uint32_t low[32], high[32];
};
template <int WARPS>
__device__ __forceinline__ void warps_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(WARPS * 32) : "memory");
}
template <int WARPS, bool PACK, class K, class H, class E>
__device__ __forceinline__ void choose(TopShared& sm, int items, int count, int forced, K key_at, H has, E emit) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool one = lane < WARPS;  // this lane has a warp's entry to add up
  uint32_t low = 0xffffffffu, high = 0;
#pragma unroll
  for (int i = 0; i < items; ++i) {
    if (has(i)) {
      const uint32_t k = key_at(i);
      low = min(low, k);
      high = max(high, k == kForced ? 0u : k);
    }
  }
  low = __reduce_min_sync(0xffffffffu, low);
  high = __reduce_max_sync(0xffffffffu, high);
  if (lane == 0) {
    sm.low[warp] = low;
    sm.high[warp] = high;
  }
  warps_sync<WARPS>();
  low = __reduce_min_sync(0xffffffffu, one ? sm.low[lane] : 0xffffffffu);
  high = __reduce_max_sync(0xffffffffu, one ? sm.high[lane] : 0u);
  // the largest x with at least `count` keys >= x: between low (all of them)
  // and the largest key that is not forced, unless the forced ones are enough
  if (forced >= count) low = high = kForced;
  int turn = 0;
  bool found = false;
  while (low < high && !found) {
    // three cuts at once: a step costs its barrier and reductions more than its counting
    const uint32_t d = high - low, q = d >> 2;
    const uint32_t m2 = low + (d >> 1) + (d & 1), m1 = max(low + q, low + 1), m3 = max(m2, high - q);
    int n12 = 0, n3 = 0;  // counts of a CTA's keys fit 16 bits (PACK), so two share a word
    int n2 = 0;
#pragma unroll
    for (int i = 0; i < items; ++i) {
      const uint32_t k = key_at(i);  // a missing key is 0, and cuts are above low, so above 0
      n12 += k >= m1;
      n2 += k >= m2;
      n3 += k >= m3;
    }
    if (PACK) {
      n12 = __reduce_add_sync(0xffffffffu, n12 | n2 << 16);
    } else {
      n12 = __reduce_add_sync(0xffffffffu, n12);
      n2 = __reduce_add_sync(0xffffffffu, n2);
    }
    n3 = __reduce_add_sync(0xffffffffu, n3);
    if (lane == 0) sm.count[turn][warp] = make_int4(n12, n2, n3, 0);
    warps_sync<WARPS>();
    const int4 c = one ? sm.count[turn][lane] : make_int4(0, 0, 0, 0);
    turn ^= 1;
    int c1 = __reduce_add_sync(0xffffffffu, c.x), c2;
    if (PACK) {
      c2 = static_cast<int>(static_cast<unsigned>(c1) >> 16);
      c1 &= 0xffff;
    } else {
      c2 = __reduce_add_sync(0xffffffffu, c.y);
    }
    const int c3 = __reduce_add_sync(0xffffffffu, c.z);
    if (c3 >= count) {
      low = m3;
      found = c3 == count;  // exactly these
    } else if (c2 >= count) {
      low = m2;
      high = m3 - 1;
      found = c2 == count;
    } else if (c1 >= count) {
      low = m1;
      high = m2 - 1;
      found = c1 == count;
    } else {
      high = m1 - 1;
    }
  }

  // keys above it are chosen, and of those equal to it the first ones (if the
  // search ended early, all of them)
  int above = 0, equal = 0;
#pragma unroll
  for (int i = 0; i < items; ++i) {
    const bool in = has(i);
    const uint32_t k = key_at(i);
    above += __popc(__ballot_sync(0xffffffffu, in && k > low));
    equal += __popc(__ballot_sync(0xffffffffu, in && k == low));
  }
  warps_sync<WARPS>();  // the search's last counts have been read
  if (lane == 0) sm.count[0][warp] = make_int4(above, equal, 0, 0);
  warps_sync<WARPS>();
  const int a = one ? sm.count[0][lane].x : 0, e = one ? sm.count[0][lane].y : 0;
  const int take = count - __reduce_add_sync(0xffffffffu, a);  // of the equal ones
  int before_above = __reduce_add_sync(0xffffffffu, lane < warp ? a : 0);
  int before_equal = __reduce_add_sync(0xffffffffu, lane < warp ? e : 0);
  const unsigned under = (1u << lane) - 1;
#pragma unroll
  for (int i = 0; i < items; ++i) {
    const bool in = has(i);
    const uint32_t k = key_at(i);
    const unsigned ma = __ballot_sync(0xffffffffu, in && k > low), me = __ballot_sync(0xffffffffu, in && k == low);
    const int ra = before_above + __popc(ma & under), re = before_equal + __popc(me & under);
    if (in && (k > low || (k == low && re < take))) emit(ra + min(re, take), i);
    before_above += __popc(ma);
    before_equal += __popc(me);
  }
}

// Forced keys: the first p.first and the last p.last of `have` > p.count blocks.
__device__ __forceinline__ int forced_in(const SelectParams& p, int have, int from, int to) {
  return max(0, min(to, p.first) - from) + max(0, to - max(from, have - p.last));
}

// Scores (unless they are in memory) and choice, up to kSelectBlocks blocks a CTA:
// a cluster of 1 to 8 CTAs has a (row, kv head), each a run of its blocks, whose
// keys stay in shared memory and then in registers.  Each chooses `count` of its own, into
// the shared memory of the first, which chooses among those; no CTA waits for
// another during a search.
constexpr int kSelectBlocks = 4 * kTopThreads;
constexpr int kChooseWarps = 16;
constexpr int kTopCtas = 8;
constexpr int kTopMost = 512;  // largest count for a cluster
template <int D>
__global__ void __launch_bounds__(kTopThreads) k_cache_select(const SelectParams p, int ctas, bool scored) {
  namespace cg = cooperative_groups;
  using S = Scorer<D, kTopThreads>;
  constexpr int kItems = kSelectBlocks / (kChooseWarps * 32);
  __shared__ typename S::Shared s_query;
  __shared__ TopShared s_top;
  __shared__ union {
    uint32_t keys[kSelectBlocks];
    struct {
      uint32_t key[kTopCtas * kTopMost];
      int block[kTopCtas * kTopMost];
    } passed;
  } sm;
  __shared__ int s_n[kTopCtas];
  cg::cluster_group cluster = cg::this_cluster();
  const int unit = blockIdx.x / ctas, rank = blockIdx.x - unit * ctas;
  const int row = unit / p.c.hkv, head = unit - row * p.c.hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int seq, have;
  const bool live = row_place(p.c, row, seq, have);
  if (scored) asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!live) return;  // the whole cluster
  int32_t* out = p.out + static_cast<size_t>(unit) * p.count;
  if (have <= p.count) {
    if (rank == 0)
      for (int i = threadIdx.x; i < p.count; i += kTopThreads) out[i] = i < have ? i : -1;
    return;
  }
  const int each = ((have + ctas - 1) / ctas + 31) / 32 * 32;  // at most kSelectBlocks
  const int from = min(have, rank * each), to = min(have, from + each), n = to - from;

  if (!scored) {
    S s(p, seq, have, head);
    s.all(s_query, row, from + warp * 32, kTopThreads, to, [&](int b, uint32_t k) { sm.keys[b - from] = k; });
    __syncthreads();
  }
  const uint32_t* keys = p.keys + static_cast<size_t>(unit) * p.c.max_pages + from;
  // The choice is up to kChooseWarps warps, which have a run of items * 32 keys each.
  const bool on = warp < kChooseWarps;
  const int items = (n + kChooseWarps * 32 - 1) / (kChooseWarps * 32);
  const int base = warp * items * 32 + lane;
  uint32_t key[kItems];
  unsigned there = 0;  // bit i: item i is one
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const bool in = on && i < items && base + i * 32 < n;
    there |= static_cast<unsigned>(in) << i;
    key[i] = !in ? 0u : scored ? __ldcg(keys + base + i * 32) : sm.keys[base + i * 32];
  }
  auto key_at = [&](int i) { return key[i]; };
  auto has = [&](int i) { return (there >> i & 1) != 0; };
  const int forced = forced_in(p, have, from, to);
  if (ctas == 1) {
    if (on)
      choose<kChooseWarps, true>(s_top, kItems, p.count, forced, key_at, has, [&](int at, int i) { out[at] = base + i * 32; });
    return;
  }
  uint32_t* to_key = cluster.map_shared_rank(sm.passed.key, 0) + rank * kTopMost;
  int* to_block = cluster.map_shared_rank(sm.passed.block, 0) + rank * kTopMost;
  auto pass_on = [&](int at, int i) {
    to_key[at] = key[i];
    to_block[at] = from + base + i * 32;
  };
  cluster.sync();  // the first CTA has its keys in registers
  if (on) {
    if (n <= p.count) {
#pragma unroll
      for (int i = 0; i < kItems; ++i)
        if (has(i)) pass_on(base + i * 32, i);
    } else {
      choose<kChooseWarps, true>(s_top, kItems, p.count, forced, key_at, has, pass_on);
    }
  }
  if (threadIdx.x == 0) cluster.map_shared_rank(s_n, 0)[rank] = min(n, p.count);
  cluster.sync();
  if (rank != 0 || !on) return;
  // slots of kTopMost for each CTA, in the order of the blocks
  const int at = warp * (kItems * 32) + lane;
  there = 0;
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const int x = at + i * 32, c = x / kTopMost;
    const bool in = c < ctas && x % kTopMost < s_n[c];
    there |= static_cast<unsigned>(in) << i;
    key[i] = in ? sm.passed.key[x] : 0u;
  }
  choose<kChooseWarps, true>(s_top, kItems, p.count, forced_in(p, have, 0, have), key_at, has,
                             [&](int place, int i) { out[place] = sm.passed.block[at + i * 32]; });
}

// The choice among keys in memory, for more blocks or a larger count than a
// cluster takes; they are read again for each step of the search.
__global__ void __launch_bounds__(kTopThreads) k_cache_top(const SelectParams p) {
  __shared__ TopShared sm;
  const int row = blockIdx.x / p.c.hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int seq, have;
  const bool live = row_place(p.c, row, seq, have);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!live) return;
  int32_t* out = p.out + static_cast<size_t>(blockIdx.x) * p.count;
  if (have <= p.count) {
    for (int i = threadIdx.x; i < p.count; i += kTopThreads) out[i] = i < have ? i : -1;
    return;
  }
  const uint32_t* keys = p.keys + static_cast<size_t>(blockIdx.x) * p.c.max_pages;
  const int items = (have + kTopThreads - 1) / kTopThreads;
  const int base = warp * items * 32 + lane;
  auto has = [&](int i) { return i < items && base + i * 32 < have; };
  choose<kTopThreads / 32, false>(sm, items, p.count, forced_in(p, have, 0, have),
                [&](int i) { return has(i) ? __ldcg(keys + base + i * 32) : 0u; }, has,
                [&](int at, int i) { out[at] = base + i * 32; });
}

// CTAs of k_cache_select for a (row, kv head), as few as hold its keys; 0: not for
// this size.  More of them cost more than they save (us a call for 8 and 64 heads
// of 2,048 blocks: 9.7 and 13.8 with one, 13.8 and 18.2 with two, 14.0 and 40.8
// with eight).
int select_ctas(int64_t units, int max_pages, int count) {
  const int least = (max_pages + kSelectBlocks - 1) / kSelectBlocks;
  int ctas = 1;
  while (ctas < least) ctas *= 2;
  if (ctas > kTopCtas || (ctas > 1 && count > kTopMost) || units * ctas > 2147483647LL) return 0;
  return ctas;
}

size_t select_bytes(int64_t rows, int hkv, int max_pages) {
  return (static_cast<size_t>(rows) * hkv * max_pages * sizeof(uint32_t) + 255) & ~size_t(255);
}

}  // namespace
}  // namespace hdp

using namespace hdp;

extern "C" hdp_status_t hdp_cache_select_workspace_bytes(const hdp_cache_t* cache, int64_t rows, size_t* bytes) {
  if (!cache || !bytes) return fail(HDP_ERR_INVALID_ARGUMENT, "hdp_cache_select_workspace_bytes: NULL argument");
  if (cache->hkv < 1 || cache->max_pages < 1 || rows < 0 || rows > 2147483647LL)
    return fail(HDP_ERR_INVALID_ARGUMENT, "hdp_cache_select_workspace_bytes: need hkv >= 1, max_pages >= 1, 0 <= rows < 2^31");
  *bytes = select_bytes(rows, cache->hkv, cache->max_pages);
  return HDP_OK;
}

extern "C" hdp_status_t hdp_cache_select(const hdp_cache_t* cache, const int32_t* cu, int64_t rows, const void* q,
                                         int32_t hq, int32_t count, int32_t keep_first, int32_t keep_last,
                                         void* workspace, size_t workspace_bytes, int32_t* blocks, void* stream) {
  SelectParams p = {};
  const hdp_status_t r = cache_view("hdp_cache_select", cache, cu, rows, &p.c);
  if (r != HDP_OK) return r;
  if (hq < 1 || hq % cache->hkv != 0)
    return fail(HDP_ERR_INVALID_ARGUMENT, "hdp_cache_select: need hq >= 1 and hq % hkv == 0");
  if (hq / cache->hkv > 128) return fail(HDP_ERR_UNSUPPORTED, "hdp_cache_select: hq / hkv must be at most 128");
  if (count < 1 || keep_first < 0 || keep_last < 0 || static_cast<int64_t>(keep_first) + keep_last > count)
    return fail(HDP_ERR_INVALID_ARGUMENT,
                "hdp_cache_select: need count >= 1, keep_first >= 0, keep_last >= 0, keep_first + keep_last <= count");
  if (rows == 0) return HDP_OK;
  if (!q || !blocks) return fail(HDP_ERR_INVALID_ARGUMENT, "hdp_cache_select: NULL argument");
  if (reinterpret_cast<uintptr_t>(q) & 15)
    return fail(HDP_ERR_INVALID_ARGUMENT, "hdp_cache_select: q must be 16-byte aligned");
  if (rows * cache->hkv > 2147483647LL / ((cache->max_pages + kScoreBlocks - 1) / kScoreBlocks))
    return fail(HDP_ERR_UNSUPPORTED, "hdp_cache_select: rows * hkv * max_pages / 256 must be below 2^31");
  const size_t need = select_bytes(rows, cache->hkv, cache->max_pages);
  if (!workspace || workspace_bytes < need)
    return fail(HDP_ERR_INVALID_ARGUMENT, "hdp_cache_select: workspace too small (need " + std::to_string(need) + " bytes)");
  if (reinterpret_cast<uintptr_t>(workspace) & 255)
    return fail(HDP_ERR_INVALID_ARGUMENT, "hdp_cache_select: workspace must be 256-byte aligned");
  p.c.err = device_error_word();
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.keys = static_cast<uint32_t*>(workspace);
  p.out = blocks;
  p.hq = hq;
  p.g = hq / cache->hkv;
  p.count = count;
  p.first = keep_first;
  p.last = keep_last;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t units = rows * cache->hkv;
  const int ctas = select_ctas(units, cache->max_pages, count);
  // Few (row, kv head)s: the scores want every SM and have a kernel of their own.
  // us a call with it and without, heads x blocks: 8 x 1,024 9.8 and 13.4, 64 x 2,048
  // 13.8 and 18.2, 64 x 4,096 19.2 and 26.9, 8 x 32,768 23.3 and 30.8.  Where the heads
  // fill the SMs themselves, one launch does: 128 x 2,048 18.9 and 18.9, 128 x 3,000
  // 29.6 and 27.5, 128 x 4,096 39.4 and 38.2 (128 x 32,768, by 8 CTAs each: 271 and 314).
  constexpr int kFewUnits = 100;
  const bool scored = !ctas || units < kFewUnits;
  if (scored) {
    const int chunks = (cache->max_pages + kScoreBlocks - 1) / kScoreBlocks;
    const unsigned grid = static_cast<unsigned>(units * chunks);
    if (cache->d == 128) k_cache_scores<128><<<grid, kScoreThreads, 0, st>>>(p, chunks);
    else k_cache_scores<64><<<grid, kScoreThreads, 0, st>>>(p, chunks);
    note_launch();
    HDP_CUDA_TRY(cudaGetLastError());
  }
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kTopThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  if (ctas) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = ctas;
    attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  if (scored) {  // the launch overlaps the scores; the kernel waits for them
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  cfg.gridDim = dim3(static_cast<unsigned>(units * std::max(1, ctas)));
  if (!ctas) HDP_CUDA_TRY(cudaLaunchKernelEx(&cfg, k_cache_top, p));
  else HDP_CUDA_TRY(cudaLaunchKernelEx(&cfg, cache->d == 128 ? k_cache_select<128> : k_cache_select<64>, p, ctas, scored));
  note_launch();
  return HDP_OK;
}
