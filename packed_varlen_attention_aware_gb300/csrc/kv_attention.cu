// Attention of the newest tokens of each sequence over the 8-bit cache.
//
// For a few query rows per sequence the work is one pass over the cache: 2 d
// bytes per (key, kv head) against 4 d multiply-adds per query head, so HBM
// bounds it as long as the arithmetic stays out of the way.
//
//   Work split.  All (sequence, kv head, tile of query rows, block of 64 keys)
//   are laid out in one flat order; each warp of a grid of one CTA per SM takes
//   an equal run of it, whatever the lengths are, and streams it without a
//   break: 16-byte asynchronous copies run two to three half blocks ahead, over
//   the ends of sequences.  Each lane copies exactly the bytes that it later
//   reads, so no barrier stands between the copies and the arithmetic.
//   SMs do not get equal shares of the memory's rate (with equal runs the
//   fastest CTAs were done at 0.78 of the slowest's time), so the last fifth of
//   every run is cut into pieces of falling size that warps take as they come
//   free.  The pieces are fixed; who computes one changes no result.
//   Products.  S^T = K Q^T with the 64 keys as rows of m16n8k16 fragments and
//   the query rows of the group as the 8 columns, so one decoded token of 8
//   query heads fills the instruction and the keys fill the rest; O^T = V^T P^T
//   likewise.  The codes become fp16 exactly (int8 by the exponent of 1024,
//   e4m3 by the conversion instruction); the cache's order of bytes is the
//   fragments' order.  The query row is shifted by a power of two to
//   [2^14, 2^15), which is exact in fp16 down to 2^-31 of its largest element
//   (below, the error is at most 2^-39 of it).  P is rounded to fp16 at 2^15 times
//   its share of the block's largest: half a step is 2^-11 of it, 1/8 of the bf16
//   rounding of the output, as long as it is one of fp16's normal numbers, down to
//   2^-29.  A block's O^T is summed alone and added to the output's in fp32 by its
//   power of two, so a key with nearly all of a row's weight costs the other blocks
//   nothing.  In its own block, keys 20 nats below it lose bits; that counts only
//   where its V is zero and theirs is the output.  So where a block's O^T is small,
//   what fp16 left of P takes further passes over the V codes, each for the next 40
//   bits, down to fp32's end.  All sums are fp32.
//   Softmax.  The row sum's reference is a whole number of bits, m.  The output's
//   takes in the V scales' exponents as well and is kept as its distance `gap` from
//   m: that stays small (-126 to 122) whatever the scores are, where the sum of the
//   two would lose it from 2^24 on.  Every rescaling is by a power of two, and
//   blocks with very different V scales lose nothing.
//   Joining.  A piece leaves a normalised O and its (m, row sum) for a unit that
//   it shares with its neighbours, not their LSE, which for the same reason could
//   not tell the row sums of large scores apart; a second small kernel joins them
//   in the order of the keys.
//
// Measured (one GB300, in a captured graph): one token over 2M cached ones, 8 kv
// heads of 128, 629 to 637 us (4.3 GB, 6.7 to 6.8 TB/s); 64 sequences of 256 to
// 29K tokens 146.5 us (843 MB, 5.8 TB/s: while the runs stream, a block takes a warp
// 5.2K cycles; the rest is the start and the ends); 64 x 32 chosen blocks 54 us
// (270 MB); 16 sequences with up to 5 drafted tokens 62 us.
#include "kv_attention.cuh"

namespace hdp {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMeta = 8;  // blocks whose scales and first key are kept
constexpr PartCount kCount = {kWarps * (1 + kMorePieces), kWarps * (1 + kMorePieces) * 2};
// Bytes of a warp's ring of half blocks.  More in flight streams a long run
// better; less leaves the memory's queues shorter, and with them every other
// access (lists, pages, query rows), which short runs wait for.  Measured at
// 24 KB and 16 KB: one 2M-token sequence 636 and 647 us, 64 sequences 146.7 and
// 148.7, 64 x 32 chosen blocks 56.4 and 53.7.  (24 KB do not fit beside two tiles' P;
// before it had a place there, 16 sequences with up to 5 drafted tokens took 67 and
// 62 us.)
template <int NT, bool SPARSE>
constexpr int kRingBytes = NT == 1 && !SPARSE ? 24576 : 16384;
// What rounding to fp16 leaves of a block's P is at most 64 * 2^-25 times its largest
// code, 127 or 448; 2^12 times that is enough of an output to forget it.
template <int FMT>
constexpr float kEnough = FMT == HDP_CACHE_INT8 ? 1.f : 4.f;

struct Meta {
  float sk, sv;
  int key0;   // first key of the block; -1: nothing of it is seen
  int piece;  // the piece that the block belongs to
};

__device__ __forceinline__ void copy8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

// The smallest magnitude.
__device__ __forceinline__ float least_of(float a, float b, float c) {
  float r;
  asm("min.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Four codes to fp16: bytes 0, 1 and bytes 2, 3.
template <int FMT>
__device__ __forceinline__ void decode4(uint32_t x, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == HDP_CACHE_INT8) {
    const uint32_t u = x ^ 0x80808080u;  // code + 128; 0x6400 | u is 1024 + u
    const __half2 off = __half2half2(__ushort_as_half(0x6480));
    lo = h2_bits(__hsub2(as_h2(__byte_perm(u, 0x64646464u, 0x4140)), off));
    hi = h2_bits(__hsub2(as_h2(__byte_perm(u, 0x64646464u, 0x4342)), off));
  } else {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(x));
  }
}

// NaN codes (only e4m3 has them) read as zero: a masked key's V byte must not
// turn 0 * code into NaN, whatever the page holds.
template <int FMT>
__device__ __forceinline__ uint32_t without_nan(uint32_t x) {
  if constexpr (FMT == HDP_CACHE_INT8) return x;
  const uint32_t full = ((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
  return x & ~((full >> 7) * 0xffu);
}

template <int FMT>
__device__ __forceinline__ uint4 without_nan(uint4 x) {
  return make_uint4(without_nan<FMT>(x.x), without_nan<FMT>(x.y), without_nan<FMT>(x.z), without_nan<FMT>(x.w));
}

template <int NT, bool SPARSE>
struct Shared {
  unsigned char ring[kWarps][kRingBytes<NT, SPARSE>];
  SeqPlace seq[kSeqs];
  Meta meta[kWarps][kMeta];
  float4 p[kWarps][NT][4][32];  // P of a block, each lane its own
  long long pre[kThreads];  // steps before each thread's sequences
  long long warp_sum[kWarps];
};

// Raw query rows of a unit, this lane's channels.
template <int D, int NT>
__device__ __forceinline__ void fetch_rows(const AttnParams& p, int row0, int head, unsigned rr0, int nrows,
                                           uint4 (&qx)[NT][D / 32]) {
  const int lane = threadIdx.x & 31, gr = lane >> 2, tc = lane & 3;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int r = t * 8 + gr;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) qx[t][i] = make_uint4(0, 0, 0, 0);
    if (r < nrows) {
      const unsigned token = (rr0 + r) / p.g;
      const uint4* src = reinterpret_cast<const uint4*>(
          p.q + (static_cast<long long>(row0 + token) * p.hq + head * p.g + (rr0 + r - token * p.g)) * D + tc * 16);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) qx[t][i] = __ldg(src + (i >> 1) * 8 + (i & 1));
    }
  }
}

// S^T = K Q^T; key_at(i, j) is chunk j of this lane's key 8 i + gr.
template <int D, int FMT, int NT, class K>
__device__ __forceinline__ void first_product(const Rows<D, NT>& rows, float (&s)[NT][4][4], K key_at) {
#pragma unroll
  for (int i = 0; i < 4; i += kTogether) {
#pragma unroll
    for (int h = 0; h < kTogether; ++h)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[t][i + h][k] = 0.f;
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      uint4 u[kTogether], w[kTogether];
#pragma unroll
      for (int h = 0; h < kTogether; ++h) {
        u[h] = key_at(2 * (i + h), j);
        w[h] = key_at(2 * (i + h) + 1, j);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int h = 0; h < kTogether; ++h) {
          uint32_t a0, a1, a2, a3;
          decode4<FMT>(word(u[h], k), a0, a2);
          decode4<FMT>(word(w[h], k), a1, a3);
#pragma unroll
          for (int t = 0; t < NT; ++t)
            mma16816(s[t][i + h], a0, a1, a2, a3, rows.q[t][j * 4 + k][0], rows.q[t][j * 4 + k][1]);
        }
      }
    }
  }
}

// Scores to P, at most 2^15, in place; brings the sums to the new references, and f
// to the power of two (<= 1) of the block in the output.
template <int D, int NT>
__device__ __forceinline__ void softmax(const Rows<D, NT>& rows, Sums<D, NT>& sums, float sk, float sv, int key0,
                                        bool masked, float (&s)[NT][4][4], float (&f)[NT][2]) {
  const int gr = (threadIdx.x & 31) >> 2;
  const int ev = static_cast<int>((__float_as_uint(sv) >> 23) & 0xff) - 127;
  const float lsv = sv == sv ? static_cast<float>(ev) : sv;  // log2 of the V scale
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float top[2] = {-__int_as_float(0x7f800000), -__int_as_float(0x7f800000)};
    // The products are below 2^31: times a scale above one they may pass fp32's end
    // where a small q brings the score back, so the row's factor goes first then.
    const bool large = sk > 1.f;
    const float first[2] = {large ? rows.scale[t][0] : sk, large ? rows.scale[t][1] : sk};
    const float second[2] = {large ? sk : rows.scale[t][0], large ? sk : rows.scale[t][1]};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float x = s[t][i][k] * first[k & 1] * second[k & 1];
        if (masked && key0 + 16 * i + 8 * (k >> 1) + gr > rows.pos[t][k & 1]) x = -__int_as_float(0x7f800000);
        s[t][i][k] = x;
        top[k & 1] = fmaxf(top[k & 1], x);
      }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int d = 4; d < 32; d *= 2) top[k] = fmaxf(top[k], __shfl_xor_sync(0xffffffffu, top[k], d));
      const bool none = top[k] == -__int_as_float(0x7f800000);
      float c = none ? 0.f : ceilf(top[k]);
      if (fabsf(c) < kBiasMost) c -= kBias;
      const float m = sums.m[t][k], gap = sums.gap[t][k];
      const float m1 = none ? m : fmaxf(m, c);
      const float down = m - m1;
      const float gap1 = none ? gap : fmaxf(gap + down, (c - m1) + lsv);
      sums.l[t][k] *= exp2_approx(down);
      const float up = exp2_approx(down + (gap - gap1));
      if (up != 1.f) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          sums.acc[t][i][k] *= up;
          sums.acc[t][i][k + 2] *= up;
        }
      }
      sums.m[t][k] = m1;
      sums.gap[t][k] = gap1;
      const float fl = none ? 0.f : exp2_approx(c - m1);
      f[t][k] = none ? 0.f : exp2_approx((c - m1) + (lsv - gap1));
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[t][i][k] = exp2_approx(s[t][i][k] - c);
        s[t][i][k + 2] = exp2_approx(s[t][i][k + 2] - c);
        sum += s[t][i][k] + s[t][i][k + 2];
      }
      sums.l[t][k] = fmaf(sum, fl, sums.l[t][k]);
    }
  }
}

// O^T += f Y, Y = V^T P^T; value_at(i) is this lane's chunk of channel 8 i + gr, least
// the smallest |Y| of this lane's rows.
template <int D, int FMT, int NT, class V>
__device__ __forceinline__ void second_product(Sums<D, NT>& sums, const uint32_t (&pf)[NT][4][2], const float (&f)[NT][2],
                                               bool masked, float (&least)[NT][2], V value_at) {
#pragma unroll
  for (int t = 0; t < NT; ++t) least[t][0] = least[t][1] = __int_as_float(0x7f800000);
#pragma unroll
  for (int i = 0; i < D / 16; i += kTogether) {
    uint4 u[kTogether], w[kTogether];
    float y[NT][kTogether][4];
#pragma unroll
    for (int h = 0; h < kTogether; ++h) {
      u[h] = value_at(2 * (i + h));
      w[h] = value_at(2 * (i + h) + 1);
      if (masked) {
        u[h] = without_nan<FMT>(u[h]);
        w[h] = without_nan<FMT>(w[h]);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
      for (int h = 0; h < kTogether; ++h) {
        uint32_t a0, a1, a2, a3;
        decode4<FMT>(word(u[h], k), a0, a2);
        decode4<FMT>(word(w[h], k), a1, a3);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if (k == 0) mma16816_first(y[t][h], a0, a1, a2, a3, pf[t][k][0], pf[t][k][1]);
          else mma16816(y[t][h], a0, a1, a2, a3, pf[t][k][0], pf[t][k][1]);
        }
      }
    }
#pragma unroll
    for (int h = 0; h < kTogether; ++h)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          sums.acc[t][i + h][k] = fmaf(y[t][h][k], f[t][k & 1], sums.acc[t][i + h][k]);
          if (k < 2) least[t][k] = least_of(least[t][k], y[t][h][k], y[t][h][k + 2]);
        }
  }
}

template <int D, int FMT, int NT, bool SPARSE>
__global__ void __launch_bounds__(kThreads, 1) k_cache_attention(const AttnParams p) {
  constexpr int kHalf = kBlock * D;               // bytes of a block's K or V codes of one head
  constexpr int kSlots = kRingBytes<NT, SPARSE> / kHalf;  // half blocks in flight
  constexpr int kKeyChunks = D / 64;              // 16-byte chunks that a lane has of a key
  constexpr int kMt = D / 16;
  constexpr int kRows = 8 * NT;
  using Cur = Cursor<SPARSE, NT>;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  auto& sm = *reinterpret_cast<Shared<NT, SPARSE>*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gr = lane >> 2, tc = lane & 3;  // fragment row group and column pair

  // ---- the flat order: total steps, and where this warp starts
  long long total;
  const int per_thread = (p.c.num_seqs + kThreads - 1) / kThreads;
  const int per_row = SPARSE ? p.c.hkv * Cur::tiles_of(1, p.g) : 0;
  if constexpr (SPARSE) {
    total = static_cast<long long>(p.c.rows) * per_row * p.count;
  } else {
    long long mine = 0;
    for (int i = 0; i < per_thread; ++i) {
      const int s = threadIdx.x * per_thread + i;
      if (s < p.c.num_seqs) {
        const SeqPlace at = seq_place(p.c, s);
        if (s < kSeqs) sm.seq[s] = at;
        mine += Cur::cost(p, at);
      }
    }
    long long run = mine;
#pragma unroll
    for (int s = 1; s < 32; s *= 2) {
      const long long up = __shfl_up_sync(0xffffffffu, run, s);
      if (lane >= s) run += up;
    }
    if (lane == 31) sm.warp_sum[warp] = run;
    __syncthreads();
    long long before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sm.warp_sum[w];
      total += sm.warp_sum[w];
    }
    sm.pre[threadIdx.x] = before + run - mine;
  }
  __syncthreads();
  const Cut cut(total, gridDim.x, kWarps, p.dynamic);
  const int used = cut.used(gridDim.x);
  if (!p.dynamic && blockIdx.x == 0 && threadIdx.x == 0) p.head[2] = cut.workers;
  if (warp >= used) return;
  const int run = blockIdx.x * used + warp;
  if (!p.dynamic && lane == 0) p.open[run].parts = 0;

  // Puts a cursor on a step of the flat order.
  auto locate = [&](Cur& cur, long long x) {
    if constexpr (SPARSE) {
      const long long row_cost = static_cast<long long>(per_row) * p.count;
      const int row = static_cast<int>(x / row_cost);
      const long long off = x - row * row_cost;
      const int head = static_cast<int>(off / (static_cast<long long>(p.count) * (per_row / p.c.hkv)));
      const int at = min(static_cast<int>(off % p.count) + lane, p.count - 1);  // of the list that comes next
      asm volatile("prefetch.global.L1 [%0];" ::"l"(p.blocks + (static_cast<long long>(row) * p.c.hkv + head) * p.count + at));
      cur.enter(p, sm.seq, row);
      cur.skip(off);
    } else {
      const int slice = find_last(kThreads, x, [&](int s) { return sm.pre[s]; });
      long long at = sm.pre[slice];
      int i = slice * per_thread;
      for (long long c; x - at >= (c = Cur::cost(p, Cur::place(p, sm.seq, i))) && i + 1 < p.c.num_seqs; ++i) at += c;
      cur.enter(p, sm.seq, i);
      cur.skip(x - at);
    }
  };

  long long start, stop;
  cut.range(run, 0, start, stop);
  if (start < total) {
    Cur cc, lc;  // of the arithmetic; of the copies, which run ahead
    locate(lc, start);
    cc = lc;
    int piece = run * cut.pieces;  // of the copies
    long long to_load = stop - start;
    int loaded = 0, done = 0;      // blocks
    int ticket = 0;                // lane 0: the next piece to take
    bool asked = false, more_pieces = p.dynamic;
    auto ask = [&]() {
      asm volatile("griddepcontrol.wait;" ::: "memory");  // the counters are zero
      if (lane == 0) ticket = atomicAdd(p.head + 1, 1);
      asked = true;
    };
    int half = 0;                 // 0: K of lc's block next, 1: V
    int load_slot = 0, load_meta = 0;
    int ids = -1, ids_at = -1;    // 32 blocks' pages (dense) or blocks and pages (sparse) of lc's unit, one a lane
    int ids_page = -1;
    int next_page = 0, next_of = -1;  // dense: a page of sequence next_of's first blocks, asked for early
    const unsigned char* cur_v = nullptr;  // V of the block whose K went last
    const uint32_t ring = smem_addr(sm.ring[warp]) + lane * 16;

    auto issue = [&]() {
      while (to_load == 0 && more_pieces) {
        if (!asked) ask();
        asked = false;
        const int j = __shfl_sync(0xffffffffu, ticket, 0);
        const int k = 1 + j / cut.workers, w = j - (k - 1) * cut.workers;
        more_pieces = k < cut.pieces;
        if (!more_pieces) break;
        long long a, z;
        cut.range(w, k, a, z);
        if (a >= z) continue;
        locate(lc, a);
        to_load = z - a;
        piece = w * cut.pieces + k;
        ids_at = -1;
      }
      if (to_load > 0) {
        if (half == 0) {
          ++loaded;
          if (ids_at != (lc.blk & ~31)) {  // a new list, or the next 32 blocks
            const int last = lc.last_pos(p.g);
            ids_at = lc.blk & ~31;
            const int b = ids_at + lane;
            ids = ids_page = -1;
            if constexpr (SPARSE) {
              if (b < lc.nb && lc.seq >= 0) {
                const int32_t* list = p.blocks + (static_cast<long long>(lc.s.row0) * p.c.hkv + lc.head) * p.count;
                const int x = __ldg(list + b), before = b ? __ldg(list + b - 1) : -1;
                if (x > before && x >= 0 && x <= last / kBlock && last >= 0) {
                  ids = x;
                  ids_page = page_of(p.c, lc.seq, x);
                }
              }
            } else {
              const bool early = next_of == lc.seq && ids_at == 0;
              if (b < lc.nb && b <= last / kBlock && last >= 0) {
                ids = b;
                ids_page = early ? next_page : __ldg(p.c.table + static_cast<long long>(lc.seq) * p.c.max_pages + b);
                if (ids_page < 0 || ids_page >= p.c.num_pages) {
                  report_table(p.c);
                  ids_page = -1;
                }
              }
              next_of = -1;
            }
          }
          if (!SPARSE && next_of < 0 && lc.last_unit(p)) {
            next_of = lc.next_seq(p, sm.seq);
            if (next_of < p.c.num_seqs && lane < p.c.max_pages)
              next_page = __ldg(p.c.table + static_cast<long long>(next_of) * p.c.max_pages + lane);
          }
          const int b = __shfl_sync(0xffffffffu, ids, lc.blk & 31);
          const int page = __shfl_sync(0xffffffffu, ids_page, lc.blk & 31);
          const bool seen = b >= 0 && page >= 0;
          Meta* meta = &sm.meta[warp][load_meta];
          if (lane == 0) meta->piece = piece;
          if (seen) {
            const size_t ph = static_cast<size_t>(page) * p.c.hkv + lc.head;
            if (lane == 0) {
              copy8(smem_addr(meta), p.c.scales + 2 * ph);
              meta->key0 = b * kBlock;
            }
            const unsigned char* kb = p.c.k + ph * kHalf + gr * D + tc * 16;
            const uint32_t dst = ring + load_slot * kHalf;
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
              for (int j = 0; j < kKeyChunks; ++j) copy16(dst + (i * kKeyChunks + j) * 512, kb + i * 8 * D + j * 64);
            cur_v = p.c.v + ph * kHalf + lane * 16;
          } else {
            if (lane == 0) meta->key0 = -1;
            cur_v = nullptr;
          }
        } else {
          if (cur_v) {
            const uint32_t dst = ring + load_slot * kHalf;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) copy16(dst + i * 512, cur_v + i * 512);
          }
          load_meta = (load_meta + 1) % kMeta;
          --to_load;
          if (to_load == 1 && more_pieces) ask();  // not earlier: a slow warp must not sit on a piece
          if (++lc.blk == lc.nb && to_load > 0) {
            // heads of a sequence share its pages: a list of up to 32 serves them all (its
            // visible blocks are those of the sequence's last rows)
            const bool same = !SPARSE && lc.nb <= 32 && lc.tiles == 1 && !lc.last_unit(p);
            lc.next_unit(p, sm.seq);
            if (!same) ids_at = -1;
          }
        }
        half ^= 1;
        load_slot = load_slot + 1 == kSlots ? 0 : load_slot + 1;
      }
      copies_commit();
    };

    int ahead = kSlots;  // half steps that the copies go in front at first

    int slot = 0, meta_at = 0, at_piece = run * cut.pieces;  // (the copies may be in a later piece already)
    long long at = start;
    uint4 qx[NT][kMt / 2];  // raw query rows of cc's unit, this lane's channels
    auto fetch_q = [&]() {  // a row of no sequence is not read
      fetch_rows<D, NT>(p, cc.s.row0, cc.head, cc.rr0(), !SPARSE || cc.seq >= 0 ? cc.nrows(p.g) : 0, qx);
    };
    fetch_q();
    while (true) {
      // ---- one unit, or the part of it that the piece has
      const bool begins = cc.blk == 0;
      const int steps = static_cast<int>(min(static_cast<long long>(cc.nb - cc.blk), stop - at));
      const bool ends = cc.blk + steps == cc.nb;
      const int nrows = cc.nrows(p.g), rr0 = cc.rr0(), row0 = cc.s.row0, head = cc.head;
      const bool live = !SPARSE || cc.seq >= 0;

      const int low_pos = cc.first_pos(p.g);
      const Rows<D, NT> rows(p, qx, cc.s.p0, rr0, nrows);
      Sums<D, NT> sums;
      sums.clear();

      // Half a step is a block's scores or its output; then the next half block is asked
      // for.  That is a page of code with a place of its own, once in the kernel: the
      // loop is bound by the fetch of its instructions as much as by what they do.  Twice
      // in the loop and once in front of it, unrolled, 64 sequences took 149.4 us against
      // 146.5, 16 drafts 66.3 against 61.8, four short documents 11.3 against 9.9.
      const Probabilities<NT> prob = {sm.p[warp]};
      float f[NT][2];
      bool seen = false, masked = false;
#pragma unroll 1
      for (int half_step = -ahead; half_step < 2 * steps; ++half_step) {
        if (half_step >= 0) {
          copies_wait<kSlots - 1>();
          if (half_step % 2 == 0) {
            __syncwarp();
            const Meta meta = sm.meta[warp][meta_at];
            meta_at = (meta_at + 1) % kMeta;
            seen = meta.key0 >= 0;
            masked = meta.key0 + kBlock - 1 > low_pos;  // some row does not see the whole block
            if (seen) {
              const uint4* kx = reinterpret_cast<const uint4*>(sm.ring[warp] + slot * kHalf) + lane;
              float s[NT][4][4];
              first_product<D, FMT, NT>(rows, s, [&](int i, int j) { return kx[(i * kKeyChunks + j) * 32]; });
              softmax<D, NT>(rows, sums, meta.sk, meta.sv, meta.key0, masked, s, f);
              prob.put(s);
            }
          } else if (seen) {
            const uint4* vx = reinterpret_cast<const uint4*>(sm.ring[warp] + slot * kHalf) + lane;
            bool sure = false;  // that further passes are needed
            while (true) {
              uint32_t pf[NT][4][2];
              float least[NT][2];
              prob.get(pf);
              second_product<D, FMT, NT>(sums, pf, f, masked, least, [&](int i) { return vx[i * 32]; });
              // Is an output so small that what fp16 leaves of P could count?
#pragma unroll
              for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                  sure |= t * 8 + 2 * tc + k < nrows && f[t][k] != 0.f && !(least[t][k] >= kEnough<FMT>);
              if (!__any_sync(0xffffffffu, sure) || !__any_sync(0xffffffffu, prob.more())) break;
              sure = true;
              prob.next();  // four times at most
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                f[t][0] *= 1.f / kNextPass;
                f[t][1] *= 1.f / kNextPass;
              }
            }
          }
          slot = slot + 1 == kSlots ? 0 : slot + 1;
        }
        issue();
      }
      ahead = 0;
      at += steps;
      done += steps;
      const int rest = cc.nb - cc.blk - steps;  // steps of the unit behind the piece
      const int this_piece = at_piece;
      const long long this_at = at;

      // ---- the next unit's query rows are asked for before this one is written
      bool more = true;
      if (at < stop) {
        cc.next_unit(p, sm.seq);
      } else {
        __syncwarp();
        more = done != loaded;
        if (more) {  // the piece that the copies went on to
          at_piece = sm.meta[warp][meta_at].piece;
          const int w = at_piece / cut.pieces;
          cut.range(w, at_piece - w * cut.pieces, at, stop);
          locate(cc, at);
        }
      }
      if (more) fetch_q();

      // ---- the unit's part is done: out, or into a partial
      const bool whole = begins && ends;
      const size_t part_at = (static_cast<size_t>(this_piece) * 2 + (begins ? 1 : 0)) * kRows;
      if (live) write_part<D, NT>(p, sums, head, row0, rr0, nrows, whole, p.part + part_at * D, p.part_sum + part_at);
      if (begins && !ends && live && lane == 0) {
        Open o = {};
        o.first = this_piece;
        o.parts = cut.piece_of(this_at + rest - 1) - this_piece + 1;
        o.row0 = row0;
        o.head = head;
        o.nrows = nrows;
        o.rr0 = rr0;
        p.open[p.dynamic ? atomicAdd(p.head, 1) : this_piece] = o;
      }
      if (!more) break;
    }
    copies_wait<0>();
  }
  // Even a call without work ends after the kernels in front of it: what comes
  // next in the stream (another thread's kernel, perhaps) waits for this one only.
  if (p.dynamic) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Zeroes the counters while the attention's CTAs are starting.
__global__ void k_cache_attention_start(const AttnParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x < 2) p.head[threadIdx.x] = 0;
}

// Joins the parts of units that several pieces share.  A CTA has every n-th
// open unit (n CTAs), and its warps take rows of up to kAlone parts in turn.  A
// 2M-token sequence leaves 600 parts for each of its few heads: the rows of such
// units are dealt to all CTAs, whose warps then share a row's parts (that call:
// 646 us with each unit's CTA joining its rows itself, 636 us so).
template <int D, int NT>
__global__ void __launch_bounds__(kJoinWarps * 32, 1) k_cache_attention_join(const AttnParams p, int pieces) {
  constexpr int kRows = 8 * NT;
  constexpr int kAlone = 48;  // most parts of a row that a warp joins alone
  constexpr int kFew = 256;   // most parts of rows that a CTA joins at once
  // Two units share at most one piece, so n units of more than kAlone parts take
  // more than n (kAlone - 1) pieces; of the others a CTA has one for each
  // gridDim.x pieces.  The host keeps both below this.
  constexpr int kMostShared = 192;
  constexpr int V = D / 32;
  __shared__ __align__(16) float s_x[kJoinWarps][D];
  __shared__ float2 s_sum[kJoinWarps];
  __shared__ int4 s_shared[kMostShared][2], s_own[kMostShared][2];  // shared units, and this CTA's others
  __shared__ int s_n, s_own_n;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) s_n = s_own_n = 0;
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int made = min(pieces, __ldcg(p.head + (p.dynamic ? 0 : 2)));
  auto at = [&](int e, int k, int r) { return (static_cast<size_t>(e + k) * 2 + (k == 0 ? 1 : 0)) * kRows + r; };

  // This CTA's open units, and all shared ones where the units are listed as they
  // came; where each piece has an entry (1,216 of them, which 152 CTAs reading all
  // would take 4 us for), a CTA keeps to its own.
  const int stride = p.dynamic ? 1 : gridDim.x, origin = p.dynamic ? 0 : blockIdx.x;
  constexpr int kScan = 2;
  for (int base = 0; base == 0 || origin + base * stride < made; base += kScan * kJoinWarps * 32) {
    int4 a[kScan], b[kScan];  // the first loads do not wait for the units' number
#pragma unroll
    for (int u = 0; u < kScan; ++u) {
      const int i = origin + (base + u * kJoinWarps * 32 + static_cast<int>(threadIdx.x)) * stride;
      a[u] = b[u] = make_int4(0, 0, 0, 0);
      if (i < pieces) {
        a[u] = __ldcg(reinterpret_cast<const int4*>(p.open + i));
        b[u] = __ldcg(reinterpret_cast<const int4*>(p.open + i) + 1);
      }
    }
#pragma unroll
    for (int u = 0; u < kScan; ++u) {
      const int i = origin + (base + u * kJoinWarps * 32 + static_cast<int>(threadIdx.x)) * stride;
      if (i >= made || a[u].x == 0) continue;
      const bool shared = a[u].x > kAlone;
      if (!shared && i % gridDim.x != blockIdx.x) continue;
      const int n = atomicAdd(shared ? &s_n : &s_own_n, 1);
      if (n >= kMostShared) continue;  // cannot be (see there)
      int4* to = shared ? s_shared[n] : s_own[n];
      to[0] = a[u];
      to[1] = b[u];
    }
  }
  __syncthreads();

  const int own = min(s_own_n, kMostShared);
  int nth = 0;
  for (int q = 0; q < own; ++q) {
    const int4 a = s_own[q][0], b = s_own[q][1];
    for (int r = 0; r < b.x; ++r) {
      if (nth++ % kJoinWarps != warp) continue;
      float x[V];
      const float2 sum = join_row<D>(
          a.x, lane, x, [&](int k) { return __ldcg(p.part_sum + at(a.y, k, r)); },
          [&](int k) { return p.part + at(a.y, k, r) * D; });
      write_o<D>(p, a.z, a.w, b.y + r, x, lse_of(sum.x, sum.y), lane);
    }
  }

  const int n = min(s_n, kMostShared);
  for (int q = 0; q < n; ++q) {
    const int4 a = s_shared[q][0], b = s_shared[q][1];
    const int m = a.x, e = a.y, nrows = b.x;
    int rank = 0;  // of its first piece: the same in every CTA, whose lists differ in order
    for (int z = lane; z < n; z += 32) rank += s_shared[z][0].y < e;
    rank = __reduce_add_sync(0xffffffffu, rank);
    // rows that a CTA joins at once, and warps for each
    const int rows = m > kFew ? 1 : min(kJoinWarps, 1 << (32 - __clz(nrows - 1)) % 32), each = kJoinWarps / rows;
    const int nr = warp / each, run = warp - nr * each;
    for (int r0 = 0; r0 < nrows; r0 += rows) {
      if (p.dynamic && (rank * nrows + r0) % static_cast<int>(gridDim.x) != static_cast<int>(blockIdx.x)) continue;
      const int r = r0 + nr;
      float x[V];
      if (r < nrows) {
        const int k0 = m * run / each, k1 = m * (run + 1) / each;
        const float2 part = join_row<D>(
            k1 - k0, lane, x, [&](int k) { return __ldcg(p.part_sum + at(e, k0 + k, r)); },
            [&](int k) { return p.part + at(e, k0 + k, r) * D; });
#pragma unroll
        for (int v = 0; v < V; ++v) s_x[warp][lane * V + v] = x[v];
        if (lane == 0) s_sum[warp] = part;
      }
      __syncthreads();
      if (r < nrows && run == 0) {
        const float2 sum = join_row<D>(each, lane, x, [&](int k) { return s_sum[warp + k]; },
                                       [&](int k) { return &s_x[warp + k][0]; });
        write_o<D>(p, a.z, a.w, b.y + r, x, lse_of(sum.x, sum.y), lane);
      }
      __syncthreads();  // the sums have been read
    }
  }
}

template <int D, int FMT, int NT, bool SPARSE>
hdp_status_t launch8(const AttnParams& p, int device, int ctas, cudaStream_t st) {
  static std::atomic<bool> ready[kDevices];
  constexpr int smem = sizeof(Shared<NT, SPARSE>);
  static_assert(smem <= 232448, "shared memory of a CTA");
  const auto kernel = k_cache_attention<D, FMT, NT, SPARSE>;
  const int pieces = ctas * kWarps * (p.dynamic ? 1 + kMorePieces : 1);
  if (pieces > 47 * 192)  // k_cache_attention_join's lists; a device of over 188 SMs
    return fail(HDP_ERR_UNSUPPORTED, "hdp_cache_attention: too many SMs");
  hdp_status_t r = allow(kernel, smem, ready, device);
  if (r != HDP_OK) return r;
  if (p.dynamic) {
    k_cache_attention_start<<<1, 32, 0, st>>>(p);
    note_launch();
    HDP_CUDA_TRY(cudaGetLastError());
    r = launch_early(kernel, dim3(ctas), kThreads, smem, st, p);
  } else {
    r = launch_attention(kernel, ctas, kThreads, smem, p, st);
  }
  if (r != HDP_OK) return r;
  return launch_early(k_cache_attention_join<D, NT>, dim3(ctas), kJoinWarps * 32, 0, st, p, pieces);
}

template <int D, int FMT>
hdp_status_t launch_for(const AttnParams& p, int nt, int device, int ctas, cudaStream_t st) {
  if (p.blocks) return nt == 1 ? launch8<D, FMT, 1, true>(p, device, ctas, st) : launch8<D, FMT, 2, true>(p, device, ctas, st);
  return nt == 1 ? launch8<D, FMT, 1, false>(p, device, ctas, st) : launch8<D, FMT, 2, false>(p, device, ctas, st);
}

}  // namespace
}  // namespace hdp

using namespace hdp;

extern "C" hdp_status_t hdp_cache_attention_workspace_bytes(const hdp_cache_t* cache, int32_t hq, size_t* bytes) {
  if (!cache || !bytes) return fail(HDP_ERR_INVALID_ARGUMENT, "hdp_cache_attention_workspace_bytes: NULL argument");
  return workspace_bytes_of("hdp_cache_attention_workspace_bytes", kCount, cache->hkv, cache->d, hq, bytes);
}

extern "C" hdp_status_t hdp_cache_attention(const hdp_cache_t* cache, const int32_t* cu, int64_t rows, const void* q,
                                            int32_t hq, float scale, const int32_t* blocks, int32_t count,
                                            void* workspace, size_t workspace_bytes, void* o, float* lse,
                                            void* stream) {
  AttnParams p = {};
  const hdp_status_t r = cache_view("hdp_cache_attention", cache, cu, rows, &p.c);
  if (r != HDP_OK) return r;
  const bool i8 = cache->format == HDP_CACHE_INT8, wide = cache->d == 128;
  return attend("hdp_cache_attention", kCount, kWarps, p, cache->d, rows, q, hq, scale, blocks, count, workspace, workspace_bytes, o, lse,
                stream, [=](const AttnParams& a, int nt, int device, int, int ctas, cudaStream_t st) {
                  if (wide)
                    return i8 ? launch_for<128, HDP_CACHE_INT8>(a, nt, device, ctas, st)
                              : launch_for<128, HDP_CACHE_E4M3>(a, nt, device, ctas, st);
                  return i8 ? launch_for<64, HDP_CACHE_INT8>(a, nt, device, ctas, st)
                            : launch_for<64, HDP_CACHE_E4M3>(a, nt, device, ctas, st);
                });
}
