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
#include <cuda_fp16.h>

#include <atomic>
#include <string>

#include "kv_cache.cuh"

namespace hdp {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
// Bytes of a warp's ring of half blocks.  More in flight streams a long run
// better; less leaves the memory's queues shorter, and with them every other
// access (lists, pages, query rows), which short runs wait for.  Measured at
// 24 KB and 16 KB: one 2M-token sequence 636 and 647 us, 64 sequences 146.7 and
// 148.7, 64 x 32 chosen blocks 56.4 and 53.7.  (24 KB do not fit beside two tiles' P;
// before it had a place there, 16 sequences with up to 5 drafted tokens took 67 and
// 62 us.)
template <int NT, bool SPARSE>
constexpr int kRingBytes = NT == 1 && !SPARSE ? 24576 : 16384;
constexpr int kMeta = 8;           // blocks whose scales and first key are kept
constexpr float kLow = -3.402823466e38f;  // reference exponent before the first key: below every finite score
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kBias = 15.f;                  // P is at most 2^15, in fp16
constexpr float kBiasMost = 1048576.f;         // references above it are not biased: far below 2^24, so exactly
constexpr float kNormal = 6.103515625e-05f;    // 2^-14, fp16's smallest normal number
constexpr float kNextPass = 1099511627776.f;   // 2^40: what rounding to fp16 leaves below kNormal, 2^-25, to 2^15
// What rounding to fp16 leaves of a block's P is at most 64 * 2^-25 times its largest
// code, 127 or 448; 2^12 times that is enough of an output to forget it.
template <int FMT>
constexpr float kEnough = FMT == HDP_CACHE_INT8 ? 1.f : 4.f;

struct Meta {
  float sk, sv;
  int key0;   // first key of the block; -1: nothing of it is seen
  int piece;  // the piece that the block belongs to
};

// A unit that several pieces share, for the kernel that joins them.
struct __align__(16) Open {
  int parts, first, row0, head;  // parts: pieces first, first + 1, ...; 0: no unit
  int nrows, rr0, pad[2];
};

struct AttnParams {
  CacheView c;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  const int32_t* blocks;
  int count, hq, g;
  float scale_log2;
  bool dynamic;      // the ends of the runs are handed out through the counter
  float* part;       // [pieces][2][rows of a tile][d]: of a unit begun before the piece, and of one begun in it
  float2* part_sum;  // [pieces][2][rows of a tile]: m, sum of 2^(score - m)
  Open* open;        // [pieces]: one for each piece, or, with a counter, as they come
  int* head;         // [0] entries of open (dynamic), [1] next ticket, [2] entries of open (static)
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The smallest magnitude.
__device__ __forceinline__ float least_of(float a, float b, float c) {
  float r;
  asm("min.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same without a sum to add to.
__device__ __forceinline__ void mma16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ uint32_t h2_bits(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }
__device__ __forceinline__ __half2 as_h2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }

// What rounding x, below fp16's normal numbers, to fp16 leaves of it, for the next pass; 0 for normal ones.
__device__ __forceinline__ float left_by_fp16(float x) {
  return fabsf(x) < kNormal ? (x - __half2float(__float2half_rn(x))) * kNextPass : 0.f;
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

constexpr int kSeqs = 512;  // sequences whose places are kept in shared memory

template <int FMT>
__device__ __forceinline__ uint4 without_nan(uint4 x) {
  return make_uint4(without_nan<FMT>(x.x), without_nan<FMT>(x.y), without_nan<FMT>(x.z), without_nan<FMT>(x.w));
}
__device__ __forceinline__ uint32_t word(const uint4& x, int k) { return k == 0 ? x.x : k == 1 ? x.y : k == 2 ? x.z : x.w; }

// A sequence's rows in the call, its tokens, and the position of its first row.
struct SeqPlace {
  int row0, n, len, p0;
};

__device__ __forceinline__ SeqPlace seq_place(const CacheView& c, int i) {
  SeqPlace s;
  seq_rows(c, i, s.row0, s.n);
  const long long len = seq_len(c, i);
  s.len = static_cast<int>(len);
  s.p0 = static_cast<int>(max(first_position(c, i, len), -2147483647LL));
  return s;
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

// A place in the flat order.  A unit is (sequence or row, kv head, tile of
// query rows); a step is one block of it.
template <bool SPARSE, int NT>
struct Cursor {
  int seq, head, tile, tiles, nb, blk;
  SeqPlace s;

  __device__ __forceinline__ static int tiles_of(int n, int g) { return static_cast<int>((n * g + 8u * NT - 1) / (8u * NT)); }
  __device__ __forceinline__ static int blocks_of(const SeqPlace& s) { return max(1, static_cast<int>((s.len + (kBlock - 1u)) / kBlock)); }
  __device__ __forceinline__ static SeqPlace place(const AttnParams& p, const SeqPlace* kept, int i) {
    return i < kSeqs ? kept[i] : seq_place(p.c, i);
  }
  // Steps of all units of a sequence.
  __device__ __forceinline__ static long long cost(const AttnParams& p, const SeqPlace& s) {
    return s.n ? static_cast<long long>(blocks_of(s)) * tiles_of(s.n, p.g) * p.c.hkv : 0;
  }
  __device__ __forceinline__ void enter(const AttnParams& p, const SeqPlace* kept, int i) {
    head = tile = blk = 0;
    if constexpr (SPARSE) {
      nb = p.count;
      seq = seq_of_row(p.c, i);
      s.len = s.p0 = 0;
      if (seq >= 0) {
        s = seq_place(p.c, seq);
        s.p0 += i - s.row0;
      }
      s.row0 = i;
      s.n = 1;
    } else {
      seq = i;
      s = place(p, kept, i);
      nb = blocks_of(s);
    }
    tiles = tiles_of(s.n, p.g);
  }
  // The sequence after this one that has rows.
  __device__ __forceinline__ int next_seq(const AttnParams& p, const SeqPlace* kept) const {
    int i = seq + 1;
    while (i < p.c.num_seqs && place(p, kept, i).n == 0) ++i;
    return i;
  }
  __device__ __forceinline__ void next_unit(const AttnParams& p, const SeqPlace* kept) {
    blk = 0;
    if (++tile < tiles) return;
    tile = 0;
    if (++head < p.c.hkv) return;
    const int i = SPARSE ? s.row0 + 1 : next_seq(p, kept);
    if (i < (SPARSE ? p.c.rows : p.c.num_seqs)) enter(p, kept, i);
  }
  // Skips `off` steps from the sequence's first.
  __device__ __forceinline__ void skip(long long off) {
    const long long unit = off / nb;
    blk = static_cast<int>(off - unit * nb);
    head = static_cast<int>(unit / tiles);
    tile = static_cast<int>(unit - static_cast<long long>(head) * tiles);
  }
  __device__ __forceinline__ bool last_unit(const AttnParams& p) const { return tile + 1 == tiles && head + 1 == p.c.hkv; }
  __device__ __forceinline__ int rr0() const { return tile * (8 * NT); }
  __device__ __forceinline__ int nrows(int g) const { return min(8 * NT, s.n * g - rr0()); }
  // Positions of the tile's first and last row.
  __device__ __forceinline__ int first_pos(int g) const { return s.p0 + static_cast<int>(static_cast<unsigned>(rr0()) / g); }
  __device__ __forceinline__ int last_pos(int g) const {
    return s.p0 + static_cast<int>((rr0() + nrows(g) - 1u) / g);
  }
};

template <int D>
__device__ __forceinline__ void write_o(const AttnParams& p, int row0, int head, unsigned rr, const float* x, float lse,
                                        int lane) {
  const unsigned token = rr / p.g;
  const long long t = row0 + token;
  const int h = head * p.g + static_cast<int>(rr - token * p.g);
  __nv_bfloat16* out = p.o + (t * p.hq + h) * D;
  if constexpr (D == 128) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    *reinterpret_cast<uint2*>(out + lane * 4) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]);
    *reinterpret_cast<uint32_t*>(out + lane * 2) = *reinterpret_cast<const uint32_t*>(&a);
  }
  if (lane == 0) p.lse[static_cast<long long>(h) * p.c.rows + t] = lse;
}

// Joins `m` normalised partials of one row in their order: with (r, l) = sum_at(k),
// x = sum 2^(r_k - R) l_k o_k / L, R = max r_k, L = sum 2^(r_k - R) l_k.  Returns (R, L).
template <int D, class S, class O>
__device__ __forceinline__ float2 join_row(int m, int lane, float (&x)[D / 32], S sum_at, O o_at) {
  constexpr int V = D / 32;
  constexpr int kAhead = 8;  // partial rows in flight (16: a spill, 64 x 32 chosen blocks 54.3 us against 53.7)
  float top = kLow, sum = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = 0.f;
  for (int base = 0; base < m; base += 32) {
    const int here = min(32, m - base);
    const float2 l = lane < here ? sum_at(base + lane) : make_float2(kLow, 0.f);
    float t = l.x;
#pragma unroll
    for (int s = 16; s; s >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, s));
    t = fmaxf(t, top);
    float w = l.y * exp2_approx(l.x - t), all = w;
#pragma unroll
    for (int s = 16; s; s >>= 1) all += __shfl_xor_sync(0xffffffffu, all, s);
    const float old = sum * exp2_approx(top - t);
    top = t;
    sum = old + all;
    // x stays normalised, so it is no larger than the largest V
    const float inv = sum == 0.f ? 0.f : 1.f / sum;  // no key so far: o = 0
    w *= inv;
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] *= old * inv;
    for (int k = 0; k < here; k += kAhead) {
      float y[kAhead][V];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {  // past the end: the last row again, with weight 0
        const float* o = o_at(base + min(k + u, here - 1)) + lane * V;
        if constexpr (V == 4) {
          const float4 z = *reinterpret_cast<const float4*>(o);
          y[u][0] = z.x;
          y[u][1] = z.y;
          y[u][2] = z.z;
          y[u][3] = z.w;
        } else {
          const float2 z = *reinterpret_cast<const float2*>(o);
          y[u][0] = z.x;
          y[u][1] = z.y;
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const float f = __shfl_sync(0xffffffffu, w, (k + u) & 31);
        const float g = k + u < here ? f : 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = k + u < here ? fmaf(g, y[u][i], x[i]) : x[i];
      }
    }
  }
  return make_float2(top, sum);
}

// Natural logarithm of sum 2^m; the bias of most references is taken out first,
// so that a single key's LSE is its score.
__device__ __forceinline__ float lse_of(float m, float sum) {
  return sum == 0.f ? -__int_as_float(0x7f800000) : ((m + kBias) + log2f(sum * (1.f / 32768.f))) * kLn2;
}

// How the flat order of `total` steps is cut.  `used` warps of each CTA have a
// run of `per` steps each; while there are fewer steps than warps, the steps
// are spread over the CTAs first.  A run is one piece, or, where pieces are
// handed out, a first piece of four fifths and up to kMorePieces more of half
// of the rest each, but not below kLeast steps (a piece costs its warp about a
// step: its query rows, its partial).  Pieces are numbered in the flat order.
constexpr int kMorePieces = 5;
constexpr int kLeast = 4;
struct Cut {
  long long total, per, tail;
  int workers, pieces;  // warps with a run, pieces of a run
  __device__ __forceinline__ Cut(long long steps, int ctas, bool dynamic) : total(steps) {
    const long long each = (total + ctas - 1) / ctas;
    const int used = static_cast<int>(min(static_cast<long long>(kWarps), max(1LL, each)));
    workers = ctas * used;
    per = max(1LL, (total + workers - 1) / workers);
    tail = dynamic && per >= 5 * kLeast ? per / 5 : 0;
    pieces = 1;
    for (long long left = tail; left > 0 && pieces <= kMorePieces; ++pieces) left -= size_of(left, pieces);
  }
  __device__ __forceinline__ int used(int ctas) const { return workers / ctas; }
  // Size of piece k >= 1 of a run when `left` steps of the tail are left.
  __device__ __forceinline__ static long long size_of(long long left, int k) {
    return k == kMorePieces || left < 2 * kLeast ? left : (left + 1) / 2;
  }
  // Steps [start, stop) of piece k of run w.
  __device__ __forceinline__ void range(int w, int k, long long& start, long long& stop) const {
    long long a = 0, size = per - tail, left = tail;
    for (int i = 1; i <= k; ++i) {
      a += size;
      size = size_of(left, i);
      left -= size;
    }
    start = w * per + a;
    stop = min(total, start + size);
  }
  // The piece that step x lies in.
  __device__ __forceinline__ int piece_of(long long x) const {
    const long long w = x / per;
    long long off = x - w * per - (per - tail), left = tail;
    int k = 0;
    while (off >= 0 && k + 1 < pieces) {
      ++k;
      const long long size = size_of(left, k);
      off -= size;
      left -= size;
    }
    return static_cast<int>(w) * pieces + k;
  }
};

// The arithmetic of one block of 64 keys for a tile of 8 NT query rows; lane (gr, tc)
// has keys 8 i + gr, i = 0..7, of rows 8 t + 2 tc and 8 t + 2 tc + 1.

constexpr int kTogether = 2;  // 16-row tiles whose chains of products are interleaved

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

template <int D, int NT>
struct Rows {
  static constexpr int kMt = D / 16;
  uint32_t q[NT][kMt][2];
  float scale[NT][2];  // scale * log2(e) * 2^(shift) of rows 2 tc and 2 tc + 1
  int pos[NT][2];      // their positions

  __device__ __forceinline__ Rows(const AttnParams& p, const uint4 (&qx)[NT][D / 32], int p0, unsigned rr0, int nrows) {
    const int tc = threadIdx.x & 3;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < kMt / 2; ++i)
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(qx[t][i].x & 0x7fff7fffu, qx[t][i].y & 0x7fff7fffu),
                                     __vmaxu2(qx[t][i].z & 0x7fff7fffu, qx[t][i].w & 0x7fff7fffu)));
      top = max(top & 0xffffu, top >> 16);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // the largest element's exponent goes to 14; infinities and NaN stay what they are
      const int e = min(max(static_cast<int>(top >> 7) - 127, -112), 127) - 14;
      const float down = pow2i(-e);
#pragma unroll
      for (int i = 0; i < kMt / 2; ++i) {
        const uint32_t w[4] = {qx[t][i].x, qx[t][i].y, qx[t][i].z, qx[t][i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const __half2 y = __floats2half2_rn(__uint_as_float(w[k] << 16) * down, __uint_as_float(w[k] & 0xffff0000u) * down);
          q[t][i * 2 + (k >> 1)][k & 1] = h2_bits(y);
        }
      }
      const float s = p.scale_log2 * pow2i(e);
      scale[t][0] = __shfl_sync(0xffffffffu, s, tc * 8);
      scale[t][1] = __shfl_sync(0xffffffffu, s, tc * 8 + 4);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const unsigned rc = rr0 + min(t * 8 + 2 * tc + k, nrows - 1);
        pos[t][k] = max(-1, p0 + static_cast<int>(rc / p.g));
      }
    }
  }
};

// What a warp keeps of a unit between blocks.
template <int D, int NT>
struct Sums {
  static constexpr int kMt = D / 16;
  float acc[NT][kMt][4];  // O^T, relative to 2^(m + gap)
  float m[NT][2], gap[NT][2], l[NT][2];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < kMt; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[t][i][k] = 0.f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        m[t][k] = gap[t][k] = kLow;
        l[t][k] = 0.f;
      }
    }
  }
};

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

// A lane's numbers of P between the softmax and the second product.  They wait in
// shared memory: the copies of the next blocks are issued in between.
template <int NT>
struct Probabilities {
  float4 (*p)[4][32];
  __device__ __forceinline__ float4& at(int i) const { return p[i >> 2][i & 3][threadIdx.x & 31]; }
  __device__ __forceinline__ void put(const float (&s)[NT][4][4]) const {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) at(t * 4 + i) = make_float4(s[t][i][0], s[t][i][1], s[t][i][2], s[t][i][3]);
  }
  // To fp16, in the second product's order.
  __device__ __forceinline__ void get(uint32_t (&pf)[NT][4][2]) const {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 x = at(t * 4 + i);
        const uint32_t a = h2_bits(__floats2half2_rn(x.x, x.y)), b = h2_bits(__floats2half2_rn(x.z, x.w));
        pf[t][i][0] = transpose8x8(a);
        pf[t][i][1] = transpose8x8(b);
      }
  }
  // Does fp16 leave something of them?
  __device__ __forceinline__ bool more() const {
    bool any = false;
#pragma unroll 1
    for (int i = 0; i < 4 * NT; ++i) {
      const float4 x = at(i);
      any |= left_by_fp16(x.x) != 0.f || left_by_fp16(x.y) != 0.f || left_by_fp16(x.z) != 0.f || left_by_fp16(x.w) != 0.f;
    }
    return any;
  }
  // To what fp16 left of them.
  __device__ __forceinline__ void next() const {
#pragma unroll 1
    for (int i = 0; i < 4 * NT; ++i) {
      const float4 x = at(i);
      at(i) = make_float4(left_by_fp16(x.x), left_by_fp16(x.y), left_by_fp16(x.z), left_by_fp16(x.w));
    }
  }
};

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

// Normalises the sums of a unit, or of a piece's part of it, and writes them.
template <int D, int NT>
__device__ __forceinline__ void write_part(const AttnParams& p, const Sums<D, NT>& sums, int head, int row0, int rr0,
                                           int nrows, bool whole, size_t part_at) {
  const int lane = threadIdx.x & 31, gr = lane >> 2, tc = lane & 3;
  constexpr int kMt = D / 16;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float l[2], inv[2], unit[2];  // two factors: 2^-126 / l would be a subnormal number of few bits
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      l[k] = sums.l[t][k];
#pragma unroll
      for (int d = 4; d < 32; d *= 2) l[k] += __shfl_xor_sync(0xffffffffu, l[k], d);
      const bool none = l[k] == 0.f;
      inv[k] = none ? 0.f : 1.f / l[k];
      unit[k] = none ? 0.f : exp2_approx(sums.gap[t][k]);
    }
    if (whole) {
      const int r = t * 8 + gr;
      const unsigned rr = rr0 + r, token = rr / p.g;
      __nv_bfloat16* out =
          p.o + (static_cast<long long>(row0 + token) * p.hq + head * p.g + (rr - token * p.g)) * D + tc * 2;
#pragma unroll
      for (int i = 0; i < kMt; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // [8 channels][8 rows] to [8 rows][8 channels]: lane then has row gr, channels 2 tc and 2 tc + 1
          const __nv_bfloat162 y = __floats2bfloat162_rn(sums.acc[t][i][2 * h] * inv[0] * unit[0],
                                                         sums.acc[t][i][2 * h + 1] * inv[1] * unit[1]);
          const uint32_t z = transpose8x8(*reinterpret_cast<const uint32_t*>(&y));
          if (r < nrows) *reinterpret_cast<uint32_t*>(out + i * 16 + h * 8) = z;
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int rc = t * 8 + 2 * tc + k;
        if (gr == 0 && rc < nrows) {
          const unsigned tk = static_cast<unsigned>(rr0 + rc) / p.g;
          p.lse[(static_cast<long long>(head) * p.g + (rr0 + rc - tk * p.g)) * p.c.rows + row0 + tk] =
              lse_of(sums.m[t][k], l[k]);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = t * 8 + 2 * tc + (k & 1);
        if (r < nrows) {
#pragma unroll
          for (int i = 0; i < kMt; ++i)
            p.part[(part_at + r) * D + i * 16 + (k >> 1) * 8 + gr] = sums.acc[t][i][k] * inv[k & 1] * unit[k & 1];
          if (gr == 0 && k < 2) p.part_sum[part_at + r] = make_float2(sums.m[t][k & 1], l[k & 1]);
        }
      }
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
  const Cut cut(total, gridDim.x, p.dynamic);
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
      if (live) write_part<D, NT>(p, sums, head, row0, rr0, nrows, whole, part_at);
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
constexpr int kJoinWarps = 16;
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

constexpr int kMaxNt = 2;
constexpr size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

constexpr int kDevices = 64;

// The current device and its SMs (asked for once).
hdp_status_t sm_count(int* device, int* sms) {
  static std::atomic<int> known[kDevices];
  HDP_CUDA_TRY(cudaGetDevice(device));
  const bool kept = *device < kDevices;
  *sms = kept ? known[*device].load(std::memory_order_relaxed) : 0;
  if (*sms > 0) return HDP_OK;
  HDP_CUDA_TRY(cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *device));
  if (kept) known[*device].store(*sms, std::memory_order_relaxed);
  return HDP_OK;
}

struct Layout {
  int pieces;
  size_t part, part_sum, open, head, bytes;
  Layout(int sms, int d) {
    const size_t rows = 8 * kMaxNt;
    pieces = sms * kWarps * (1 + kMorePieces);
    part = 0;
    part_sum = part + align256(pieces * 2 * rows * d * sizeof(float));
    open = part_sum + align256(pieces * 2 * rows * sizeof(float2));
    head = open + align256(pieces * sizeof(Open));
    bytes = head + 256;
  }
};

// A launch that may begin before the kernel in front of it has ended; it waits
// for that kernel's results itself.
template <class... T>
hdp_status_t launch_early(void (*kernel)(T...), dim3 grid, int threads, int smem, cudaStream_t st, T... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  HDP_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, args...));
  note_launch();
  return HDP_OK;
}

template <int D, int FMT, int NT, bool SPARSE>
hdp_status_t launch(const AttnParams& p, int device, int ctas, cudaStream_t st) {
  auto* kernel = k_cache_attention<D, FMT, NT, SPARSE>;
  constexpr int smem = sizeof(Shared<NT, SPARSE>);
  static_assert(smem <= 232448, "shared memory of a CTA");
  static std::atomic<bool> ready[kDevices];
  if (device >= kDevices || !ready[device].load(std::memory_order_relaxed)) {
    HDP_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    if (device < kDevices) ready[device].store(true, std::memory_order_relaxed);
  }
  const int pieces = ctas * kWarps * (p.dynamic ? 1 + kMorePieces : 1);
  if (pieces > 47 * 192)  // k_cache_attention_join's lists; a device of over 188 SMs
    return fail(HDP_ERR_UNSUPPORTED, "hdp_cache_attention: too many SMs");
  if (p.dynamic) {
    k_cache_attention_start<<<1, 32, 0, st>>>(p);
    note_launch();
    HDP_CUDA_TRY(cudaGetLastError());
    const hdp_status_t r = launch_early(kernel, dim3(ctas), kThreads, smem, st, p);
    if (r != HDP_OK) return r;
  } else {
    kernel<<<ctas, kThreads, smem, st>>>(p);
    note_launch();
    HDP_CUDA_TRY(cudaGetLastError());
  }
  return launch_early(k_cache_attention_join<D, NT>, dim3(ctas), kJoinWarps * 32, 0, st, p, pieces);
}

template <int D, int FMT>
hdp_status_t launch_for(const AttnParams& p, int nt, int device, int ctas, cudaStream_t st) {
  if (p.blocks) return nt == 1 ? launch<D, FMT, 1, true>(p, device, ctas, st) : launch<D, FMT, 2, true>(p, device, ctas, st);
  return nt == 1 ? launch<D, FMT, 1, false>(p, device, ctas, st) : launch<D, FMT, 2, false>(p, device, ctas, st);
}

}  // namespace
}  // namespace hdp

using namespace hdp;

extern "C" hdp_status_t hdp_cache_attention_workspace_bytes(const hdp_cache_t* cache, int32_t hq, size_t* bytes) {
  if (!cache || !bytes) return fail(HDP_ERR_INVALID_ARGUMENT, "hdp_cache_attention_workspace_bytes: NULL argument");
  if (cache->hkv < 1 || hq < 1 || hq % cache->hkv != 0)
    return fail(HDP_ERR_INVALID_ARGUMENT, "hdp_cache_attention_workspace_bytes: need hq >= 1 and hq % hkv == 0");
  if (cache->d != 64 && cache->d != 128)
    return fail(HDP_ERR_UNSUPPORTED, "hdp_cache_attention_workspace_bytes: d must be 64 or 128");
  int device = 0, sms = 0;
  const hdp_status_t r = sm_count(&device, &sms);
  if (r != HDP_OK) return r;
  *bytes = Layout(sms, cache->d).bytes;
  return HDP_OK;
}

extern "C" hdp_status_t hdp_cache_attention(const hdp_cache_t* cache, const int32_t* cu, int64_t rows, const void* q,
                                            int32_t hq, float scale, const int32_t* blocks, int32_t count,
                                            void* workspace, size_t workspace_bytes, void* o, float* lse,
                                            void* stream) {
  AttnParams p = {};
  hdp_status_t r = cache_view("hdp_cache_attention", cache, cu, rows, &p.c);
  if (r != HDP_OK) return r;
  if (hq < 1 || hq % cache->hkv != 0)
    return fail(HDP_ERR_INVALID_ARGUMENT, "hdp_cache_attention: need hq >= 1 and hq % hkv == 0");
  if (!(scale > 0.f)) return fail(HDP_ERR_INVALID_ARGUMENT, "hdp_cache_attention: scale must be > 0");
  // a list for no rows may be an empty tensor, which has no address
  if (blocks ? count < 1 : count < 0 || (count > 0 && rows > 0))
    return fail(HDP_ERR_INVALID_ARGUMENT, "hdp_cache_attention: count must be >= 1 with blocks and 0 without");
  if (rows == 0) return HDP_OK;
  if (rows * (hq / cache->hkv) > 2147483647LL)
    return fail(HDP_ERR_UNSUPPORTED, "hdp_cache_attention: rows * hq / hkv must be below 2^31");
  if (!q || !o || !lse) return fail(HDP_ERR_INVALID_ARGUMENT, "hdp_cache_attention: NULL argument");
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(o)) & 15)
    return fail(HDP_ERR_INVALID_ARGUMENT, "hdp_cache_attention: q and o must be 16-byte aligned");
  int device = 0, sms = 0;
  r = sm_count(&device, &sms);
  if (r != HDP_OK) return r;
  const Layout lay(sms, cache->d);
  if (!workspace || workspace_bytes < lay.bytes)
    return fail(HDP_ERR_INVALID_ARGUMENT, "hdp_cache_attention: workspace too small (need " +
                                              std::to_string(lay.bytes) + " bytes)");
  if (reinterpret_cast<uintptr_t>(workspace) & 255)
    return fail(HDP_ERR_INVALID_ARGUMENT, "hdp_cache_attention: workspace must be 256-byte aligned");
  p.c.err = device_error_word();
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.blocks = blocks;
  p.count = count;
  p.hq = hq;
  p.g = hq / cache->hkv;
  p.scale_log2 = scale * 1.4426950408889634f;
  char* ws = static_cast<char*>(workspace);
  p.part = reinterpret_cast<float*>(ws + lay.part);
  p.part_sum = reinterpret_cast<float2*>(ws + lay.part_sum);
  p.open = reinterpret_cast<Open*>(ws + lay.open);
  p.head = reinterpret_cast<int*>(ws + lay.head);

  // Tiles of 8 query rows while they hold a sequence's rows on average, of 16
  // beyond: a second tile reads the cache again.
  const int64_t each = blocks ? 1 : (rows + cache->num_seqs - 1) / cache->num_seqs;
  const int nt = each * p.g <= 8 ? 1 : 2;
  // No more CTAs than there can be steps.
  const double tiles = blocks ? static_cast<double>(rows) * ((p.g + 8 * nt - 1) / (8 * nt))
                              : static_cast<double>(rows) * p.g / (8 * nt) + cache->num_seqs;
  const double steps = tiles * cache->hkv * (blocks ? count : cache->max_pages);
  const int ctas = steps < sms ? static_cast<int>(steps) + 1 : sms;
  // Handing out the ends of runs costs one more small launch: from 16 steps a
  // warp on, where the runs' ends are more than a step.
  p.dynamic = steps >= 16.0 * kWarps * sms;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool i8 = cache->format == HDP_CACHE_INT8;
  if (cache->d == 128)
    return i8 ? launch_for<128, HDP_CACHE_INT8>(p, nt, device, ctas, st) : launch_for<128, HDP_CACHE_E4M3>(p, nt, device, ctas, st);
  return i8 ? launch_for<64, HDP_CACHE_INT8>(p, nt, device, ctas, st) : launch_for<64, HDP_CACHE_E4M3>(p, nt, device, ctas, st);
}
