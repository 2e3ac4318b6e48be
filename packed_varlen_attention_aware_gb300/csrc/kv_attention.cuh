// Attention of the newest tokens of each sequence over a paged cache: what the
// kernels for 8 and for 4 bits share.  How the work is cut, the softmax's references
// and the joining are explained in kv_attention.cu.  Lists of blocks (SPARSE) and pieces
// that are handed out at run time (`dynamic`) are the 8-bit kernel's alone.
#pragma once
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <string>

#include "kv_cache.cuh"

namespace hdp {
namespace {

constexpr float kLow = -3.402823466e38f;  // reference exponent before the first key: below every finite score
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kBias = 15.f;                  // P is at most 2^15, in fp16
constexpr float kBiasMost = 1048576.f;         // references above it are not biased: far below 2^24, so exactly
constexpr float kNormal = 6.103515625e-05f;    // 2^-14, fp16's smallest normal number
constexpr float kNextPass = 1099511627776.f;   // 2^40: what rounding to fp16 leaves below kNormal, 2^-25, to 2^15
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
  const uint8_t* scale_bytes;  // of a 4-bit cache
  bool alone;                  // a CTA of its kernel has a whole unit
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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

constexpr int kSeqs = 512;  // sequences whose places are kept in shared memory

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

__device__ __forceinline__ uint32_t word(const uint4& x, int k) { return k == 0 ? x.x : k == 1 ? x.y : k == 2 ? x.z : x.w; }

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
  __device__ __forceinline__ Cut(long long steps, int ctas, int warps, bool dynamic) : total(steps) {
    const long long each = (total + ctas - 1) / ctas;
    const int used = static_cast<int>(min(static_cast<long long>(warps), max(1LL, each)));
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
      // the largest element's exponent goes to 14
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
      // A row with an infinity or NaN is NaN whatever the keys are: products that are all
      // -infinity would read as a row that sees no key.
      const float s = top >= 0x7f80u ? __int_as_float(0x7fc00000) : p.scale_log2 * pow2i(e);
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

// Normalises the sums of a unit, or of a piece's part of it, and writes them (a part to
// part and part_sum, row by row).
template <int D, int NT>
__device__ __forceinline__ void write_part(const AttnParams& p, const Sums<D, NT>& sums, int head, int row0, int rr0,
                                           int nrows, bool whole, float* part, float2* part_sum) {
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
            part[r * D + i * 16 + (k >> 1) * 8 + gr] = sums.acc[t][i][k] * inv[k & 1] * unit[k & 1];
          if (gr == 0 && k < 2) part_sum[r] = make_float2(sums.m[t][k & 1], l[k & 1]);
        }
      }
    }
  }
}

constexpr int kJoinWarps = 16;  // of a CTA that joins parts

constexpr int kMaxNt = 2;
// For each SM: entries of open, and parts of 16 rows.
struct PartCount {
  int open, parts;
};
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
  size_t part, part_sum, open, head, bytes;
  Layout(const PartCount& n, int sms, int d) {
    const size_t pieces = static_cast<size_t>(sms) * n.open, rows = static_cast<size_t>(sms) * n.parts * 8 * kMaxNt;
    part = 0;
    part_sum = part + align256(rows * d * sizeof(float));
    open = part_sum + align256(rows * sizeof(float2));
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

// `kernel` may have `smem` bytes of shared memory; `ready`: the devices on which it has been told so.
hdp_status_t allow(void (*kernel)(AttnParams), int smem, std::atomic<bool> (&ready)[kDevices], int device) {
  if (device >= kDevices || !ready[device].load(std::memory_order_relaxed)) {
    HDP_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    if (device < kDevices) ready[device].store(true, std::memory_order_relaxed);
  }
  return HDP_OK;
}

hdp_status_t launch_attention(void (*kernel)(AttnParams), int ctas, int threads, int smem, const AttnParams& p, cudaStream_t st) {
  kernel<<<ctas, threads, smem, st>>>(p);
  note_launch();
  HDP_CUDA_TRY(cudaGetLastError());
  return HDP_OK;
}

// Checks and launches a call whose view is in p.c; hand_out: warps of a CTA that can hand
// out the ends of their runs, or 0.
template <class Launch>
hdp_status_t attend(const char* entry, const PartCount& count_of, int hand_out, AttnParams& p, int d, int64_t rows, const void* q, int32_t hq, float scale,
                    const int32_t* blocks, int32_t count, void* workspace, size_t workspace_bytes, void* o, float* lse,
                    void* stream, Launch launch_with) {
  const std::string name(entry);
  if (hq < 1 || hq % p.c.hkv != 0) return fail(HDP_ERR_INVALID_ARGUMENT, name + ": need hq >= 1 and hq % hkv == 0");
  if (!(scale > 0.f)) return fail(HDP_ERR_INVALID_ARGUMENT, name + ": scale must be > 0");
  // a list for no rows may be an empty tensor, which has no address
  if (blocks ? count < 1 : count < 0 || (count > 0 && rows > 0))
    return fail(HDP_ERR_INVALID_ARGUMENT, name + ": count must be >= 1 with blocks and 0 without");
  if (rows == 0) return HDP_OK;
  if (rows * (hq / p.c.hkv) > 2147483647LL)
    return fail(HDP_ERR_UNSUPPORTED, name + ": rows * hq / hkv must be below 2^31");
  if (!q || !o || !lse) return fail(HDP_ERR_INVALID_ARGUMENT, name + ": NULL argument");
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(o)) & 15)
    return fail(HDP_ERR_INVALID_ARGUMENT, name + ": q and o must be 16-byte aligned");
  int device = 0, sms = 0;
  const hdp_status_t r = sm_count(&device, &sms);
  if (r != HDP_OK) return r;
  const Layout lay(count_of, sms, d);
  if (!workspace || workspace_bytes < lay.bytes)
    return fail(HDP_ERR_INVALID_ARGUMENT, name + ": workspace too small (need " + std::to_string(lay.bytes) + " bytes)");
  if (reinterpret_cast<uintptr_t>(workspace) & 255)
    return fail(HDP_ERR_INVALID_ARGUMENT, name + ": workspace must be 256-byte aligned");
  p.c.err = device_error_word();
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.blocks = blocks;
  p.count = count;
  p.hq = hq;
  p.g = hq / p.c.hkv;
  p.scale_log2 = scale * 1.4426950408889634f;
  char* ws = static_cast<char*>(workspace);
  p.part = reinterpret_cast<float*>(ws + lay.part);
  p.part_sum = reinterpret_cast<float2*>(ws + lay.part_sum);
  p.open = reinterpret_cast<Open*>(ws + lay.open);
  p.head = reinterpret_cast<int*>(ws + lay.head);

  // Tiles of 8 query rows while they hold a sequence's rows on average, of 16
  // beyond: a second tile reads the cache again.
  const int64_t each = blocks ? 1 : (rows + p.c.num_seqs - 1) / p.c.num_seqs;
  const int nt = each * p.g <= 8 ? 1 : 2;
  // No more CTAs than there can be steps.
  const double tiles = blocks ? static_cast<double>(rows) * ((p.g + 8 * nt - 1) / (8 * nt))
                              : static_cast<double>(rows) * p.g / (8 * nt) + p.c.num_seqs;
  const double steps = tiles * p.c.hkv * (blocks ? count : p.c.max_pages);
  const int ctas = steps < sms ? static_cast<int>(steps) + 1 : sms;
  // Handing out the ends of runs costs one more small launch: from 16 steps a
  // warp on, where the runs' ends are more than a step.
  p.dynamic = hand_out > 0 && steps >= 16.0 * hand_out * sms;
  return launch_with(p, nt, device, sms, ctas, static_cast<cudaStream_t>(stream));
}

// Bytes of the workspace.
inline hdp_status_t workspace_bytes_of(const char* entry, const PartCount& count_of, int32_t hkv, int32_t d, int32_t hq,
                                       size_t* bytes) {
  const std::string name(entry);
  if (hkv < 1 || hq < 1 || hq % hkv != 0) return fail(HDP_ERR_INVALID_ARGUMENT, name + ": need hq >= 1 and hq % hkv == 0");
  if (d != 64 && d != 128) return fail(HDP_ERR_UNSUPPORTED, name + ": d must be 64 or 128");
  int device = 0, sms = 0;
  const hdp_status_t r = sm_count(&device, &sms);
  if (r != HDP_OK) return r;
  *bytes = Layout(count_of, sms, d).bytes;
  return HDP_OK;
}

}  // namespace
}  // namespace hdp
