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
//   Products.  S^T = K Q^T with the 64 keys as rows of m16n8k16 fragments and
//   the query rows of the group as the 8 columns, so one decoded token of 8
//   query heads fills the instruction and the keys fill the rest; O^T = V^T P^T
//   likewise.  The codes become fp16 exactly (int8 by the exponent of 1024,
//   e4m3 by the conversion instruction); the cache's order of bytes is the
//   fragments' order.  The query row is shifted by a power of two to
//   [2^14, 2^15), which is exact in fp16 down to 2^-38 of its largest element
//   (below, the error is at most 2^-39 of it).  P <= 1 is rounded to fp16:
//   half a step is 2^-12 of a probability (2^-25 absolute below 2^-14), 1/16 of
//   the bf16 rounding of the output.  All sums are fp32.
//   Softmax.  The reference exponents are whole numbers: m of the row sum, M of
//   the output, which also takes in the V scales' exponents; every rescaling is
//   then by a power of two, and blocks with very different V scales lose nothing.
//   Joining.  Warps leave a normalised (O, LSE) for a unit that they share with
//   a neighbour; each CTA joins those of its own warps, and a second small
//   kernel joins those of neighbouring CTAs, always in the order of the keys.
#include <cuda_fp16.h>

#include <string>

#include "kv_cache.cuh"

namespace hdp {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRingBytes = 24576;  // of each warp: 3 (d = 128) or 6 (d = 64) half blocks
constexpr int kMeta = 8;           // blocks whose scales and first key are kept
constexpr float kLow = -1.0e30f;   // reference exponent before the first key
constexpr float kLn2 = 0.6931471805599453f;

struct Meta {
  float sk, sv;
  int key0;  // first key of the block; -1: nothing of it is seen
  int pad;
};

// What a CTA leaves for its right neighbours: the unit that begins here and
// ends in CTA `last`.
struct Open {
  int active, last, row0, head, nrows, pad;
  long long rr0;
};

struct AttnParams {
  CacheView c;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  const int32_t* blocks;
  int count, hq, g;
  float scale_log2;
  float* part;      // [ctas][2][rows of a tile][d]
  float* part_lse;  // [ctas][2][rows of a tile]
  float* warp_part; // [ctas][warps][rows of a tile][d], tiles of 16 rows only
  Open* open;       // [ctas]
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

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ uint32_t h2_bits(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }
__device__ __forceinline__ __half2 as_h2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }

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

// A place in the flat order.  A unit is (sequence or row, kv head, tile of
// query rows); a step is one block of it.
template <bool SPARSE, int NT>
struct Cursor {
  int seq, row0, n, head, tile, tiles, nb, blk;
  long long len, p0;

  __device__ __forceinline__ static int tiles_of(long long n, int g) {
    return static_cast<int>((n * g + 8 * NT - 1) / (8 * NT));
  }
  // Blocks of all units of sequence i.
  __device__ __forceinline__ static long long cost(const AttnParams& p, int i) {
    int row0, n;
    seq_rows(p.c, i, row0, n);
    if (n == 0) return 0;
    const long long nb = max(1LL, (seq_len(p.c, i) + kBlock - 1) / kBlock);
    return nb * tiles_of(n, p.g) * p.c.hkv;
  }
  __device__ __forceinline__ void enter(const AttnParams& p, int i) {
    head = tile = blk = 0;
    if constexpr (SPARSE) {
      row0 = i;
      n = 1;
      nb = p.count;
      seq = seq_of_row(p.c, i);
      if (seq >= 0) {
        len = seq_len(p.c, seq);
        const int first = p.c.cu ? __ldg(p.c.cu + seq) : i;
        p0 = first_position(p.c, seq, len) + (i - first);
      } else {
        len = p0 = 0;
      }
    } else {
      seq = i;
      seq_rows(p.c, i, row0, n);
      len = seq_len(p.c, i);
      p0 = first_position(p.c, i, len);
      nb = static_cast<int>(max(1LL, (len + kBlock - 1) / kBlock));
    }
    tiles = tiles_of(n, p.g);
  }
  __device__ __forceinline__ void next_unit(const AttnParams& p) {
    blk = 0;
    if (++tile < tiles) return;
    tile = 0;
    if (++head < p.c.hkv) return;
    int i = (SPARSE ? row0 : seq) + 1;
    if constexpr (SPARSE) {
      if (i < p.c.rows) enter(p, i);
    } else {
      while (i < p.c.num_seqs && cost(p, i) == 0) ++i;
      if (i < p.c.num_seqs) enter(p, i);
    }
  }
  // Skips `off` steps from the sequence's first.
  __device__ __forceinline__ void skip(long long off) {
    const long long unit = off / nb;
    blk = static_cast<int>(off - unit * nb);
    head = static_cast<int>(unit / tiles);
    tile = static_cast<int>(unit - static_cast<long long>(head) * tiles);
  }
  __device__ __forceinline__ long long rr0() const { return static_cast<long long>(tile) * (8 * NT); }
  __device__ __forceinline__ int nrows(int g) const {
    return static_cast<int>(min(static_cast<long long>(8 * NT), static_cast<long long>(n) * g - rr0()));
  }
  // Positions of the tile's first and last row.
  __device__ __forceinline__ long long first_pos(int g) const { return p0 + rr0() / g; }
  __device__ __forceinline__ long long last_pos(int g) const { return p0 + (rr0() + nrows(g) - 1) / g; }
};

struct Seg {
  int valid, begins, ends, row0, head, nrows;
  long long rr0, unit_end;  // unit_end: flat end of the unit
};

template <int D, int NT>
struct Shared {
  static constexpr int kRows = 8 * NT;
  unsigned char ring[kWarps][kRingBytes];
  union {
    long long pre[kThreads + 1];  // steps before each thread's sequences; read before the first part is written
    float part[NT == 1 ? kWarps : 1][NT == 1 ? kRows : 1][D];
  };
  float lse[kWarps][2][kRows];
  Meta meta[kWarps][kMeta];
  Seg seg[kWarps][2];
  long long warp_sum[kWarps];
};

template <int D>
__device__ __forceinline__ void write_o(const AttnParams& p, int row0, int head, long long rr, const float* x, float lse,
                                        int lane) {
  const long long t = row0 + rr / p.g;
  const int h = head * p.g + static_cast<int>(rr % p.g);
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

// Joins `m` normalised partials of one row (lse in bits of 2) in their order:
// x = sum 2^(lse_k - L) o_k, L = log2 sum 2^lse_k.  o_at(k) points at the row.
template <int D, class L, class O>
__device__ __forceinline__ float join_row(int m, int lane, float (&x)[D / 32], L lse_at, O o_at) {
  float top = -__int_as_float(0x7f800000);
  bool nan = false;
  for (int k = lane; k < m; k += 32) {
    const float l = lse_at(k);
    nan |= l != l;
    top = fmaxf(top, l);
  }
#pragma unroll
  for (int s = 16; s; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
  nan = __any_sync(0xffffffffu, nan);
#pragma unroll
  for (int i = 0; i < D / 32; ++i) x[i] = 0.f;
  if (top == -__int_as_float(0x7f800000) && !nan) return top;  // no key in any of them: o = 0
  float sum = 0.f;
#pragma unroll 4
  for (int k = 0; k < m; ++k) {
    const float l = lse_at(k);
    const float w = exp2_approx(l - top);
    sum += w;
    const float* o = o_at(k) + lane * (D / 32);
    if constexpr (D == 128) {
      const float4 y = *reinterpret_cast<const float4*>(o);
      x[0] = fmaf(w, y.x, x[0]);
      x[1] = fmaf(w, y.y, x[1]);
      x[2] = fmaf(w, y.z, x[2]);
      x[3] = fmaf(w, y.w, x[3]);
    } else {
      const float2 y = *reinterpret_cast<const float2*>(o);
      x[0] = fmaf(w, y.x, x[0]);
      x[1] = fmaf(w, y.y, x[1]);
    }
  }
  const float inv = 1.f / sum;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) x[i] *= inv;
  return top + log2f(sum);
}

// How the flat order of `total` steps is cut: `used` warps of each CTA take
// `per` steps each.  While there are fewer steps than warps, the steps are
// spread over the CTAs first.
struct Cut {
  int used;
  long long per;
  __device__ __forceinline__ Cut(long long total, int ctas) {
    const long long each = (total + ctas - 1) / ctas;
    used = static_cast<int>(min(static_cast<long long>(kWarps), max(1LL, each)));
    const long long workers = static_cast<long long>(ctas) * used;
    per = max(1LL, (total + workers - 1) / workers);
  }
};

template <int D, int FMT, int NT, bool SPARSE>
__global__ void __launch_bounds__(kThreads, 1) k_cache_attention(const AttnParams p) {
  constexpr int kHalf = kBlock * D;               // bytes of a block's K or V codes of one head
  constexpr int kSlots = kRingBytes / kHalf;      // half blocks in flight
  constexpr int kKeyChunks = D / 64;              // 16-byte chunks that a lane has of a key
  constexpr int kMt = D / 16;
  constexpr int kRows = 8 * NT;
  using Cur = Cursor<SPARSE, NT>;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  Shared<D, NT>& sm = *reinterpret_cast<Shared<D, NT>*>(smem_raw);
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
      if (s < p.c.num_seqs) mine += Cur::cost(p, s);
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
  if (lane < 2) sm.seg[warp][lane].valid = 0;
  if (threadIdx.x == 0) p.open[blockIdx.x].active = 0;
  __syncthreads();
  const Cut cut(total, gridDim.x);
  const long long start = (static_cast<long long>(blockIdx.x) * cut.used + warp) * cut.per;
  const long long stop = warp < cut.used ? min(total, start + cut.per) : 0;

  Cur cc;  // of the arithmetic
  if (start < stop) {
    if constexpr (SPARSE) {
      const long long row_cost = static_cast<long long>(per_row) * p.count;
      const int row = static_cast<int>(start / row_cost);
      cc.enter(p, row);
      cc.skip(start - row * row_cost);
    } else {
      const int slice = find_last(kThreads, start, [&](int s) { return sm.pre[s]; });
      long long at = sm.pre[slice];
      int i = slice * per_thread;
      for (long long c = Cur::cost(p, i); start - at >= c && i + 1 < p.c.num_seqs; c = Cur::cost(p, i)) {
        at += c;
        ++i;
      }
      cc.enter(p, i);
      cc.skip(start - at);
    }
  }
  __syncthreads();

  if (start < stop) {
    Cur lc = cc;  // of the copies, which run ahead
    long long to_load = stop - start;
    int half = 0;                 // 0: K of lc's block next, 1: V
    int load_slot = 0, load_meta = 0;
    int ids = -1, ids_at = -1;    // 32 blocks' pages (dense) or blocks and pages (sparse) of lc's unit, one a lane
    int ids_page = -1;
    const unsigned char* cur_v = nullptr;  // V of the block whose K went last
    const uint32_t ring = smem_addr(sm.ring[warp]) + lane * 16;

    auto issue = [&]() {
      if (to_load > 0) {
        if (half == 0) {
          const long long last = lc.last_pos(p.g);
          if (ids_at != (lc.blk & ~31)) {  // a new unit, or the next 32 blocks
            ids_at = lc.blk & ~31;
            const int b = ids_at + lane;
            ids = ids_page = -1;
            if (b < lc.nb) {
              if constexpr (SPARSE) {
                if (lc.seq >= 0) {
                  const int32_t* list = p.blocks + (static_cast<long long>(lc.row0) * p.c.hkv + lc.head) * p.count;
                  const int x = __ldg(list + b), before = b ? __ldg(list + b - 1) : -1;
                  if (x > before && x >= 0 && static_cast<long long>(x) * kBlock <= last) {
                    ids = x;
                    ids_page = page_of(p.c, lc.seq, x);
                  }
                }
              } else if (static_cast<long long>(b) * kBlock <= last) {
                ids = b;
                ids_page = page_of(p.c, lc.seq, b);
              }
            }
          }
          const int b = __shfl_sync(0xffffffffu, ids, lc.blk & 31);
          const int page = __shfl_sync(0xffffffffu, ids_page, lc.blk & 31);
          const bool seen = b >= 0 && page >= 0;
          Meta* meta = &sm.meta[warp][load_meta];
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
          if (++lc.blk == lc.nb) {
            lc.next_unit(p);
            ids_at = -1;
          }
        }
        half ^= 1;
        load_slot = load_slot + 1 == kSlots ? 0 : load_slot + 1;
      }
      copies_commit();
    };

#pragma unroll
    for (int i = 0; i < kSlots; ++i) issue();

    int slot = 0, meta_at = 0, segs = 0;
    long long at = start;
    while (at < stop) {
      // ---- one unit, or the part of it that this warp has
      const bool begins = cc.blk == 0;
      const int steps = static_cast<int>(min(static_cast<long long>(cc.nb - cc.blk), stop - at));
      const bool ends = cc.blk + steps == cc.nb;
      const int nrows = cc.nrows(p.g);
      const long long rr0 = cc.rr0();
      const bool live = !SPARSE || cc.seq >= 0;

      uint32_t qf[NT][kMt][2];
      float qs[NT][2];   // scale * log2(e) * 2^(shift) of columns 2 tc and 2 tc + 1
      int pos[NT][2];    // their positions
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int r = t * 8 + gr;
        uint4 x[kMt / 2];
#pragma unroll
        for (int i = 0; i < kMt / 2; ++i) x[i] = make_uint4(0, 0, 0, 0);
        if (r < nrows) {
          const long long rr = rr0 + r;
          const uint4* src = reinterpret_cast<const uint4*>(
              p.q + ((cc.row0 + rr / p.g) * p.hq + cc.head * p.g + rr % p.g) * D + tc * 16);
#pragma unroll
          for (int i = 0; i < kMt / 2; ++i) x[i] = __ldg(src + (i >> 1) * 8 + (i & 1));
        }
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kMt / 2; ++i)
          top = __vmaxu2(top, __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                                       __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu)));
        top = max(top & 0xffffu, top >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // the largest element's exponent goes to 14; infinities and NaN stay what they are
        const int e = min(max(static_cast<int>(top >> 7) - 127, -112), 127) - 14;
        const float down = pow2i(-e);
#pragma unroll
        for (int i = 0; i < kMt / 2; ++i) {
          const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const __half2 y = __floats2half2_rn(__uint_as_float(w[k] << 16) * down, __uint_as_float(w[k] & 0xffff0000u) * down);
            qf[t][i * 2 + (k >> 1)][k & 1] = h2_bits(y);
          }
        }
        const float s = p.scale_log2 * pow2i(e);
        qs[t][0] = __shfl_sync(0xffffffffu, s, tc * 8);
        qs[t][1] = __shfl_sync(0xffffffffu, s, tc * 8 + 4);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int rc = min(t * 8 + 2 * tc + k, nrows - 1);
          pos[t][k] = static_cast<int>(max(-1LL, cc.p0 + (rr0 + rc) / p.g));
        }
      }
      const long long low_pos = cc.first_pos(p.g);

      float acc[NT][kMt][4], m[NT][2], M[NT][2], l[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int i = 0; i < kMt; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[t][i][k] = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          m[t][k] = M[t][k] = kLow;
          l[t][k] = 0.f;
        }
      }

      for (int step = 0; step < steps; ++step) {
        copies_wait<kSlots - 1>();
        __syncwarp();
        const Meta meta = sm.meta[warp][meta_at];
        meta_at = (meta_at + 1) % kMeta;
        const bool seen = meta.key0 >= 0;
        const bool masked = meta.key0 + kBlock - 1 > low_pos;  // some row does not see the whole block
        uint32_t pf[NT][4][2];
        if (seen) {
          const uint4* kx = reinterpret_cast<const uint4*>(sm.ring[warp] + slot * kHalf) + lane;
          float s[NT][4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int k = 0; k < 4; ++k) s[t][i][k] = 0.f;
#pragma unroll
            for (int j = 0; j < kKeyChunks; ++j) {
              const uint4 u = kx[((2 * i) * kKeyChunks + j) * 32], w = kx[((2 * i + 1) * kKeyChunks + j) * 32];
              const uint32_t uw[4] = {u.x, u.y, u.z, u.w}, ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t a0, a1, a2, a3;
                decode4<FMT>(uw[k], a0, a2);
                decode4<FMT>(ww[k], a1, a3);
#pragma unroll
                for (int t = 0; t < NT; ++t) mma16816(s[t][i], a0, a1, a2, a3, qf[t][j * 4 + k][0], qf[t][j * 4 + k][1]);
              }
            }
          }
          const int ev = static_cast<int>((__float_as_uint(meta.sv) >> 23) & 0xff) - 127;
          const float lsv = meta.sv == meta.sv ? static_cast<float>(ev) : meta.sv;  // log2 of the V scale
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            float top[2] = {-__int_as_float(0x7f800000), -__int_as_float(0x7f800000)};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                float x = s[t][i][k] * meta.sk * qs[t][k & 1];
                if (masked && meta.key0 + 16 * i + 8 * (k >> 1) + gr > pos[t][k & 1]) x = -__int_as_float(0x7f800000);
                s[t][i][k] = x;
                top[k & 1] = fmaxf(top[k & 1], x);
              }
            float f[2], ref[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
              for (int d = 4; d < 32; d *= 2) top[k] = fmaxf(top[k], __shfl_xor_sync(0xffffffffu, top[k], d));
              const bool none = top[k] == -__int_as_float(0x7f800000);
              const float c = none ? 0.f : ceilf(top[k]);
              ref[k] = c;
              const float m1 = none ? m[t][k] : fmaxf(m[t][k], c);
              const float M1 = none ? M[t][k] : fmaxf(M[t][k], c + lsv);
              l[t][k] *= exp2_approx(m[t][k] - m1);
              const float up = exp2_approx(M[t][k] - M1);
              if (M1 != M[t][k]) {
#pragma unroll
                for (int i = 0; i < kMt; ++i) {
                  acc[t][i][k] *= up;
                  acc[t][i][k + 2] *= up;
                }
              }
              m[t][k] = m1;
              M[t][k] = M1;
              const float fl = none ? 0.f : exp2_approx(c - m1);
              f[k] = none ? 0.f : exp2_approx(c + lsv - M1);
              float sum = 0.f;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                s[t][i][k] = exp2_approx(s[t][i][k] - c);
                s[t][i][k + 2] = exp2_approx(s[t][i][k + 2] - c);
                sum += s[t][i][k] + s[t][i][k + 2];
              }
              l[t][k] = fmaf(sum, fl, l[t][k]);
            }
            const __half2 ff = __floats2half2_rn(f[0], f[1]);  // a power of two <= 1
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              pf[t][i][0] = transpose8x8(h2_bits(__hmul2(__floats2half2_rn(s[t][i][0], s[t][i][1]), ff)));
              pf[t][i][1] = transpose8x8(h2_bits(__hmul2(__floats2half2_rn(s[t][i][2], s[t][i][3]), ff)));
            }
          }
        }
        slot = slot + 1 == kSlots ? 0 : slot + 1;
        issue();

        copies_wait<kSlots - 1>();
        if (seen) {
          const uint4* vx = reinterpret_cast<const uint4*>(sm.ring[warp] + slot * kHalf) + lane;
#pragma unroll
          for (int i = 0; i < kMt; ++i) {
            const uint4 u = vx[(2 * i) * 32], w = vx[(2 * i + 1) * 32];
            uint32_t uw[4] = {u.x, u.y, u.z, u.w}, ww[4] = {w.x, w.y, w.z, w.w};
            if (masked) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uw[k] = without_nan<FMT>(uw[k]);
                ww[k] = without_nan<FMT>(ww[k]);
              }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t a0, a1, a2, a3;
              decode4<FMT>(uw[k], a0, a2);
              decode4<FMT>(ww[k], a1, a3);
#pragma unroll
              for (int t = 0; t < NT; ++t) mma16816(acc[t][i], a0, a1, a2, a3, pf[t][k][0], pf[t][k][1]);
            }
          }
        }
        slot = slot + 1 == kSlots ? 0 : slot + 1;
        issue();
      }
      at += steps;

      // ---- the unit's part is done: normalise, then out, or into a partial
      const bool whole = begins && ends;
      float* part = segs == 0 ? (NT == 1 ? &sm.part[warp][0][0]
                                         : p.warp_part + (static_cast<size_t>(blockIdx.x) * kWarps + warp) * kRows * D)
                              : reinterpret_cast<float*>(sm.ring[warp]);
      if (!whole && segs > 0) {
        copies_wait<0>();  // the ring becomes the partial's place: this is the warp's last unit
        __syncwarp();
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float inv[2], lse2[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int d = 4; d < 32; d *= 2) l[t][k] += __shfl_xor_sync(0xffffffffu, l[t][k], d);
          const bool none = l[t][k] == 0.f;
          inv[k] = none ? 0.f : exp2_approx(M[t][k] - m[t][k]) / l[t][k];
          lse2[k] = none ? -__int_as_float(0x7f800000) : m[t][k] + log2f(l[t][k]);
        }
        if (whole) {
#pragma unroll
          for (int i = 0; i < kMt; ++i) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              // [8 channels][8 rows] to [8 rows][8 channels]: lane then has row gr, channels 2 tc and 2 tc + 1
              const __nv_bfloat162 y = __floats2bfloat162_rn(acc[t][i][2 * h] * inv[0], acc[t][i][2 * h + 1] * inv[1]);
              const uint32_t z = transpose8x8(*reinterpret_cast<const uint32_t*>(&y));
              const int r = t * 8 + gr;
              if (r < nrows && live) {
                const long long rr = rr0 + r;
                __nv_bfloat16* out = p.o + ((cc.row0 + rr / p.g) * p.hq + cc.head * p.g + rr % p.g) * D;
                *reinterpret_cast<uint32_t*>(out + i * 16 + h * 8 + tc * 2) = z;
              }
            }
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int r = t * 8 + 2 * tc + k;
            if (gr == 0 && r < nrows && live) {
              const long long rr = rr0 + r;
              p.lse[(static_cast<long long>(cc.head) * p.g + rr % p.g) * p.c.rows + cc.row0 + rr / p.g] = lse2[k] * kLn2;
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < kMt; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              part[(t * 8 + 2 * tc + (k & 1)) * D + i * 16 + (k >> 1) * 8 + gr] = acc[t][i][k] * inv[k & 1];
          if (gr == 0) {
            sm.lse[warp][min(segs, 1)][t * 8 + 2 * tc] = lse2[0];
            sm.lse[warp][min(segs, 1)][t * 8 + 2 * tc + 1] = lse2[1];
          }
        }
      }
      if (!whole && lane == 0) {
        Seg& sg = sm.seg[warp][min(segs, 1)];
        sg.valid = 1;
        sg.begins = begins;
        sg.ends = ends;
        sg.row0 = live ? cc.row0 : -1;
        sg.head = cc.head;
        sg.nrows = nrows;
        sg.rr0 = rr0;
        sg.unit_end = at + (cc.nb - cc.blk - steps);
      }
      segs = 1;
      cc.blk += steps;
      if (cc.blk == cc.nb && at < stop) cc.next_unit(p);
    }
    copies_wait<0>();
  }
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- units that warps of this CTA share: a group is a run of parts (w, s),
  // (w + 1, 0), ...; all warps take rows of the groups in turn
  int item = 0;
  for (int w0 = 0; w0 < cut.used; ++w0) {
#pragma unroll
    for (int s0 = 0; s0 < 2; ++s0) {
      const Seg& a = sm.seg[w0][s0];
      if (!a.valid || (!a.begins && !(w0 == 0 && s0 == 0))) continue;
      int w1 = w0;
      bool ends = a.ends;
      while (!ends && w1 + 1 < cut.used && sm.seg[w1 + 1][0].valid) ends = sm.seg[++w1][0].ends;
      const bool whole = a.begins && ends;
      for (int r = 0; r < a.nrows; ++r, ++item) {
        if (item % kWarps != warp) continue;
        float x[D / 32];
        const float lse2 = join_row<D>(
            w1 - w0 + 1, lane, x, [&](int k) { return sm.lse[w0 + k][k ? 0 : s0][r]; },
            [&](int k) {
              const float* base = (k == 0 && s0 == 1) ? reinterpret_cast<const float*>(sm.ring[w0])
                                  : NT == 1 ? &sm.part[w0 + k][0][0]
                                            : p.warp_part + (static_cast<size_t>(blockIdx.x) * kWarps + w0 + k) * kRows * D;
              return base + r * D;
            });
        if (whole) {
          if (a.row0 >= 0) write_o<D>(p, a.row0, a.head, a.rr0 + r, x, lse2 * kLn2, lane);
        } else {
          const size_t at = (static_cast<size_t>(blockIdx.x) * 2 + (a.begins ? 1 : 0)) * kRows + r;
#pragma unroll
          for (int i = 0; i < D / 32; ++i) p.part[at * D + lane * (D / 32) + i] = x[i];
          if (lane == 0) p.part_lse[at] = lse2;
        }
      }
      if (a.begins && !ends && threadIdx.x == 0) {
        Open o;
        o.active = a.row0 >= 0;
        o.last = static_cast<int>((a.unit_end - 1) / cut.per / cut.used);
        o.row0 = a.row0;
        o.head = a.head;
        o.nrows = a.nrows;
        o.pad = 0;
        o.rr0 = a.rr0;
        p.open[blockIdx.x] = o;
      }
    }
  }
}

// Joins the parts of units that several CTAs share: CTA e takes the unit that
// begins in the attention's CTA e and goes on in CTAs e + 1 .. last.
template <int D, int NT>
__global__ void __launch_bounds__(kThreads) k_cache_attention_join(const AttnParams p) {
  constexpr int kRows = 8 * NT;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Open o = p.open[blockIdx.x];
  if (!o.active) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int r = warp; r < o.nrows; r += kWarps) {
    float x[D / 32];
    auto at = [&](int k) { return (static_cast<size_t>(blockIdx.x + k) * 2 + (k == 0 ? 1 : 0)) * kRows + r; };
    const float lse2 = join_row<D>(
        o.last - static_cast<int>(blockIdx.x) + 1, lane, x, [&](int k) { return p.part_lse[at(k)]; },
        [&](int k) { return p.part + at(k) * D; });
    write_o<D>(p, o.row0, o.head, o.rr0 + r, x, lse2 * kLn2, lane);
  }
}

constexpr int kMaxNt = 2;
constexpr size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

hdp_status_t sm_count(int* sms) {
  int dev = 0;
  HDP_CUDA_TRY(cudaGetDevice(&dev));
  HDP_CUDA_TRY(cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev));
  return HDP_OK;
}

struct Layout {
  size_t part, part_lse, warp_part, open, bytes;
  Layout(int ctas, int d) {
    const size_t rows = 8 * kMaxNt;
    part = 0;
    part_lse = part + align256(ctas * 2 * rows * d * sizeof(float));
    warp_part = part_lse + align256(ctas * 2 * rows * sizeof(float));
    open = warp_part + align256(ctas * kWarps * rows * d * sizeof(float));
    bytes = open + align256(ctas * sizeof(Open));
  }
};

template <int D, int FMT, int NT, bool SPARSE>
hdp_status_t launch(const AttnParams& p, int ctas, cudaStream_t st) {
  auto* kernel = k_cache_attention<D, FMT, NT, SPARSE>;
  constexpr int smem = sizeof(Shared<D, NT>);
  static_assert(smem <= 232448, "shared memory of a CTA");
  HDP_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
  kernel<<<ctas, kThreads, smem, st>>>(p);
  note_launch();
  HDP_CUDA_TRY(cudaGetLastError());
  // The join's launch overlaps the attention's tail; it waits for its results.
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  HDP_CUDA_TRY(cudaLaunchKernelEx(&cfg, k_cache_attention_join<D, NT>, p));
  note_launch();
  return HDP_OK;
}

template <int D, int FMT>
hdp_status_t launch_for(const AttnParams& p, int nt, int ctas, cudaStream_t st) {
  if (p.blocks) return nt == 1 ? launch<D, FMT, 1, true>(p, ctas, st) : launch<D, FMT, 2, true>(p, ctas, st);
  return nt == 1 ? launch<D, FMT, 1, false>(p, ctas, st) : launch<D, FMT, 2, false>(p, ctas, st);
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
  int sms = 0;
  const hdp_status_t r = sm_count(&sms);
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
  if (blocks ? count < 1 : count != 0)
    return fail(HDP_ERR_INVALID_ARGUMENT, "hdp_cache_attention: count must be >= 1 with blocks and 0 without");
  if (rows == 0) return HDP_OK;
  if (!q || !o || !lse) return fail(HDP_ERR_INVALID_ARGUMENT, "hdp_cache_attention: NULL argument");
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(o)) & 15)
    return fail(HDP_ERR_INVALID_ARGUMENT, "hdp_cache_attention: q and o must be 16-byte aligned");
  int sms = 0;
  r = sm_count(&sms);
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
  p.part_lse = reinterpret_cast<float*>(ws + lay.part_lse);
  p.warp_part = reinterpret_cast<float*>(ws + lay.warp_part);
  p.open = reinterpret_cast<Open*>(ws + lay.open);

  // Tiles of 8 query rows while they hold a sequence's rows on average, of 16
  // beyond: a second tile reads the cache again.
  const int64_t each = blocks ? 1 : (rows + cache->num_seqs - 1) / cache->num_seqs;
  const int nt = each * p.g <= 8 ? 1 : 2;
  // No more CTAs than there can be steps.
  const double tiles = blocks ? static_cast<double>(rows) * ((p.g + 8 * nt - 1) / (8 * nt))
                              : static_cast<double>(rows) * p.g / (8 * nt) + cache->num_seqs;
  const double steps = tiles * cache->hkv * (blocks ? count : cache->max_pages);
  const int ctas = steps < sms ? static_cast<int>(steps) + 1 : sms;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool i8 = cache->format == HDP_CACHE_INT8;
  if (cache->d == 128)
    return i8 ? launch_for<128, HDP_CACHE_INT8>(p, nt, ctas, st) : launch_for<128, HDP_CACHE_E4M3>(p, nt, ctas, st);
  return i8 ? launch_for<64, HDP_CACHE_INT8>(p, nt, ctas, st) : launch_for<64, HDP_CACHE_E4M3>(p, nt, ctas, st);
}
