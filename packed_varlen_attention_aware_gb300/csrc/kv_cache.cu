// Writing rows into the 8-bit cache and reading them back.
//
// One CTA has the new rows of one (block of 64 tokens, kv head): 128 threads hold
// its K, then its V rows in registers (16 bytes = 8 channels of a row each, d / 16
// rows), so the largest magnitude, the scale, the bounds and the codes come from
// one read.
//
// The scale is 2^e with the smallest e that fits the largest magnitude ever
// written, so x / s is a shift of the exponent and the code is the only
// rounding; a block whose scale grows has its codes shifted and rounded again.
//
// V codes lie [channel][token] with the tokens in the order in which a 16-row
// matrix fragment takes its k index (the attention then feeds 16-byte loads
// straight to the tensor cores).  Two (d = 128) or four (d = 64) lanes here have
// the tokens of one 16-byte chunk, so the transposition is a byte shuffle
// between them and the chunk is stored whole; nothing goes through shared memory.
//
// With one token for each sequence (a decoding step) a warp has one (sequence,
// kv head) instead, half of it the K row and half the V row: nothing but the
// latencies of the length, the page and the old scale stands in its way, and all
// warps of an ordinary batch run at once.
#include <cuda_fp8.h>

#include <cstring>
#include <string>

#include "kv_cache.cuh"

namespace hdp {

hdp_status_t cache_view(const char* call, const hdp_cache_t* c, const int32_t* cu, int64_t rows, CacheView* out) {
  const std::string name(call);
  if (!c) return fail(HDP_ERR_INVALID_ARGUMENT, name + ": cache is NULL");
  if (!c->k || !c->v || !c->scales || !c->bounds || !c->page_table || !c->lens)
    return fail(HDP_ERR_INVALID_ARGUMENT, name + ": the cache has a NULL pointer");
  if (c->num_pages < 1 || c->hkv < 1 || c->num_seqs < 1 || c->max_pages < 1)
    return fail(HDP_ERR_INVALID_ARGUMENT, name + ": num_pages, hkv, num_seqs and max_pages must be >= 1");
  if (c->num_seqs > (1 << 24)) return fail(HDP_ERR_UNSUPPORTED, name + ": num_seqs must be at most 2^24");
  if (c->hkv > 65535) return fail(HDP_ERR_UNSUPPORTED, name + ": hkv must be at most 65535");
  if (c->d != 64 && c->d != 128) return fail(HDP_ERR_UNSUPPORTED, name + ": d must be 64 or 128");
  if (c->format != HDP_CACHE_E4M3 && c->format != HDP_CACHE_INT8)
    return fail(HDP_ERR_INVALID_ARGUMENT, name + ": unknown cache format");
  if ((reinterpret_cast<uintptr_t>(c->k) | reinterpret_cast<uintptr_t>(c->v) |
       reinterpret_cast<uintptr_t>(c->bounds)) & 15 ||
      reinterpret_cast<uintptr_t>(c->scales) & 7)
    return fail(HDP_ERR_INVALID_ARGUMENT,
                name + ": k, v and bounds must be 16-byte and scales 8-byte aligned");
  if (rows < 0 || rows > 2147483647LL)
    return fail(HDP_ERR_INVALID_ARGUMENT, name + ": rows must be 0 .. 2^31-1");
  if (!cu && rows != c->num_seqs)
    return fail(HDP_ERR_INVALID_ARGUMENT, name + ": without cu, rows must equal num_seqs");
  out->k = static_cast<uint8_t*>(c->k);
  out->v = static_cast<uint8_t*>(c->v);
  out->scales = c->scales;
  out->bounds = c->bounds;
  out->table = c->page_table;
  out->lens = c->lens;
  out->cu = cu;
  out->num_pages = c->num_pages;
  out->hkv = c->hkv;
  out->num_seqs = c->num_seqs;
  out->max_pages = c->max_pages;
  out->rows = static_cast<int>(rows);
  return HDP_OK;
}

namespace {

constexpr int kThreads = 128;

// Code of x (already divided by the scale): nearest, ties to even.
template <int FMT>
__device__ __forceinline__ uint32_t code_pair(float a, float b) {
  if constexpr (FMT == HDP_CACHE_INT8) {
    // 1.5 * 2^23 + x: the sum is rounded to a whole number, ties to even, and its low byte is the code
    return __byte_perm(__float_as_uint(a + 12582912.f), __float_as_uint(b + 12582912.f), 0x0040) & 0xffffu;
  } else {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  }
}

// Four codes in a word.
template <int FMT>
__device__ __forceinline__ uint32_t code_quad(float a, float b, float c, float d) {
  if constexpr (FMT == HDP_CACHE_INT8) {
    const uint32_t ab = __byte_perm(__float_as_uint(a + 12582912.f), __float_as_uint(b + 12582912.f), 0x0040);
    const uint32_t cd = __byte_perm(__float_as_uint(c + 12582912.f), __float_as_uint(d + 12582912.f), 0x0040);
    return __byte_perm(ab, cd, 0x5410);
  } else {
    return __byte_perm(code_pair<FMT>(a, b), code_pair<FMT>(c, d), 0x5410);
  }
}

template <int FMT>
__device__ __forceinline__ float2 value_pair(uint32_t two) {
  if constexpr (FMT == HDP_CACHE_INT8) {
    const uint32_t u = two ^ 0x8080u;  // code + 128; 0x4b000000 | u is 2^23 + u
    return make_float2(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440)) - 8388736.f,
                       __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7441)) - 8388736.f);
  } else {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two & 0xffff), __NV_E4M3);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
  }
}

// Four codes at a new scale (`ratio` = old scale / new scale).
template <int FMT>
__device__ __forceinline__ uint32_t rescale4(uint32_t x, float ratio) {
  const float2 a = value_pair<FMT>(x), b = value_pair<FMT>(x >> 16);
  return code_quad<FMT>(a.x * ratio, a.y * ratio, b.x * ratio, b.y * ratio);
}

// Exponent of the smallest power of two 2^e, e >= -126, with |x| <= M 2^e, for
// the bf16 bits of |x|: M is 1.984375 * 2^6 (int8) or 1.75 * 2^8 (e4m3).
template <int FMT>
__device__ __forceinline__ int scale_exponent(uint32_t abs_bits) {
  const int x = static_cast<int>(abs_bits >> 7) - 127, m = abs_bits & 0x7f;
  const int e = FMT == HDP_CACHE_INT8 ? x - 6 + (m > 0x7e) : x - 8 + (m > 0x60);
  return max(e, -126);
}

// x * unit (a power of two) to the whole number below and above.  The product is exact
// but where it is below fp32's range; rounded outwards there too, it keeps its side
// of zero, so that rounding nests (bounds depend on the rows alone).
__device__ __forceinline__ float below(float x, float unit) { return floorf(__fmul_rd(x, unit)); }
__device__ __forceinline__ float above(float x, float unit) { return ceilf(__fmul_ru(x, unit)); }

__device__ __forceinline__ __nv_bfloat162 as_bf2(uint32_t x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); }
__device__ __forceinline__ uint32_t bits(__nv_bfloat162 x) { return *reinterpret_cast<const uint32_t*>(&x); }
__device__ __forceinline__ float bf_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// Words of byte x of each of four words: (a.x, b.x, c.x, d.x) for x = 0..3.
__device__ __forceinline__ void transpose4(uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t (&t)[4]) {
  const uint32_t ab0 = __byte_perm(a, b, 0x5140), ab1 = __byte_perm(a, b, 0x7362);
  const uint32_t cd0 = __byte_perm(c, d, 0x5140), cd1 = __byte_perm(c, d, 0x7362);
  t[0] = __byte_perm(ab0, cd0, 0x5410);
  t[1] = __byte_perm(ab0, cd0, 0x7632);
  t[2] = __byte_perm(ab1, cd1, 0x5410);
  t[3] = __byte_perm(ab1, cd1, 0x7632);
}

// Where a thread's rows and channels lie: pass p of a thread has 8 channels of
// token
//   d = 128: 8 p + 2 c + e
//   d =  64: 16 p + 8 h + 2 c + e
// of the block, so 2 or 4 lanes have exactly the tokens of V chunk c.  With
// d = 128, either 16 lanes have a row (WIDE, c = warp: whole rows), or 8 have
// half of one and the next lanes the chunk beside it (whole 32-byte sectors of V).
template <int D, bool WIDE>
struct Place {
  static constexpr int kLanes = D == 128 && WIDE ? 16 : 8;  // lanes of a row
  int c, e, h, ch;
  __device__ __forceinline__ Place() {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    e = lane / kLanes & 1;
    h = D == 64 ? lane >> 4 : 0;
    c = D == 64 || WIDE ? warp : 2 * (warp & 1) + (lane >> 4);
    ch = lane % kLanes * 8 + (D == 64 || WIDE ? 0 : (warp >> 1) * 64);
  }
  __device__ __forceinline__ int token(int p) const { return D == 128 ? 8 * p + 2 * c + e : 16 * p + 8 * h + 2 * c + e; }
  // Byte of token(p) inside a channel's 64 bytes of V.
  __device__ __forceinline__ int v_byte(int p) const {
    const int j = D == 128 ? p >> 1 : p, hh = D == 128 ? p & 1 : h;
    return 16 * c + 4 * j + 2 * hh + e;
  }
};

// Row-wise codes w[p][2] (8 channels of token(p)) to whole 16-byte chunks of
// channels (out[x] belongs to channel v_channel(x)) and back.
template <int D, bool W>
__device__ __forceinline__ void to_chunks(const Place<D, W>& pl, const uint32_t (&w)[D / 16][2],
                                          uint32_t (&out)[D / 32][4]) {
  constexpr int P = D / 16;
  uint32_t lo[P], hi[P];  // of this lane's four channels: tokens with e = 0 and e = 1
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const uint32_t mine = pl.e ? w[p][1] : w[p][0];
    const uint32_t got = __shfl_xor_sync(0xffffffffu, pl.e ? w[p][0] : w[p][1], Place<D, W>::kLanes);
    lo[p] = pl.e ? got : mine;
    hi[p] = pl.e ? mine : got;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t t[4];
    if constexpr (D == 128) {
      transpose4(lo[2 * j], hi[2 * j], lo[2 * j + 1], hi[2 * j + 1], t);
#pragma unroll
      for (int x = 0; x < 4; ++x) out[x][j] = t[x];
    } else {
      const uint32_t lo2 = __shfl_xor_sync(0xffffffffu, lo[j], 16), hi2 = __shfl_xor_sync(0xffffffffu, hi[j], 16);
      if (pl.h) transpose4(lo2, hi2, lo[j], hi[j], t);
      else transpose4(lo[j], hi[j], lo2, hi2, t);
#pragma unroll
      for (int x = 0; x < 2; ++x) out[x][j] = pl.h ? t[2 + x] : t[x];
    }
  }
}

template <int D, bool W>
__device__ __forceinline__ int v_channel(const Place<D, W>& pl, int x) {
  return pl.ch + 4 * pl.e + (D == 64 ? 2 * pl.h : 0) + x;
}

template <int D, bool W>
__device__ __forceinline__ void from_chunks(const Place<D, W>& pl, const uint32_t (&in)[D / 32][4],
                                            uint32_t (&w)[D / 16][2]) {
  constexpr int P = D / 16;
  uint32_t lo[P], hi[P];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t t[4];
    if constexpr (D == 128) {
      transpose4(in[0][j], in[1][j], in[2][j], in[3][j], t);  // its own inverse
      lo[2 * j] = t[0];
      hi[2 * j] = t[1];
      lo[2 * j + 1] = t[2];
      hi[2 * j + 1] = t[3];
    } else {
      const uint32_t a = __shfl_xor_sync(0xffffffffu, in[0][j], 16), b = __shfl_xor_sync(0xffffffffu, in[1][j], 16);
      if (pl.h) transpose4(a, b, in[0][j], in[1][j], t);
      else transpose4(in[0][j], in[1][j], a, b, t);
      lo[j] = pl.h ? t[2] : t[0];
      hi[j] = pl.h ? t[3] : t[1];
    }
  }
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const uint32_t mine = pl.e ? hi[p] : lo[p];
    const uint32_t got = __shfl_xor_sync(0xffffffffu, pl.e ? lo[p] : hi[p], Place<D, W>::kLanes);
    w[p][0] = pl.e ? got : mine;
    w[p][1] = pl.e ? mine : got;
  }
}

// The new K rows (W = 0) or V rows (W = 1) of one (block, kv head).
template <int D, int FMT, int W>
__device__ __forceinline__ void append_rows(const CacheView& c, const Touched& t, int page, int head,
                                            const uint4* __restrict__ rows) {
  constexpr int P = D / 16;
  using Pl = Place<D, W == 0>;
  __shared__ uint32_t s_amax[4];
  __shared__ __align__(16) __nv_bfloat16 s_bound[W == 0 ? 4 : 1][2][D];
  const Pl pl;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t ph = static_cast<size_t>(page) * c.hkv + head;
  uint4 x[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int r = pl.token(p) - t.first;
    const size_t at = ((static_cast<size_t>(t.row) + r) * c.hkv + head) * (D / 8) + pl.ch / 8;
    x[p] = r >= 0 && r < t.count ? __ldg(rows + at) : make_uint4(0, 0, 0, 0);
  }
  const float before = t.fresh ? 0.f : c.scales[2 * ph + W];

  // Largest magnitudes, as bf16 bits: their order is the values' order, with
  // infinity and NaN (>= 0x7f80) on top.  K takes them from the channel-wise
  // minimum and maximum, which keep a NaN.
  uint32_t m = 0;
  if constexpr (W == 0) {
    const __nv_bfloat162 inf = __halves2bfloat162(__ushort_as_bfloat16(0x7f80), __ushort_as_bfloat16(0x7f80));
    __nv_bfloat162 lo[4] = {inf, inf, inf, inf}, hi[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) hi[i] = __hneg2(inf);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int r = pl.token(p) - t.first;
      if (r >= 0 && r < t.count) {
        const uint32_t q[4] = {x[p].x, x[p].y, x[p].z, x[p].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          lo[i] = __hmin2_nan(lo[i], as_bf2(q[i]));
          hi[i] = __hmax2_nan(hi[i], as_bf2(q[i]));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int o = Pl::kLanes; o < 32; o *= 2) {
        lo[i] = __hmin2_nan(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], o));
        hi[i] = __hmax2_nan(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], o));
      }
      // a warp may have no row at all: +inf and -inf say nothing then
      if (__hgt2_mask(lo[i], hi[i]) == 0u) m = __vmaxu2(m, __vmaxu2(bits(lo[i]) & 0x7fff7fffu, bits(hi[i]) & 0x7fff7fffu));
    }
    if (lane < Pl::kLanes) {
      *reinterpret_cast<uint4*>(&s_bound[warp][0][pl.ch]) = make_uint4(bits(lo[0]), bits(lo[1]), bits(lo[2]), bits(lo[3]));
      *reinterpret_cast<uint4*>(&s_bound[warp][1][pl.ch]) = make_uint4(bits(hi[0]), bits(hi[1]), bits(hi[2]), bits(hi[3]));
    }
  } else {
#pragma unroll
    for (int p = 0; p < P; ++p)
      m = __vmaxu2(m, __vmaxu2(__vmaxu2(x[p].x & 0x7fff7fffu, x[p].y & 0x7fff7fffu),
                               __vmaxu2(x[p].z & 0x7fff7fffu, x[p].w & 0x7fff7fffu)));
  }
  uint32_t top = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
  if (lane == 0) s_amax[warp] = top;
  __syncthreads();

  top = max(max(s_amax[0], s_amax[1]), max(s_amax[2], s_amax[3]));
  const bool lost = top >= 0x7f80u || before != before;
  const float scale = lost ? __int_as_float(0x7fc00000) : fmaxf(pow2i(scale_exponent<FMT>(top)), before);
  // 1 / scale: the scale is a power of two, so its exponent changes sign
  const float inv = lost ? 1.f : __int_as_float((254 << 23) - __float_as_int(scale));
  const bool grown = !t.fresh && !lost && scale != before;
  const float ratio = grown ? before * inv : 1.f;

  uint8_t* block = (W ? c.v : c.k) + ph * (kBlock * D);
  // A larger scale: the codes that are there are rounded to it (every byte of
  // the block is one, written or zero).
  if (grown) {
    uint4* b = reinterpret_cast<uint4*>(block);
    for (int i = threadIdx.x; i < kBlock * D / 16; i += kThreads) {
      uint4 y = b[i];
      y.x = rescale4<FMT>(y.x, ratio);
      y.y = rescale4<FMT>(y.y, ratio);
      y.z = rescale4<FMT>(y.z, ratio);
      y.w = rescale4<FMT>(y.w, ratio);
      b[i] = y;
    }
    __syncthreads();  // the new rows go over them
  }

  uint32_t code[P][2];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const uint4 y = x[p];
    code[p][0] = code_quad<FMT>(bf_lo(y.x) * inv, bf_hi(y.x) * inv, bf_lo(y.y) * inv, bf_hi(y.y) * inv);
    code[p][1] = code_quad<FMT>(bf_lo(y.z) * inv, bf_hi(y.z) * inv, bf_lo(y.w) * inv, bf_hi(y.w) * inv);
  }
  if constexpr (W == 0) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int r = pl.token(p) - t.first;
      if (t.fresh || (r >= 0 && r < t.count))
        *reinterpret_cast<uint2*>(block + pl.token(p) * D + pl.ch) = make_uint2(code[p][0], code[p][1]);
    }
    // Bounds, in whole units (one K scale, four for e4m3): rounding outwards
    // nests, so a change of unit loses nothing but the finer grid.
    if (threadIdx.x < D) {
      const int i = threadIdx.x;
      const float unit = FMT == HDP_CACHE_INT8 ? inv : inv * 0.25f;
      const __nv_bfloat16 lo = __hmin(__hmin(s_bound[0][0][i], s_bound[1][0][i]), __hmin(s_bound[2][0][i], s_bound[3][0][i]));
      const __nv_bfloat16 hi = __hmax(__hmax(s_bound[0][1][i], s_bound[1][1][i]), __hmax(s_bound[2][1][i], s_bound[3][1][i]));
      float a = below(__bfloat162float(lo), unit), b = above(__bfloat162float(hi), unit);
      int8_t* out = c.bounds + ph * (2 * D) + i;
      if (!t.fresh) {
        // before * inv alone may be below fp32's range
        a = fminf(a, below(static_cast<float>(out[0]) * before, inv));
        b = fmaxf(b, above(static_cast<float>(out[D]) * before, inv));
      }
      out[0] = static_cast<int8_t>(fminf(fmaxf(a, -127.f), 127.f));
      out[D] = static_cast<int8_t>(fminf(fmaxf(b, -127.f), 127.f));
    }
  } else if (t.fresh) {
    uint32_t chunk[D / 32][4];
    to_chunks(pl, code, chunk);
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
      *reinterpret_cast<uint4*>(block + v_channel(pl, i) * kBlock + pl.c * 16) =
          make_uint4(chunk[i][0], chunk[i][1], chunk[i][2], chunk[i][3]);
  } else {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int r = pl.token(p) - t.first;
      if (r >= 0 && r < t.count) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          block[(pl.ch + i) * kBlock + pl.v_byte(p)] = static_cast<uint8_t>(code[p][i >> 2] >> (8 * (i & 3)));
      }
    }
  }
  if (threadIdx.x == 0) c.scales[2 * ph + W] = scale;
}

// K, then V: one of them in registers at a time leaves room for 7 CTAs an SM (83K
// prompt tokens, 8 heads of 128, int8: 85 us; both at once 93, a CTA for each 91).
template <int D, int FMT>
__global__ void __launch_bounds__(kThreads) k_cache_append(CacheView c, const uint4* __restrict__ k,
                                                           const uint4* __restrict__ v) {
  Touched t;
  if (!touched_block(c, blockIdx.x, t)) return;
  const int page = page_of(c, t.seq, t.block);
  if (page < 0) return;
  append_rows<D, FMT, 0>(c, t, page, blockIdx.y, k);
  append_rows<D, FMT, 1>(c, t, page, blockIdx.y, v);
}

// One token for each sequence.
template <int D, int FMT>
__global__ void __launch_bounds__(kThreads) k_cache_append_one(CacheView c, const uint4* __restrict__ k,
                                                               const uint4* __restrict__ v) {
  constexpr int kRow = D / 8;  // lanes of a row: K in the first, V in the next
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long unit = static_cast<long long>(blockIdx.x) * (kThreads / 32) + warp;
  if (unit >= static_cast<long long>(c.num_seqs) * c.hkv) return;
  const int seq = static_cast<int>(unit / c.hkv), head = static_cast<int>(unit - static_cast<long long>(seq) * c.hkv);
  const int w = lane / kRow, ch = lane % kRow * 8;
  const bool on = w < 2;
  uint4 x = make_uint4(0, 0, 0, 0);
  if (on) x = __ldg((w ? v : k) + static_cast<size_t>(unit) * kRow + ch / 8);
  const long long p0 = seq_len(c, seq) - 1;
  if (p0 < 0) return;
  const int page = page_of(c, seq, static_cast<int>(p0 / kBlock)), t = static_cast<int>(p0 % kBlock);
  if (page < 0) return;
  const size_t ph = static_cast<size_t>(page) * c.hkv + head;
  const bool fresh = t == 0;
  uint8_t* codes = (w == 1 ? c.v : c.k) + ph * (kBlock * D);
  int8_t* bounds = c.bounds + ph * (2 * D) + ch;
  float before = 0.f;
  uint2 blo = make_uint2(0, 0), bhi = blo;
  if (!fresh && on) {
    before = c.scales[2 * ph + w];
    if (w == 0) {
      blo = *reinterpret_cast<const uint2*>(bounds);
      bhi = *reinterpret_cast<const uint2*>(bounds + D);
    }
  }
  const uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
  uint32_t top = max(m & 0xffffu, m >> 16);
#pragma unroll
  for (int o = 1; o < kRow; o *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  const bool lost = top >= 0x7f80u || before != before;
  const float scale = lost ? __int_as_float(0x7fc00000) : fmaxf(pow2i(scale_exponent<FMT>(top)), before);
  const float inv = lost ? 1.f : __int_as_float((254 << 23) - __float_as_int(scale));
  const bool grown = !fresh && !lost && scale != before;
  const float ratio = grown ? before * inv : 1.f;

  // The block begins: zero codes; or its scale grows: its codes rounded to it.
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const bool grows = __shfl_sync(0xffffffffu, static_cast<int>(grown), side * kRow) != 0;
    const float r = __shfl_sync(0xffffffffu, ratio, side * kRow);
    if (!fresh && !grows) continue;
    uint4* b = reinterpret_cast<uint4*>((side ? c.v : c.k) + ph * (kBlock * D));
#pragma unroll 4
    for (int i = lane; i < kBlock * D / 16; i += 32) {
      uint4 y = make_uint4(0, 0, 0, 0);
      if (!fresh) {
        y = b[i];
        y.x = rescale4<FMT>(y.x, r);
        y.y = rescale4<FMT>(y.y, r);
        y.z = rescale4<FMT>(y.z, r);
        y.w = rescale4<FMT>(y.w, r);
      }
      b[i] = y;
    }
  }
  __syncwarp();  // the new row goes over them
  if (!on) return;
  const float f[8] = {bf_lo(x.x), bf_hi(x.x), bf_lo(x.y), bf_hi(x.y), bf_lo(x.z), bf_hi(x.z), bf_lo(x.w), bf_hi(x.w)};
  const uint2 code = make_uint2(code_quad<FMT>(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                                code_quad<FMT>(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
  if (w == 0) {
    *reinterpret_cast<uint2*>(codes + t * D + ch) = code;
    const float unit_inv = FMT == HDP_CACHE_INT8 ? inv : inv * 0.25f;
    int8_t lo[8], hi[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float a = below(f[i], unit_inv), b = above(f[i], unit_inv);
      if (!fresh) {
        const uint32_t ol = (i < 4 ? blo.x : blo.y) >> (8 * (i & 3)), oh = (i < 4 ? bhi.x : bhi.y) >> (8 * (i & 3));
        a = fminf(a, below(static_cast<float>(static_cast<int8_t>(ol & 0xff)) * before, inv));
        b = fmaxf(b, above(static_cast<float>(static_cast<int8_t>(oh & 0xff)) * before, inv));
      }
      lo[i] = static_cast<int8_t>(fminf(fmaxf(a, -127.f), 127.f));
      hi[i] = static_cast<int8_t>(fminf(fmaxf(b, -127.f), 127.f));
    }
    uint2 pl, ph2;
    memcpy(&pl, lo, 8);
    memcpy(&ph2, hi, 8);
    *reinterpret_cast<uint2*>(bounds) = pl;
    *reinterpret_cast<uint2*>(bounds + D) = ph2;
  } else {
    const int byte = 16 * (t / 2 % 4) + 4 * (t / 16) + 2 * (t / 8 % 2) + t % 2;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      codes[(ch + i) * kBlock + byte] = static_cast<uint8_t>((i < 4 ? code.x : code.y) >> (8 * (i & 3)));
  }
  if (ch == 0) c.scales[2 * ph + w] = scale;
}

template <int FMT>
__device__ __forceinline__ uint32_t bf16_pair(uint32_t two, float s) {
  const float2 a = value_pair<FMT>(two);
  const __nv_bfloat162 r = __floats2bfloat162_rn(a.x * s, a.y * s);  // exact: 7 significant bits
  return *reinterpret_cast<const uint32_t*>(&r);
}

template <int D, int FMT>
__global__ void __launch_bounds__(kThreads) k_cache_read(CacheView c, uint4* __restrict__ k, uint4* __restrict__ v) {
  constexpr int P = D / 16;
  Touched t;
  const bool any = touched_block(c, blockIdx.x, t);
  const int head = blockIdx.y;
  for (long long i = threadIdx.x; i < t.before * (D / 8); i += kThreads) {  // negative positions: zeros
    const size_t at = (static_cast<size_t>(t.row0 + i / (D / 8)) * c.hkv + head) * (D / 8) + i % (D / 8);
    k[at] = v[at] = make_uint4(0, 0, 0, 0);
  }
  if (!any) return;
  const int page = page_of(c, t.seq, t.block);
  const Place<D, true> pl;
  uint32_t code[2][P][2] = {};
  float2 scale = make_float2(0.f, 0.f);
  if (page >= 0) {
    const size_t ph = static_cast<size_t>(page) * c.hkv + head;
    const uint8_t* kb = c.k + ph * (kBlock * D);
    const uint8_t* vb = c.v + ph * (kBlock * D);
    uint32_t chunk[D / 32][4];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint4 y = __ldg(reinterpret_cast<const uint4*>(vb + v_channel(pl, i) * kBlock + pl.c * 16));
      chunk[i][0] = y.x;
      chunk[i][1] = y.y;
      chunk[i][2] = y.z;
      chunk[i][3] = y.w;
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int r = pl.token(p) - t.first;
      if (r >= 0 && r < t.count) {
        const uint2 y = __ldg(reinterpret_cast<const uint2*>(kb + pl.token(p) * D + pl.ch));
        code[0][p][0] = y.x;
        code[0][p][1] = y.y;
      }
    }
    scale = __ldg(reinterpret_cast<const float2*>(c.scales + 2 * ph));
    from_chunks(pl, chunk, code[1]);
  }
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const float s = w ? scale.y : scale.x;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int r = pl.token(p) - t.first;
      if (r < 0 || r >= t.count) continue;
      const size_t at = ((static_cast<size_t>(t.row) + r) * c.hkv + head) * (D / 8) + pl.ch / 8;
      const uint32_t* y = code[w][p];
      (w ? v : k)[at] = make_uint4(bf16_pair<FMT>(y[0], s), bf16_pair<FMT>(y[0] >> 16, s), bf16_pair<FMT>(y[1], s),
                                   bf16_pair<FMT>(y[1] >> 16, s));
    }
  }
}

hdp_status_t check_rows(const char* call, const void* k, const void* v, int64_t rows) {
  if (rows > 0 && (!k || !v)) return fail(HDP_ERR_INVALID_ARGUMENT, std::string(call) + ": k or v is NULL");
  if ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15)
    return fail(HDP_ERR_INVALID_ARGUMENT, std::string(call) + ": k and v must be 16-byte aligned");
  return HDP_OK;
}

// CTAs in x: a slot for every block that the call may touch (below 2^25 + 2^25).
dim3 slot_grid(const CacheView& c) {
  const long long slots = c.cu ? c.rows / kBlock + 2LL * c.num_seqs : c.num_seqs;
  return dim3(static_cast<unsigned>(slots), c.hkv);
}

}  // namespace
}  // namespace hdp

using namespace hdp;

#define HDP_TRY(expr)                    \
  do {                                   \
    const hdp_status_t s_ = (expr);      \
    if (s_ != HDP_OK) return s_;         \
  } while (0)

extern "C" hdp_status_t hdp_cache_append(const hdp_cache_t* cache, const int32_t* cu, int64_t rows, const void* k,
                                         const void* v, void* stream) {
  CacheView c;
  HDP_TRY(cache_view("hdp_cache_append", cache, cu, rows, &c));
  HDP_TRY(check_rows("hdp_cache_append", k, v, rows));
  if (rows == 0) return HDP_OK;
  c.err = device_error_word();
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 g = slot_grid(c);
  const uint4* kp = static_cast<const uint4*>(k);
  const uint4* vp = static_cast<const uint4*>(v);
  const bool i8 = cache->format == HDP_CACHE_INT8;
  const bool one = !cu;
  // one token for each sequence: a warp for each (sequence, kv head), at most 2^24 * 65535 / 4 CTAs
  const int64_t ones = (int64_t(c.num_seqs) * c.hkv + kThreads / 32 - 1) / (kThreads / 32);
  if (one && ones > 2147483647LL) return fail(HDP_ERR_UNSUPPORTED, "hdp_cache_append: num_seqs * hkv must be below 2^33");
  const dim3 grid = one ? dim3(static_cast<unsigned>(ones)) : g;
  void (*kernel)(CacheView, const uint4*, const uint4*);
  if (cache->d == 128) {
    if (one) kernel = i8 ? k_cache_append_one<128, HDP_CACHE_INT8> : k_cache_append_one<128, HDP_CACHE_E4M3>;
    else kernel = i8 ? k_cache_append<128, HDP_CACHE_INT8> : k_cache_append<128, HDP_CACHE_E4M3>;
  } else {
    if (one) kernel = i8 ? k_cache_append_one<64, HDP_CACHE_INT8> : k_cache_append_one<64, HDP_CACHE_E4M3>;
    else kernel = i8 ? k_cache_append<64, HDP_CACHE_INT8> : k_cache_append<64, HDP_CACHE_E4M3>;
  }
  kernel<<<grid, kThreads, 0, st>>>(c, kp, vp);
  note_launch();
  HDP_CUDA_TRY(cudaGetLastError());
  return HDP_OK;
}

extern "C" hdp_status_t hdp_cache_read(const hdp_cache_t* cache, const int32_t* cu, int64_t rows, void* k, void* v,
                                       void* stream) {
  CacheView c;
  HDP_TRY(cache_view("hdp_cache_read", cache, cu, rows, &c));
  HDP_TRY(check_rows("hdp_cache_read", k, v, rows));
  if (rows == 0) return HDP_OK;
  c.err = device_error_word();
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 g = slot_grid(c);
  uint4* kp = static_cast<uint4*>(k);
  uint4* vp = static_cast<uint4*>(v);
  const bool i8 = cache->format == HDP_CACHE_INT8;
  if (cache->d == 128) {
    if (i8) k_cache_read<128, HDP_CACHE_INT8><<<g, kThreads, 0, st>>>(c, kp, vp);
    else k_cache_read<128, HDP_CACHE_E4M3><<<g, kThreads, 0, st>>>(c, kp, vp);
  } else {
    if (i8) k_cache_read<64, HDP_CACHE_INT8><<<g, kThreads, 0, st>>>(c, kp, vp);
    else k_cache_read<64, HDP_CACHE_E4M3><<<g, kThreads, 0, st>>>(c, kp, vp);
  }
  note_launch();
  HDP_CUDA_TRY(cudaGetLastError());
  return HDP_OK;
}
