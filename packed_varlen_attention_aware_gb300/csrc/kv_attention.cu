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

template <int D, int FMT>
struct Codes8 {
  static constexpr int kD = D;
  static constexpr int kSlot = kBlock * D;       // bytes of a block's K or V codes of one head
  static constexpr int kKeyChunks = D / 64;      // 16-byte chunks that a lane has of a key
  template <int NT, bool SPARSE>
  static constexpr int kSlots = kRingBytes<NT, SPARSE> / kSlot;
  static constexpr float kEnough = hdp::kEnough<FMT>;

  template <int NT>
  __device__ __forceinline__ static void fetch_rows(const AttnParams& p, int row0, int head, unsigned rr0, int nrows,
                                                    uint4 (&qx)[NT][D / 32]) {
    hdp::fetch_rows<D, NT>(p, row0, head, rr0, nrows, qx);
  }
  __device__ __forceinline__ static void copy_k(const AttnParams& p, size_t ph, uint32_t dst, Meta* meta) {
    const int lane = threadIdx.x & 31, gr = lane >> 2, tc = lane & 3;
    if (lane == 0) copy8(smem_addr(meta), p.c.scales + 2 * ph);
    const unsigned char* kb = p.c.k + ph * kSlot + gr * D + tc * 16;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < kKeyChunks; ++j) copy16(dst + (i * kKeyChunks + j) * 512, kb + i * 8 * D + j * 64);
  }
  __device__ __forceinline__ static const unsigned char* v_of(const AttnParams& p, size_t ph) {
    return p.c.v + ph * kSlot + (threadIdx.x & 31) * 16;
  }
  __device__ __forceinline__ static void copy_v(const unsigned char* v, uint32_t dst) {
#pragma unroll
    for (int i = 0; i < D / 8; ++i) copy16(dst + i * 512, v + i * 512);
  }
  template <int NT>
  __device__ __forceinline__ static void scores(const Rows<D, NT>& rows, Sums<D, NT>& sums, const unsigned char* slot,
                                                const Meta& meta, bool masked, const Probabilities<NT>& prob,
                                                float (&f)[NT][2]) {
    const uint4* kx = reinterpret_cast<const uint4*>(slot) + (threadIdx.x & 31);
    float s[NT][4][4];
    first_product<D, FMT, NT>(rows, s, [&](int i, int j) { return kx[(i * kKeyChunks + j) * 32]; });
    softmax<D, NT>(rows, sums, meta.sk, meta.sv, meta.key0, masked, s, f);
    prob.put(s);
  }
  template <int NT>
  __device__ __forceinline__ static void output(Sums<D, NT>& sums, const uint32_t (&pf)[NT][4][2], const float (&f)[NT][2],
                                                const unsigned char* slot, bool masked, float (&least)[NT][2]) {
    const uint4* vx = reinterpret_cast<const uint4*>(slot) + (threadIdx.x & 31);
    second_product<D, FMT, NT>(sums, pf, f, masked, least, [&](int i) { return vx[i * 32]; });
  }
};

template <class F>
hdp_status_t launch_for(const AttnParams& p, int nt, int device, int ctas, cudaStream_t st) {
  if (p.blocks) return nt == 1 ? launch<F, 1, true>(p, device, ctas, st) : launch<F, 2, true>(p, device, ctas, st);
  return nt == 1 ? launch<F, 1, false>(p, device, ctas, st) : launch<F, 2, false>(p, device, ctas, st);
}

}  // namespace
}  // namespace hdp

using namespace hdp;

extern "C" hdp_status_t hdp_cache_attention_workspace_bytes(const hdp_cache_t* cache, int32_t hq, size_t* bytes) {
  if (!cache || !bytes) return fail(HDP_ERR_INVALID_ARGUMENT, "hdp_cache_attention_workspace_bytes: NULL argument");
  return workspace_bytes_of("hdp_cache_attention_workspace_bytes", cache->hkv, cache->d, hq, bytes);
}

extern "C" hdp_status_t hdp_cache_attention(const hdp_cache_t* cache, const int32_t* cu, int64_t rows, const void* q,
                                            int32_t hq, float scale, const int32_t* blocks, int32_t count,
                                            void* workspace, size_t workspace_bytes, void* o, float* lse,
                                            void* stream) {
  AttnParams p = {};
  const hdp_status_t r = cache_view("hdp_cache_attention", cache, cu, rows, &p.c);
  if (r != HDP_OK) return r;
  const bool i8 = cache->format == HDP_CACHE_INT8, wide = cache->d == 128;
  return attend("hdp_cache_attention", p, cache->d, rows, q, hq, scale, blocks, count, workspace, workspace_bytes, o, lse,
                stream, [=](const AttnParams& a, int nt, int device, int ctas, cudaStream_t st) {
                  if (wide)
                    return i8 ? launch_for<Codes8<128, HDP_CACHE_INT8>>(a, nt, device, ctas, st)
                              : launch_for<Codes8<128, HDP_CACHE_E4M3>>(a, nt, device, ctas, st);
                  return i8 ? launch_for<Codes8<64, HDP_CACHE_INT8>>(a, nt, device, ctas, st)
                            : launch_for<Codes8<64, HDP_CACHE_E4M3>>(a, nt, device, ctas, st);
                });
}
