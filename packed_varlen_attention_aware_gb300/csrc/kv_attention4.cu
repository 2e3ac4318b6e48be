// Attention of the newest tokens of each sequence over the 4-bit cache.
//
// How the work is cut, handed out and joined, and what carries the softmax over scores
// and V scales of any size, is the 8-bit cache's (kv_attention.cu).  Here are a block's
// products.  A key and kv head is d + d / 32 + 1 bytes, half of the 8-bit cache's, so the
// same memory rate leaves half the time for each, and instructions bound the loop, not
// bytes: on this GPU an m16n8k16 product takes a scheduler 8.3 cycles, and conversions and
// multiply-adds between products add a cycle each rather than hide behind them (measured
// in isolation), so the 64 products and 256 conversions of a block are 800 cycles of the
// 1,450 that HBM takes for it.
//
//   Codes.  e2m1 is exact in fp16, and the conversion instruction takes a byte: one
//   for two codes, where the 8-bit kinds need four and seven cycles for as many.  The
//   cache's order of bytes is the fragments': K's words have one group of 32 channels
//   each, so the two products of a group share an accumulator.
//   Scales of K.  A group's sum is multiplied by its scale in fp32 and added to the
//   score's: no rounding of a code to a scaled one.  Where that passes fp32's end and a
//   scale is 2^65 or more, the block is computed again with all scales 2^-32 times as
//   large and the score back up behind the row's factor, so that only scores beyond
//   fp32's end pass it; what the smallest scales lose by that is below such a score's
//   last bit.
//   Scales of V go into P, as powers of two relative to the output's reference.
//   References.  Where every P of a block, under the references that the sums have, is a
//   normal number of fp16 (2^-14 to 2^15), it stays under them: nothing is rescaled, no
//   product can lose a small P, and the second product adds to the output in place.
//   Fresh references are 4 bits above what needs them, so that is all but the first blocks
//   of a run unless a block's scores are spread over more than 17 nats.  Else P is taken
//   from the block's own largest, the sums come to new references, and what fp16 leaves of
//   P takes further passes where an output is small enough for it to count, as in the
//   8-bit kernel.
#include "kv_attention.cuh"
#include "kv_cache4.cuh"

namespace hdp {
namespace {

// Eight codes to fp16, a byte's two to a register.
__device__ __forceinline__ void decode8(uint32_t x, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(x));
}

// A lane's scales of one group: of its keys 8 j + gr, byte j.
__device__ __forceinline__ uint32_t scale_word(const uint2& x, int j) { return j < 4 ? x.x : x.y; }
// 2^(byte j - 127)
__device__ __forceinline__ float scale_at(const uint2& x, int j) {
  const uint32_t w = scale_word(x, j);
  const int b = j & 3;
  return __uint_as_float((b == 3 ? w >> 1 : w << (23 - 8 * b)) & 0x7f800000u);
}
// 2^23 + byte j: 8388735 more than its exponent
__device__ __forceinline__ float exponent_bits(const uint2& x, int j) {
  return __uint_as_float(__byte_perm(scale_word(x, j), 0x4b000000u, 0x7650 + (j & 3)));
}
// Of bytes: the top bit of those that are 192 (2^65) or more, of those that are 255.
__device__ __forceinline__ uint32_t large_bytes(uint32_t w) { return w & (w << 1); }
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & w & 0x80808080u; }

// Bytes of a block whose scales go up to 2^126, times 2^-32; bit j of the result: some
// scale of key j is NaN.
template <int G>
__device__ __forceinline__ uint32_t lower_scales(uint2 (&ks)[G]) {
  uint32_t lost = 0;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    uint32_t w[2] = {ks[g].x, ks[g].y};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t y = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const uint32_t e = w[h] >> (8 * b) & 0xffu;
        if (e == 255) lost |= 1u << (4 * h + b);
        y |= (e > 32 ? e - 32 : 0) << (8 * b);
      }
      w[h] = y;
    }
    ks[g] = make_uint2(w[0], w[1]);
  }
  return lost;
}

// Warps of a CTA for one tile of query rows and for two.
constexpr int kWarpsOf[kMaxNt] = {8, 8};

constexpr float kHeadroom = 4.f;    // bits of a fresh reference above what needs it
constexpr float kCommon = 8.f;      // most bits that an output's reference is raised to be its neighbours', or above a V scale
// What fp16 leaves of a block's P is at most 64 * 2^-25 times its largest code, 6; 2^12 times that.
constexpr float kEnough4 = 0.0625f;

// A block's place in the ring: codes of K, scales, codes of V.
template <int D>
constexpr int kBlock4 = 2 * kCodes4<D> + kScales4<D>;

template <int D, int NT>
struct Shared4 {
  static constexpr int kWarps = kWarpsOf[NT - 1];
  // P of a block on its way round takes the place of the codes of K, if it fits.
  static constexpr bool kOwnP = NT * 2048 > kCodes4<D>;
  static constexpr int kSlots = D == 128 ? 3 : kOwnP ? 5 : 6;
  unsigned char ring[kWarps][kSlots][kBlock4<D>];
  float4 p[kOwnP ? kWarps : 1][NT][4][32];
  SeqPlace seq[kSeqs];
  int piece[kWarps][kSlots];
  long long pre[kWarps * 32];  // steps before each thread's sequences
  long long warp_sum[kWarps];
};

// Query rows of a unit: of each group of channels this lane's 8.
template <int D, int NT>
__device__ __forceinline__ void fetch_rows(const AttnParams& p, int row0, int head, unsigned rr0, int nrows,
                                           uint4 (&qx)[NT][D / 32]) {
  const int lane = threadIdx.x & 31, gr = lane >> 2, tc = lane & 3;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int r = t * 8 + gr;
#pragma unroll
    for (int g = 0; g < D / 32; ++g) qx[t][g] = make_uint4(0, 0, 0, 0);
    if (r < nrows) {
      const unsigned token = (rr0 + r) / p.g;
      const uint4* src = reinterpret_cast<const uint4*>(
          p.q + (static_cast<long long>(row0 + token) * p.hq + head * p.g + (rr0 + r - token * p.g)) * D + tc * 8);
#pragma unroll
      for (int g = 0; g < D / 32; ++g) qx[t][g] = __ldg(src + g * 4);
    }
  }
}

// Words of a key's codes, one for each group.
template <int D>
__device__ __forceinline__ void key_words(const unsigned char* slot, int lane, int j, uint32_t (&w)[D / 32]) {
  if constexpr (D == 128) {
    const uint4 x = reinterpret_cast<const uint4*>(slot)[j * 32 + lane];
    w[0] = x.x;
    w[1] = x.y;
    w[2] = x.z;
    w[3] = x.w;
  } else {
    const uint2 x = reinterpret_cast<const uint2*>(slot)[j * 32 + lane];
    w[0] = x.x;
    w[1] = x.y;
  }
}

// S^T = K Q^T, group by group.
template <int D, int NT>
__device__ __forceinline__ void first_product(const Rows<D, NT>& rows, const unsigned char* slot, int lane,
                                              const uint2 (&ks)[D / 32], float (&s)[NT][4][4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t u[D / 32], w[D / 32];
    key_words<D>(slot, lane, 2 * i, u);
    key_words<D>(slot, lane, 2 * i + 1, w);
#pragma unroll
    for (int g = 0; g < D / 32; ++g) {
      uint32_t a[4], b[4];
      decode8(u[g], a);
      decode8(w[g], b);
      const float lo = scale_at(ks[g], 2 * i), hi = scale_at(ks[g], 2 * i + 1);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float y[4];
        mma16816_first(y, a[0], b[0], a[1], b[1], rows.q[t][2 * g][0], rows.q[t][2 * g][1]);
        mma16816(y, a[2], b[2], a[3], b[3], rows.q[t][2 * g + 1][0], rows.q[t][2 * g + 1][1]);
#pragma unroll
        for (int k = 0; k < 4; ++k) s[t][i][k] = g == 0 ? y[k] * (k < 2 ? lo : hi) : fmaf(y[k], k < 2 ? lo : hi, s[t][i][k]);
      }
    }
  }
}

// Y += V^T P^T for the channels 16 i .. 16 i + 16 kTogether - 1; FIRST: there is no sum to add to.
template <bool FIRST, int NT>
__device__ __forceinline__ void second_product(const uint4* vx, int i, const uint32_t (&pf)[NT][4][2],
                                               float (&y)[NT][kTogether][4]) {
  uint4 u[kTogether];
#pragma unroll
  for (int h = 0; h < kTogether; ++h) u[h] = vx[(i + h) * 32];
#pragma unroll
  for (int k = 0; k < 4; k += 2)
#pragma unroll
    for (int h = 0; h < kTogether; ++h) {
      uint32_t a[4], b[4];  // channels 16 i + gr and 8 more: tokens of steps k and k + 1
      decode8(word(u[h], k >> 1), a);
      decode8(word(u[h], 2 + (k >> 1)), b);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (FIRST && k == 0) mma16816_first(y[t][h], a[0], b[0], a[1], b[1], pf[t][k][0], pf[t][k][1]);
        else mma16816(y[t][h], a[0], b[0], a[1], b[1], pf[t][k][0], pf[t][k][1]);
        mma16816(y[t][h], a[2], b[2], a[3], b[3], pf[t][k + 1][0], pf[t][k + 1][1]);
      }
    }
}

// What the outputs of a warp's rows have in common: their distance from the row sums'
// references (Sums::gap), if it is the same for all of them.
struct Common {
  bool any;
  int gap;  // + 127, as a scale's byte; below 0: no block yet
};

// Scores of a block to P under the references that the sums have.  True, and the row sums
// have their share, if every P is a normal number of fp16.
template <int D, int NT>
__device__ __forceinline__ bool as_is(const Rows<D, NT>& rows, Sums<D, NT>& sums, const Common& common,
                                      const unsigned char* scales, int lane, const float (&s)[NT][4][4],
                                      uint32_t (&pf)[NT][4][2]) {
  const uint2 vs = reinterpret_cast<const uint2*>(scales + (D / 32) * kBlock)[lane >> 2];
  // V scales of the block, two a lane: 2^-14 to 1 of the output's reference, as normal numbers of fp16
  const uint32_t two = reinterpret_cast<const uint16_t*>(scales + (D / 32) * kBlock)[lane];
  bool ok = static_cast<uint32_t>(common.gap) - (two & 0xffu) <= 14u && static_cast<uint32_t>(common.gap) - (two >> 8) <= 14u;
  const uint32_t back = (15u - static_cast<uint32_t>(common.gap)) * 0x04000400u;
  float l[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float high = -__int_as_float(0x7f800000);
    __half2 least = __half2half2(__ushort_as_half(0x7c00));
    l[t][0] = l[t][1] = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float e[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float y = fmaf(s[t][j >> 1][k + 2 * (j & 1)], rows.scale[t][k], -sums.m[t][k]);
        high = fmaxf(high, y);
        e[k] = exp2_approx(y);
        l[t][k] += e[k];
      }
      const uint32_t w = __byte_perm(scale_word(vs, j), 0u, 0x4440 + (j & 3)) * 0x04000400u + back;
      const __half2 x = __hmul2(__floats2half2_rn(e[0], e[1]), as_h2(w));
      least = __hmin2(least, x);
      pf[t][j >> 1][j & 1] = h2_bits(x);
    }
    // (a NaN is in the sum, and in neither of the extremes)
    ok = ok && high <= kBias && __hbge2(least, __half2half2(__ushort_as_half(0x0400))) && l[t][0] == l[t][0] && l[t][1] == l[t][1];
  }
  if (!__all_sync(0xffffffffu, ok)) return false;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int k = 0; k < 2; ++k) sums.l[t][k] += l[t][k];
#pragma unroll
    for (int j = 0; j < 8; ++j) pf[t][j >> 1][j & 1] = transpose8x8(pf[t][j >> 1][j & 1]);
  }
  return true;
}

// Brings the sums to references that are kHeadroom above the block's scores and a bit above
// its V scales, where they are not that high already.
template <int D, int NT>
__device__ __forceinline__ void refer(const Rows<D, NT>& rows, Sums<D, NT>& sums, Common& common, const unsigned char* scales,
                                      int lane, const float (&s)[NT][4][4]) {
  const uint32_t two = reinterpret_cast<const uint16_t*>(scales + (D / 32) * kBlock)[lane];
  int above = static_cast<int>(max(two & 0xffu, two >> 8));
  above = __reduce_max_sync(0xffffffffu, above);
  if (above > common.gap) common.gap = above + 1;
  const float gap = static_cast<float>(common.gap - 127);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float top = -__int_as_float(0x7f800000);
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmaxf(top, s[t][j >> 1][k + 2 * (j & 1)] * rows.scale[t][k]);
#pragma unroll
      for (int d = 4; d < 32; d *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      const float c = ceilf(top) - kBias, m = sums.m[t][k];
      const float m1 = c > m && fabsf(c) < kBiasMost ? c + kHeadroom : m;  // (larger ones are not for here)
      const float turn = exp2_approx((m - m1) + (sums.gap[t][k] - gap));
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        sums.acc[t][i][k] *= turn;
        sums.acc[t][i][k + 2] *= turn;
      }
      sums.l[t][k] *= exp2_approx(m - m1);
      sums.m[t][k] = m1;
      sums.gap[t][k] = gap;
    }
}

// Scores of any kind to P from the block's own largest, at most 2^15, in place; brings the
// sums to new references, and f to the power of two (<= 1) of the block in the output.
template <int D, int NT>
__device__ __forceinline__ void softmax(const Rows<D, NT>& rows, Sums<D, NT>& sums, Common& common, const unsigned char* scales,
                                        int key0, bool masked, bool careful, uint32_t lost, float (&s)[NT][4][4],
                                        float (&f)[NT][2]) {
  const float inf = __int_as_float(0x7f800000), nan = __int_as_float(0x7fc00000);
  const int gr = (threadIdx.x & 31) >> 2;
  const uint2 vs = reinterpret_cast<const uint2*>(scales + (D / 32) * kBlock)[gr];
  bool fresh = false;
  float most_gap = -inf;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float top[2] = {-inf, -inf};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float r = rows.scale[t][k & 1], back = 4294967296.f;  // 2^32
        float x = s[t][i][k];
        if (careful) x = x * (r < 1.f ? r : back) * (r < 1.f ? back : r);
        else x *= r;
        if (lost >> (2 * i + (k >> 1)) & 1) x = nan;
        if (masked && key0 + 16 * i + 8 * (k >> 1) + gr > rows.pos[t][k & 1]) x = -inf;
        s[t][i][k] = x;
        top[k & 1] = fmaxf(top[k & 1], x);
      }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int d = 4; d < 32; d *= 2) top[k] = fmaxf(top[k], __shfl_xor_sync(0xffffffffu, top[k], d));
      const bool none = top[k] == -inf;
      float ref = none ? 0.f : ceilf(top[k]);
      const bool biased = fabsf(ref) < kBiasMost;
      if (biased) ref -= kBias;
      // the row sum's share, and the exponents of P with the V scales
      float sum = 0.f, most = -inf;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float& x = s[t][j >> 1][k + 2 * (j & 1)];
        const float y = x - ref;
        sum += exp2_approx(y);
        x = y + (exponent_bits(vs, j) - 8388735.f);
        most = fmaxf(most, x);
      }
#pragma unroll
      for (int d = 4; d < 32; d *= 2) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
      const float e = most == -inf ? 0.f : ceilf(most) - kBias;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[t][i][k] = exp2_approx(s[t][i][k] - e);
        s[t][i][k + 2] = exp2_approx(s[t][i][k + 2] - e);
      }
      const float m = sums.m[t][k], gap = sums.gap[t][k];
      const float m1 = none || ref <= m ? m : ref + (biased ? kHeadroom : 0.f);
      const float down = m - m1, up = none ? -inf : ref - m1;
      const float gap1 = none ? gap : fmaxf(gap + down, up + e);
      fresh |= gap1 > gap + down;
      most_gap = fmaxf(most_gap, gap1);
      sums.l[t][k] = fmaf(sum, exp2_approx(up), sums.l[t][k] * exp2_approx(down));
      f[t][k] = exp2_approx(up + (e - gap1));  // 0 where no key is seen
      const float turn = exp2_approx(down + (gap - gap1));
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        sums.acc[t][i][k] *= turn;
        sums.acc[t][i][k + 2] *= turn;
      }
      sums.m[t][k] = m1;
      sums.gap[t][k] = gap1;
    }
  }
  // One distance for all rows, as long as it is not far above what a row needs.
#pragma unroll
  for (int d = 1; d < 4; d *= 2) most_gap = fmaxf(most_gap, __shfl_xor_sync(0xffffffffu, most_gap, d));
  // It is above the scales of V too, which quick blocks need, if they are not far above it.
  int scale = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    bool seen = !masked;
#pragma unroll
    for (int t = 0; t < NT; ++t) seen = seen || key0 + 8 * j + gr <= max(rows.pos[t][0], rows.pos[t][1]);
    if (seen) scale = max(scale, static_cast<int>(scale_word(vs, j) >> (8 * (j & 3)) & 0xffu));
  }
  const float above = static_cast<float>(__reduce_max_sync(0xffffffffu, scale) - 126);
  const float least_gap = most_gap;
  if (__any_sync(0xffffffffu, fresh)) most_gap += kHeadroom;
  if (above <= least_gap + kCommon) most_gap = fmaxf(most_gap, above);
  bool same = true;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const bool near = most_gap - sums.gap[t][k] <= kCommon;
      const float turn = near ? exp2_approx(sums.gap[t][k] - most_gap) : 1.f;
      same = same && near;
      f[t][k] *= turn;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        sums.acc[t][i][k] *= turn;
        sums.acc[t][i][k + 2] *= turn;
      }
      if (near) sums.gap[t][k] = most_gap;
    }
  common.any = __all_sync(0xffffffffu, same);
  common.gap = static_cast<int>(fminf(fmaxf(most_gap, -1126.f), 999.f)) + 127;
  // A NaN scale of a V row that a query row sees makes its output NaN.
  if (__any_sync(0xffffffffu, (nan_bytes(vs.x) | nan_bytes(vs.y)) != 0)) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        int bad = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          bad |= (scale_word(vs, j) >> (8 * (j & 3)) & 0xffu) == 255u && key0 + 8 * j + gr <= rows.pos[t][k];
#pragma unroll
        for (int d = 4; d < 32; d *= 2) bad |= __shfl_xor_sync(0xffffffffu, bad, d);
        if (bad) f[t][k] = nan;
      }
  }
}

// What the block that is not quick needs and changes.
template <int D, int NT>
struct Slow {
  Rows<D, NT> rows;
  Sums<D, NT> sums;
  Common common;
  float s[NT][4][4];
};

// A block with scores of any kind.  Not inlined: the loop over quick blocks would lose its
// registers to it (12 warps an SM, 2M tokens: 855 us with it inlined).
template <int D, int NT>
__device__ __noinline__ void any_block(Slow<D, NT>& slow, int warp, int slot, int key0, bool masked, int nrows) {
  using Sh = Shared4<D, NT>;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  auto& sm = *reinterpret_cast<Sh*>(smem_raw);
  const int lane = threadIdx.x & 31, tc = lane & 3;  // fragment column pair
  unsigned char* block = sm.ring[warp][slot];
  const unsigned char* scales = block + kCodes4<D>;
  const uint4* vx = reinterpret_cast<const uint4*>(scales + kScales4<D>) + lane;
  uint2 ks[D / 32];
  uint32_t large = 0, lost = 0;
#pragma unroll
  for (int g = 0; g < D / 32; ++g) {
    ks[g] = reinterpret_cast<const uint2*>(scales + g * kBlock)[lane >> 2];
    large |= large_bytes(ks[g].x) | large_bytes(ks[g].y);
  }
  const bool careful = __any_sync(0xffffffffu, (large & 0x80808080u) != 0);
  if (careful) {  // scales from 2^65 on
    lost = lower_scales<D / 32>(ks);
    first_product<D, NT>(slow.rows, block, lane, ks, slow.s);
  }
  float f[NT][2];
  softmax<D, NT>(slow.rows, slow.sums, slow.common, scales, key0, masked, careful, lost, slow.s, f);
  copies_wait<2 * Sh::kSlots - 2>();
  __syncwarp();  // V is there, and the codes of K have been read
  const Probabilities<NT> prob = {Sh::kOwnP ? sm.p[Sh::kOwnP ? warp : 0] : reinterpret_cast<float4(*)[4][32]>(block)};
  prob.put(slow.s);
  bool sure = false;  // that further passes are needed
#pragma unroll 1
  while (true) {
    uint32_t pf[NT][4][2];
    prob.get(pf);
#pragma unroll
    for (int i = 0; i < D / 16; i += kTogether) {
      float y[NT][kTogether][4];
      second_product<true, NT>(vx, i, pf, y);
#pragma unroll
      for (int h = 0; h < kTogether; ++h)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            slow.sums.acc[t][i + h][k] = fmaf(y[t][h][k], f[t][k & 1], slow.sums.acc[t][i + h][k]);
            // is an output so small that what fp16 leaves of P could count?
            sure |= t * 8 + 2 * tc + (k & 1) < nrows && f[t][k & 1] != 0.f && !(fabsf(y[t][h][k]) >= kEnough4);
          }
    }
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

template <int D, int NT>
__global__ void __launch_bounds__(kWarpsOf[NT - 1] * 32, 1) k_cache4_attention(const AttnParams p) {
  using Sh = Shared4<D, NT>;
  using Cur = Cursor<false, NT>;
  constexpr int kWarps = Sh::kWarps, kThreads = kWarps * 32, kSlots = Sh::kSlots;
  constexpr int kRows = 8 * NT;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  auto& sm = *reinterpret_cast<Sh*>(smem_raw);
  int thread;  // kept in a register: not read again wherever it is used
  asm volatile("mov.u32 %0, %%tid.x;" : "=r"(thread));
  const int warp = thread >> 5, lane = thread & 31;

  // ---- the flat order: total steps, and where this warp starts
  const int per_thread = (p.c.num_seqs + kThreads - 1) / kThreads;
  long long mine = 0;
  for (int i = 0; i < per_thread; ++i) {
    const int s = threadIdx.x * per_thread + i;
    if (s < p.c.num_seqs) {
      const SeqPlace at = seq_place(p.c, s);
      if (s < kSeqs) sm.seq[s] = at;
      mine += Cur::cost(p, at);
    }
  }
  long long upto = mine;
#pragma unroll
  for (int s = 1; s < 32; s *= 2) {
    const long long x = __shfl_up_sync(0xffffffffu, upto, s);
    if (lane >= s) upto += x;
  }
  if (lane == 31) sm.warp_sum[warp] = upto;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sm.warp_sum[w];
    total += sm.warp_sum[w];
  }
  sm.pre[threadIdx.x] = before + upto - mine;
  __syncthreads();
  const Cut cut(total, gridDim.x, kWarps, p.dynamic);
  const int used = cut.used(gridDim.x);
  if (!p.dynamic && blockIdx.x == 0 && threadIdx.x == 0) p.head[2] = cut.workers;
  if (warp >= used) return;
  const int run = blockIdx.x * used + warp;
  if (!p.dynamic && lane == 0) p.open[run].parts = 0;

  // Puts a cursor on a step of the flat order.
  auto locate = [&](Cur& cur, long long x) {
    const int slice = find_last(kThreads, x, [&](int s) { return sm.pre[s]; });
    long long at = sm.pre[slice];
    int i = slice * per_thread;
    for (long long c; x - at >= (c = Cur::cost(p, Cur::place(p, sm.seq, i))) && i + 1 < p.c.num_seqs; ++i) at += c;
    cur.enter(p, sm.seq, i);
    cur.skip(x - at);
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
    int load_slot = 0;
    int left = 0;                  // blocks that can be asked for without a look at anything else
    uint32_t unseen = 0;           // a bit for each slot whose block is on no page of the pool
    int pages = -1, pages_at = -1; // of 32 blocks of lc's unit, one a lane
    int next_page = 0, next_of = -1;  // a page of sequence next_of's first blocks, asked for early
    const uint32_t ring = smem_addr(sm.ring[warp]) + lane * 16;
    const unsigned char *k_at = nullptr, *v_at = nullptr, *s_at = nullptr;  // lc's head in page 0, this lane's bytes
    const unsigned char* values = nullptr;  // V of the block whose K went last
    const long long page_codes = static_cast<long long>(p.c.hkv) * kCodes4<D>, page_scales = static_cast<long long>(p.c.hkv) * kScales4<D>;

    // The end of a unit, of a list of pages or of a piece: what comes next.  left stays 0
    // where nothing does, and before a block that is on no page of the pool.
    auto refill = [&]() {
      while (to_load == 0) {
        if (!more_pieces) return;
        if (!asked) ask();
        asked = false;
        const int j = __shfl_sync(0xffffffffu, ticket, 0);
        const int k = 1 + j / cut.workers, w = j - (k - 1) * cut.workers;
        more_pieces = k < cut.pieces;
        if (!more_pieces) return;
        long long a, z;
        cut.range(w, k, a, z);
        if (a >= z) continue;
        locate(lc, a);
        to_load = z - a;
        piece = w * cut.pieces + k;
        if (lane == 0) sm.piece[warp][load_slot] = piece;
        pages_at = -1;
      }
      if (lc.blk == lc.nb) {
        // heads of a sequence share its pages: a list of up to 32 serves them all
        const bool same = lc.nb <= 32 && lc.tiles == 1 && !lc.last_unit(p);
        lc.next_unit(p, sm.seq);
        if (!same) pages_at = -1;
      }
      k_at = p.c.k + static_cast<long long>(lc.head) * kCodes4<D> + lane * 16;
      v_at = p.c.v + static_cast<long long>(lc.head) * kCodes4<D> + lane * 16;
      s_at = p.scale_bytes + static_cast<long long>(lc.head) * kScales4<D> + lane * 16;
      if (to_load == 1 && more_pieces && !asked) ask();  // not earlier: a slow warp must not sit on a piece
      if (pages_at != (lc.blk & ~31)) {  // a new unit, or the next 32 blocks
        const int last = lc.last_pos(p.g);
        const bool early = next_of == lc.seq && (lc.blk & ~31) == 0;
        pages_at = lc.blk & ~31;
        const int b = pages_at + lane;
        pages = -1;
        if (b < lc.nb && last >= 0 && b <= last / kBlock) {
          pages = early ? next_page : __ldg(p.c.table + static_cast<long long>(lc.seq) * p.c.max_pages + b);
          if (pages < 0 || pages >= p.c.num_pages) {
            report_table(p.c);
            pages = -1;
          }
        }
        next_of = -1;
      }
      if (next_of < 0 && lc.last_unit(p)) {
        next_of = lc.next_seq(p, sm.seq);
        if (next_of < p.c.num_seqs && lane < p.c.max_pages)
          next_page = __ldg(p.c.table + static_cast<long long>(next_of) * p.c.max_pages + lane);
      }
      const uint32_t bad = __ballot_sync(0xffffffffu, pages < 0) >> (lc.blk & 31);
      const int good = min(bad ? __ffs(bad) - 1 : 32, min(lc.nb - lc.blk, 32 - (lc.blk & 31)));
      left = static_cast<int>(min(static_cast<long long>(good), to_load > 1 && more_pieces ? to_load - 1 : to_load));
      to_load -= left;
    };
    // Asks for K of the next block, if there is one, and then for its V.
    auto issue_k = [&]() {
      __syncwarp();  // lanes read what others have copied: the slot's last readers are done
      values = nullptr;
      if (left == 0) {
        refill();
        if (left == 0 && to_load > 0) {
          unseen |= 1u << load_slot;
          --to_load;
          ++lc.blk;
          ++loaded;
          load_slot = load_slot + 1 == kSlots ? 0 : load_slot + 1;
        }
      }
      if (left > 0) {
        const long long page = __shfl_sync(0xffffffffu, pages, lc.blk & 31);
        const uint32_t dst = ring + load_slot * kBlock4<D>;
        const unsigned char* k = k_at + page * page_codes;
        values = v_at + page * page_codes;
#pragma unroll
        for (int i = 0; i < kCodes4<D> / 512; ++i) copy16(dst + i * 512, k + i * 512);
        if (lane < kScales4<D> / 16) copy16(dst + kCodes4<D>, s_at + page * page_scales);
        --left;
        ++lc.blk;
        ++loaded;
      }
      copies_commit();
    };
    auto issue_v = [&]() {
      __syncwarp();
      if (values) {
        const uint32_t dst = ring + load_slot * kBlock4<D> + kCodes4<D> + kScales4<D>;
#pragma unroll
        for (int i = 0; i < kCodes4<D> / 512; ++i) copy16(dst + i * 512, values + i * 512);
        load_slot = load_slot + 1 == kSlots ? 0 : load_slot + 1;
      }
      copies_commit();
    };
#pragma unroll 1
    for (int i = 0; i < kSlots; ++i) {
      issue_k();
      issue_v();
    }

    int slot = 0, at_piece = run * cut.pieces;  // (the copies may be in a later piece already)
    long long at = start;
    uint4 qx[NT][D / 32];  // raw query rows of cc's unit, this lane's channels
    auto fetch_q = [&]() { fetch_rows<D, NT>(p, cc.s.row0, cc.head, cc.rr0(), cc.nrows(p.g), qx); };
    fetch_q();
    while (true) {
      // ---- one unit, or the part of it that the piece has
      const bool begins = cc.blk == 0;
      const int steps = static_cast<int>(min(static_cast<long long>(cc.nb - cc.blk), stop - at));
      const bool ends = cc.blk + steps == cc.nb;
      const int nrows = cc.nrows(p.g), rr0 = cc.rr0(), row0 = cc.s.row0, head = cc.head;
      const int clear = (cc.first_pos(p.g) + 1) / kBlock - cc.blk;  // blocks that every row sees whole
      const Rows<D, NT> rows(p, qx, cc.s.p0, rr0, nrows);
      Sums<D, NT> sums;
      sums.clear();
      Common common = {true, -999};
#pragma unroll 1
      for (int step = 0; step < steps; ++step) {
        unsigned char* block = sm.ring[warp][slot];
        const unsigned char* scales = block + kCodes4<D>;
        uint32_t pf[NT][4][2];
        bool quick = false;
        copies_wait<2 * kSlots - 1>();
        __syncwarp();
        if (!(unseen >> slot & 1)) {
          uint2 ks[D / 32];
#pragma unroll
          for (int g = 0; g < D / 32; ++g) ks[g] = reinterpret_cast<const uint2*>(scales + g * kBlock)[lane >> 2];
          float s[NT][4][4];
          first_product<D, NT>(rows, block, lane, ks, s);
          if (step < clear && common.any) {
            quick = as_is<D, NT>(rows, sums, common, scales, lane, s, pf);
            if (!quick) {
              refer<D, NT>(rows, sums, common, scales, lane, s);
              quick = as_is<D, NT>(rows, sums, common, scales, lane, s, pf);
            }
          }
          if (!quick) {
            Slow<D, NT> slow = {rows, sums, common, {}};
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) slow.s[t][i][k] = s[t][i][k];
            any_block<D, NT>(slow, warp, slot, (cc.blk + step) * kBlock, step >= clear, nrows);
            sums = slow.sums;
            common = slow.common;
          }
        }
        unseen &= ~(1u << slot);
        issue_k();
        copies_wait<2 * kSlots - 1>();
        __syncwarp();
        if (quick) {
          const uint4* vx = reinterpret_cast<const uint4*>(scales + kScales4<D>) + lane;
#pragma unroll
          for (int i = 0; i < D / 16; i += kTogether) {
            float y[NT][kTogether][4];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int h = 0; h < kTogether; ++h)
#pragma unroll
                for (int k = 0; k < 4; ++k) y[t][h][k] = sums.acc[t][i + h][k];
            second_product<false, NT>(vx, i, pf, y);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int h = 0; h < kTogether; ++h)
#pragma unroll
                for (int k = 0; k < 4; ++k) sums.acc[t][i + h][k] = y[t][h][k];
          }
        }
        issue_v();
        slot = slot + 1 == kSlots ? 0 : slot + 1;
      }
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
          at_piece = sm.piece[warp][slot];
          const int w = at_piece / cut.pieces;
          cut.range(w, at_piece - w * cut.pieces, at, stop);
          locate(cc, at);
        }
      }
      if (more) fetch_q();

      // ---- the unit's part is done: out, or into a partial
      const size_t part_at = (static_cast<size_t>(this_piece) * 2 + (begins ? 1 : 0)) * kRows;
      write_part<D, NT>(p, sums, head, row0, rr0, nrows, begins && ends, part_at);
      if (begins && !ends && lane == 0) {
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
  // Even a call without work ends after the kernels in front of it (see the 8-bit kernel).
  if (p.dynamic) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <int D, int NT>
hdp_status_t launch4(const AttnParams& p, int device, int ctas, cudaStream_t st) {
  static std::atomic<bool> ready[kDevices];
  constexpr int smem = sizeof(Shared4<D, NT>);
  static_assert(smem <= 232448, "shared memory of a CTA");
  return launch<D, NT>(k_cache4_attention<D, NT>, kWarpsOf[NT - 1], smem, ready, p, device, ctas, st);
}

template <int D>
hdp_status_t launch_for(const AttnParams& p, int nt, int device, int ctas, cudaStream_t st) {
  return nt == 1 ? launch4<D, 1>(p, device, ctas, st) : launch4<D, 2>(p, device, ctas, st);
}

}  // namespace
}  // namespace hdp

using namespace hdp;

extern "C" hdp_status_t hdp_fourbit_attention_workspace_bytes(const hdp_fourbit_cache_t* cache, int32_t hq, size_t* bytes) {
  if (!cache || !bytes) return fail(HDP_ERR_INVALID_ARGUMENT, "hdp_fourbit_attention_workspace_bytes: NULL argument");
  return workspace_bytes_of("hdp_fourbit_attention_workspace_bytes", kWarpsOf, cache->hkv, cache->d, hq, bytes);
}

extern "C" hdp_status_t hdp_fourbit_attention(const hdp_fourbit_cache_t* cache, const int32_t* cu, int64_t rows,
                                              const void* q, int32_t hq, float scale, void* workspace,
                                              size_t workspace_bytes, void* o, float* lse, void* stream) {
  Cache4View c;
  const hdp_status_t r = cache4_view("hdp_fourbit_attention", cache, cu, rows, &c);
  if (r != HDP_OK) return r;
  AttnParams p = {};
  p.c = c;
  p.scale_bytes = c.scale_bytes;
  const bool wide = cache->d == 128;
  return attend("hdp_fourbit_attention", kWarpsOf, p, cache->d, rows, q, hq, scale, nullptr, 0, workspace, workspace_bytes, o, lse,
                stream, [=](const AttnParams& a, int nt, int device, int ctas, cudaStream_t st) {
                  return wide ? launch_for<128>(a, nt, device, ctas, st)
                              : launch_for<64>(a, nt, device, ctas, st);
                });
}
