// Attention of the newest tokens of each sequence over the 4-bit cache.
//
// The flat order of (sequence, head, tile, block), and what carries the softmax over scores
// and V scales of any size, are the 8-bit cache's (kv_attention.cu).  A key and kv head is
// d + d / 32 + 1 bytes, half of the 8-bit cache's, so the same memory rate leaves half the
// time for each: on this GPU an m16n8k16 product takes a scheduler 8.3 cycles, and
// conversions and multiply-adds between products add a cycle each rather than hide behind
// them (measured in isolation), so the 64 products and 256 conversions of a block are 800
// cycles of the 1,450 that HBM takes for it.
//
//   Work.  Each of 8 warps an SM has an equal run of the order and a ring of blocks in
//   shared memory of its own, K and V of a block asked for apart; no barrier stands in the
//   loop.  Parts of a unit are joined within the CTA, then between CTAs by a small kernel.
//   Measured (32 / 8 heads of 128, in a captured graph): 2,097,152 tokens 341 us, 6.5 TB/s,
//   0.97 of the copy rate; 64 sequences of 411,000 tokens 93 us, 0.80: 4 to 8 us until data
//   flows, SMs that end 9 us apart, 4 us for the join.
//   Codes.  e2m1 is exact in fp16, and the conversion instruction takes a byte: one
//   for two codes, where the 8-bit kinds need four and seven cycles for as many.  The
//   cache's order of bytes is the fragments': K's words have one group of 32 channels
//   each, so the two products of a group share an accumulator.
//   Scales of K.  A group's sum is multiplied by its scale in fp32 and added to the
//   score's: no rounding of a code to a scaled one.  Where that passes fp32's end and a
//   scale is 2^65 or more, the block is computed again with all scales 2^-32 times as
//   large (those below 2^-94 count as 0) and the score back up behind the row's factor,
//   so that only scores beyond fp32's end pass it.
//   Scales of V go into P, as powers of two relative to the output's reference.
//   References.  Where every P of a block, under the references that the sums have, is a
//   normal number of fp16 (2^-14 to 2^15), it stays under them: nothing is rescaled, no
//   product can lose a small P, and the second product's sums are added to the output's.
//   (Added in fp32, to nearest: the matrix instruction cuts its sums off.  With the output
//   as its accumulator an instruction less an element is needed, and 2M tokens take 338 us,
//   64 sequences 92.0 and 16 drafts of 4 tokens 38.5, but all that is cut off has one sign:
//   2^-12 of the output where a warp has 131,072 tokens, 2^-6 at 2M.)
//   Fresh references are 4 bits above what needs them, so that is all but the first blocks
//   of a run unless a block's scores are spread over more than 17 nats.  Else P is taken
//   from the block's own largest, the sums come to new references, and what fp16 leaves of
//   P takes further passes where an output is small enough for it to count, as in the
//   8-bit kernel.  That takes a block many times as long, so it is not done for each block
//   of a peaked row: what fp16 leaves of a small P counts only in a channel where the keys
//   that weigh more are zero, and a block on that path also forms the sum of P |v| for each
//   row and channel.  The smallest of them is a budget: so many blocks with small P stay
//   quick that all they lose is 2^-12 of that sum (a P's rounding is up to 2^-11 of it).
//   64 sequences of random codes whose scores deviate by 1.7, 2.5 and 3.4 nats: 165, 322 and
//   478 us; 299, 792 and 802 without a budget and with all sums rescaled for each block; by
//   0.85, 93.  Of normally distributed V, with fewer zeros: 96, 130 and 282.
//   Scores past fp32's end.  A sum of products may pass it before the row's factor brings it
//   back, and a NaN scale makes it infinite: such a block goes to the general path.  As
//   -infinity it would pass for a masked one.  Only blocks that are not all normal are
//   searched for it: in them its P is 0.
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
// The top bit of bytes that are 192 (2^65) or more.
__device__ __forceinline__ uint32_t large_bytes(uint32_t w) { return w & (w << 1); }

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

constexpr int kWarps = 8;
// A part for each warp, and two for each CTA in front of them.
constexpr PartCount kCount = {1, kWarps + 2};

constexpr float kHeadroom = 4.f;    // bits of a fresh reference above what needs it
// What fp16 leaves of a block's P below its normal numbers (2^-25 each, twice rounded) is at
// most 64 * 2^-24 times the largest code; 2^12 times that.
constexpr float kSmallLoss = 0.09375f;
constexpr int kMostGap = 254;       // of Common::gap, so that a NaN's byte, 255, is above it: no block with one is quick
constexpr float kFactorBias = 24.f;  // of a block's factor in the output, for the same reason: a product is at most 2^24
constexpr float kCommon = 8.f;      // most bits that an output's reference is raised to be its neighbours', or above a V scale
// What fp16 leaves of a block's P is at most 64 * 2^-25 times its largest code, 6; 2^12 times that.
constexpr float kEnough4 = 0.0625f;

// A block's place in the ring: codes of K, scales, codes of V.
template <int D>
constexpr int kBlock4 = 2 * kCodes4<D> + kScales4<D>;

// What a warp's run leaves of units that it shares with its neighbours: [0] of one begun
// before it, [1] of one begun in it that goes on behind it.
struct RunEnds {
  bool has[2];
  bool ends;           // [0] is the unit's last
  const float* o[2];   // the part's rows
  int row0[2], head[2], nrows[2], rr0[2];
  long long last;      // [1]: the unit's last step
};

template <int D, int NT>
struct Shared4 {
  // P of a block on its way round takes the place of the codes of K, if it fits.
  static constexpr bool kOwnP = NT * 2048 > kCodes4<D>;
  static constexpr int kSlots = D == 128 ? 3 : kOwnP ? 5 : 6;
  unsigned char ring[kWarps][kSlots][kBlock4<D>];
  float4 p[kOwnP ? kWarps : 1][NT][4][32];
  SeqPlace seq[kSeqs];
  longlong2 pre[kWarps * 32];  // steps, and blocks, before each thread's sequences
  longlong2 warp_sum[kWarps];
  long long last_blocks;  // of the last thread's sequences
  RunEnds ends[kWarps];
  float2 part_sum[kWarps][2][8 * NT];
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

// Y = V^T P^T for the channels 16 i .. 16 i + 16 kTogether - 1; SIZE: of |V|.
template <int NT, bool SIZE = false>
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
      if constexpr (SIZE) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          a[x] &= 0x7fff7fffu;
          b[x] &= 0x7fff7fffu;
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (k == 0) mma16816_first(y[t][h], a[0], b[0], a[1], b[1], pf[t][k][0], pf[t][k][1]);
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
  float budget;  // blocks that may lose what fp16 leaves of small P
};

// A whole power of two as two factors, so that a sum is only lost where the result is: 2^-126 ends one.
__device__ __forceinline__ float2 exp2_far(float z) {
  return make_float2(exp2_approx(fmaxf(z, -100.f)), exp2_approx(fminf(z + 100.f, 0.f)));
}

// What stands behind it in a rare branch is not computed in front of the branch.
__device__ __forceinline__ void stay_here() { asm volatile("" ::: "memory"); }

// A place in a row of scales (of a lane's two, at 2 lane) to its token.
__device__ __forceinline__ int place_token(int place) { return 8 * (place & 7) + (place >> 3); }

// Scores of a block to P under the references that the sums have.  True, and the row sums
// have their share, if every P is a normal number of fp16, or the budget allows for small
// ones, and no seen score has passed fp32's end.  (Infinity and NaN are noticed as such; the
// P of -infinity is 0, which is not normal, as a masked key's may be.)  Of a block that is
// not seen whole (`masked`) the scores that a row does not see are -infinity already, no
// others are, and the tokens from `limit` on, which no row sees, may hold anything.
template <int D, int NT>
__device__ __forceinline__ bool as_is(const Rows<D, NT>& rows, Sums<D, NT>& sums, Common& common,
                                      const unsigned char* scales, int lane, bool masked, int limit,
                                      const float (&s)[NT][4][4], uint32_t (&pf)[NT][4][2]) {
  uint2 vs = reinterpret_cast<const uint2*>(scales + (D / 32) * kBlock)[lane >> 2];
  // V scales of the block, two a lane: 2^-14 to 1 of the output's reference, as normal numbers of fp16
  uint32_t two = reinterpret_cast<const uint16_t*>(scales + (D / 32) * kBlock)[lane];
  if (masked) {
    stay_here();
    const uint32_t any = static_cast<uint32_t>(common.gap) & 0xffu;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (8 * j + (lane >> 2) >= limit) {
        uint32_t& w = j < 4 ? vs.x : vs.y;
        w = (w & ~(0xffu << (8 * (j & 3)))) | any << (8 * (j & 3));
      }
    if (place_token(2 * lane) >= limit) two = (two & 0xff00u) | any;
    if (place_token(2 * lane + 1) >= limit) two = (two & 0x00ffu) | any << 8;
  }
  bool ok = static_cast<uint32_t>(common.gap) - (two & 0xffu) <= 14u && static_cast<uint32_t>(common.gap) - (two >> 8) <= 14u;
  const uint32_t back = (15u - static_cast<uint32_t>(common.gap)) * 0x04000400u;
  float l[NT][2];
  bool normal = true;
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
    if (masked) {  // a score of -infinity may have its 0
      stay_here();
      least = __half2half2(__ushort_as_half(0x7c00));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t low = s[t][j >> 1][2 * (j & 1)] == -__int_as_float(0x7f800000) ? 0x7c00u : 0u;
        const uint32_t up = s[t][j >> 1][1 + 2 * (j & 1)] == -__int_as_float(0x7f800000) ? 0x7c000000u : 0u;
        least = __hmin2(least, as_h2(pf[t][j >> 1][j & 1] | low | up));
      }
    }
    // (a NaN is in the sum, and in neither of the extremes)
    ok = ok && high <= kBias && l[t][0] == l[t][0] && l[t][1] == l[t][1];
    normal = normal && __hbge2(least, __half2half2(__ushort_as_half(0x0400)));
  }
  if (!__all_sync(0xffffffffu, ok && normal)) {
    if (!(common.budget >= 1.f)) return false;
    stay_here();
    if (!masked) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) ok = ok && s[t][i][k] != -__int_as_float(0x7f800000);
    }
    if (!__all_sync(0xffffffffu, ok)) return false;
    // (a lane has 8 of a row's 64 P)
    common.budget -= fminf(0.125f * __popc(__ballot_sync(0xffffffffu, !normal)), 1.f);
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int k = 0; k < 2; ++k) sums.l[t][k] += l[t][k];
#pragma unroll
    for (int j = 0; j < 8; ++j) pf[t][j >> 1][j & 1] = transpose8x8(pf[t][j >> 1][j & 1]);
  }
  return true;
}

__device__ __forceinline__ float lowest(float x) {
#pragma unroll
  for (int d = 16; d; d >>= 1) x = fminf(x, __shfl_xor_sync(0xffffffffu, x, d));
  return x;
}

// Brings the sums to references that are kHeadroom above the block's scores and a bit above
// its V scales, where they are not that high already.  Nothing is changed where that does not
// make the block quick (its V scales are too far apart), or where V scales of keys that weigh
// little would take a reference over kCommon bits above what needs it: the sums' range, down
// to 2^-126 of the largest product, would go to what is not there.
template <int D, int NT>
__device__ __forceinline__ void refer(const Rows<D, NT>& rows, Sums<D, NT>& sums, Common& common, const unsigned char* scales,
                                      int lane, int limit, const float (&s)[NT][4][4]) {
  const uint32_t two = reinterpret_cast<const uint16_t*>(scales + (D / 32) * kBlock)[lane];
  const bool seen = place_token(2 * lane) < limit, other = place_token(2 * lane + 1) < limit;
  const int above = __reduce_max_sync(0xffffffffu, static_cast<int>(max(seen ? two & 0xffu : 0u, other ? two >> 8 : 0u)));
  const int below = __reduce_min_sync(0xffffffffu, static_cast<int>(min(seen ? two & 0xffu : 255u, other ? two >> 8 : 255u)));
  const int byte = above > common.gap ? above + 1 : common.gap;
  if (byte > kMostGap || byte - below > 14) return;
  const float gap = static_cast<float>(byte - 127);
  float m1[NT][2];
  bool far = false;
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
      m1[t][k] = c > m && fabsf(c) < kBiasMost ? c + kHeadroom : m;  // (larger ones are not for here)
      far |= (m1[t][k] - m) + (gap - sums.gap[t][k]) > kCommon && (m1[t][k] - c) + (byte - above) > kCommon;
    }
  if (__any_sync(0xffffffffu, far)) return;
  common.gap = byte;
  float down = 0.f;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float m = sums.m[t][k], by = (m - m1[t][k]) + (sums.gap[t][k] - gap);
      const float2 turn = exp2_far(by);
      down = fminf(down, by);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        sums.acc[t][i][k] = sums.acc[t][i][k] * turn.x * turn.y;
        sums.acc[t][i][k + 2] = sums.acc[t][i][k + 2] * turn.x * turn.y;
      }
      sums.l[t][k] *= exp2_approx(m - m1[t][k]);
      sums.m[t][k] = m1[t][k];
      sums.gap[t][k] = gap;
    }
  common.budget *= exp2_approx(lowest(down));
}

// What a block that is not quick needs and changes.
template <int D, int NT>
struct Slow {
  Rows<D, NT> rows;
  Sums<D, NT> sums;
  Common common;
  float s[NT][4][4];
};

// A block with scores of any kind: P from the block's own largest, at most 2^15, the sums
// brought to new references.  Not inlined: the loop over quick blocks would lose its
// registers to it (12 warps an SM, 2M tokens: 855 us with it inlined); and written as loops:
// few calls come here, and fetch their instructions from far.
template <int D, int NT>
__device__ __noinline__ void any_block(Slow<D, NT>& slow, int warp, int slot, int key0, bool masked, int nrows) {
  using Sh = Shared4<D, NT>;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  auto& sm = *reinterpret_cast<Sh*>(smem_raw);
  const float inf = __int_as_float(0x7f800000), nan = __int_as_float(0x7fc00000);
  const int lane = threadIdx.x & 31, gr = lane >> 2, tc = lane & 3;
  unsigned char* block = sm.ring[warp][slot];
  const unsigned char* scales = block + kCodes4<D>;
  const uint4* vx = reinterpret_cast<const uint4*>(scales + kScales4<D>) + lane;
  const uint2 vs = reinterpret_cast<const uint2*>(scales + (D / 32) * kBlock)[gr];
  uint2 ks[D / 32];
  uint32_t large = 0, lost = 0;
#pragma unroll
  for (int g = 0; g < D / 32; ++g) {
    ks[g] = reinterpret_cast<const uint2*>(scales + g * kBlock)[gr];
    large |= large_bytes(ks[g].x) | large_bytes(ks[g].y);
  }
  bool past = false;  // fp32's end
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int k = 0; k < 2; ++k)
        past |= (!masked || key0 + 8 * j + gr <= slow.rows.pos[t][k]) && !(fabsf(slow.s[t][j >> 1][k + 2 * (j & 1)]) < inf);
  const bool careful = __any_sync(0xffffffffu, (large & 0x80808080u) != 0) && __any_sync(0xffffffffu, past);
  if (careful) {  // by scales from 2^65 on
    lost = lower_scales<D / 32>(ks);
    first_product<D, NT>(slow.rows, block, lane, ks, slow.s);
  }
  int scale = 0;  // the largest V scale that a row sees
  float f[NT][2];  // the power of two (<= 1) of the block in the output, times 2^kFactorBias
  float most_gap = -inf, shrunk = 0.f;  // the largest step of a row's sums to new references
  bool fresh = false;
#pragma unroll 1
  for (int tk = 0; tk < 2 * NT; ++tk) {
    const int t = tk >> 1, k = tk & 1;
    const float r = slow.rows.scale[t][k], back = 4294967296.f;  // 2^32
    const int pos = slow.rows.pos[t][k];
    float x[8], top = -inf;
    int bad = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] = slow.s[t][j >> 1][k + 2 * (j & 1)];
      if (careful) x[j] = x[j] * (r < 1.f ? r : back) * (r < 1.f ? back : r);
      else x[j] *= r;
      if (lost >> j & 1) x[j] = nan;
      const bool seen = !masked || key0 + 8 * j + gr <= pos;
      if (!seen) x[j] = -inf;
      top = fmaxf(top, x[j]);
      const int byte = static_cast<int>(scale_word(vs, j) >> (8 * (j & 3)) & 0xffu);
      if (seen) scale = max(scale, byte);
      bad |= seen && byte == 255;
    }
#pragma unroll
    for (int d = 4; d < 32; d *= 2) {
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      bad |= __shfl_xor_sync(0xffffffffu, bad, d);
    }
    const bool none = top == -inf;
    float ref = none ? 0.f : ceilf(top);
    const bool biased = fabsf(ref) < kBiasMost;
    if (biased) ref -= kBias;
    // the row sum's share, and the exponents of P with the V scales
    float sum = 0.f, most = -inf;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float y = x[j] - ref;
      sum += exp2_approx(y);
      x[j] = y + (exponent_bits(vs, j) - 8388735.f);
      most = fmaxf(most, x[j]);
    }
#pragma unroll
    for (int d = 4; d < 32; d *= 2) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
    const float e = most == -inf ? 0.f : ceilf(most) - kBias;
#pragma unroll
    for (int j = 0; j < 8; ++j) slow.s[t][j >> 1][k + 2 * (j & 1)] = exp2_approx(x[j] - e);
    const float m = slow.sums.m[t][k], gap = slow.sums.gap[t][k];
    const float m1 = none || ref <= m ? m : ref + (biased ? kHeadroom : 0.f);
    const float down = m - m1, up = none ? -inf : ref - m1;
    const float gap1 = none ? gap : fmaxf(gap + down, up + e);
    fresh |= gap1 > gap + down;
    most_gap = fmaxf(most_gap, gap1);
    slow.sums.l[t][k] = fmaf(sum, exp2_approx(up), slow.sums.l[t][k] * exp2_approx(down));
    // 0 where no key is seen; NaN where the scale of a seen V row is
    f[t][k] = bad ? nan : exp2_approx(up + (e - gap1) + kFactorBias);
    const float2 turn = exp2_far(down + (gap - gap1));
    shrunk = fminf(shrunk, down + (gap - gap1));
    if (down + (gap - gap1) != 0.f) {  // (the sums are in local memory here: a fourth of a block's time)
#pragma unroll 1
      for (int i = 0; i < D / 16; ++i) {
        slow.sums.acc[t][i][k] = slow.sums.acc[t][i][k] * turn.x * turn.y;
        slow.sums.acc[t][i][k + 2] = slow.sums.acc[t][i][k + 2] * turn.x * turn.y;
      }
    }
    slow.sums.m[t][k] = m1;
    slow.sums.gap[t][k] = gap1;
  }
  // One distance for all rows, as long as it is not far above what a row needs.  It is
  // above the scales of V too, which quick blocks need, if they are not far above it.
#pragma unroll
  for (int d = 1; d < 4; d *= 2) most_gap = fmaxf(most_gap, __shfl_xor_sync(0xffffffffu, most_gap, d));
  const float above = static_cast<float>(__reduce_max_sync(0xffffffffu, scale) - 126);
  const float least_gap = most_gap;
  if (__any_sync(0xffffffffu, fresh)) most_gap += kHeadroom;
  if (above <= least_gap + kCommon) most_gap = fmaxf(most_gap, above);
  bool same = true;
  float common_by = 0.f;
#pragma unroll 1
  for (int tk = 0; tk < 2 * NT; ++tk) {
    const int t = tk >> 1, k = tk & 1;
    const bool near = most_gap - slow.sums.gap[t][k] <= kCommon;
    const float turn = near ? exp2_approx(slow.sums.gap[t][k] - most_gap) : 1.f;
    if (near) common_by = fminf(common_by, slow.sums.gap[t][k] - most_gap);
    same = same && near;
    f[t][k] *= turn;
    if (turn != 1.f) {
#pragma unroll 1
      for (int i = 0; i < D / 16; ++i) {
        slow.sums.acc[t][i][k] *= turn;
        slow.sums.acc[t][i][k + 2] *= turn;
      }
    }
    if (near) slow.sums.gap[t][k] = most_gap;
  }
  slow.common.gap = static_cast<int>(fminf(fmaxf(most_gap, -1126.f), 999.f)) + 127;
  slow.common.any = __all_sync(0xffffffffu, same) && slow.common.gap <= kMostGap;

  copies_wait<2 * Sh::kSlots - 2>();
  __syncwarp();  // V is there, and the codes of K have been read
  const Probabilities<NT> prob = {Sh::kOwnP ? sm.p[Sh::kOwnP ? warp : 0] : reinterpret_cast<float4(*)[4][32]>(block)};
  prob.put(slow.s);
  bool sure = false;  // that further passes are needed
  bool first = true;  // pass: the same in all lanes, as the products need
  float least = inf;  // sum of P |v| over rows and channels
  float pass = 1.f / (1 << static_cast<int>(kFactorBias));  // what this one's P count
#pragma unroll 1
  while (true) {
    uint32_t pf[NT][4][2];
    prob.get(pf);
#pragma unroll 1
    for (int i = 0; i < D / 16; i += kTogether) {
      float y[NT][kTogether][4];
      if (first) {
        second_product<NT, true>(vx, i, pf, y);
#pragma unroll
        for (int h = 0; h < kTogether; ++h)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (t * 8 + 2 * tc + (k & 1) < nrows) least = fminf(least, y[t][h][k] * pass * f[t][k & 1]);
      }
      second_product<NT>(vx, i, pf, y);
#pragma unroll
      for (int h = 0; h < kTogether; ++h)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            slow.sums.acc[t][i + h][k] = fmaf(y[t][h][k] * pass, f[t][k & 1], slow.sums.acc[t][i + h][k]);
            // is an output so small that what fp16 leaves of P could count?
            sure |= t * 8 + 2 * tc + (k & 1) < nrows && f[t][k & 1] != 0.f && !(fabsf(y[t][h][k]) >= kEnough4);
          }
    }
    if (!__any_sync(0xffffffffu, sure) || !__any_sync(0xffffffffu, prob.more())) break;
    sure = true;
    prob.next();  // three times at most: P are 0 or above 2^-126
    pass *= 1.f / kNextPass;
    first = false;
  }
  slow.common.budget = slow.common.budget * exp2_approx(lowest(shrunk + common_by)) + lowest(least) * (1.f / kSmallLoss);
}

// A unit takes a warp its blocks and about three blocks' time more: its query rows, its
// first references, its output.  The flat order has that many steps in front of it (64
// sequences of 256 to 29K tokens: 110.6 us with none, 97.1 with two, 93.5 with three).
constexpr int kUnitSteps = 3;

// a / b of a >= 0, b > 0: in 32 bits where a has no more.
__device__ __forceinline__ long long quotient(long long a, int b) {
  return a >> 32 ? a / b : static_cast<long long>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
}

// Steps of all units of a sequence.
template <int NT>
__device__ __forceinline__ long long steps_of(const AttnParams& p, const SeqPlace& s) {
  using Cur = Cursor<false, NT>;
  return s.n ? static_cast<long long>(Cur::blocks_of(s) + kUnitSteps) * Cur::tiles_of(s.n, p.g) * p.c.hkv : 0;
}

// join_row of at most kWarps parts, in few instructions: a CTA runs them once or twice, and
// waits for each to be fetched.  Lane k (and k + 8, ..) has part k's sum and place.  (Of a
// CTA's time a joined unit of 16 rows took 1.9 us with join_row and 1.2 so; 16 drafts of 4
// tokens 43.1 and 38.8, 64 sequences 93.4 and 92.4.)
static_assert(kWarps == 8, "eight lanes' parts");
template <int D>
__device__ __forceinline__ float2 join_few(int m, int lane, float (&x)[D / 32], float2 l, const float* o) {
  constexpr int V = D / 32;
  float top = l.x;
#pragma unroll
  for (int s = 1; s < kWarps; s *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
  float w = l.y * exp2_approx(l.x - top), sum = w;
#pragma unroll
  for (int s = 1; s < kWarps; s *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, s);
  w *= sum == 0.f ? 0.f : 1.f / sum;  // no key: o = 0
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = 0.f;
#pragma unroll 2
  for (int k = 0; k < m; ++k) {
    const float f = __shfl_sync(0xffffffffu, w, k);
    const float* y = reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(o), k)) + lane * V;
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float2 z = *reinterpret_cast<const float2*>(y + i);
      x[i] = fmaf(f, z.x, x[i]);
      x[i + 1] = fmaf(f, z.y, x[i + 1]);
    }
  }
  return make_float2(top, sum);
}

template <int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, 1) k_cache4_attention(const AttnParams p) {
  using Sh = Shared4<D, NT>;
  using Cur = Cursor<false, NT>;
  constexpr int kThreads = kWarps * 32, kSlots = Sh::kSlots;
  constexpr int kRows = 8 * NT;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  auto& sm = *reinterpret_cast<Sh*>(smem_raw);
  int thread;  // kept in a register: not read again wherever it is used
  asm volatile("mov.u32 %0, %%tid.x;" : "=r"(thread));
  const int warp = thread >> 5, lane = thread & 31;

  // ---- the blocks of this warp: `todo` from cc's on, of the `used` runs of the CTA
  long long todo = 0, stop = 0, total = 0;
  int used;
  Cur cc, lc;  // of the arithmetic; of the copies, which run ahead
  if (lane < 2) sm.ends[warp].has[lane] = false;
  __syncwarp();
  if (p.alone) {  // one unit for the CTA
    cc.tiles = Cur::tiles_of(1, p.g);
    const int row = static_cast<int>(blockIdx.x) / (p.c.hkv * cc.tiles);
    cc.seq = row;
    cc.s = seq_place(p.c, row);
    cc.nb = Cur::blocks_of(cc.s);
    cc.head = (static_cast<int>(blockIdx.x) - row * p.c.hkv * cc.tiles) / cc.tiles;
    cc.tile = static_cast<int>(blockIdx.x) % cc.tiles;
    used = min(cc.nb, kWarps);
    if (warp < used) {
      cc.blk = cc.nb * warp / used;
      todo = cc.nb * (warp + 1) / used - cc.blk;
    }
  } else {  // an equal run of the flat order for each warp
    const int per_thread = (p.c.num_seqs + kThreads - 1) / kThreads;
    longlong2 mine = make_longlong2(0, 0);
    for (int i = 0; i < per_thread; ++i) {
      const int s = threadIdx.x * per_thread + i;
      if (s < p.c.num_seqs) {
        const SeqPlace at = seq_place(p.c, s);
        if (s < kSeqs) sm.seq[s] = at;
        mine.x += steps_of<NT>(p, at);
        mine.y += Cur::cost(p, at);
      }
    }
    longlong2 upto = mine;
#pragma unroll
    for (int s = 1; s < 32; s *= 2) {
      const long long x = __shfl_up_sync(0xffffffffu, upto.x, s), y = __shfl_up_sync(0xffffffffu, upto.y, s);
      if (lane >= s) {
        upto.x += x;
        upto.y += y;
      }
    }
    if (lane == 31) sm.warp_sum[warp] = upto;
    __syncthreads();
    longlong2 before = make_longlong2(0, 0);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) {
        before.x += sm.warp_sum[w].x;
        before.y += sm.warp_sum[w].y;
      }
      total += sm.warp_sum[w].x;
    }
    if (threadIdx.x == kThreads - 1) sm.last_blocks = mine.y;
    sm.pre[threadIdx.x] = make_longlong2(before.x + upto.x - mine.x, before.y + upto.y - mine.y);
    __syncthreads();
    if (threadIdx.x == 0) p.open[blockIdx.x].parts = 0;
    // Puts a cursor on a step of the flat order, and says how many blocks lie before it.
    auto locate = [&](Cur& cur, long long x) -> long long {
      const int slice = find_last(kThreads, x, [&](int s) { return sm.pre[s].x; });
      longlong2 at = sm.pre[slice];
      int i = slice * per_thread;
      SeqPlace s = Cur::place(p, sm.seq, i);
      for (long long c; x - at.x >= (c = steps_of<NT>(p, s)) && i + 1 < p.c.num_seqs; s = Cur::place(p, sm.seq, ++i)) {
        at.x += c;
        at.y += Cur::cost(p, s);
      }
      cur.enter(p, sm.seq, i);
      const int each = cur.nb + kUnitSteps;
      const long long off = x - at.x, unit = quotient(off, each);
      cur.blk = max(0, static_cast<int>(off - unit * each) - kUnitSteps);
      cur.head = static_cast<int>(quotient(unit, cur.tiles));
      cur.tile = static_cast<int>(unit - static_cast<long long>(cur.head) * cur.tiles);
      return at.y + unit * cur.nb + cur.blk;
    };

    const Cut cut(total, gridDim.x, kWarps, false);  // a run is one piece
    used = cut.used(gridDim.x);
    long long start;
    cut.range(blockIdx.x * used + warp, 0, start, stop);
    if (warp < used && start < total) {
      const long long end = stop < total ? locate(cc, stop) : sm.pre[kThreads - 1].y + sm.last_blocks;
      todo = end - locate(cc, start);
    }
  }
  const int run = blockIdx.x * used + warp;
  if (todo > 0) {
    lc = cc;
    long long to_load = todo;
    int load_slot = 0;
    int left = 0;                  // blocks that can be asked for without a look at anything else
    uint32_t unseen = 0;           // a bit for each slot whose block is on no page of the pool
    int pages = -1, pages_at = -1; // of 32 blocks of lc's unit, one a lane
    int next_page = 0, next_of = -1;  // a page of sequence next_of's first blocks, asked for early
    const uint32_t ring = smem_addr(sm.ring[warp]) + lane * 16;
    const unsigned char *k_at = nullptr, *v_at = nullptr, *s_at = nullptr;  // lc's head in page 0, this lane's bytes
    const unsigned char* values = nullptr;  // V of the block whose K went last
    const long long page_codes = static_cast<long long>(p.c.hkv) * kCodes4<D>, page_scales = static_cast<long long>(p.c.hkv) * kScales4<D>;

    // The end of a unit or of a list of pages: what comes next.  left stays 0 where nothing
    // does, and before a block that is on no page of the pool.
    auto refill = [&]() {
      if (to_load == 0) return;
      if (lc.blk == lc.nb) {
        // heads of a sequence share its pages: a list of up to 32 serves them all
        const bool same = lc.nb <= 32 && lc.tiles == 1 && !lc.last_unit(p);
        lc.next_unit(p, sm.seq);
        if (!same) pages_at = -1;
      }
      k_at = p.c.k + static_cast<long long>(lc.head) * kCodes4<D> + lane * 16;
      v_at = p.c.v + static_cast<long long>(lc.head) * kCodes4<D> + lane * 16;
      s_at = p.scale_bytes + static_cast<long long>(lc.head) * kScales4<D> + lane * 16;
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
      if (next_of < 0 && !p.alone && lc.last_unit(p)) {
        next_of = lc.next_seq(p, sm.seq);
        if (next_of < p.c.num_seqs && lane < p.c.max_pages)
          next_page = __ldg(p.c.table + static_cast<long long>(next_of) * p.c.max_pages + lane);
      }
      const uint32_t bad = __ballot_sync(0xffffffffu, pages < 0) >> (lc.blk & 31);
      const int good = min(bad ? __ffs(bad) - 1 : 32, min(lc.nb - lc.blk, 32 - (lc.blk & 31)));
      left = static_cast<int>(min(static_cast<long long>(good), to_load));
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

    int slot = 0;
    uint4 qx[NT][D / 32];  // raw query rows of cc's unit, this lane's channels
    auto fetch_q = [&]() { fetch_rows<D, NT>(p, cc.s.row0, cc.head, cc.rr0(), cc.nrows(p.g), qx); };
    fetch_q();
    while (true) {
      // ---- one unit, or the part of it that the piece has
      const bool begins = cc.blk == 0;
      const int steps = static_cast<int>(min(static_cast<long long>(cc.nb - cc.blk), todo));
      const bool ends = cc.blk + steps == cc.nb;
      const int nrows = cc.nrows(p.g), rr0 = cc.rr0(), row0 = cc.s.row0, head = cc.head;
      const int clear = (cc.first_pos(p.g) + 1) / kBlock - cc.blk;  // blocks that every row sees whole
      const int last_pos = cc.last_pos(p.g);
      const Rows<D, NT> rows(p, qx, cc.s.p0, rr0, nrows);
      Sums<D, NT> sums;
      sums.clear();
      Common common = {true, -999, 0.f};
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
          const bool masked = step >= clear;
          const int key0 = (cc.blk + step) * kBlock, limit = last_pos + 1 - key0;
          if (masked) {
            stay_here();
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  // a seen score that is -infinity has passed fp32's end: NaN, lest it pass for masked
                  float& x = s[t][i][k];
                  if (x == -__int_as_float(0x7f800000)) x = __int_as_float(0x7fc00000);
                  if (key0 + 16 * i + 8 * (k >> 1) + (lane >> 2) > rows.pos[t][k & 1]) x = -__int_as_float(0x7f800000);
                }
          }
          if (common.any) {
            quick = as_is<D, NT>(rows, sums, common, scales, lane, masked, limit, s, pf);
            if (!quick) {
              refer<D, NT>(rows, sums, common, scales, lane, limit, s);
              quick = as_is<D, NT>(rows, sums, common, scales, lane, masked, limit, s, pf);
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
            any_block<D, NT>(slow, warp, slot, key0, masked, nrows);
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
            second_product<NT>(vx, i, pf, y);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int h = 0; h < kTogether; ++h)
#pragma unroll
                for (int k = 0; k < 4; ++k) sums.acc[t][i + h][k] += y[t][h][k];
          }
        }
        issue_v();
        slot = slot + 1 == kSlots ? 0 : slot + 1;
      }
      todo -= steps;
      const int rest = cc.nb - cc.blk - steps;  // steps of the unit behind the run
      // ---- the next unit's query rows are asked for before this one is written
      const bool more = todo > 0;
      if (more) cc.next_unit(p, sm.seq);
      if (more) fetch_q();

      // ---- the unit's part is done: out, or into a partial
      // (at the end of the run the ring is free for it)
      float* part = p.part + (static_cast<size_t>(gridDim.x) * 2 + run) * kRows * D;
      if (!more) {
        copies_wait<0>();
        __syncwarp();
        part = reinterpret_cast<float*>(sm.ring[warp][0]);
      }
      write_part<D, NT>(p, sums, head, row0, rr0, nrows, begins && ends, part, sm.part_sum[warp][begins]);
      if (!(begins && ends) && lane == 0) {
        RunEnds& e = sm.ends[warp];
        e.has[begins] = true;
        if (!begins) e.ends = ends;
        e.o[begins] = part;
        e.row0[begins] = row0;
        e.head[begins] = head;
        e.nrows[begins] = nrows;
        e.rr0[begins] = rr0;
        e.last = stop + rest - 1;
      }
      if (!more) break;
    }
  }

  // ---- units that the warps of this CTA share are joined, row by row; which they are, all
  // lanes know from the warps' flags (a walk through them took 0.6 us)
  __syncthreads();
  const int other = min(lane, kWarps - 1);
  const uint32_t older = __ballot_sync(0xffffffffu, sm.ends[other].has[0]) & ((1u << used) - 1);
  const uint32_t newer = __ballot_sync(0xffffffffu, sm.ends[other].has[1]) & ((1u << used) - 1);
  const uint32_t last = __ballot_sync(0xffffffffu, sm.ends[other].ends) & older;
  int nth = 0;
#pragma unroll 1
  for (uint32_t left = newer << 1 | (older & 1u); left; left &= left - 1) {
    const int kind = left & 1u ? 0 : 1, w0 = max(__ffs(left) - 2, 0);  // begun in this CTA, by run w0, or before it
    // the parts behind it: of runs that have one of an older unit, up to the unit's last
    const uint32_t behind = older >> (w0 + 1), stops = last >> (w0 + 1);
    const bool single = !kind && (last & 1u);
    const int most = single ? 0 : __ffs(~behind) - 1, to_last = single || !stops ? kWarps : __ffs(stops);
    const bool whole = single || to_last <= most;
    const int m = 1 + min(most, to_last);
    const RunEnds& e = sm.ends[w0];
    const int nrows = e.nrows[kind];
    const int mine = min(lane & (kWarps - 1), m - 1), which = mine == 0 ? kind : 0;
    const float* o = sm.ends[w0 + mine].o[which];
    for (int r = (warp - nth) & (kWarps - 1); r < nrows; r += kWarps) {
      float x[D / 32];
      float2 l = sm.part_sum[w0 + mine][which][r];
      if ((lane & (kWarps - 1)) >= m) l = make_float2(kLow, 0.f);
      const float2 sum = join_few<D>(m, lane, x, l, o + r * D);
      if (kind && whole) {
        write_o<D>(p, e.row0[1], e.head[1], e.rr0[1] + r, x, lse_of(sum.x, sum.y), lane);
      } else {
        const size_t at = (static_cast<size_t>(blockIdx.x) * 2 + kind) * kRows + r;
#pragma unroll
        for (int v = 0; v < D / 32; ++v) p.part[at * D + lane * (D / 32) + v] = x[v];
        if (lane == 0) p.part_sum[at] = sum;
      }
    }
    nth += nrows;
    if (kind && !whole && threadIdx.x == 0) {
      Open o = {};
      o.first = blockIdx.x;
      o.parts = Cut(total, gridDim.x, kWarps, false).piece_of(e.last) / used - blockIdx.x + 1;
      o.row0 = e.row0[1];
      o.head = e.head[1];
      o.nrows = nrows;
      o.rr0 = e.rr0[1];
      p.open[blockIdx.x] = o;
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Joins the unit that a CTA began and did not end, if there is one, with its parts in the
// CTAs behind it: up to eight warps share a row's parts.  No lists of units are made, which
// the join of handed-out pieces needs (16 drafts of 4 tokens 37.9 us, 38.9 by that).
template <int D, int NT>
__global__ void __launch_bounds__(kJoinWarps * 32, 1) k_cache4_join(const AttnParams p) {
  constexpr int kRows = 8 * NT;
  static_assert(kRows <= kJoinWarps, "a warp for each row");
  __shared__ __align__(16) float s_x[kJoinWarps][D];
  __shared__ float2 s_sum[kJoinWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4* open = reinterpret_cast<const int4*>(p.open + blockIdx.x);
  const int4 a = __ldcg(open), b = __ldcg(open + 1);
  const int m = a.x, nrows = b.x;
  if (m == 0) return;
  const int each = min(kWarps, kJoinWarps >> (nrows > 1 ? 32 - __clz(nrows - 1) : 0));  // warps of a row
  const int r = warp / each, run = warp - r * each;
  auto at = [&](int k) { return (static_cast<size_t>(a.y + k) * 2 + (k == 0)) * kRows + r; };
  float x[D / 32];
  float2 sum;
  if (r < nrows) {
    const int k0 = m * run / each, k1 = m * (run + 1) / each;
    sum = join_row<D>(k1 - k0, lane, x, [&](int k) { return __ldcg(p.part_sum + at(k0 + k)); },
                      [&](int k) { return p.part + at(k0 + k) * D; });
  }
  if (each > 1) {
#pragma unroll
    for (int v = 0; v < D / 32; ++v) s_x[warp][lane * (D / 32) + v] = x[v];
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    if (run > 0 || r >= nrows) return;
    const int mine = min(lane & (kWarps - 1), each - 1);
    float2 l = s_sum[warp + mine];
    if ((lane & (kWarps - 1)) >= each) l = make_float2(kLow, 0.f);
    sum = join_few<D>(each, lane, x, l, s_x[warp + mine]);
  }
  if (r < nrows) write_o<D>(p, a.z, a.w, b.y + r, x, lse_of(sum.x, sum.y), lane);
}

template <int D, int NT>
hdp_status_t launch4(AttnParams p, int device, int sms, int ctas, cudaStream_t st) {
  static std::atomic<bool> ready[kDevices];
  constexpr int smem = sizeof(Shared4<D, NT>);
  static_assert(smem <= 232448, "shared memory of a CTA");
  // One token for each sequence, no more units than SMs and at most four blocks for each
  // warp of a unit: a CTA takes a unit, and nothing is left to join.  Measured (in a captured
  // graph, so and by runs): four documents of 64 to 512 tokens, 4 heads of 64, 6.6 and 11.2
  // us; 16 of 2,000 tokens, 8 heads of 128, 13.0 and 17.9; one of 2,048, 12.5 and 12.7; one
  // of 2,000 and 15 of 60, 12.6 and 12.3.
  const int64_t units = static_cast<int64_t>(p.c.num_seqs) * p.c.hkv * ((p.g + 8 * NT - 1) / (8 * NT));
  p.alone = !p.c.cu && units <= sms && p.c.max_pages <= 4 * kWarps;
  if (p.alone) ctas = static_cast<int>(units);
  hdp_status_t r = allow(k_cache4_attention<D, NT>, smem, ready, device);
  if (r == HDP_OK) r = launch_attention(k_cache4_attention<D, NT>, ctas, kWarps * 32, smem, p, st);
  if (r != HDP_OK || p.alone) return r;
  return launch_early(k_cache4_join<D, NT>, dim3(ctas), kJoinWarps * 32, 0, st, p);
}

template <int D>
hdp_status_t launch_for(const AttnParams& p, int nt, int device, int sms, int ctas, cudaStream_t st) {
  return nt == 1 ? launch4<D, 1>(p, device, sms, ctas, st) : launch4<D, 2>(p, device, sms, ctas, st);
}

}  // namespace
}  // namespace hdp

using namespace hdp;

extern "C" hdp_status_t hdp_fourbit_attention_workspace_bytes(const hdp_fourbit_cache_t* cache, int32_t hq, size_t* bytes) {
  if (!cache || !bytes) return fail(HDP_ERR_INVALID_ARGUMENT, "hdp_fourbit_attention_workspace_bytes: NULL argument");
  return workspace_bytes_of("hdp_fourbit_attention_workspace_bytes", kCount, cache->hkv, cache->d, hq, bytes);
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
  return attend("hdp_fourbit_attention", kCount, 0, p, cache->d, rows, q, hq, scale, nullptr, 0, workspace, workspace_bytes, o, lse,
                stream, [=](const AttnParams& a, int nt, int device, int sms, int ctas, cudaStream_t st) {
                  return wide ? launch_for<128>(a, nt, device, sms, ctas, st)
                              : launch_for<64>(a, nt, device, sms, ctas, st);
                });
}
