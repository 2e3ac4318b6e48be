// Attention of the newest tokens of each sequence over the 4-bit cache.
//
// How the work is cut, copied ahead, handed out and joined, and what carries the
// softmax over scores and V scales of any size, is the 8-bit cache's (kv_attention.cu).
// Here are a block's products.  A key and kv head is d + d / 32 + 1 bytes, half of the
// 8-bit cache's, so the same memory rate leaves half the instructions for each.
//
//   Codes.  e2m1 is exact in fp16, and the conversion instruction takes a byte: one
//   for two codes, where the 8-bit kinds need four and seven cycles for as many.  The
//   cache's order of bytes is the fragments': K's words have one group of 32 channels
//   each, so the two products of a group share an accumulator.
//   Scales of K.  A group's sum is multiplied by its scale in fp32 and added to the
//   score's: 64 multiply-adds a block and lane, which the 32-bit pipe has free, and no
//   rounding of a code to a scaled one.  Where a scale is 2^65 or more (checked for the
//   block), all scales of the block are taken 2^-32 times as large and the score back up
//   behind the row's factor, so that only scores beyond fp32's end pass it; what the
//   smallest scales lose by that is below such a score's last bit.
//   Scales of V go into P: 2^(score + e) against the block's largest of these, which a
//   second maximum over the keys finds, beside 2^score for the row sum.  P is then fp16
//   at up to 2^15 as in the 8-bit kernel, and what fp16 leaves of it takes further
//   passes where an output is small enough for it to count.
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
// byte j - 127, as a float
__device__ __forceinline__ float exponent_at(const uint2& x, int j) {
  return __uint_as_float(__byte_perm(scale_word(x, j), 0x4b000000u, 0x7650 + (j & 3))) - 8388735.f;
}
// Of bytes: the top bit of those that are 192 (2^65) or more, of those that are 255.
__device__ __forceinline__ uint32_t large_bytes(uint32_t w) { return w & (w << 1); }
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & w & 0x80808080u; }

// Bytes of a block whose scales go up to 2^126, times 2^-32; bit j of the result: some
// scale of key j is NaN.
template <int G>
__device__ __noinline__ uint32_t lower_scales(uint2 (&ks)[G]) {
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

template <int D>
struct Codes4 {
  static constexpr int kD = D;
  static constexpr int kGroups = D / 32;
  static constexpr int kSlot = kCodes4<D> + kScales4<D>;  // scales behind the codes of K
  // About 22 KB for each warp, as many as fit beside two tiles' P.
  template <int NT, bool SPARSE>
  static constexpr int kSlots = D == 128 ? 5 : 10;
  // What fp16 leaves of a block's P is at most 64 * 2^-25 times its largest code, 6; 2^12 times that.
  static constexpr float kEnough = 0.0625f;

  // Query rows: of each group this lane's 8 channels.
  template <int NT>
  __device__ __forceinline__ static void fetch_rows(const AttnParams& p, int row0, int head, unsigned rr0, int nrows,
                                                    uint4 (&qx)[NT][D / 32]) {
    const int lane = threadIdx.x & 31, gr = lane >> 2, tc = lane & 3;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = t * 8 + gr;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) qx[t][g] = make_uint4(0, 0, 0, 0);
      if (r < nrows) {
        const unsigned token = (rr0 + r) / p.g;
        const uint4* src = reinterpret_cast<const uint4*>(
            p.q + (static_cast<long long>(row0 + token) * p.hq + head * p.g + (rr0 + r - token * p.g)) * D + tc * 8);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) qx[t][g] = __ldg(src + g * 4);
      }
    }
  }

  __device__ __forceinline__ static void copy_k(const AttnParams& p, size_t ph, uint32_t dst, Meta*) {
    const int lane = threadIdx.x & 31;
    __syncwarp();  // lanes read what others have copied: the slot's last readers are done
    const unsigned char* src = p.c.k + ph * kCodes4<D> + lane * 16;
#pragma unroll
    for (int i = 0; i < kCodes4<D> / 512; ++i) copy16(dst + i * 512, src + i * 512);
    if (lane < kScales4<D> / 16) copy16(dst + kCodes4<D>, p.scale_bytes + ph * kScales4<D> + lane * 16);
  }
  __device__ __forceinline__ static const unsigned char* v_of(const AttnParams& p, size_t ph) {
    return p.c.v + ph * kCodes4<D> + (threadIdx.x & 31) * 16;
  }
  __device__ __forceinline__ static void copy_v(const unsigned char* v, uint32_t dst) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kCodes4<D> / 512; ++i) copy16(dst + i * 512, v + i * 512);
  }

  // Words of a key's codes, one for each group.
  __device__ __forceinline__ static void key_words(const unsigned char* slot, int j, uint32_t (&w)[kGroups]) {
    const int lane = threadIdx.x & 31;
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
  template <int NT>
  __device__ __forceinline__ static void first_product(const Rows<D, NT>& rows, const unsigned char* slot,
                                                       const uint2 (&ks)[kGroups], float (&s)[NT][4][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t u[kGroups], w[kGroups];
      key_words(slot, 2 * i, u);
      key_words(slot, 2 * i + 1, w);
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
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

  // Scores to P times the V scales, at most 2^15; brings the sums to the new references,
  // and f to the power of two (<= 1) of the block in the output.
  template <int NT>
  __device__ __forceinline__ static void scores(const Rows<D, NT>& rows, Sums<D, NT>& sums, const unsigned char* slot,
                                                const Meta& meta, bool masked, const Probabilities<NT>& prob,
                                                float (&f)[NT][2]) {
    const float inf = __int_as_float(0x7f800000);
    const int gr = (threadIdx.x & 31) >> 2;
    const uint2* scales = reinterpret_cast<const uint2*>(slot + kCodes4<D>) + gr;
    uint2 ks[kGroups];
    uint32_t large = 0;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      ks[g] = scales[g * 8];
      large |= large_bytes(ks[g].x) | large_bytes(ks[g].y);
    }
    const uint2 vs = scales[kGroups * 8];
    const bool careful = __any_sync(0xffffffffu, (large & 0x80808080u) != 0);
    uint32_t lost = 0;
    if (careful) lost = lower_scales<kGroups>(ks);
    float s[NT][4][4];
    first_product<NT>(rows, slot, ks, s);

#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float top[2] = {-inf, -inf};
      float row[2] = {rows.scale[t][0], rows.scale[t][1]};
      if (careful) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float r = row[k & 1], back = 4294967296.f;  // 2^32
            s[t][i][k] = lost >> (2 * i + (k >> 1)) & 1 ? __int_as_float(0x7fc00000)
                                                        : s[t][i][k] * (r < 1.f ? r : back) * (r < 1.f ? back : r);
          }
        row[0] = row[1] = 1.f;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float x = s[t][i][k] * row[k & 1];
          if (masked && meta.key0 + 16 * i + 8 * (k >> 1) + gr > rows.pos[t][k & 1]) x = -inf;
          s[t][i][k] = x;
          top[k & 1] = fmaxf(top[k & 1], x);
        }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int d = 4; d < 32; d *= 2) top[k] = fmaxf(top[k], __shfl_xor_sync(0xffffffffu, top[k], d));
        const bool none = top[k] == -inf;
        float c = none ? 0.f : ceilf(top[k]);
        if (fabsf(c) < kBiasMost) c -= kBias;
        // the row sum's share, and the exponents of P with the V scales
        float sum = 0.f, most = -inf;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float y = s[t][i][k + 2 * h] - c;
            sum += exp2_approx(y);
            s[t][i][k + 2 * h] = y + exponent_at(vs, 2 * i + h);
            most = fmaxf(most, s[t][i][k + 2 * h]);
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
        const float m1 = none ? m : fmaxf(m, c);
        const float down = m - m1;
        const float gap1 = none ? gap : fmaxf(gap + down, (c - m1) + e);
        const float up = exp2_approx(down + (gap - gap1));
        if (up != 1.f) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            sums.acc[t][i][k] *= up;
            sums.acc[t][i][k + 2] *= up;
          }
        }
        const float fl = none ? 0.f : exp2_approx(c - m1);
        f[t][k] = none ? 0.f : exp2_approx((c - m1) + (e - gap1));
        sums.l[t][k] = fmaf(sum, fl, sums.l[t][k] * exp2_approx(down));
        sums.m[t][k] = m1;
        sums.gap[t][k] = gap1;
      }
    }
    // A NaN scale of a V row that a query row sees makes its output NaN.
    if (__any_sync(0xffffffffu, (nan_bytes(vs.x) | nan_bytes(vs.y)) != 0)) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          bool bad = false;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            bad |= (scale_word(vs, j) >> (8 * (j & 3)) & 0xffu) == 255u && meta.key0 + 8 * j + gr <= rows.pos[t][k];
          int any = bad;
#pragma unroll
          for (int d = 4; d < 32; d *= 2) any |= __shfl_xor_sync(0xffffffffu, any, d);
          if (any) f[t][k] = __int_as_float(0x7fc00000);
        }
    }
    prob.put(s);
  }

  // O^T += f Y, Y = V^T P^T; least: the smallest |Y| of this lane's rows.
  template <int NT>
  __device__ __forceinline__ static void output(Sums<D, NT>& sums, const uint32_t (&pf)[NT][4][2], const float (&f)[NT][2],
                                                const unsigned char* slot, bool, float (&least)[NT][2]) {
    const uint4* vx = reinterpret_cast<const uint4*>(slot) + (threadIdx.x & 31);
#pragma unroll
    for (int t = 0; t < NT; ++t) least[t][0] = least[t][1] = __int_as_float(0x7f800000);
#pragma unroll
    for (int i = 0; i < D / 16; i += kTogether) {
      uint4 u[kTogether];
      float y[NT][kTogether][4];
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
            if (k == 0) mma16816_first(y[t][h], a[0], b[0], a[1], b[1], pf[t][k][0], pf[t][k][1]);
            else mma16816(y[t][h], a[0], b[0], a[1], b[1], pf[t][k][0], pf[t][k][1]);
            mma16816(y[t][h], a[2], b[2], a[3], b[3], pf[t][k + 1][0], pf[t][k + 1][1]);
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
};

template <class F>
hdp_status_t launch_for(const AttnParams& p, int nt, int device, int ctas, cudaStream_t st) {
  return nt == 1 ? launch<F, 1, false>(p, device, ctas, st) : launch<F, 2, false>(p, device, ctas, st);
}

}  // namespace
}  // namespace hdp

using namespace hdp;

extern "C" hdp_status_t hdp_fourbit_attention_workspace_bytes(const hdp_fourbit_cache_t* cache, int32_t hq, size_t* bytes) {
  if (!cache || !bytes) return fail(HDP_ERR_INVALID_ARGUMENT, "hdp_fourbit_attention_workspace_bytes: NULL argument");
  return workspace_bytes_of("hdp_fourbit_attention_workspace_bytes", cache->hkv, cache->d, hq, bytes);
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
  return attend("hdp_fourbit_attention", p, cache->d, rows, q, hq, scale, nullptr, 0, workspace, workspace_bytes, o, lse,
                stream, [=](const AttnParams& a, int nt, int device, int ctas, cudaStream_t st) {
                  return wide ? launch_for<Codes4<128>>(a, nt, device, ctas, st)
                              : launch_for<Codes4<64>>(a, nt, device, ctas, st);
                });
}
