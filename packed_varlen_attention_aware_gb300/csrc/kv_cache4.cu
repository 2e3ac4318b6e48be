// Writing rows into the 4-bit cache and reading them back.
//
// A row's codes depend on that row alone: 32 channels of K, or a token's whole V
// row, share the smallest power of two 2^e, e >= -126, with |x| <= 6 2^e; x / 2^e
// is a shift of the exponent and the code its only rounding.  So rows may come in
// any order and nothing that is there is ever rounded again.
//
// One CTA has the rows of one (block of 64 tokens, kv head).  A row is d / 8 lanes
// of 8 channels, whose codes make one 32-bit word.  K's words go straight to their
// places.  V's bytes hold two tokens of one channel (the pair that a matrix fragment
// takes along its k index): the words go through shared memory, and a thread turns
// the words of 8 tokens x 8 channels around, nibble by nibble, into 8 words of
// 8 tokens.  Bytes that also hold tokens of earlier calls are read and merged.
//
// With one token for each sequence a warp has one (sequence, kv head), half of it
// the K row and half the V row, as in the 8-bit cache.
//
// HBM bounds both ways (645 bytes a token and kv head of 128), the ALUs come next.
// Measured, 8 kv heads of 128: 83,000 tokens written 73 us, 5.9 TB/s; 131,072
// written 108.5 us and read 108, 6.2 TB/s, 0.92 of the copy rate; 256 sequences, one
// token each, written 3.6 us and read 5.0, latency.
#include <cuda_bf16.h>

#include <string>

#include "kv_cache4.cuh"

namespace hdp {

hdp_status_t cache4_view(const char* call, const hdp_fourbit_cache_t* c, const int32_t* cu, int64_t rows, Cache4View* out) {
  const std::string name(call);
  if (!c) return fail(HDP_ERR_INVALID_ARGUMENT, name + ": cache is NULL");
  if (!c->k || !c->v || !c->scales || !c->page_table || !c->lens)
    return fail(HDP_ERR_INVALID_ARGUMENT, name + ": the cache has a NULL pointer");
  if (c->num_pages < 1 || c->hkv < 1 || c->num_seqs < 1 || c->max_pages < 1)
    return fail(HDP_ERR_INVALID_ARGUMENT, name + ": num_pages, hkv, num_seqs and max_pages must be >= 1");
  if (c->num_seqs > (1 << 24)) return fail(HDP_ERR_UNSUPPORTED, name + ": num_seqs must be at most 2^24");
  if (c->hkv > 65535) return fail(HDP_ERR_UNSUPPORTED, name + ": hkv must be at most 65535");
  if (c->d != 64 && c->d != 128) return fail(HDP_ERR_UNSUPPORTED, name + ": d must be 64 or 128");
  if ((reinterpret_cast<uintptr_t>(c->k) | reinterpret_cast<uintptr_t>(c->v) | reinterpret_cast<uintptr_t>(c->scales)) & 15)
    return fail(HDP_ERR_INVALID_ARGUMENT, name + ": k, v and scales must be 16-byte aligned");
  if (rows < 0 || rows > 2147483647LL) return fail(HDP_ERR_INVALID_ARGUMENT, name + ": rows must be 0 .. 2^31-1");
  if (!cu && rows != c->num_seqs)
    return fail(HDP_ERR_INVALID_ARGUMENT, name + ": without cu, rows must equal num_seqs");
  *out = {};
  out->k = static_cast<uint8_t*>(c->k);
  out->v = static_cast<uint8_t*>(c->v);
  out->scale_bytes = c->scales;
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

__device__ __forceinline__ float bf_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// Largest magnitude of a lane's 8 channels, as bf16 bits (infinity and NaN, >= 0x7f80, on top).
__device__ __forceinline__ uint32_t largest(const uint4& x) {
  const uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
  return max(m & 0xffffu, m >> 16);
}

// The scale's byte, e + 127, for the bf16 bits of the largest magnitude: 6 is 1.5 * 2^2.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  if (top >= 0x7f80u) return 255;
  return max(static_cast<int>(top >> 7) - 2 + ((top & 0x7f) > 0x40), 1);
}

// 1 / 2^(byte - 127); the scale of a row with an infinity or NaN is NaN and its codes are zeros.
__device__ __forceinline__ float inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Magnitudes of two channels, at most 3 * 2^126.
__device__ __forceinline__ uint32_t bounded(uint32_t x) { return (x & 0x80008000u) | __vminu2(x & 0x7fff7fffu, 0x7f407f40u); }

// Codes of a lane's 8 channels, the first in the low four bits.
__device__ __forceinline__ uint32_t codes_of(uint4 x, uint32_t byte) {
  if (byte >= 253) {
    if (byte == 255) return 0;
    x = make_uint4(bounded(x.x), bounded(x.y), bounded(x.z), bounded(x.w));  // 4 * 2^126 is past bf16's end
  }
  const float inv = inverse(byte);
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(bf_lo(x.x) * inv), "f"(bf_hi(x.x) * inv), "f"(bf_lo(x.y) * inv), "f"(bf_hi(x.y) * inv),
        "f"(bf_lo(x.z) * inv), "f"(bf_hi(x.z) * inv), "f"(bf_lo(x.w) * inv), "f"(bf_hi(x.w) * inv));
  return r;
}

// 2^(byte - 127), down to bf16's range.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  if (byte == 255) return __int_as_float(0x7fc00000);
  return byte ? __uint_as_float(byte << 23) : __uint_as_float(0x00400000u);
}

__device__ __forceinline__ uint32_t bf16_pair(__half2 x, float s) {
  const float2 f = __half22float2(x);
  const __nv_bfloat162 r = __floats2bfloat162_rn(f.x * s, f.y * s);  // exact: two significant bits
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Values of 8 codes in bf16.
__device__ __forceinline__ uint4 values_of(uint32_t codes, float s) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
  const __half2* x = reinterpret_cast<const __half2*>(h);
  return make_uint4(bf16_pair(x[0], s), bf16_pair(x[1], s), bf16_pair(x[2], s), bf16_pair(x[3], s));
}

// Nibble k of word i becomes nibble i of word k.
__device__ __forceinline__ void transpose8(uint32_t (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const uint32_t a = w[i], b = w[i + 1];
    w[i] = (a & 0x0f0f0f0fu) | (b << 4 & 0xf0f0f0f0u);
    w[i + 1] = (a >> 4 & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i & 2) continue;
    const uint32_t a = w[i], b = w[i + 2];
    w[i] = __byte_perm(a, b, 0x6240);
    w[i + 2] = __byte_perm(a, b, 0x7351);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = w[i], b = w[i + 4];
    w[i] = __byte_perm(a, b, 0x5410);
    w[i + 4] = __byte_perm(a, b, 0x7632);
  }
}

// A thread's part of a block's V codes: 8 tokens (32 a + 16 s + 8 p + 2 c + e for word
// 4 s + 2 p + e) of the 8 channels 16 i + 8 h + r, whose words of tokens stand 64 bytes apart.
template <int D>
struct VPart {
  static constexpr int kParts = D / 16 * 16;  // threads that have one
  int a, h, c, i;
  __device__ __forceinline__ VPart() {
    a = threadIdx.x & 1;
    h = threadIdx.x >> 1 & 1;
    c = threadIdx.x >> 2 & 3;
    i = threadIdx.x >> 4;
  }
  __device__ __forceinline__ int token(int k) const { return 32 * a + 16 * (k >> 2) + 8 * (k >> 1 & 1) + 2 * c + (k & 1); }
  __device__ __forceinline__ int byte(int r) const { return 512 * i + 64 * r + 16 * c + 8 * h + 4 * a; }
  __device__ __forceinline__ int word() const { return 2 * i + h; }  // of a token's row
};

template <int D>
__global__ void __launch_bounds__(kThreads) k_cache4_append(const Cache4View c, const uint4* __restrict__ k,
                                                            const uint4* __restrict__ v) {
  constexpr int kLanes = D / 8;                   // of a row
  constexpr int kRows = kThreads / kLanes;        // at once
  constexpr int kPasses = kBlock / kRows;
  __shared__ uint32_t s_word[kBlock][kLanes + 1];
  Touched t;
  if (!touched_block(c, blockIdx.x, t)) return;
  const int page = page_of(c, t.seq, t.block), head = blockIdx.y;
  if (page < 0) return;
  const size_t ph = static_cast<size_t>(page) * c.hkv + head;
  const int l = threadIdx.x % kLanes, mine = threadIdx.x / kLanes;
  uint8_t* scales = c.scale_bytes + ph * kScales4<D>;
  uint8_t* kc = c.k + ph * kCodes4<D> + D / 8 * (l & 3) + 4 * (l >> 2);
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int token = p * kRows + mine, r = token - t.first;
    const bool here = r >= 0 && r < t.count;
    uint4 x = make_uint4(0, 0, 0, 0), y = x;
    if (here) {
      const size_t at = ((static_cast<size_t>(t.row) + r) * c.hkv + head) * kLanes + l;
      x = __ldg(k + at);
      y = __ldg(v + at);
    }
    uint32_t kt = largest(x), vt = largest(y);
#pragma unroll
    for (int o = 1; o < kLanes; o *= 2) {
      if (o < 4) kt = max(kt, __shfl_xor_sync(0xffffffffu, kt, o));
      vt = max(vt, __shfl_xor_sync(0xffffffffu, vt, o));
    }
    const uint32_t kb = scale_byte(kt), vb = scale_byte(vt);
    s_word[token][l] = codes_of(y, vb);
    if (here) {
      *reinterpret_cast<uint32_t*>(kc + token * (D / 2)) = codes_of(x, kb);
      if ((l & 3) == 0) scales[(l >> 2) * kBlock + scale_place(token)] = static_cast<uint8_t>(kb);
      if (l == 0) scales[(D / 32) * kBlock + scale_place(token)] = static_cast<uint8_t>(vb);
    }
  }
  __syncthreads();
  if (threadIdx.x >= VPart<D>::kParts) return;
  const VPart<D> part;
  uint32_t w[8], keep = 0;  // halves of bytes that the call does not write
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int token = part.token(i), r = token - t.first;
    w[i] = s_word[token][part.word()];
    if (r < 0 || r >= t.count) keep |= 15u << (4 * i);
  }
  transpose8(w);
  uint8_t* vc = c.v + ph * kCodes4<D>;
  if (keep == 0xffffffffu) return;
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    uint32_t* to = reinterpret_cast<uint32_t*>(vc + part.byte(r));
    *to = keep ? (*to & keep) | (w[r] & ~keep) : w[r];
  }
}

// One token for each sequence.
template <int D>
__global__ void __launch_bounds__(kThreads) k_cache4_append_one(const Cache4View c, const uint4* __restrict__ k,
                                                                const uint4* __restrict__ v) {
  constexpr int kLanes = D / 8;  // of a row: K in the first, V in the next
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long unit = static_cast<long long>(blockIdx.x) * (kThreads / 32) + warp;
  if (unit >= static_cast<long long>(c.num_seqs) * c.hkv) return;
  const int seq = static_cast<int>(unit / c.hkv), head = static_cast<int>(unit - static_cast<long long>(seq) * c.hkv);
  const int l = lane % kLanes;
  const bool is_v = lane / kLanes == 1, on = lane < 2 * kLanes;
  uint4 x = make_uint4(0, 0, 0, 0);
  if (on) x = __ldg((is_v ? v : k) + static_cast<size_t>(unit) * kLanes + l);
  const long long p0 = seq_len(c, seq) - 1;
  if (p0 < 0) return;
  const int page = page_of(c, seq, static_cast<int>(p0 / kBlock)), t = static_cast<int>(p0 % kBlock);
  if (page < 0) return;
  const size_t ph = static_cast<size_t>(page) * c.hkv + head;
  uint8_t* vc = c.v + ph * kCodes4<D> + 512 * (l >> 1) + 16 * (t >> 1 & 3) + 8 * (l & 1) + 2 * (t >> 4) + (t >> 3 & 1);
  uint32_t old[8] = {};
  if (is_v) {
#pragma unroll
    for (int r = 0; r < 8; ++r) old[r] = vc[64 * r];
  }
  uint32_t top = largest(x);
#pragma unroll
  for (int o = 1; o < kLanes; o *= 2) {
    const uint32_t other = __shfl_xor_sync(0xffffffffu, top, o);
    if (is_v || o < 4) top = max(top, other);
  }
  if (!on) return;
  const uint32_t byte = scale_byte(top), codes = codes_of(x, byte);
  uint8_t* scales = c.scale_bytes + ph * kScales4<D> + scale_place(t);
  if (is_v) {
    const int shift = (t & 1) * 4;
#pragma unroll
    for (int r = 0; r < 8; ++r)
      vc[64 * r] = static_cast<uint8_t>((old[r] & (0xf0u >> shift)) | ((codes >> (4 * r) & 15u) << shift));
    if (l == 0) scales[D / 32 * kBlock] = static_cast<uint8_t>(byte);
  } else {
    *reinterpret_cast<uint32_t*>(c.k + ph * kCodes4<D> + t * (D / 2) + D / 8 * (l & 3) + 4 * (l >> 2)) = codes;
    if ((l & 3) == 0) scales[(l >> 2) * kBlock] = static_cast<uint8_t>(byte);
  }
}

// Everything that a block has is asked for before anything of it is used: 16 words of codes
// and a word of scales a thread.
template <int D>
__global__ void __launch_bounds__(kThreads) k_cache4_read(const Cache4View c, uint4* __restrict__ k, uint4* __restrict__ v) {
  constexpr int kLanes = D / 8;
  constexpr int kRows = kThreads / kLanes;
  constexpr int kPasses = kBlock / kRows;
  __shared__ uint32_t s_word[kBlock][kLanes + 1];
  __shared__ uint32_t s_scale[kScales4<D> / 4];
  Touched t;
  const bool any = touched_block(c, blockIdx.x, t);
  const int head = blockIdx.y;
  for (long long i = threadIdx.x; i < t.before * kLanes; i += kThreads) {  // negative positions: zeros
    const size_t at = (static_cast<size_t>(t.row0 + i / kLanes) * c.hkv + head) * kLanes + i % kLanes;
    k[at] = v[at] = make_uint4(0, 0, 0, 0);
  }
  if (!any) return;
  const int page = page_of(c, t.seq, t.block);
  const size_t ph = static_cast<size_t>(max(page, 0)) * c.hkv + head;
  const int l = threadIdx.x % kLanes, mine = threadIdx.x / kLanes;
  uint32_t word[kPasses];
  if (page >= 0) {
    const VPart<D> part;
    uint32_t w[8];
    if (threadIdx.x < VPart<D>::kParts) {
#pragma unroll
      for (int r = 0; r < 8; ++r) w[r] = __ldg(reinterpret_cast<const uint32_t*>(c.v + ph * kCodes4<D> + part.byte(r)));
    }
    const uint8_t* kc = c.k + ph * kCodes4<D> + D / 8 * (l & 3) + 4 * (l >> 2);
#pragma unroll
    for (int p = 0; p < kPasses; ++p) word[p] = __ldg(reinterpret_cast<const uint32_t*>(kc + (p * kRows + mine) * (D / 2)));
    if (threadIdx.x < kScales4<D> / 4)
      s_scale[threadIdx.x] = __ldg(reinterpret_cast<const uint32_t*>(c.scale_bytes + ph * kScales4<D>) + threadIdx.x);
    if (threadIdx.x < VPart<D>::kParts) {
      transpose8(w);
#pragma unroll
      for (int i = 0; i < 8; ++i) s_word[part.token(i)][part.word()] = w[i];
    }
  }
  __syncthreads();
  const uint8_t* scales = reinterpret_cast<const uint8_t*>(s_scale);
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int token = p * kRows + mine, r = token - t.first;
    if (r < 0 || r >= t.count) continue;
    uint4 x = make_uint4(0, 0, 0, 0), y = x;
    if (page >= 0) {
      x = values_of(word[p], scale_value(scales[(l >> 2) * kBlock + scale_place(token)]));
      y = values_of(s_word[token][l], scale_value(scales[(D / 32) * kBlock + scale_place(token)]));
    }
    const size_t at = ((static_cast<size_t>(t.row) + r) * c.hkv + head) * kLanes + l;
    k[at] = x;
    v[at] = y;
  }
}

hdp_status_t check_rows(const char* call, const void* k, const void* v, int64_t rows) {
  if (rows > 0 && (!k || !v)) return fail(HDP_ERR_INVALID_ARGUMENT, std::string(call) + ": k or v is NULL");
  if ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15)
    return fail(HDP_ERR_INVALID_ARGUMENT, std::string(call) + ": k and v must be 16-byte aligned");
  return HDP_OK;
}

// CTAs in x: a slot for every block that the call may touch.
dim3 slot_grid(const Cache4View& c) {
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

extern "C" hdp_status_t hdp_fourbit_append(const hdp_fourbit_cache_t* cache, const int32_t* cu, int64_t rows, const void* k,
                                           const void* v, void* stream) {
  Cache4View c;
  HDP_TRY(cache4_view("hdp_fourbit_append", cache, cu, rows, &c));
  HDP_TRY(check_rows("hdp_fourbit_append", k, v, rows));
  if (rows == 0) return HDP_OK;
  c.err = device_error_word();
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const uint4* kp = static_cast<const uint4*>(k);
  const uint4* vp = static_cast<const uint4*>(v);
  if (cu) {
    (cache->d == 128 ? k_cache4_append<128> : k_cache4_append<64>)<<<slot_grid(c), kThreads, 0, st>>>(c, kp, vp);
  } else {
    const int64_t ctas = (int64_t(c.num_seqs) * c.hkv + kThreads / 32 - 1) / (kThreads / 32);
    if (ctas > 2147483647LL)
      return fail(HDP_ERR_UNSUPPORTED, "hdp_fourbit_append: num_seqs * hkv must be below 2^33");
    (cache->d == 128 ? k_cache4_append_one<128> : k_cache4_append_one<64>)<<<static_cast<unsigned>(ctas), kThreads, 0, st>>>(
        c, kp, vp);
  }
  note_launch();
  HDP_CUDA_TRY(cudaGetLastError());
  return HDP_OK;
}

extern "C" hdp_status_t hdp_fourbit_read(const hdp_fourbit_cache_t* cache, const int32_t* cu, int64_t rows, void* k, void* v,
                                         void* stream) {
  Cache4View c;
  HDP_TRY(cache4_view("hdp_fourbit_read", cache, cu, rows, &c));
  HDP_TRY(check_rows("hdp_fourbit_read", k, v, rows));
  if (rows == 0) return HDP_OK;
  c.err = device_error_word();
  (cache->d == 128 ? k_cache4_read<128> : k_cache4_read<64>)<<<slot_grid(c), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      c, static_cast<uint4*>(k), static_cast<uint4*>(v));
  note_launch();
  HDP_CUDA_TRY(cudaGetLastError());
  return HDP_OK;
}
