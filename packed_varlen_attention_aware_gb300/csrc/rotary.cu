// Rotary positions of query and key rows, and their gradient.
//
// A pair (a, b) of a head's first `rot` channels at position p becomes
//   (f (a cos x - b sin x), f (b cos x + a sin x)),   x = p theta_i,
// and the gradient of a is f times the turn by -x.  2 d bytes in and out for each
// element of q and k against a few operations: HBM bounds it.
//
//   Angles.  p theta in fp32 is off by 0.1 radians at two million positions.  The
//   angle is kept in turns instead, as a 64-bit fraction: theta / 2 pi mod 1 times
//   2^64 is a whole number, p times it mod 2^64 is exact, and what is left is the
//   angle's fraction of a turn to 2^-33 for any 31-bit p (theta / 2 pi is rounded at
//   2^-53 of itself).  As a signed number it is within half a turn, which sincospi
//   takes in fp32.
//   Sharing.  A token's cosines and sines serve all its heads: a CTA works them out
//   for a tile of tokens, one pair a thread, and its threads then go over the
//   tile's (token, head) units, 16 bytes of each half of a pair at a time.
//   Rows whose layout does not allow 16 bytes go by one pair of elements a thread.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>
#include <string>

#include "internal.h"

namespace hdp {
namespace {

constexpr int kThreads = 256;
constexpr int kMostD = 256;
constexpr int kMostTile = 8;  // tokens of a CTA

struct RotaryTensor {
  const char* in;
  char* out;
  long long in_row, in_head, out_row, out_head;  // in elements
};

struct Rotary {
  RotaryTensor x[2];
  int heads[2];
  const int32_t* pos;
  const double* freqs;
  int rows, d, rot, tile;
  float factor, sign;
  bool copy;  // channels behind rot are copied
};

template <class T>
__device__ __forceinline__ float to_float(T x) {
  if constexpr (sizeof(T) == 4) return x;
  else if constexpr (std::is_same<T, __half>::value) return __half2float(x);
  else return __bfloat162float(x);
}
template <class T>
__device__ __forceinline__ T from_float(float x) {
  if constexpr (sizeof(T) == 4) return x;
  else if constexpr (std::is_same<T, __half>::value) return __float2half_rn(x);
  else return __float2bfloat16_rn(x);
}

// a c + b s, rounded alike whichever kernel a row takes.
__device__ __forceinline__ float turned(float a, float c, float b, float s) { return fmaf(b, s, __fmul_rn(a, c)); }

template <class T, int V>
struct alignas(sizeof(T) * V) Vec {
  T v[V];
};

template <class T, int V>
__device__ __forceinline__ Vec<T, V> get(const T* p) {
  return *reinterpret_cast<const Vec<T, V>*>(p);
}
template <class T, int V>
__device__ __forceinline__ void put(T* p, const Vec<T, V>& x) {
  *reinterpret_cast<Vec<T, V>*>(p) = x;
}

template <class T, int V, bool NEIGHBOURS>
__global__ void __launch_bounds__(kThreads) k_rotary(const Rotary p) {
  __shared__ __align__(16) float s_cos[kMostTile * kMostD / 2];
  __shared__ __align__(16) float s_sin[kMostTile * kMostD / 2];
  __shared__ int s_pos[kMostTile];
  const int half = p.rot / 2;
  const long long row0 = static_cast<long long>(blockIdx.x) * p.tile;
  const int n = static_cast<int>(min(static_cast<long long>(p.tile), p.rows - row0));

  for (int x = threadIdx.x; x < n * half; x += kThreads) {
    const int t = x / half, i = x - t * half;
    const int at = __ldg(p.pos + row0 + t);
    double turn = __ldg(p.freqs + i) * 0.15915494309189535;  // 1 / 2 pi
    turn -= floor(turn);
    const unsigned long long step = static_cast<unsigned long long>(turn * 18446744073709551616.0);
    const unsigned long long fraction = step * static_cast<unsigned long long>(static_cast<long long>(at));
    float s, c;
    sincospif(__ll2float_rn(static_cast<long long>(fraction)) * 1.0842021724855044e-19f, &s, &c);  // 2^-63
    s_cos[x] = c * p.factor;
    s_sin[x] = s * p.factor * p.sign;
    if (i == 0) s_pos[t] = at;
  }
  __syncthreads();

  // A unit is one head of one token: `pairs` threads with V pairs each, then those that copy.
  const int pairs = half / V, group = pairs + (p.copy ? (p.d - p.rot + 2 * V - 1) / (2 * V) : 0);
  const int groups = kThreads / group;
  const int g = threadIdx.x / group, j = threadIdx.x - g * group;
  if (g >= groups) return;
  const int all = p.heads[0] + p.heads[1], units = n * all;
#pragma unroll 4
  for (int u = g; u < units; u += groups) {
    const int t = u / all;
    int h = u - t * all;
    if (s_pos[t] < 0) continue;
    const bool second = h >= p.heads[0];
    if (second) h -= p.heads[0];
    const RotaryTensor& x = p.x[second];
    const T* in = reinterpret_cast<const T*>(x.in) + (row0 + t) * x.in_row + h * x.in_head;
    T* out = reinterpret_cast<T*>(x.out) + (row0 + t) * x.out_row + h * x.out_head;
    if (j < pairs) {
      const int a0 = NEIGHBOURS ? 2 * V * j : V * j, b0 = NEIGHBOURS ? a0 + V : half + V * j;
      Vec<T, V> a = get<T, V>(in + a0), b = get<T, V>(in + b0);
      const float* cos = s_cos + t * half + V * j;
      const float* sin = s_sin + t * half + V * j;
      if constexpr (NEIGHBOURS && V > 1) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
          Vec<T, V>& y = k < V / 2 ? a : b;
          const int m = 2 * k % V;
          const float c = cos[k], s = sin[k], y0 = to_float(y.v[m]), y1 = to_float(y.v[m + 1]);
          y.v[m] = from_float<T>(turned(y0, c, -y1, s));
          y.v[m + 1] = from_float<T>(turned(y1, c, y0, s));
        }
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float c = cos[k], s = sin[k], y0 = to_float(a.v[k]), y1 = to_float(b.v[k]);
          a.v[k] = from_float<T>(turned(y0, c, -y1, s));
          b.v[k] = from_float<T>(turned(y1, c, y0, s));
        }
      }
      put(out + a0, a);
      put(out + b0, b);
    } else {
      const int c0 = p.rot + (j - pairs) * 2 * V;
      put(out + c0, get<T, V>(in + c0));
      if (c0 + V < p.d) put(out + c0 + V, get<T, V>(in + c0 + V));
    }
  }
}

template <class T, int V>
void launch(const Rotary& p, bool neighbours, cudaStream_t st) {
  const unsigned ctas = static_cast<unsigned>((p.rows + p.tile - 1) / p.tile);
  if (neighbours) k_rotary<T, V, true><<<ctas, kThreads, 0, st>>>(p);
  else k_rotary<T, V, false><<<ctas, kThreads, 0, st>>>(p);
}

template <class T>
void launch_for(const Rotary& p, int bytes, bool neighbours, cudaStream_t st) {
  constexpr int wide = 16 / sizeof(T);
  if (bytes >= 16) launch<T, wide>(p, neighbours, st);
  else launch<T, 1>(p, neighbours, st);
}

}  // namespace
}  // namespace hdp

using namespace hdp;

extern "C" hdp_status_t hdp_rotary(const hdp_rotary_rows_t* q, const hdp_rotary_rows_t* k, int64_t rows, int32_t d,
                                   int32_t type, const int32_t* position, const double* freqs, int32_t rot, int32_t flags,
                                   float factor, void* stream) {
  const std::string name = "hdp_rotary: ";
  if (!q && !k) return fail(HDP_ERR_INVALID_ARGUMENT, name + "q and k are NULL");
  if (rows < 0 || rows > 2147483647LL) return fail(HDP_ERR_INVALID_ARGUMENT, name + "rows must be 0 .. 2^31-1");
  if (d < 2 || rot < 2 || rot % 2 || rot > d) return fail(HDP_ERR_INVALID_ARGUMENT, name + "need an even rot, 2 <= rot <= d");
  if (d > kMostD) return fail(HDP_ERR_UNSUPPORTED, name + "d must be at most 256");
  if (type != HDP_TYPE_BF16 && type != HDP_TYPE_FP16 && type != HDP_TYPE_FP32)
    return fail(HDP_ERR_INVALID_ARGUMENT, name + "unknown type");
  if (flags & ~(HDP_ROTARY_NEIGHBOURS | HDP_ROTARY_BACKWARD)) return fail(HDP_ERR_INVALID_ARGUMENT, name + "unknown flag");
  if (!(factor > 0.f) || !(factor < __builtin_inff()))
    return fail(HDP_ERR_INVALID_ARGUMENT, name + "factor must be a positive number");
  const int size = type == HDP_TYPE_FP32 ? 4 : 2;
  const bool neighbours = flags & HDP_ROTARY_NEIGHBOURS;
  Rotary p = {};
  uintptr_t bits = 0;  // of everything that 16-byte accesses need to be a multiple of 16
  const hdp_rotary_rows_t* both[2] = {q, k};
  for (int i = 0; i < 2; ++i) {
    const hdp_rotary_rows_t* x = both[i];
    if (!x || x->heads == 0) continue;
    if (x->heads < 0 || x->heads > (1 << 20)) return fail(HDP_ERR_INVALID_ARGUMENT, name + "heads must be 0 .. 2^20");
    if (rows > 0 && (!x->in || !x->out)) return fail(HDP_ERR_INVALID_ARGUMENT, name + "NULL argument");
    if ((reinterpret_cast<uintptr_t>(x->in) | reinterpret_cast<uintptr_t>(x->out)) % size)
      return fail(HDP_ERR_INVALID_ARGUMENT, name + "rows must be aligned to their elements");
    if (rows > 0 && x->in == x->out && (x->in_row_stride != x->out_row_stride || x->in_head_stride != x->out_head_stride))
      return fail(HDP_ERR_INVALID_ARGUMENT, name + "in place, the strides of both sides must be the same");
    p.x[i] = {static_cast<const char*>(x->in), static_cast<char*>(x->out), x->in_row_stride, x->in_head_stride,
              x->out_row_stride, x->out_head_stride};
    p.heads[i] = x->heads;
    bits |= reinterpret_cast<uintptr_t>(x->in) | reinterpret_cast<uintptr_t>(x->out);
    bits |= static_cast<uintptr_t>(x->in_row_stride | x->in_head_stride | x->out_row_stride | x->out_head_stride) * size;
    p.copy = p.copy || x->in != x->out;
  }
  if (rows == 0 || p.heads[0] + p.heads[1] == 0) return HDP_OK;
  if (!position || !freqs) return fail(HDP_ERR_INVALID_ARGUMENT, name + "position or freqs is NULL");
  if (reinterpret_cast<uintptr_t>(freqs) & 7) return fail(HDP_ERR_INVALID_ARGUMENT, name + "freqs must be 8-byte aligned");
  p.copy = p.copy && rot < d;
  bits |= static_cast<uintptr_t>(rot / 2) * size;
  if (p.copy) bits |= static_cast<uintptr_t>(d - rot) * size;
  p.pos = position;
  p.freqs = freqs;
  p.rows = static_cast<int>(rows);
  p.d = d;
  p.rot = rot;
  p.factor = factor;
  p.sign = flags & HDP_ROTARY_BACKWARD ? -1.f : 1.f;
  p.tile = rows <= 4 * 152 ? 1 : 4;
  const int bytes = bits & 15 ? size : 16;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (type == HDP_TYPE_BF16) launch_for<__nv_bfloat16>(p, bytes, neighbours, st);
  else if (type == HDP_TYPE_FP16) launch_for<__half>(p, bytes, neighbours, st);
  else launch_for<float>(p, bytes, neighbours, st);
  note_launch();
  HDP_CUDA_TRY(cudaGetLastError());
  return HDP_OK;
}
