// Rotary positions of query and key rows, and their gradient.
//
// A pair (a, b) of a head's first `rot` channels at position p becomes
//   (f (a cos x - b sin x), f (b cos x + a sin x)),   x = p theta_i,
// and the gradient of a is f times the turn by -x.  2 d bytes in and out for each
// element of q and k against a few operations: HBM bounds it.
//
//   Angles.  p theta in fp32 is off by 0.1 radians at two million positions.  The
//   angle is kept in turns instead, as a 64-bit fraction: theta / 2 pi mod 1 times
//   2^64 is a whole number, cut off from the exact product of theta's 53 bits and 128
//   bits of 1 / 2 pi; p times it mod 2^64 is exact, and what is left is the angle's
//   fraction of a turn to 2^-33 for any 31-bit p and |theta| < 2^53.  (A double holds
//   theta / 2 pi to 2^-53 of itself only: times 2^31 that is 2^-18 of a turn at 100
//   radians a position.)  As a signed number it is within half a turn, which sincospi
//   takes in fp32.
//   Sharing.  A token's cosines and sines serve all its heads: a CTA works them out
//   for a tile of tokens, one pair a thread, and its threads then go over the
//   tile's (token, head) units, 16 bytes of each half of a pair at a time.
//   Where only rot does not allow 16 bytes of each half, a lane has 16 bytes of a head and
//   looks for their partners in it or in shared memory; other rows go by two elements or
//   one at a time.
//
// Measured: 40,121 rows of 40 heads of 128 bf16, 124 us, 0.97 of the copy rate; 131,072 of
// 40 heads with 64 of 128 channels turned, the gradient, 418 us, 0.95; 131,072 of 10
// heads, as many turned, 117 us, 0.85: there a token's angles count.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cstdlib>
#include <string>
#include <type_traits>

#include "internal.h"

namespace hdp {
namespace {

constexpr int kThreads = 256;
constexpr int kMostD = 256;
constexpr int kMostTile = 16;  // tokens of a CTA

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

// Cosines, sines and positions of a tile.
extern __shared__ __align__(16) float s_angles[];

int shared_bytes(const Rotary& p) { return p.tile * (p.rot + 1) * 4; }

// theta / 2 pi mod 1 in units of 2^-64, cut off: theta = m 2^e, and m / 2 pi, with the digits
// of 1 / 2 pi as whole numbers (Payne and Hanek, 1983), has 64 bits in front of the point and
// 128 behind it.
__device__ __forceinline__ unsigned long long turns(double theta) {
  using u64 = unsigned long long;
  constexpr u64 kHigh = 0x28be60db9391054aull, kLow = 0x7f09d5f47d4d3770ull;  // 2^128 / 2 pi
  const u64 bits = static_cast<u64>(__double_as_longlong(theta));
  const int e = static_cast<int>(bits >> 52 & 0x7ff) - 1075;
  const u64 m = (bits & 0xfffffffffffffull) | 1ull << 52;
  const u64 p0 = kLow * m, p1 = __umul64hi(kLow, m) + kHigh * m;
  const u64 p2 = __umul64hi(kHigh, m) + (p1 < kHigh * m);
  const int shift = 64 - e;  // (of a subnormal theta's too: nothing is left)
  u64 x = 0;
  if (shift >= 128) x = shift < 192 ? p2 >> (shift - 128) : 0;
  else if (shift > 64) x = p1 >> (shift - 64) | p2 << (128 - shift);
  else if (shift == 64) x = p1;
  else if (shift > 0) x = p0 >> shift | p1 << (64 - shift);
  return theta < 0 ? 0 - x : x;
}

// Positions of the tile's tokens, and cosines and sines of their pairs.
__device__ __forceinline__ void angles(const Rotary& p, long long row0, int n, float* s_cos, float* s_sin, int* s_pos) {
  const int half = p.rot / 2, tokens = kThreads / half;  // at a time
  const int t0 = threadIdx.x / half, i = threadIdx.x - t0 * half;
  if (t0 < tokens && t0 < n) {
    int at = __ldg(p.pos + row0 + t0);
    const unsigned long long step = turns(__ldg(p.freqs + i));
    for (int t = t0, now; t < n; t += tokens) {
      now = at;
      if (t + tokens < n) at = __ldg(p.pos + row0 + t + tokens);
      const unsigned long long fraction = step * static_cast<unsigned long long>(static_cast<long long>(now));
      float s, c;
      sincospif(__ll2float_rn(static_cast<long long>(fraction)) * 1.0842021724855044e-19f, &s, &c);  // 2^-63
      s_cos[t * half + i] = c * p.factor;
      s_sin[t * half + i] = s * p.factor * p.sign;
      if (i == 0) s_pos[t] = now;
    }
  }
  __syncthreads();
}

// A thread has V pairs of a unit, W elements at a time: W = V, but for one pair of
// neighbours, whose two elements may be one access (W = 2).
template <class T, int V, int W, bool NEIGHBOURS>
__global__ void __launch_bounds__(kThreads) k_rotary(const Rotary p) {
  const int half = p.rot / 2;
  float* s_cos = s_angles;
  float* s_sin = s_angles + p.tile * half;
  int* s_pos = reinterpret_cast<int*>(s_angles + 2 * p.tile * half);
  const long long row0 = static_cast<long long>(blockIdx.x) * p.tile;
  const int n = static_cast<int>(min(static_cast<long long>(p.tile), p.rows - row0));
  angles(p, row0, n, s_cos, s_sin, s_pos);

  // A unit is one head of one token: `pairs` threads with V pairs each, then those that copy.
  const int pairs = half / V, group = pairs + (p.copy ? (p.d - p.rot + 2 * W - 1) / (2 * W) : 0);
  const int groups = kThreads / group;
  const int g = threadIdx.x / group, j = threadIdx.x - g * group;
  if (g >= groups) return;
  const int all = p.heads[0] + p.heads[1], units = n * all;
  // Other warps hide a unit's latency better than its neighbours do: unrolled by four, 131,072
  // rows of 40 heads with half of their channels turned took 471 us, not 417.
#pragma unroll 1
  for (int u = g; u < units; u += groups) {
    const int t = u / all;
    int h = u - t * all;
    if (s_pos[t] < 0) continue;
    const bool second = h >= p.heads[0];
    if (second) h -= p.heads[0];
    const RotaryTensor& x = p.x[second];
    const T* in = reinterpret_cast<const T*>(x.in) + (row0 + t) * x.in_row + h * x.in_head;
    T* out = reinterpret_cast<T*>(x.out) + (row0 + t) * x.out_row + h * x.out_head;
    if (j < pairs && W == 2 * V) {
      Vec<T, W> a = get<T, W>(in + 2 * j);
      const float c = s_cos[t * half + j], s = s_sin[t * half + j], y0 = to_float(a.v[0]), y1 = to_float(a.v[W - 1]);
      a.v[0] = from_float<T>(turned(y0, c, -y1, s));
      a.v[W - 1] = from_float<T>(turned(y1, c, y0, s));
      put(out + 2 * j, a);
    } else if (j < pairs) {
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
      const int c0 = p.rot + (j - pairs) * 2 * W;
      put(out + c0, get<T, W>(in + c0));
      if (c0 + W < p.d) put(out + c0 + W, get<T, W>(in + c0 + W));
    }
  }
}

// Rows that allow 16 bytes but for rot: a unit is whole 16-byte pieces of a head, a lane
// each.  Neighbours are in one piece; halves are found in shared memory, where the warp
// puts its pieces.  Channels behind rot keep their bits.
template <class T, bool NEIGHBOURS>
__global__ void __launch_bounds__(kThreads) k_rotary_pieces(const Rotary p) {
  constexpr int V = 16 / sizeof(T);
  __shared__ __align__(16) T s_x[NEIGHBOURS ? 1 : kThreads * V];
  const int half = p.rot / 2;
  float* s_cos = s_angles;
  float* s_sin = s_angles + p.tile * half;
  int* s_pos = reinterpret_cast<int*>(s_angles + 2 * p.tile * half);
  const long long row0 = static_cast<long long>(blockIdx.x) * p.tile;
  const int n = static_cast<int>(min(static_cast<long long>(p.tile), p.rows - row0));
  angles(p, row0, n, s_cos, s_sin, s_pos);

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int pieces = p.d / V, each = 32 / pieces;  // of a unit; units of a warp
  const int mine = lane / pieces, j = lane - mine * pieces;
  const int all = p.heads[0] + p.heads[1], units = n * all;
  T* x0 = s_x + (NEIGHBOURS ? 0 : (warp * 32 + mine * pieces) * V);  // the unit's channels
  for (int u0 = warp * each; u0 < units; u0 += kThreads / 32 * each) {
    const int u = u0 + mine;
    const bool on = mine < each && u < units && s_pos[u / all] >= 0 && (p.copy || j * V < p.rot);
    const int t = u / all;
    int h = u - t * all;
    const bool second = h >= p.heads[0];
    if (second) h -= p.heads[0];
    const RotaryTensor& x = p.x[second];
    Vec<T, V> y;
    if (on) y = get<T, V>(reinterpret_cast<const T*>(x.in) + (row0 + t) * x.in_row + h * x.in_head + j * V);
    if constexpr (!NEIGHBOURS) {
      __syncwarp();
      if (on) put(x0 + j * V, y);
      __syncwarp();
    }
    if (!on) continue;
    const float* cos = s_cos + t * half;
    const float* sin = s_sin + t * half;
    if constexpr (NEIGHBOURS) {
#pragma unroll
      for (int k = 0; k < V; k += 2) {
        const int i = (j * V + k) / 2;
        if (i >= half) continue;
        const float c = cos[i], s = sin[i], y0 = to_float(y.v[k]), y1 = to_float(y.v[k + 1]);
        y.v[k] = from_float<T>(turned(y0, c, -y1, s));
        y.v[k + 1] = from_float<T>(turned(y1, c, y0, s));
      }
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int ch = j * V + k;
        if (ch >= p.rot) continue;
        const bool up = ch >= half;
        const int i = up ? ch - half : ch;
        const float other = to_float(x0[up ? i : ch + half]);
        y.v[k] = from_float<T>(turned(to_float(y.v[k]), cos[i], up ? other : -other, sin[i]));
      }
    }
    put(reinterpret_cast<T*>(x.out) + (row0 + t) * x.out_row + h * x.out_head + j * V, y);
  }
}

template <class T, int V, int W, bool NEIGHBOURS>
void launch(const Rotary& p, cudaStream_t st) {
  k_rotary<T, V, W, NEIGHBOURS><<<static_cast<unsigned>((p.rows + p.tile - 1) / p.tile), kThreads, shared_bytes(p), st>>>(p);
}

// `bits`: of addresses and strides, `lengths`: of rot / 2 and what is copied, in bytes: an
// access of a size needs both to be multiples of it, pieces need the former only.  Measured
// on 4,687 rows of 72 heads of 64 bf16 (12.7 us at the copy rate): 30 channels turned, by
// pieces 25 us (neighbours) and 37 (halves), by two elements 39 (neighbours), one at a time
// 47 and 51; 36 channels, halves, by two elements 29 us, by pieces 38.
template <class T>
void launch_for(const Rotary& p, uintptr_t bits, uintptr_t lengths, bool neighbours, cudaStream_t st) {
  constexpr int wide = 16 / sizeof(T);
  const int two = 2 * sizeof(T);
  const unsigned ctas = static_cast<unsigned>((p.rows + p.tile - 1) / p.tile);
  const bool pieces = !(bits & 15) && p.d % wide == 0 && p.d / wide <= 32;
  if (!((bits | lengths) & 15)) {
    if (neighbours) launch<T, wide, wide, true>(p, st);
    else launch<T, wide, wide, false>(p, st);
  } else if (neighbours) {
    if (pieces) k_rotary_pieces<T, true><<<ctas, kThreads, shared_bytes(p), st>>>(p);
    else if (bits % two == 0 && (!p.copy || (p.d - p.rot) % 2 == 0)) launch<T, 1, 2, true>(p, st);
    else launch<T, 1, 1, true>(p, st);
  } else {
    if ((bits | lengths) % two == 0) launch<T, 2, 2, false>(p, st);
    else if (pieces) k_rotary_pieces<T, false><<<ctas, kThreads, shared_bytes(p), st>>>(p);
    else launch<T, 1, 1, false>(p, st);
  }
}

// Rows of a tensor as the host sees them, in elements.
struct Places {
  long long at, row, head;
  int heads;
};

// Is |x + n step| < d for an n in [-most, most]?
bool comes_near(long long x, long long step, long long most, int d) {
  if (step < 0) step = -step;
  long long n = 0;  // the largest with x + n step <= 0
  if (step > 0) n = x > 0 ? -((x + step - 1) / step) : -x / step;
  for (int i = 0; i < 2; ++i) {
    const long long y = x + std::min(std::max(n + i, -most), most) * step;
    if (-d < y && y < d) return true;
  }
  return false;
}

// First and last element; false if they are not places in memory.
bool ends_of(const Places& x, long long rows, int d, long long& first, long long& last) {
  __int128 lo = x.at, hi = lo + d - 1;
  for (const __int128 far : {static_cast<__int128>(x.row) * (rows - 1), static_cast<__int128>(x.head) * (x.heads - 1)})
    (far < 0 ? lo : hi) += far;
  constexpr long long kMost = 1LL << 61;
  if (lo < -kMost || hi > kMost) return false;
  first = static_cast<long long>(lo);
  last = static_cast<long long>(hi);
  return true;
}

// May a and b have an element in common?  A "no" is sure, and so is a "yes" but for rows
// with different strides, or more heads than are worth comparing, within the same memory.
bool may_meet(Places a, Places b, long long rows, int d) {
  long long a0, a1, b0, b1;
  if (!ends_of(a, rows, d, a0, a1) || !ends_of(b, rows, d, b0, b1)) return true;
  if (a1 < b0 || b1 < a0) return false;
  if (rows > 1 && a.row != b.row) return true;
  if (a.heads == 1) a.head = b.head;
  if (b.heads == 1) b.head = a.head;
  const long long x = a.at - b.at;
  if (a.head == b.head) {
    for (int m = 1 - b.heads; m < a.heads; ++m)
      if (comes_near(x + m * a.head, a.row, rows - 1, d)) return true;
    return false;
  }
  if (static_cast<long long>(a.heads) * b.heads > 1 << 16) return true;
  for (int h = 0; h < a.heads; ++h)
    for (int g = 0; g < b.heads; ++g)
      if (comes_near(x + h * a.head - g * b.head, a.row, rows - 1, d)) return true;
  return false;
}

// Do two heads of two rows of x have an element in common?
bool meets_itself(const Places& x, long long rows, int d) {
  long long first, last;
  if (!ends_of(x, rows, d, first, last)) return true;
  const long long row = std::abs(x.row), head = std::abs(x.head);
  if (rows > 1 && row < d) return true;
  if (x.heads == 1 || (head >= d && (rows == 1 || row >= head * (x.heads - 1) + d))) return false;
  for (int m = 1; m < x.heads; ++m)
    if (comes_near(m * x.head, x.row, rows - 1, d)) return true;
  return false;
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
  uintptr_t bits = 0;  // of addresses and strides in bytes
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
  Places in[2], out[2];
  for (int i = 0; i < 2; ++i) {
    if (!p.heads[i]) continue;
    const RotaryTensor& x = p.x[i];
    const auto places = [&](const char* at, long long row, long long head) -> Places {  // (a stride to nowhere says nothing)
      return {static_cast<long long>(reinterpret_cast<intptr_t>(at) / size), rows > 1 ? row : 0, p.heads[i] > 1 ? head : 0, p.heads[i]};
    };
    in[i] = places(x.in, x.in_row, x.in_head);
    out[i] = places(x.out, x.out_row, x.out_head);
    if (meets_itself(out[i], rows, d))
      return fail(HDP_ERR_INVALID_ARGUMENT, name + "rows and heads of an output must not overlap");
    if (x.in != x.out && may_meet(in[i], out[i], rows, d))
      return fail(HDP_ERR_INVALID_ARGUMENT, name + "an output must be its input or not overlap it");
  }
  if (p.heads[0] && p.heads[1] &&
      (may_meet(out[0], out[1], rows, d) || (p.x[1].in != p.x[1].out && may_meet(out[0], in[1], rows, d)) ||
       (p.x[0].in != p.x[0].out && may_meet(out[1], in[0], rows, d))))
    return fail(HDP_ERR_INVALID_ARGUMENT, name + "what is written for q and k must not be rows of the other");
  if (!position || !freqs) return fail(HDP_ERR_INVALID_ARGUMENT, name + "position or freqs is NULL");
  if (reinterpret_cast<uintptr_t>(freqs) & 7) return fail(HDP_ERR_INVALID_ARGUMENT, name + "freqs must be 8-byte aligned");
  p.copy = p.copy && rot < d;
  uintptr_t lengths = static_cast<uintptr_t>(rot / 2) * size;
  if (p.copy) lengths |= static_cast<uintptr_t>(d - rot) * size;
  p.pos = position;
  p.freqs = freqs;
  p.rows = static_cast<int>(rows);
  p.d = d;
  p.rot = rot;
  p.factor = factor;
  p.sign = flags & HDP_ROTARY_BACKWARD ? -1.f : 1.f;
  // Tokens of a CTA: as many as make 1,280 accesses of 16 bytes of each half, and as leave
  // four CTAs for each SM.  Measured with 1, 2, 4, 8, 16: 40,121 rows of 40 heads of 128,
  // 160, 135, 125, 127, 130 us; 50,000 of 20, 137, 106, 88, 81, 85; 131,072 of 10, half of their channels turned,
  // 317, 200, 166, 138, 126; 608 of 40, 4.6, 4.6, 5.1, 7.4, 12.
  const int64_t accesses = static_cast<int64_t>(p.heads[0] + p.heads[1]) * (((p.copy ? d : rot) * size + 31) / 32);
  for (p.tile = 1; p.tile < kMostTile && p.tile * accesses < 1280 && rows > 4 * 152 * p.tile;) p.tile *= 2;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (type == HDP_TYPE_BF16) launch_for<__nv_bfloat16>(p, bits, lengths, neighbours, st);
  else if (type == HDP_TYPE_FP16) launch_for<__half>(p, bits, lengths, neighbours, st);
  else launch_for<float>(p, bits, lengths, neighbours, st);
  note_launch();
  HDP_CUDA_TRY(cudaGetLastError());
  return HDP_OK;
}
