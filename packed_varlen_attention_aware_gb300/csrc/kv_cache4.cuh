// The 4-bit key/value cache as the kernels see it.
#pragma once
#include "kv_cache.cuh"

namespace hdp {

// Device-side view of an hdp_fourbit_cache_t (the float scales and bounds of CacheView stay unused).
struct Cache4View : CacheView {
  uint8_t* scale_bytes;
};

// Bytes of a block's codes (of K, and of V) and scales for one kv head.
template <int D>
constexpr int kCodes4 = kBlock * D / 2;
template <int D>
constexpr int kPlanes4 = D / 32 + 1;  // a row of 64 bytes for 32 channels of K each, then V's
template <int D>
constexpr int kScales4 = kPlanes4<D> * kBlock;

// Place of token t in a row of 64 scales: a lane of a matrix fragment has tokens 8 j + r of one r.
__device__ __forceinline__ int scale_place(int t) { return (t & 7) * 8 + (t >> 3); }

// Host: checks what every call needs and fills the view (kv_cache4.cu).
hdp_status_t cache4_view(const char* call, const hdp_fourbit_cache_t* c, const int32_t* cu, int64_t rows, Cache4View* out);

}  // namespace hdp
