// Element loads and stores shared by the expert-FFN kernels: bf16, f16 or
// f32 in memory, float32 in registers.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "reshard.h"

namespace rs {

typedef uint32_t ou32x4 __attribute__((ext_vector_type(4)));
// The same at any address that suits its elements: the device's loads and
// stores of 8 and 16 bytes need no alignment of their own, so rows of any
// stride go eight elements at a time (4000 x 4099 bf16 values quantised: 14 us,
// an element at a time 25; six rows of 2049 a token combined: 28 and 68).
typedef ou32x4 ou32x4_2 __attribute__((aligned(2)));
typedef uint64_t ou64_1 __attribute__((aligned(1)));

__host__ __device__ inline int64_t dtype_size(int dtype) { return dtype == RS_F32 ? 4 : 2; }

__device__ __forceinline__ float bf16_float(uint32_t b) { return __uint_as_float(b << 16); }
__device__ __forceinline__ float f16_float(uint32_t b) {
  return float(__builtin_bit_cast(_Float16, uint16_t(b)));
}
// Round to nearest even; NaN stays NaN.
__device__ __forceinline__ uint32_t float_bf16(float f) { return __builtin_bit_cast(uint16_t, __bf16(f)); }
__device__ __forceinline__ uint32_t float_f16(float f) { return __builtin_bit_cast(uint16_t, _Float16(f)); }

__device__ __forceinline__ float load1(const void* p, int dtype, int64_t i) {
  if (dtype == RS_F32) return static_cast<const float*>(p)[i];
  const uint32_t b = static_cast<const uint16_t*>(p)[i];
  return dtype == RS_BF16 ? bf16_float(b) : f16_float(b);
}
__device__ __forceinline__ void store1(void* p, int dtype, int64_t i, float v) {
  if (dtype == RS_F32) static_cast<float*>(p)[i] = v;
  else static_cast<uint16_t*>(p)[i] = uint16_t(dtype == RS_BF16 ? float_bf16(v) : float_f16(v));
}

// Eight consecutive elements as they lie in memory, so that loads can be under
// way before the first is widened.  NT: non-temporal, for data read once.
template <int DTYPE>
struct Raw8 {
  ou32x4 a, b;
  // n (1..8) elements from index i, zeros behind them.
  template <bool NT = true>
  __device__ __forceinline__ void load(const void* p, int64_t i, int n) {
    const char* at = static_cast<const char*>(p) + i * dtype_size(DTYPE);
    if (n == 8) {
      const ou32x4_2* q = reinterpret_cast<const ou32x4_2*>(at);
      a = NT ? __builtin_nontemporal_load(q) : q[0];
      if (DTYPE == RS_F32) b = NT ? __builtin_nontemporal_load(q + 1) : q[1];
      return;
    }
    a = b = ou32x4{0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < 7; ++k) {
      if (k >= n) break;
      if (DTYPE == RS_F32) (k < 4 ? a : b)[k & 3] = reinterpret_cast<const uint32_t*>(at)[k];
      else a[k / 2] |= uint32_t(reinterpret_cast<const uint16_t*>(at)[k]) << (16 * (k & 1));
    }
  }
  __device__ __forceinline__ float get(int k) const {
    if (DTYPE == RS_F32) return __uint_as_float(k < 4 ? a[k & 3] : b[k & 3]);
    const uint32_t h = k & 1 ? a[k / 2] >> 16 : a[k / 2] & 0xFFFFu;
    return DTYPE == RS_BF16 ? bf16_float(h) : f16_float(h);
  }
};

// Eight elements from index i as float32.
__device__ __forceinline__ void load8(const void* p, int dtype, int64_t i, float v[8]) {
  if (dtype == RS_F32) {
    Raw8<RS_F32> r;
    r.load<false>(p, i, 8);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = r.get(k);
  } else {
    Raw8<RS_BF16> r;  // the bits
    r.load<false>(p, i, 8);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t h = k & 1 ? r.a[k / 2] >> 16 : r.a[k / 2] & 0xFFFFu;
      v[k] = dtype == RS_BF16 ? bf16_float(h) : f16_float(h);
    }
  }
}

// n (1..8) elements to index i, by non-temporal stores if there are eight
// (combining 8192 tokens' rows: 216 us with cached stores, 199 us with these).
template <bool NT = true>
__device__ __forceinline__ void store8(void* p, int dtype, int64_t i, int n, const float v[8]) {
  if (n < 8) {
#pragma unroll
    for (int k = 0; k < 7; ++k)
      if (k < n) store1(p, dtype, i + k, v[k]);
    return;
  }
  ou32x4_2* q = reinterpret_cast<ou32x4_2*>(static_cast<char*>(p) + i * dtype_size(dtype));
  ou32x4 a, b;
  if (dtype == RS_F32) {
#pragma unroll
    for (int k = 0; k < 4; ++k) a[k] = __float_as_uint(v[k]), b[k] = __float_as_uint(v[4 + k]);
    if (NT) __builtin_nontemporal_store(b, q + 1);
    else q[1] = b;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      a[k] = dtype == RS_BF16 ? float_bf16(v[2 * k]) | float_bf16(v[2 * k + 1]) << 16
                              : float_f16(v[2 * k]) | float_f16(v[2 * k + 1]) << 16;
  }
  if (NT) __builtin_nontemporal_store(a, q);
  else q[0] = a;
}

}  // namespace rs
