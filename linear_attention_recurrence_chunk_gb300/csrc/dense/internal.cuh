// The dense half of a decoder layer: the launchers behind include/kda_dense.h
// and the device helpers that its kernels share.
#pragma once

#include <cuda_fp8.h>

#include "kda_dense.h"
#include "kda_internal.cuh"

namespace kda {
namespace dense {

constexpr int kBlock = 128;   // columns of a scale

// ------------------------------------------------------------------ 8-bit values
// Scale byte of a block whose largest |value| has the fp32 bits `top`: the exponent field b
// of the least 2^(b - 127), b >= 1, with top <= 448 * 2^(b - 127); 255 for an inf or NaN.
// 448 = 1.75 * 2^8: top = m 2^(E - 127) fits b = E - 8 when m <= 1.75, else E - 7, so b is the
// exponent field of top + 0x1fffff, minus 8 (a mantissa above 0x600000 carries).
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  if (top >= 0x7f800000u) return 255u;
  return (uint32_t)max(1, (int)((top + 0x1fffffu) >> 23) - 8);
}
// 1 / scale, exact: 2^(127 - byte) for the bytes that scale_byte gives below 255 (1 .. 247).
__device__ __forceinline__ float scale_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }
// 2^(byte - 127) of any byte; NaN for 255.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7fc00000u : byte << 23);
}
// Two values (at most 448 in size) to E4M3, the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 e4m3x2_values(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// --------------------------------------------------- eight values of a row per lane
// A warp takes 256 columns of a row at a time.  kWide: lane l has columns 8 l .. 8 l + 7 (one
// 16-byte load of bf16), and 16 lanes hold a block of 128.  Otherwise (rows of any alignment) lane l
// has columns l, l + 32, ..., so that neighbours stay neighbours; values 0 .. 3 are of the first block
// of 128, 4 .. 7 of the second.
template <bool kWide>
__device__ __forceinline__ int column(int lane, int i) {
  return kWide ? 8 * lane + i : lane + 32 * i;
}

template <typename T, bool kWide>
__device__ __forceinline__ void load8(const T* row, int64_t c0, int64_t C, int lane, float (&v)[8]) {
  if constexpr (kWide) {
    const int64_t c = c0 + 8 * lane;
    if (c >= C) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
    } else if constexpr (sizeof(T) == 2) {
      const uint4 u = __ldcs(reinterpret_cast<const uint4*>(row + c));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    } else {
      const float4 a = __ldcs(reinterpret_cast<const float4*>(row + c)), b = __ldcs(reinterpret_cast<const float4*>(row + c) + 1);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t c = c0 + lane + 32 * i;
      v[i] = c < C ? to_f32<T>(row[c]) : 0.f;
    }
  }
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 z = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&z);
}

template <typename T, bool kWide>
__device__ __forceinline__ void store8(T* row, int64_t c0, int64_t C, int lane, const float (&v)[8]) {
  if constexpr (kWide) {
    const int64_t c = c0 + 8 * lane;
    if (c >= C) return;
    if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<uint4*>(row + c) = make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
    } else {
      reinterpret_cast<float4*>(row + c)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(row + c)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t c = c0 + lane + 32 * i;
      if (c < C) row[c] = from_f32<T>(v[i]);
    }
  }
}

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// Largest |value| bits of each lane's block or blocks: `a` of values 0 .. 3, `b` of 4 .. 7
// (kWide: the same block).
template <bool kWide>
__device__ __forceinline__ void block_tops(const float (&v)[8], uint32_t& a, uint32_t& b) {
  a = max(max(magnitude(v[0]), magnitude(v[1])), max(magnitude(v[2]), magnitude(v[3])));
  b = max(max(magnitude(v[4]), magnitude(v[5])), max(magnitude(v[6]), magnitude(v[7])));
  if constexpr (kWide) {
    a = max(a, b);
#pragma unroll
    for (int m = 8; m > 0; m >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, m));
    b = a;
  } else {
    a = __reduce_max_sync(0xffffffffu, a);
    b = __reduce_max_sync(0xffffffffu, b);
  }
}

// The values' codes under the scale bytes of their blocks, as two words of four.
__device__ __forceinline__ uint2 codes8(const float (&v)[8], uint32_t byte_a, uint32_t byte_b) {
  const float ia = scale_inverse(byte_a), ib = scale_inverse(byte_b);
  uint2 w;
  w.x = e4m3x2(v[0] * ia, v[1] * ia) | e4m3x2(v[2] * ia, v[3] * ia) << 16;
  w.y = e4m3x2(v[4] * ib, v[5] * ib) | e4m3x2(v[6] * ib, v[7] * ib) << 16;
  if (byte_a == 255u) w.x = 0;
  if (byte_b == 255u) w.y = 0;
  return w;
}

template <bool kWide>
__device__ __forceinline__ void store_codes(uint8_t* row, int64_t c0, int64_t C, int lane, uint2 w) {
  if constexpr (kWide) {
    const int64_t c = c0 + 8 * lane;
    if (c < C) *reinterpret_cast<uint2*>(row + c) = w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t c = c0 + lane + 32 * i;
      if (c < C) row[c] = (uint8_t)((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
    }
  }
}

// The 256 columns' values in 8 bits: codes, and a scale byte for each block of 128.
template <bool kWide>
__device__ __forceinline__ void store_fp8(uint8_t* codes_row, uint8_t* scales_row, int64_t c0, int64_t C, int lane,
                                          const float (&v)[8]) {
  uint32_t a, b;
  block_tops<kWide>(v, a, b);
  const uint32_t ba = scale_byte(a), bb = scale_byte(b);
  store_codes<kWide>(codes_row, c0, C, lane, codes8(v, ba, bb));
  const int64_t c = c0 + (kWide ? 8 * lane : 0);
  if constexpr (kWide) {
    if ((lane & 15) == 0 && c < C) scales_row[c / kBlock] = (uint8_t)ba;
  } else if (lane < 2 && c0 + kBlock * lane < C) {
    scales_row[c0 / kBlock + lane] = (uint8_t)(lane ? bb : ba);
  }
}

// ---------------------------------------------------------------------- launchers
struct QuantProblem {
  const void* x;
  int64_t stride, T, C;
  int32_t rows;
  kda_dtype dt;
  uint8_t *codes, *scales;
};
cudaError_t launch_quant(const QuantProblem& p, cudaStream_t stream);

struct ValuesProblem {
  const uint8_t *codes, *scales;
  int64_t T, C;
  int32_t rows;
  kda_dtype dt;
  void* y;
};
cudaError_t launch_values(const ValuesProblem& p, cudaStream_t stream);

constexpr int64_t kNormMost = 32768;
struct NormProblem {
  const void* x;
  int64_t xs;
  const void* r;
  int64_t rs;
  const float* w;
  float eps;
  int64_t T, C;
  kda_dtype dt;
  void *h, *y;
  uint8_t *codes, *scales;
};
cudaError_t launch_norm(const NormProblem& p, cudaStream_t stream);

struct MatmulProblem {
  const uint8_t *a, *sa, *w, *sw;
  int64_t lda, ldw, M, N, K;
  kda_dtype dt;
  void* out;
  int64_t ldo;
  int32_t* dev_err;
};
cudaError_t launch_matmul(const MatmulProblem& p, cudaStream_t stream);
cudaError_t launch_matmul_pair(const MatmulProblem& p, int sms, cudaStream_t stream);   // many rows

struct RotaryPart {   // queries or keys
  const void* x;
  void* y;
  int64_t xt, xh, yt, yh;   // strides in elements
  int32_t H;
};
struct RotaryProblem {
  RotaryPart q, k;
  const int32_t* pos;
  const double* freqs;
  int64_t T;
  int32_t D, rot;
  float amplitude;
  int32_t flags;
  kda_dtype dt;
};
cudaError_t launch_rotary(const RotaryProblem& p, cudaStream_t stream);

}  // namespace dense
}  // namespace kda
