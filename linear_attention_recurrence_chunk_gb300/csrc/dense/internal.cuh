// The dense half of a decoder layer: the launchers behind include/kda_dense.h
// and the device helpers that its kernels share.
#pragma once

#include <cuda_fp8.h>

#include "kda_dense.h"
#include "kda_internal.cuh"

namespace kda {
namespace dense {

constexpr int kBlock = 128;   // columns of a scale

// -------------------------------------------------------------- launches one behind another
// Every kernel here is launched so that it may start while the one before it in the stream ends, and lets the next one
// do so at once (one thread of a CTA says so for it); a product only when it has its tensor memory.  CTAs of the next
// product take theirs before they wait and give it back after this one has ended: were this one still without its own,
// each could wait for the other.  No kernel touches global memory before all that ran before it is complete and visible, or
// loads by the read-only path or through __restrict__ pointers, since what they read may be written while it waits.  Taken in
// turn with plain launches: a product of one row, 16,416 x 4,096, 13.0 us a call against 15.6, 8 x 2,052 x 512 in
// a graph 2.4 against 3.2, 8,192 x 12,288 to 8 bits and back 92.6 against 96.9.  CTAs that wait keep their threads,
// registers and shared memory from other streams as long as the kernel before them runs (not timed).
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// cluster: CTAs of a cluster, 0 for what the kernel itself says.
template <typename... P, typename... A>
cudaError_t launch_kernel(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

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

// The eight values as they lie in memory (zeros behind C), and as fp32.
template <typename T, bool kWide>
struct Eight {
  alignas(kWide ? 16 : sizeof(T)) T x[8];
  __device__ __forceinline__ void load(const T* row, int64_t c0, int64_t C, int lane) {
    if constexpr (kWide) {
      const int64_t c = c0 + 8 * lane;
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i)
        reinterpret_cast<uint4*>(x)[i] = c < C ? __ldcs(reinterpret_cast<const uint4*>(row + c) + i) : make_uint4(0, 0, 0, 0);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t c = c0 + lane + 32 * i;
        x[i] = c < C ? row[c] : from_f32<T>(0.f);
      }
    }
  }
  __device__ __forceinline__ float at(int i) const { return to_f32<T>(x[i]); }
};

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

// Largest size of three or two values, a NaN above all.
__device__ __forceinline__ float top3(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(fabsf(a)), "f"(fabsf(b)), "f"(fabsf(c)));
  return d;
}
__device__ __forceinline__ float top2(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(fabsf(a)), "f"(fabsf(b)));
  return d;
}

// The fp32 bits of the largest size of each lane's block or blocks: `a` of values 0 .. 3, `b` of 4 .. 7
// (kWide: the same block, of 16 lanes).
__device__ __forceinline__ uint32_t half_warp_max(uint32_t t) {
#pragma unroll
  for (int m = 8; m > 0; m >>= 1) t = max(t, __shfl_xor_sync(0xffffffffu, t, m));
  return t;
}
template <bool kWide>
__device__ __forceinline__ void block_tops(const float (&v)[8], uint32_t& a, uint32_t& b) {
  const float lo = top2(v[3], top3(v[0], v[1], v[2])), hi = top2(v[7], top3(v[4], v[5], v[6]));
  if constexpr (kWide) {
    a = b = half_warp_max(__float_as_uint(top2(lo, hi)));
  } else {
    a = __reduce_max_sync(0xffffffffu, __float_as_uint(lo));
    b = __reduce_max_sync(0xffffffffu, __float_as_uint(hi));
  }
}
// The lane's own largest size.
template <typename T, bool kWide>
__device__ __forceinline__ uint32_t lane_top(const Eight<T, kWide>& v) {
  if constexpr (sizeof(T) == 2 && kWide) {   // two values a word: sizes compare as whole numbers
    const uint32_t* w = reinterpret_cast<const uint32_t*>(v.x);
    const uint32_t m = 0x7fff7fffu, t = __vmaxu2(__vmaxu2(w[0] & m, w[1] & m), __vmaxu2(w[2] & m, w[3] & m));
    return max(t << 16, t & 0xffff0000u);
  } else {
    return __float_as_uint(top3(top3(v.at(0), v.at(1), v.at(2)), top3(v.at(3), v.at(4), v.at(5)), top2(v.at(6), v.at(7))));
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
template <typename T, bool kWide>
__device__ __forceinline__ uint2 codes8(const Eight<T, kWide>& v, uint32_t byte) {
  float f[8];
  if constexpr (sizeof(T) == 2 && kWide) {
    // scaled in bf16: exact but below 2^-126, where every code is 0
    const __nv_bfloat16 i1 = __float2bfloat16_rn(scale_inverse(byte));
    const __nv_bfloat162 i2 = __halves2bfloat162(i1, i1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 z = __hmul2(reinterpret_cast<const __nv_bfloat162*>(v.x)[i], i2);
      const uint32_t w = *reinterpret_cast<const uint32_t*>(&z);
      f[2 * i] = __uint_as_float(w << 16);
      f[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
    }
    uint2 w;
    w.x = e4m3x2(f[0], f[1]) | e4m3x2(f[2], f[3]) << 16;
    w.y = e4m3x2(f[4], f[5]) | e4m3x2(f[6], f[7]) << 16;
    return byte == 255u ? make_uint2(0, 0) : w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = v.at(i);
    return codes8(f, byte, byte);
  }
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
// How a product is cut: tiles of `rows` rows of A (a power of two from 16 to 256; 0: the kernel of many rows), the parts of
// K of a tile (1, 2, 4 or 8, each with a group of four K blocks at least), and one CTA an SM or two.
struct Cut {
  int32_t rows, split;
  bool deep;
};
Cut choose_cut(const MatmulProblem& p, int sms);
bool cut_fits(const MatmulProblem& p, const Cut& c);   // a grid's limits
cudaError_t launch_matmul(const MatmulProblem& p, const Cut* cut, cudaStream_t stream);   // cut NULL: the one chosen by sizes
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

// For tests, and no part of the headers that a user includes: the cut {rows, split, deep} that kda_fp8_matmul takes on a device
// of so many SMs, and kda_fp8_matmul with a given one.  KDA_ERR_INVALID_ARG for a cut that there is not,
// KDA_ERR_UNSUPPORTED for one beyond a grid's limits.
extern "C" {
KDA_API kda_status kda_fp8_matmul_choice(int64_t M, int64_t N, int64_t K, kda_dtype dt, int32_t sms, int32_t* cut);
KDA_API kda_status kda_fp8_matmul_cut(const uint8_t* a, int64_t a_stride, const uint8_t* a_scales, const uint8_t* w, int64_t w_stride,
                                      const uint8_t* w_scales, int64_t M, int64_t N, int64_t K, kda_dtype dt, void* out, int64_t out_stride,
                                      int32_t rows, int32_t split, int32_t deep, cudaStream_t stream);
}
