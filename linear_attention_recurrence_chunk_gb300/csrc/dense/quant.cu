// Matrices to 8 bits and back.
//
//   e = least e >= -126 with max |x| <= 448 * 2^e over a block,  code = E4M3(x * 2^-e),  value = code * 2^e
//
// Both scalings are exact and the hardware's conversion rounds once, so that the result is
// defined bit by bit.  Bound: HBM.  Blocks of 1 x 128: a warp takes 4 x 256 columns of a row, all loads
// first.  Blocks of 128 x 128: a CTA holds one in registers between its maximum and its codes.
#include "internal.cuh"

namespace kda {
namespace dense {
namespace {

constexpr int kJ = 4;          // 256-column chunks of a warp
constexpr int kWarps = 4;

template <typename T, bool kWide>
__global__ void __launch_bounds__(32 * kWarps)
    fp8_quant_kernel(const T* __restrict__ x, int64_t xs, int64_t rows, int64_t C, int64_t per_row, uint8_t* codes, uint8_t* scales) {
  const int lane = threadIdx.x & 31;
  const int64_t task = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5), row = task / per_row;
  if (row >= rows) return;
  const int64_t c0 = (task - row * per_row) * (256 * kJ);
  float v[kJ][8];
#pragma unroll
  for (int j = 0; j < kJ; ++j) load8<T, kWide>(x + row * xs, c0 + 256 * j, C, lane, v[j]);
#pragma unroll
  for (int j = 0; j < kJ; ++j)
    if (c0 + 256 * j < C)
      store_fp8<kWide>(codes + row * C, scales + row * ((C + kBlock - 1) / kBlock), c0 + 256 * j, C, lane, v[j]);
}

// A block of 128 x 128: 256 threads, half a warp's 16 lanes a row of 128 columns, 8 values each, 8 rows a
// thread (kWide); else a warp a row, 4 values a lane, 16 rows.
template <typename T, bool kWide>
__global__ void __launch_bounds__(256)
    fp8_quant_square_kernel(const T* __restrict__ x, int64_t xs, int64_t rows, int64_t C, uint8_t* codes, uint8_t* scales) {
  __shared__ uint32_t part[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t blocks = (C + kBlock - 1) / kBlock, br = blockIdx.x / blocks, bc = blockIdx.x - br * blocks;
  const int64_t r0 = br * kBlock, c0 = bc * kBlock;
  float v[8][8];
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (kWide) {
      // load8's lane stands for 8 columns: 16 lanes of two rows
      const int64_t row = r0 + 16 * j + 2 * warp + (lane >> 4);
      const bool in = row < rows;
      load8<T, true>(x + (in ? row : r0) * xs, c0, in ? C : 0, lane & 15, v[j]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t row = r0 + 16 * j + 2 * warp + (i >> 2), c = c0 + lane + 32 * (i & 3);
        v[j][i] = row < rows && c < C ? to_f32<T>(x[row * xs + c]) : 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, magnitude(v[j][i]));
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) part[warp] = top;
  __syncthreads();
  top = __reduce_max_sync(0xffffffffu, part[lane & 7]);
  const uint32_t byte = scale_byte(top);
  if (threadIdx.x == 0) scales[br * blocks + bc] = (uint8_t)byte;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint2 w = codes8(v[j], byte, byte);
    if constexpr (kWide) {
      const int64_t row = r0 + 16 * j + 2 * warp + (lane >> 4);
      if (row < rows) store_codes<true>(codes + row * C, c0, C, lane & 15, w);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t row = r0 + 16 * j + 2 * warp + (i >> 2), c = c0 + lane + 32 * (i & 3);
        if (row < rows && c < C) codes[row * C + c] = (uint8_t)((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
      }
    }
  }
}

template <typename T, bool kWide>
__global__ void __launch_bounds__(32 * kWarps)
    fp8_values_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t rows, int64_t C, int32_t block_rows,
                      int64_t per_row, T* y) {
  const int lane = threadIdx.x & 31;
  const int64_t task = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5), row = task / per_row;
  if (row >= rows) return;
  const int64_t c0 = (task - row * per_row) * (256 * kJ);
  const uint8_t* in = codes + row * C;
  const uint8_t* sc = scales + (block_rows == 1 ? row : row / kBlock) * ((C + kBlock - 1) / kBlock);
  uint2 w[kJ];
  uint32_t s[kJ][2];
#pragma unroll
  for (int j = 0; j < kJ; ++j) {
    const int64_t c = c0 + 256 * j;
    w[j] = make_uint2(0, 0);
    if constexpr (kWide) {
      const bool in_row = c + 8 * lane < C;
      if (in_row) w[j] = __ldcs(reinterpret_cast<const uint2*>(in + c) + lane);
      s[j][0] = s[j][1] = in_row ? sc[(c + 8 * lane) / kBlock] : 127u;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t b = c + lane + 32 * i < C ? in[c + lane + 32 * i] : 0u;
        (i < 4 ? w[j].x : w[j].y) |= b << (8 * (i & 3));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) s[j][i] = c + kBlock * i < C ? sc[c / kBlock + i] : 127u;
    }
  }
#pragma unroll
  for (int j = 0; j < kJ; ++j) {
    float v[8];
    const float a = scale_value(s[j][0]), b = scale_value(s[j][1]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 z = e4m3x2_values((i < 2 ? w[j].x : w[j].y) >> (16 * (i & 1)) & 0xffffu);
      v[2 * i] = z.x * (i < 2 ? a : b);
      v[2 * i + 1] = z.y * (i < 2 ? a : b);
    }
    store8<T, kWide>(y + row * C, c0 + 256 * j, C, lane, v);
  }
}

bool at(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

template <typename T>
cudaError_t quant(const QuantProblem& p, cudaStream_t stream) {
  const bool wide = p.C % 8 == 0 && p.stride % (16 / sizeof(T)) == 0 && at(p.x, 16) && at(p.codes, 8);
  const T* x = static_cast<const T*>(p.x);
  prof_begin(stream, "fp8_quant_kernel");
  if (p.rows == 1) {
    const int64_t per_row = (p.C + 256 * kJ - 1) / (256 * kJ);
    const unsigned grid = (unsigned)((p.T * per_row + kWarps - 1) / kWarps);
    if (wide) fp8_quant_kernel<T, true><<<grid, 32 * kWarps, 0, stream>>>(x, p.stride, p.T, p.C, per_row, p.codes, p.scales);
    else fp8_quant_kernel<T, false><<<grid, 32 * kWarps, 0, stream>>>(x, p.stride, p.T, p.C, per_row, p.codes, p.scales);
  } else {
    const unsigned grid = (unsigned)(((p.T + kBlock - 1) / kBlock) * ((p.C + kBlock - 1) / kBlock));
    if (wide) fp8_quant_square_kernel<T, true><<<grid, 256, 0, stream>>>(x, p.stride, p.T, p.C, p.codes, p.scales);
    else fp8_quant_square_kernel<T, false><<<grid, 256, 0, stream>>>(x, p.stride, p.T, p.C, p.codes, p.scales);
  }
  prof_end(stream);
  return cudaGetLastError();
}

template <typename T>
cudaError_t values(const ValuesProblem& p, cudaStream_t stream) {
  const bool wide = p.C % 8 == 0 && at(p.codes, 8) && at(p.y, 16);
  const int64_t per_row = (p.C + 256 * kJ - 1) / (256 * kJ);
  const unsigned grid = (unsigned)((p.T * per_row + kWarps - 1) / kWarps);
  prof_begin(stream, "fp8_values_kernel");
  if (wide) fp8_values_kernel<T, true><<<grid, 32 * kWarps, 0, stream>>>(p.codes, p.scales, p.T, p.C, p.rows, per_row, static_cast<T*>(p.y));
  else fp8_values_kernel<T, false><<<grid, 32 * kWarps, 0, stream>>>(p.codes, p.scales, p.T, p.C, p.rows, per_row, static_cast<T*>(p.y));
  prof_end(stream);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quant(const QuantProblem& p, cudaStream_t stream) {
  return p.dt == KDA_F32 ? quant<float>(p, stream) : quant<__nv_bfloat16>(p, stream);
}
cudaError_t launch_values(const ValuesProblem& p, cudaStream_t stream) {
  return p.dt == KDA_F32 ? values<float>(p, stream) : values<__nv_bfloat16>(p, stream);
}

}  // namespace dense
}  // namespace kda
