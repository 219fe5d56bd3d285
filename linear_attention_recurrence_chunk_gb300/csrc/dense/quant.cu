// Matrices to 8 bits and back.
//
//   e = least e >= -126 with max |x| <= 448 * 2^e over a block,  code = E4M3(x * 2^-e),  value = code * 2^e
//
// Both scalings are exact and the hardware's conversion rounds once, so that the result is
// defined bit by bit.  Bound: HBM.  Blocks of 1 x 128: half a warp has a block (eight values a lane; any
// alignment: a warp, four values a lane), four of them at once, whatever rows they lie in.  Blocks of 128 x 128: a CTA
// holds one in registers between its maximum and its codes.
// Measured (replayed from a graph), 32,768 x 4,096 of bf16: 62.9 us (6.4 TB/s) by rows, 65.5 us (6.2 TB/s) by
// squares, read back 61 us (6.6 TB/s); 16,384 x 4,096 of fp32 48 us (6.9 TB/s) and 52 us (6.5 TB/s).  By rows the instructions count (issue slots 69 %): with the sizes compared
// and the values scaled as packed bf16, and the places of a warp's blocks taken from one row, 76 -> 63 us.
// bf16 rows of odd width, by 2-byte accesses, 2.9 TB/s (8,192 x 8,001).
#include <type_traits>

#include "internal.cuh"

namespace kda {
namespace dense {
namespace {

constexpr int kJ = 4;          // blocks of 1 x 128 of half a warp (kWide) or twice as many of a warp
constexpr int kWarps = 4, kSquareThreads = 512;

// Where the blocks of a warp lie: block i of its kBlocks follows on block i - 1, row after row.
template <bool kWide>
struct Walk {
  static constexpr int kBlocks = 2 * kJ;
  int64_t row0, C;
  uint32_t b0, per_row, magic;
  __device__ __forceinline__ Walk(int64_t C_, uint32_t per_row_, uint32_t magic_) : C(C_), per_row(per_row_), magic(magic_) {
    const int64_t first = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * kBlocks;
    row0 = first / per_row;
    b0 = (uint32_t)(first - row0 * per_row);
  }
  __device__ __forceinline__ void at(uint32_t i, int64_t& row, int64_t& c) const {
    const uint32_t b = b0 + i, down = magic ? __umulhi(b, magic) : per_row == 1 ? b : b / per_row;
    row = row0 + down;
    c = (int64_t)(b - down * per_row) * kBlock;
  }
};
// ceil(2^32 / d) where n / d = n magic >> 32 for every n < d + 2^8; else 0.
uint32_t walk_magic(int64_t d) { return d > 1 && d < 60000 ? (uint32_t)((0x100000000ull + d - 1) / d) : 0u; }

template <typename T, bool kWide>
__global__ void __launch_bounds__(32 * kWarps)
    fp8_quant_kernel(const T* x, int64_t xs, int64_t rows, int64_t C, uint32_t per_row, uint32_t magic, uint8_t* codes, uint8_t* scales) {
  let_next_start();
  wait_for_previous();
  const Walk<kWide> walk(C, per_row, magic);
  const int lane = threadIdx.x & 31;
  if constexpr (kWide) {
    Eight<T, true> v[kJ];
    // one block's place after another, or (all in one row) 256 columns on each time
    const bool whole = walk.b0 + walk.kBlocks <= per_row;
    int64_t row, c;
    walk.at(lane >> 4, row, c);
    if (whole) {
      if (row >= rows) return;
      const T* from = x + row * xs;
#pragma unroll
      for (int j = 0; j < kJ; ++j) v[j].load(from, c + 256 * j, C, lane & 15);
    } else {
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        walk.at(2 * j + (lane >> 4), row, c);
        v[j].load(x + (row < rows ? row : 0) * xs, c, row < rows ? C : 0, lane & 15);
      }
      walk.at(lane >> 4, row, c);
    }
    uint8_t* to = codes + row * C + c;
    uint8_t* sc = scales + row * per_row + c / kBlock;
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      const uint32_t byte = scale_byte(half_warp_max(lane_top(v[j])));
      const uint2 w = codes8(v[j], byte);
      if (whole) {
        store_codes<true>(to + 256 * j, 0, C - c - 256 * j, lane & 15, w);
        if ((lane & 15) == 0) sc[2 * j] = (uint8_t)byte;
      } else {
        walk.at(2 * j + (lane >> 4), row, c);
        if (row < rows) {
          store_codes<true>(codes + row * C, c, C, lane & 15, w);
          if ((lane & 15) == 0) scales[row * per_row + c / kBlock] = (uint8_t)byte;
        }
      }
    }
  } else {
    T v[2 * kJ][4];
#pragma unroll
    for (int j = 0; j < 2 * kJ; ++j) {
      int64_t row, c;
      walk.at(j, row, c);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j][i] = row < rows && c + lane + 32 * i < C ? x[row * xs + c + lane + 32 * i] : from_f32<T>(0.f);
    }
#pragma unroll
    for (int j = 0; j < kJ; ++j) {   // two blocks at a time
      float f[8];
      uint32_t a, b;
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = to_f32<T>(v[2 * j + (i >> 2)][i & 3]);
      block_tops<false>(f, a, b);
      const uint32_t byte[2] = {scale_byte(a), scale_byte(b)};
      const uint2 w = codes8(f, byte[0], byte[1]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        int64_t row, c;
        walk.at(2 * j + k, row, c);
        if (row >= rows) break;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c + lane + 32 * i < C) codes[row * C + c + lane + 32 * i] = (uint8_t)((k ? w.y : w.x) >> (8 * i));
        if (lane == 0) scales[row * per_row + c / kBlock] = (uint8_t)byte[k];
      }
    }
  }
}

// Blocks of 128 x 128, kSide of them side by side, so that a row gives a line of 512 bytes: two of bf16 (one took 81 us
// for 32,768 x 4,096, two 66), one of fp32 (4,096 x 4,096: two took 19.7 us); and one where there are no more.  16
// warps have a row each at a time, or (kSide 1) two.
template <typename T, bool kWide, int kSide>
__global__ void __launch_bounds__(kSquareThreads)
    fp8_quant_square_kernel(const T* x, int64_t xs, int64_t rows, int64_t C, uint8_t* codes, uint8_t* scales) {
  let_next_start();
  wait_for_previous();
  constexpr int W = kSquareThreads / 32, kAtOnce = 2 / kSide, kSteps = kBlock / (W * kAtOnce);
  __shared__ uint32_t part[2][W];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t across = (C + kSide * kBlock - 1) / (kSide * kBlock), br = blockIdx.x / across, bc = blockIdx.x - br * across;
  const int64_t r0 = br * kBlock + kAtOnce * warp, c0 = bc * kSide * kBlock;
  // kWide: lane `sub` of a row has eight columns; else value i lies in row_of(i), column_of(i)
  const int sub = kSide == 2 ? lane : lane & 15, half = kSide == 2 ? 0 : lane >> 4;
  const auto row_of = [&](int j, int i) { return r0 + W * kAtOnce * j + (kSide == 2 ? 0 : kWide ? half : i >> 2); };
  const auto column_of = [&](int i) { return c0 + lane + 32 * (kSide == 2 ? i : i & 3); };
  Eight<T, kWide> v[kSteps];
#pragma unroll
  for (int j = 0; j < kSteps; ++j) {
    if constexpr (kWide) {
      const int64_t row = row_of(j, 0);
      v[j].load(x + (row < rows ? row : 0) * xs, c0, row < rows ? C : 0, sub);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[j].x[i] = row_of(j, i) < rows && column_of(i) < C ? x[row_of(j, i) * xs + column_of(i)] : from_f32<T>(0.f);
    }
  }
  // the largest of each half warp (kWide), or of values 0 .. 3 and 4 .. 7: of the first and the second block, or both of one
  uint32_t top[2] = {0, 0};
  if constexpr (kWide) {
#pragma unroll
    for (int j = 0; j < kSteps; ++j) top[0] = max(top[0], lane_top(v[j]));
    top[0] = half_warp_max(top[0]);
    if ((lane & 15) == 0) part[lane >> 4][warp] = top[0];
  } else {
#pragma unroll
    for (int j = 0; j < kSteps; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) top[i >> 2] = max(top[i >> 2], __float_as_uint(top2(v[j].at(i), 0.f)));
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      top[k] = __reduce_max_sync(0xffffffffu, top[k]);
      if (lane == 0) part[k][warp] = top[k];
    }
  }
  __syncthreads();
  uint32_t byte[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) byte[k] = __reduce_max_sync(0xffffffffu, part[k][lane & (W - 1)]);
  if constexpr (kSide == 1) byte[0] = byte[1] = max(byte[0], byte[1]);
#pragma unroll
  for (int k = 0; k < 2; ++k) byte[k] = scale_byte(byte[k]);
  if (threadIdx.x < kSide && c0 + kBlock * threadIdx.x < C)
    scales[br * ((C + kBlock - 1) / kBlock) + c0 / kBlock + threadIdx.x] = (uint8_t)(threadIdx.x ? byte[1] : byte[0]);
#pragma unroll
  for (int j = 0; j < kSteps; ++j) {
    if constexpr (kWide) {
      const int64_t row = row_of(j, 0);
      if (row < rows) store_codes<true>(codes + row * C, c0, C, sub, codes8(v[j], lane < 16 ? byte[0] : byte[1]));
    } else {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = v[j].at(i);
      const uint2 w = codes8(f, byte[0], byte[1]);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (row_of(j, i) < rows && column_of(i) < C) codes[row_of(j, i) * C + column_of(i)] = (uint8_t)((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
    }
  }
}

template <typename T, bool kWide>
__global__ void __launch_bounds__(32 * kWarps)
    fp8_values_kernel(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t C, int32_t block_rows,
                      uint32_t per_row, uint32_t magic, T* y) {
  let_next_start();
  wait_for_previous();
  const Walk<kWide> walk(C, per_row, magic);
  const int lane = threadIdx.x & 31;
  constexpr int kN = kWide ? kJ : 2 * kJ, kPer = kWide ? 2 : 1;   // blocks of a lane; half a warp or a warp each
  const int sub = kWide ? lane >> 4 : 0;
  uint2 w[kN];
  uint32_t s[kN];
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    int64_t row, c;
    walk.at(kPer * j + sub, row, c);
    w[j] = make_uint2(0, 0);
    s[j] = row < rows ? scales[(block_rows == 1 ? row : row / kBlock) * per_row + c / kBlock] : 127u;
    if constexpr (kWide) {
      c += 8 * (lane & 15);
      if (row < rows && c < C) w[j] = __ldcs(reinterpret_cast<const uint2*>(codes + row * C + c));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (row < rows && c + lane + 32 * i < C) w[j].x |= (uint32_t)codes[row * C + c + lane + 32 * i] << (8 * i);
    }
  }
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    int64_t row, c;
    walk.at(kPer * j + sub, row, c);
    if (row >= rows) continue;
    const float f = scale_value(s[j]);
    float v[8];
#pragma unroll
    for (int i = 0; i < (kWide ? 4 : 2); ++i) {
      const float2 z = e4m3x2_values((i < 2 ? w[j].x : w[j].y) >> (16 * (i & 1)) & 0xffffu);
      v[2 * i] = z.x * f;
      v[2 * i + 1] = z.y * f;
    }
    if constexpr (kWide) {
      store8<T, true>(y + row * C, c, C, lane & 15, v);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + lane + 32 * i < C) y[row * C + c + lane + 32 * i] = from_f32<T>(v[i]);
    }
  }
}

bool at(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

template <typename T>
cudaError_t quant(const QuantProblem& p, cudaStream_t stream) {
  const bool wide = p.C % 8 == 0 && p.stride % (16 / sizeof(T)) == 0 && at(p.x, 16) && at(p.codes, 8);
  const T* x = static_cast<const T*>(p.x);
  cudaError_t e;
  prof_begin(stream, "fp8_quant_kernel");
  if (p.rows == 1) {
    const uint32_t per_row = (uint32_t)((p.C + kBlock - 1) / kBlock);
    const unsigned grid = (unsigned)((p.T * per_row + 2 * kJ * kWarps - 1) / (2 * kJ * kWarps));
    e = launch_kernel(wide ? fp8_quant_kernel<T, true> : fp8_quant_kernel<T, false>, dim3(grid), 32 * kWarps, 0, 0, stream, x, p.stride, p.T, p.C, per_row,
                      walk_magic(per_row), p.codes, p.scales);
  } else {
    const auto go = [&](auto side) {
      constexpr int kSide = decltype(side)::value;
      const unsigned grid = (unsigned)(((p.T + kBlock - 1) / kBlock) * ((p.C + kSide * kBlock - 1) / (kSide * kBlock)));
      return launch_kernel(wide ? fp8_quant_square_kernel<T, true, kSide> : fp8_quant_square_kernel<T, false, kSide>, dim3(grid), kSquareThreads, 0, 0,
                           stream, x, p.stride, p.T, p.C, p.codes, p.scales);
    };
    if constexpr (sizeof(T) == 4) e = go(std::integral_constant<int, 1>{});
    else e = p.C <= kBlock ? go(std::integral_constant<int, 1>{}) : go(std::integral_constant<int, 2>{});
  }
  prof_end(stream);
  return e;
}

template <typename T>
cudaError_t values(const ValuesProblem& p, cudaStream_t stream) {
  const bool wide = p.C % 8 == 0 && at(p.codes, 8) && at(p.y, 16);
  const uint32_t per_row = (uint32_t)((p.C + kBlock - 1) / kBlock);
  const unsigned grid = (unsigned)((p.T * per_row + 2 * kJ * kWarps - 1) / (2 * kJ * kWarps));
  prof_begin(stream, "fp8_values_kernel");
  const cudaError_t e = launch_kernel(wide ? fp8_values_kernel<T, true> : fp8_values_kernel<T, false>, dim3(grid), 32 * kWarps, 0, 0, stream, p.codes,
                                      p.scales, p.T, p.C, p.rows, per_row, walk_magic(per_row), static_cast<T*>(p.y));
  prof_end(stream);
  return e;
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
