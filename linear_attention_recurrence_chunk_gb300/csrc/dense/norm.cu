// The residual's addition and a root-mean-square norm, in the input's type or in 8 bits.
//
//   s = x + r,   h = round(s),   y = s / sqrt(mean s^2 + eps) * w
//
// Bound: HBM, each value read and written once.  A row stays in registers between its sum and
// its output: W warps of a CTA have J x 256 columns each (one warp alone for narrow rows), all
// loads of a row on their way before the first is used; the 8-bit form takes its block maxima from
// the same registers, so that nothing is read twice.  Rows of a head's size share a warp.
// Measured (replayed from a graph), with a residual, of bf16: 32,768 x 4,096 156 us (6.9 TB/s), in 8 bits 142 us (6.6 TB/s;
// DRAM 80 %, issue slots 73 %); 1,000,000 x 128 153 us (6.7 TB/s); 32,000 x 768 32 us (6.1 TB/s); rows of odd width by
// 2-byte accesses 4.4 TB/s, 3.1 without a residual (8,192 x 8,001).  256 x 4,096 3.1 us, one row 1.9 us: launch and
// latency.  Of fp32: 16,384 x 2,001 79 us (6.7 TB/s); 4,096 x 32,768 333 us (6.5 TB/s); 4,096 x 20,000 232 us (5.7
// TB/s: 79 chunks are 20 warps of 64 registers, one block an SM), x 20,001 276 us (4.8 TB/s: 116 bytes a thread spill too).
// Slower: a block with row after row and the next one's loads ahead (32,768 x 4,096 172 us: half the warps an SM).
#include <type_traits>

#include "internal.cuh"

namespace kda {
namespace dense {
namespace {

constexpr int kRowsPerBlock = 4;   // of the one-warp form

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

// Sum over the W warps of a row, the same in each thread (warps in order: the same bits every time).
template <bool kOneWarp>
__device__ __forceinline__ float row_sum(float x, float* part, int warp, int lane, int W) {
  x = warp_sum(x);
  if constexpr (!kOneWarp) {
    __syncthreads();   // the last sum's readers are done
    if (lane == 0) part[warp] = x;
    __syncthreads();
    x = warp_sum(lane < W ? part[lane] : 0.f);
  }
  return x;
}

template <typename T, int J, bool kAdd, bool kFp8, bool kWide, bool kOneWarp>
__global__ void __launch_bounds__(kOneWarp ? 32 * kRowsPerBlock : 1024)
    add_rmsnorm_kernel(const T* x, int64_t xs, const T* r, int64_t rs, const float* w, float eps,
                       int64_t rows, int64_t C, T* h, T* y, uint8_t* codes, uint8_t* scales) {
  __shared__ float part[32];
  let_next_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31, warp = kOneWarp ? 0 : threadIdx.x >> 5, W = kOneWarp ? 1 : blockDim.x >> 5;
  const int64_t row = kOneWarp ? (int64_t)blockIdx.x * kRowsPerBlock + (threadIdx.x >> 5) : blockIdx.x;
  if (kOneWarp && row >= rows) return;
  float v[J][8];
  {
    Eight<T, kWide> a[J], b[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      a[j].load(x + row * xs, 256 * (int64_t)(warp + W * j), C, lane);
      if constexpr (kAdd) b[j].load(r + row * rs, 256 * (int64_t)(warp + W * j), C, lane);
    }
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = kAdd ? a[j].at(i) + b[j].at(i) : a[j].at(i);
  }
  if constexpr (kAdd) {
#pragma unroll
    for (int j = 0; j < J; ++j) store8<T, kWide>(h + row * C, 256 * (int64_t)(warp + W * j), C, lane, v[j]);
  }
  auto squares = [&](float t) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(v[j][i] * t, v[j][i] * t, s);
    return row_sum<kOneWarp>(s, part, warp, lane, W);
  };
  const float ss = squares(1.f);
  const float mean = ss / (float)C + eps;
  float inv = 1.f / sqrtf(mean);
  // Squares beyond fp32's range, alone or with eps, or below it with an eps that does not cover them: the row once more,
  // scaled by a power of two (every thread of the row has the same ss).  The values of a large row take half of its
  // scaling, their squares and the factor the rest: those 2^126 below its largest would lose bits as subnormal numbers.
  const bool high = !(mean < __uint_as_float(0x7f800000u)), low = ss < 0x1p-60f && eps < 0x1p-100f;
  if (high || low) {
    const float f = high ? 0x1p-40f : 0x1p80f, t = high ? f : 1.f;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] *= f;
    inv = t / sqrtf(squares(t) / (float)C + eps * (f * t) * (f * t));   // (what underflows beside a mean or an eps of 2^113 and more does not count there)
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int64_t c0 = 256 * (int64_t)(warp + W * j);
    if (c0 >= C) continue;
    if (w) {
      float g[8];
      if constexpr (kWide) {
        const int64_t c = c0 + 8 * lane;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
        if (c < C) a = reinterpret_cast<const float4*>(w + c)[0], b = reinterpret_cast<const float4*>(w + c)[1];
        g[0] = a.x, g[1] = a.y, g[2] = a.z, g[3] = a.w, g[4] = b.x, g[5] = b.y, g[6] = b.z, g[7] = b.w;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int64_t c = c0 + lane + 32 * i;
          g[i] = c < C ? w[c] : 0.f;
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = v[j][i] * inv * g[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] *= inv;
    }
    if constexpr (kFp8) {
      // a row with a sum that is not finite has NaN in the columns behind C as well: they belong to no block
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c0 + column<kWide>(lane, i) >= C) v[j][i] = 0.f;
      store_fp8<kWide>(codes + row * C, scales + row * ((C + kBlock - 1) / kBlock), c0, C, lane, v[j]);
    } else {
      store8<T, kWide>(y + row * C, c0, C, lane, v[j]);
    }
  }
}

// Rows of at most 128 values (a head's channels): the least power of two L of lanes that holds one at eight values a lane,
// so 32 / L rows a warp, and two such sets of rows at once.  kWide: lane l of a row has columns 8 l ..; else l, l + L, ...
constexpr int kNarrow = 128, kSets = 2;

template <typename T, bool kAdd, bool kFp8, bool kWide>
__global__ void __launch_bounds__(32 * kRowsPerBlock)
    add_rmsnorm_narrow_kernel(const T* x, int64_t xs, const T* r, int64_t rs, const float* w, float eps, int64_t rows, int32_t C,
                              int32_t L, T* h, T* y, uint8_t* codes, uint8_t* scales) {
  let_next_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31, l = lane & (L - 1), per_warp = 32 / L;
  const int64_t row0 = ((int64_t)blockIdx.x * kRowsPerBlock + (threadIdx.x >> 5)) * (kSets * per_warp) + lane / L;
  const auto column = [&](int i) { return kWide ? 8 * l + i : l + L * i; };
  const auto load = [&](Eight<T, kWide>& v, const T* row) {
    if constexpr (kWide) {
      v.load(row, 0, C, l);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v.x[i] = column(i) < C ? row[column(i)] : from_f32<T>(0.f);
    }
  };
  const auto store = [&](T* row, const float(&v)[8]) {
    if constexpr (kWide) {
      store8<T, true>(row, 0, C, l, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (column(i) < C) row[column(i)] = from_f32<T>(v[i]);
    }
  };
  Eight<T, kWide> a[kSets], b[kAdd ? kSets : 1];
#pragma unroll
  for (int j = 0; j < kSets; ++j) {
    const int64_t at = min(row0 + j * per_warp, rows - 1);   // (the last row again behind it: not stored)
    load(a[j], x + at * xs);
    if constexpr (kAdd) load(b[j], r + at * rs);
  }
  float g[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) g[i] = w && column(i) < C ? w[column(i)] : 1.f;
#pragma unroll
  for (int j = 0; j < kSets; ++j) {
    const int64_t row = row0 + j * per_warp;
    const bool live = row < rows;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = kAdd ? a[j].at(i) + b[j].at(i) : a[j].at(i);
    if constexpr (kAdd)
      if (live) store(h + row * C, v);
    const auto squares = [&](float t) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(v[i] * t, v[i] * t, s);
      for (int m = L >> 1; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
      return s;
    };
    const float ss = squares(1.f);
    const float mean = ss / (float)C + eps;
    float inv = 1.f / sqrtf(mean);
    // as in add_rmsnorm_kernel, each row for itself
    const bool high = !(mean < __uint_as_float(0x7f800000u)), low = ss < 0x1p-60f && eps < 0x1p-100f;
    if (__any_sync(0xffffffffu, high || low)) {
      const float f = high ? 0x1p-40f : low ? 0x1p80f : 1.f, t = high ? f : 1.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= f;
      inv = t / sqrtf(squares(t) / (float)C + eps * (f * t) * (f * t));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = column(i) < C ? v[i] * inv * g[i] : 0.f;
    if constexpr (kFp8) {
      uint32_t top = __float_as_uint(top3(top3(v[0], v[1], v[2]), top3(v[3], v[4], v[5]), top2(v[6], v[7])));
      for (int m = L >> 1; m > 0; m >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, m));
      const uint32_t byte = scale_byte(top);
      const uint2 c = codes8(v, byte, byte);
      if (live) {
        uint8_t* to = codes + row * C;
        if constexpr (kWide) {
          store_codes<true>(to, 0, C, l, c);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (column(i) < C) to[column(i)] = (uint8_t)((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
        }
        if (l == 0) scales[row] = (uint8_t)byte;
      }
    } else if (live) {
      store(y + row * C, v);
    }
  }
}

template <typename T, bool kWide>
cudaError_t launch_narrow(const NormProblem& p, cudaStream_t stream) {
  int L = 1;
  while (8 * L < p.C) L *= 2;
  const int64_t per_block = (int64_t)kRowsPerBlock * kSets * (32 / L);
  auto go = [&](auto add, auto fp8) {
    return launch_kernel(add_rmsnorm_narrow_kernel<T, decltype(add)::value, decltype(fp8)::value, kWide>, dim3((unsigned)((p.T + per_block - 1) / per_block)),
                         32 * kRowsPerBlock, 0, 0, stream, static_cast<const T*>(p.x), p.xs, static_cast<const T*>(p.r), p.rs, p.w, p.eps, p.T, p.C, L,
                         static_cast<T*>(p.h), static_cast<T*>(p.y), p.codes, p.scales);
  };
  const std::true_type yes;
  const std::false_type no;
  prof_begin(stream, "add_rmsnorm_narrow_kernel");
  const cudaError_t e = p.r ? (p.codes ? go(yes, yes) : go(yes, no)) : (p.codes ? go(no, yes) : go(no, no));
  prof_end(stream);
  return e;
}

template <typename T, int J, bool kAdd, bool kFp8, bool kWide>
cudaError_t launch4(const NormProblem& p, int warps, cudaStream_t stream) {
  auto go = [&](auto one) {
    constexpr bool kOne = decltype(one)::value;
    return launch_kernel(add_rmsnorm_kernel<T, J, kAdd, kFp8, kWide, kOne>, dim3((unsigned)(kOne ? (p.T + kRowsPerBlock - 1) / kRowsPerBlock : p.T)),
                         kOne ? 32 * kRowsPerBlock : 32 * warps, 0, 0, stream, static_cast<const T*>(p.x), p.xs, static_cast<const T*>(p.r), p.rs, p.w,
                         p.eps, p.T, p.C, static_cast<T*>(p.h), static_cast<T*>(p.y), p.codes, p.scales);
  };
  prof_begin(stream, "add_rmsnorm_kernel");
  const cudaError_t e = warps == 1 ? go(std::true_type{}) : go(std::false_type{});
  prof_end(stream);
  return e;
}

template <typename T, int J, bool kWide>
cudaError_t launch2(const NormProblem& p, int warps, cudaStream_t stream) {
  if (p.r) return p.codes ? launch4<T, J, true, true, kWide>(p, warps, stream) : launch4<T, J, true, false, kWide>(p, warps, stream);
  return p.codes ? launch4<T, J, false, true, kWide>(p, warps, stream) : launch4<T, J, false, false, kWide>(p, warps, stream);
}

template <typename T>
cudaError_t launch1(const NormProblem& p, cudaStream_t stream) {
  const auto at = [](const void* q, size_t n) { return reinterpret_cast<uintptr_t>(q) % n == 0; };
  const int64_t step = 16 / sizeof(T);
  const bool wide = p.C % 8 == 0 && p.xs % step == 0 && at(p.x, 16) && (!p.r || (p.rs % step == 0 && at(p.r, 16) && at(p.h, 16))) &&
                    at(p.w, 16) && (p.codes ? at(p.codes, 8) : at(p.y, 16));
  if (p.C <= kNarrow) return wide ? launch_narrow<T, true>(p, stream) : launch_narrow<T, false>(p, stream);
  const int chunks = (int)((p.C + 255) / 256);   // 256 columns each, at most 128
  // One or two chunks: a warp a row; three or four too where there are many rows of at most 3,584 bytes to read (32,000 x
  // 520 of bf16: 14 us, 34 with two warps, whose blocks start too slowly; 32,000 x 768 with a residual 33 and 37; but
  // 1,024 with a residual 43 and 42, of fp32 83 and 79, and 500 x 768 2.4 and 2.3).  Else two chunks a warp, four where
  // 32 warps are not enough and for 8-bit output of
  // many rows (32,768 x 4,096: 157 us with two, 143 with four; 16,384 x 8,192: 182 and 147; but 1 x 4,096: 3.0 and
  // 3.6, 256 x 8,192: 5.5 and 5.9; in the input's type the two differ by 1 %).
  if (chunks <= 1) return wide ? launch2<T, 1, true>(p, 1, stream) : launch2<T, 1, false>(p, 1, stream);
  if (chunks > 2 && chunks <= 4 && p.T >= 4096 && p.C * (int64_t)sizeof(T) * (p.r ? 2 : 1) <= 3584)
    return wide ? launch2<T, 4, true>(p, 1, stream) : launch2<T, 4, false>(p, 1, stream);
  const int J = chunks > 64 || (p.codes && chunks > 8 && p.T >= 1024) ? 4 : 2, warps = (chunks + J - 1) / J;
  if (J == 2) return wide ? launch2<T, 2, true>(p, warps, stream) : launch2<T, 2, false>(p, warps, stream);
  return wide ? launch2<T, 4, true>(p, warps, stream) : launch2<T, 4, false>(p, warps, stream);
}

}  // namespace

cudaError_t launch_norm(const NormProblem& p, cudaStream_t stream) {
  return p.dt == KDA_F32 ? launch1<float>(p, stream) : launch1<__nv_bfloat16>(p, stream);
}

}  // namespace dense
}  // namespace kda
