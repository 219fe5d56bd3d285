// Rotary positions.
//
//   (a, b) -> amplitude (a cos t - b sin t, a sin t + b cos t),   t = position * frequency
//
// The angle is wanted modulo a turn, and positions go to 2^31: the frequency in turns, modulo 1, is held
// as a 64-bit fixed-point fraction (from fp64 once per block), so that its product with the position p
// modulo 2^64 is the fraction of a turn to p 2^-63, with no reduction and no table.  The top 32 bits, signed,
// are half turns in [-1, 1) for sincospi, rounded to fp32's 24 bits: 4.1e-8 radians rms, 9.4e-8 at most.
// (fp32 outputs are off by 3.9e-8 of their size, with exact angles they would be by 2.9e-8.)
//
// Bound: HBM, each value read and written once.  A warp takes a token at a time (a part of its heads when there are
// few tokens): the first loads go out, then the token's cosines and sines into the warp's shared memory, each once,
// then all heads of queries and keys, eight pairs (two 16-byte loads of bf16) a lane and three such items on their
// way at once.
// Measured (replayed from a graph): 65,536 tokens, 32 + 4 heads of 128 in bf16 187 us (6.5 TB/s), either order of the pairs,
// half of each head turned 189 us; 256 tokens of 96 + 8 heads 4.4 us, 6.1 where the frequencies come from HBM too; one token
// 2.8 us.  Pairs that are no multiple of 8, one value a load: 65,536 tokens, 8 + 2 heads of 80, 20 channels turned, 171
// us (1.2 TB/s), of 96 with 24 turned 183 us; with 32 turned 50 us (5.0 TB/s).  A block that first makes the
// cosines of a few tokens together and then turns their heads took 328 us: its phases waited for one another.
#include <algorithm>
#include <type_traits>

#include "internal.cuh"

namespace kda {
namespace dense {
namespace {

constexpr int kWarps = 8, kItems = 3;

// n / d for n d < 2^32, m = ceil(2^32 / d) (d = 1: m = 0).
__device__ __forceinline__ uint32_t divide(uint32_t n, uint32_t m) { return m ? __umulhi(n, m) : n; }

// x modulo 1 in units of 2^-64 (0 for what is not finite).
__device__ __forceinline__ uint64_t fraction(double x) {
  x -= floor(x);
  return x < 1.0 ? (uint64_t)(x * 0x1p64) : 0;
}

struct Shape {
  RotaryPart q, k;
  const int32_t* pos;
  const double* freqs;
  int64_t T;
  int32_t D, rot, half;   // half = rot / 2 pairs
  float amplitude;
  int32_t split, heads;   // warps of a token, heads of each
  int32_t tokens;         // of a warp at a time (1 where split > 1)
  int32_t parts, turned;  // items of a head: of pairs first, then of channels that stay
  uint32_t m_parts, m_token;   // (tokens > 1: a token has at most 128 items)
};

// kE consecutive values of one side of kE pairs.
template <typename T, int kE>
struct Values {
  alignas(kE > 1 ? 16 : sizeof(T)) T x[kE];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kE == 1) {
      x[0] = *p;
    } else {
#pragma unroll
      for (int i = 0; i < (int)(kE * sizeof(T) / 16); ++i) reinterpret_cast<uint4*>(x)[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (kE == 1) {
      *p = x[0];
    } else {
#pragma unroll
      for (int i = 0; i < (int)(kE * sizeof(T) / 16); ++i) reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(x)[i];
    }
  }
};

// kMany: several tokens a warp at a time (or whatever the sizes ask for); else one, or a part of its heads.
template <typename T, int kE, bool kNext, bool kInverse, bool kMany>
__global__ void __launch_bounds__(32 * kWarps, 2) rotary_kernel(const Shape s) {
  extern __shared__ uint64_t sm[];
  let_next_start();
  wait_for_previous();
  uint64_t* turn = sm;   // [half] turns per position, 2^-64 each
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // its tokens' (cos, sin), of each kE / 2 blocks of [turned][2 pairs] (kE = 1: [half]): lanes of neighbouring parts read neighbouring banks
  float2* cs = reinterpret_cast<float2*>(turn + s.half) + (size_t)warp * s.tokens * s.half;
  for (int i = threadIdx.x; i < s.half; i += 32 * kWarps) {
    // freq / (2 pi) as a rounded product and what it lacks: 1 / (2 pi) = kHi + kLo to 2^-110
    constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;
    const double w = s.freqs[i], f = w * kHi, low = fma(w, kHi, -f) + w * kLo;
    turn[i] = fraction(f) + fraction(low);
  }
  __syncthreads();
  const int H = s.q.H + s.k.H;
  const int64_t units = s.split == 1 ? (s.T + s.tokens - 1) / s.tokens : s.T * s.split, step = (int64_t)gridDim.x * kWarps;
  int64_t u = (int64_t)blockIdx.x * kWarps + warp;
  // lane g has the position of the unit's token g
  auto token = [&](int64_t unit) { return s.split == 1 ? unit * s.tokens : unit / s.split; };
  auto position = [&](int64_t unit) {
    const int64_t t = token(unit) + lane;
    return unit < units && lane < s.tokens && t < s.T ? s.pos[t] : -1;
  };
  int32_t next = position(u);
  for (; u < units; u += step) {
    const int64_t t = token(u);
    const int h0 = s.split == 1 ? 0 : (int)(u - t * s.split) * s.heads, nh = min(H - h0, s.heads);
    const int32_t p = next;
    next = position(u + step);
    const T *xq = static_cast<const T*>(s.q.x) + t * s.q.xt, *xk = static_cast<const T*>(s.k.x) + t * s.k.xt;
    T *yq = static_cast<T*>(s.q.y) + t * s.q.yt, *yk = static_cast<T*>(s.k.y) + t * s.k.yt;
    const int nt = kMany ? (int)min((int64_t)s.tokens, s.T - t) : 1, n = s.split == 1 ? nt * nh * s.parts : nh * s.parts;
    Values<T, kE> a[kItems], b[kItems];
    T *ya[kItems], *yb[kItems];   // NULL: nothing to write
    int c[kItems];                // negative: the values stay
    auto load = [&](int i0) {
#pragma unroll
      for (int j = 0; j < kItems; ++j) {
        ya[j] = yb[j] = nullptr;
        c[j] = -1;
        const uint32_t i = i0 + 32 * j, g = kMany && s.tokens > 1 ? divide(i, s.m_token) : 0, r = i - g * s.heads * s.parts, hl = divide(r, s.m_parts);
        const int part = (int)(r - hl * s.parts), h = h0 + (int)hl, hk = h - s.q.H;
        const int32_t at = __shfl_sync(0xffffffffu, p, kMany ? g & 31 : 0);
        if ((int)i >= n) continue;
        const T* x = hk < 0 ? xq + g * s.q.xt + h * s.q.xh : xk + g * s.k.xt + hk * s.k.xh;
        T* y = hk < 0 ? yq + g * s.q.yt + h * s.q.yh : yk + g * s.k.yt + hk * s.k.yh;
        const bool pairs = part < s.turned, turned = pairs && at >= 0;
        const int ca = !pairs ? s.rot + 2 * kE * (part - s.turned) : kNext ? 2 * kE * part : kE * part;
        const int cb = pairs && !kNext ? s.half + ca : ca + kE;
        if (!turned && x == y) continue;   // in place
        a[j].load(x + ca);
        ya[j] = y + ca;
        if (cb < s.D) {
          b[j].load(x + cb);
          yb[j] = y + cb;
        }
        if (turned) c[j] = (int)g * s.half + (kE == 1 ? part : 2 * part);
      }
    };
    load(lane);
    __syncwarp();   // the last token's cosines have been read
    for (int g = 0; g < nt; ++g) {
      const int32_t at = __shfl_sync(0xffffffffu, p, g);
      if (at < 0) continue;
      for (int i = lane; i < s.half; i += 32) {
        const int32_t frac = (int32_t)((uint64_t)(uint32_t)at * turn[i] >> 32);
        float sn, cc;
        sincospif((float)frac * 0x1p-31f, &sn, &cc);
        // pair i is pair i % kE of part i / kE
        const int to = kE == 1 ? i : ((i % kE >> 1) * s.turned + i / kE) * 2 + (i & 1);
        cs[g * s.half + to] = make_float2(cc * s.amplitude, (kInverse ? -sn : sn) * s.amplitude);
      }
    }
    __syncwarp();
    for (int i0 = lane;;) {
#pragma unroll
      for (int j = 0; j < kItems; ++j) {
        if (c[j] >= 0) {
          if constexpr (kE == 1) {
            const float2 z = cs[c[j]];
            const float x0 = to_f32<T>(a[j].x[0]), x1 = to_f32<T>(b[j].x[0]);
            a[j].x[0] = from_f32<T>(x0 * z.x - x1 * z.y);
            b[j].x[0] = from_f32<T>(x0 * z.y + x1 * z.x);
          } else {
#pragma unroll
            for (int e = 0; e < kE; e += 2) {
              const float4 z = *reinterpret_cast<const float4*>(cs + c[j] + e * s.turned);
#pragma unroll
              for (int d = 0; d < 2; ++d) {
                // kNext: pair e is values 2 e, 2 e + 1 of a and b together
                T& u0 = kNext ? (2 * (e + d) < kE ? a[j].x[2 * (e + d) % kE] : b[j].x[2 * (e + d) % kE]) : a[j].x[e + d];
                T& u1 = kNext ? (2 * (e + d) < kE ? a[j].x[(2 * (e + d) + 1) % kE] : b[j].x[(2 * (e + d) + 1) % kE]) : b[j].x[e + d];
                const float x0 = to_f32<T>(u0), x1 = to_f32<T>(u1), cc = d ? z.z : z.x, sn = d ? z.w : z.y;
                u0 = from_f32<T>(x0 * cc - x1 * sn);
                u1 = from_f32<T>(x0 * sn + x1 * cc);
              }
            }
          }
        }
        if (ya[j]) a[j].store(ya[j]);
        if (yb[j]) b[j].store(yb[j]);
      }
      i0 += 32 * kItems;
      if (i0 - lane >= n) break;
      load(i0);
    }
  }
}

uint32_t magic(uint32_t d) { return d == 1 ? 0u : (uint32_t)((0x100000000ull + d - 1) / d); }

template <typename T, int kE>
cudaError_t launch(const RotaryProblem& p, cudaStream_t stream) {
  Shape s{p.q, p.k, p.pos, p.freqs, p.T, p.D, p.rot, p.rot / 2, p.amplitude, 1, 0, 1, 0, 0, 0, 0};
  const int H = p.q.H + p.k.H;
  s.turned = s.half / kE;
  s.parts = s.turned + (p.D - p.rot + 2 * kE - 1) / (2 * kE);
  s.m_parts = magic((uint32_t)s.parts);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  // Two blocks an SM.  With fewer tokens than warps, several warps a token, each with an item a lane at least;
  // with few items a token (a round of a warp has 96), as many tokens a warp as fill its rounds, and the rounds of all
  // warps, best (2 + 1 heads of 64, 65,536 tokens: 16 us, 34 with one token at a time; 12 + 1 heads of 64, 43,045 tokens:
  // 31 and 37 us; of 24 + 2 heads of 128 in fp32, 208 items, 65 and 61).
  const int64_t warps = (int64_t)2 * sms * kWarps, items = (int64_t)H * s.parts;
  const int64_t split = std::min<int64_t>(std::max<int64_t>(1, warps / p.T), std::max<int64_t>(1, items / 32));
  s.heads = (int)((H + split - 1) / split);
  s.split = (H + s.heads - 1) / s.heads;
  if (s.split == 1 && items <= 128) {
    double most = 0;   // of the places in all rounds, those with an item
    for (int64_t k = 1; k <= std::min<int64_t>(8, 512 / std::max(s.half, 1)); ++k) {
      const int64_t rounds = (k * items + 32 * kItems - 1) / (32 * kItems), turns = ((p.T + k - 1) / k + warps - 1) / warps;
      const double full = (double)(p.T * items) / (double)(turns * warps * rounds * 32 * kItems);
      if (full > 1.03 * most) most = full, s.tokens = (int)k;
    }
  }
  if (s.tokens > 1) s.m_token = magic((uint32_t)(s.heads * s.parts));
  const size_t smem = (size_t)s.half * 8 * (1 + kWarps * s.tokens);   // 36 KB at most
  const int64_t units = s.split == 1 ? (p.T + s.tokens - 1) / s.tokens : p.T * s.split;
  const unsigned grid = (unsigned)std::min<int64_t>(2 * sms, (units + kWarps - 1) / kWarps);
  auto go = [&](auto kernel) -> cudaError_t {
    return launch_kernel(kernel, dim3(grid), 32 * kWarps, smem, 0, stream, s);
  };
  prof_begin(stream, "rotary_kernel");
  auto pick = [&](auto many) -> cudaError_t {
    constexpr bool kMany = decltype(many)::value;
    const bool inverse = (p.flags & KDA_ROTARY_INVERSE) != 0;
    if (p.flags & KDA_ROTARY_INTERLEAVED) return inverse ? go(rotary_kernel<T, kE, true, true, kMany>) : go(rotary_kernel<T, kE, true, false, kMany>);
    return inverse ? go(rotary_kernel<T, kE, false, true, kMany>) : go(rotary_kernel<T, kE, false, false, kMany>);
  };
  if constexpr (kE == 1) e = pick(std::true_type{});
  else e = s.tokens > 1 ? pick(std::true_type{}) : pick(std::false_type{});
  prof_end(stream);
  return e;
}

bool steps16(const RotaryPart& p, size_t eb) {
  if (p.H == 0) return true;
  const int64_t step = (int64_t)(16 / eb);
  return reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && reinterpret_cast<uintptr_t>(p.y) % 16 == 0 && p.xt % step == 0 && p.xh % step == 0 &&
         p.yt % step == 0 && p.yh % step == 0;
}

template <typename T>
cudaError_t pick(const RotaryProblem& p, cudaStream_t stream) {
  const bool wide = p.D % 8 == 0 && p.rot % 16 == 0 && steps16(p.q, sizeof(T)) && steps16(p.k, sizeof(T));
  return wide ? launch<T, 8>(p, stream) : launch<T, 1>(p, stream);
}

}  // namespace

cudaError_t launch_rotary(const RotaryProblem& p, cudaStream_t stream) {
  return p.dt == KDA_F32 ? pick<float>(p, stream) : pick<__nv_bfloat16>(p, stream);
}

}  // namespace dense
}  // namespace kda
