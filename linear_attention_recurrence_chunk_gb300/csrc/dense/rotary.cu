// Rotary positions.
//
//   (a, b) -> amplitude (a cos t - b sin t, a sin t + b cos t),   t = position * frequency
//
// The angle is wanted modulo a turn, and positions go to 2^31: the frequency in turns, modulo 1, is held
// as a 64-bit fixed-point fraction (from fp64 once per block), so that its product with the position p
// modulo 2^64 is the fraction of a turn to p 2^-63, with no reduction and no table.  The top 32 bits, signed,
// are half turns in [-1, 1) for sincospi.
//
// Bound: HBM, each value read and written once.  A block takes a few tokens: their cosines and sines
// once into shared memory, then all heads of queries and keys, eight pairs (two 16-byte loads of bf16) a
// thread and four such items on their way at once.
#include <algorithm>

#include "internal.cuh"

namespace kda {
namespace dense {
namespace {

constexpr int kThreads = 256, kItems = 4;

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
  int32_t tokens;         // of a block
  int32_t heads;          // of a block (blockIdx.y)
  int32_t parts, turned;  // items of a head: of pairs, then of channels that stay
  uint32_t m_heads, m_parts;
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

template <typename T, int kE, bool kNext, bool kInverse>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const Shape s) {
  extern __shared__ uint64_t sm[];
  uint64_t* turn = sm;                                          // [half] turns per position, 2^-64 each
  float2* cs = reinterpret_cast<float2*>(turn + s.half);        // [tokens][half]
  int32_t* pos = reinterpret_cast<int32_t*>(cs + s.tokens * s.half);
  const int64_t t0 = (int64_t)blockIdx.x * s.tokens;
  const int nt = (int)(s.T - t0 < s.tokens ? s.T - t0 : s.tokens);
  const int H = s.q.H + s.k.H, h0 = blockIdx.y * s.heads, nh = H - h0 < s.heads ? H - h0 : s.heads;
  const int tid = threadIdx.x;
  for (int i = tid; i < s.half; i += kThreads) {
    // freq / (2 pi) as a rounded product and what it lacks: 1 / (2 pi) = kHi + kLo to 2^-110
    constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;
    const double w = s.freqs[i], f = w * kHi, low = fma(w, kHi, -f) + w * kLo;
    turn[i] = fraction(f) + fraction(low);
  }
  for (int i = tid; i < nt; i += kThreads) pos[i] = s.pos[t0 + i];
  __syncthreads();
  for (int i = tid; i < nt * s.half; i += kThreads) {
    const int t = i / s.half, e = i - t * s.half;
    const int32_t frac = (int32_t)((uint64_t)(uint32_t)pos[t] * turn[e] >> 32);
    float sn, c;
    sincospif((float)frac * 0x1p-31f, &sn, &c);
    cs[i] = make_float2(c * s.amplitude, (kInverse ? -sn : sn) * s.amplitude);
  }
  __syncthreads();

  const uint32_t n = (uint32_t)(nt * s.heads * s.parts);
  for (uint32_t i0 = tid; i0 < n; i0 += kThreads * kItems) {
    Values<T, kE> a[kItems], b[kItems];
    T *ya[kItems], *yb[kItems];                                  // NULL: nothing to write
    const float2* c[kItems];                                     // NULL: the values stay
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
      ya[j] = yb[j] = nullptr;
      c[j] = nullptr;
      const uint32_t i = i0 + kThreads * j, th = divide(i, s.m_parts), part = i - th * s.parts;
      const uint32_t t = divide(th, s.m_heads), hl = th - t * s.heads;
      if (i >= n || (int)hl >= nh) continue;
      const int h = h0 + (int)hl;
      const bool isq = h < s.q.H;
      const RotaryPart& p = isq ? s.q : s.k;
      const int hh = isq ? h : h - s.q.H;
      const T* x = static_cast<const T*>(p.x) + (t0 + t) * p.xt + hh * p.xh;
      T* y = static_cast<T*>(p.y) + (t0 + t) * p.yt + hh * p.yh;
      const bool turned = (int)part < s.turned && pos[t] >= 0;
      int ca, cb;
      if ((int)part < s.turned) {
        ca = kNext ? 2 * kE * part : kE * part;
        cb = kNext ? ca + kE : s.half + ca;
      } else {
        ca = s.rot + 2 * kE * (part - s.turned);
        cb = ca + kE < s.D ? ca + kE : -1;
      }
      if (!turned && x == y) continue;                           // in place
      a[j].load(x + ca);
      ya[j] = y + ca;
      if (cb >= 0) {
        b[j].load(x + cb);
        yb[j] = y + cb;
      }
      if (turned) c[j] = cs + t * s.half + kE * part;
    }
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
      if (c[j]) {
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          // kNext: pair e is values 2 e, 2 e + 1 of a and b together
          T& u = kNext && kE > 1 ? (2 * e < kE ? a[j].x[(2 * e) % kE] : b[j].x[(2 * e) % kE]) : a[j].x[e];
          T& w = kNext && kE > 1 ? (2 * e < kE ? a[j].x[(2 * e + 1) % kE] : b[j].x[(2 * e + 1) % kE]) : b[j].x[e];
          const float2 z = c[j][e];
          const float x0 = to_f32<T>(u), x1 = to_f32<T>(w);
          u = from_f32<T>(x0 * z.x - x1 * z.y);
          w = from_f32<T>(x0 * z.y + x1 * z.x);
        }
      }
      if (ya[j]) a[j].store(ya[j]);
      if (yb[j]) b[j].store(yb[j]);
    }
  }
}

uint32_t magic(uint32_t d) { return d == 1 ? 0u : (uint32_t)((0x100000000ull + d - 1) / d); }

template <typename T, int kE>
cudaError_t launch(const RotaryProblem& p, cudaStream_t stream) {
  Shape s{p.q, p.k, p.pos, p.freqs, p.T, p.D, p.rot, p.rot / 2, p.amplitude, 1, 0, 0, 0, 0, 0};
  const int H = p.q.H + p.k.H;
  s.turned = s.half / kE;
  s.parts = s.turned + (p.D - p.rot + 2 * kE - 1) / (2 * kE);
  // Tokens of a block: 32 KB of values or more, as long as that leaves 1,024 blocks; few tokens: their heads
  // over several blocks, at least one item a thread.
  const int64_t per_token = (int64_t)H * p.D * (int64_t)sizeof(T);
  s.tokens = (int)std::max<int64_t>(1, std::min<int64_t>({16, (32768 + per_token - 1) / per_token, p.T / 1024}));
  int split = 1;
  if (p.T < 512) split = (int)std::min<int64_t>(std::max<int64_t>(1, (int64_t)H * s.parts / kThreads), (512 + p.T - 1) / p.T);
  s.heads = (H + split - 1) / split;
  split = (H + s.heads - 1) / s.heads;
  s.m_heads = magic((uint32_t)s.heads);
  s.m_parts = magic((uint32_t)s.parts);
  const size_t smem = (size_t)s.half * 8 + (size_t)s.tokens * s.half * 8 + (size_t)s.tokens * 4;
  const dim3 grid((unsigned)((p.T + s.tokens - 1) / s.tokens), (unsigned)split);
  auto go = [&](auto kernel) -> cudaError_t {
    if (smem > 48 * 1024) {
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 72 * 1024);
      if (e != cudaSuccess) return e;
    }
    kernel<<<grid, kThreads, smem, stream>>>(s);
    return cudaGetLastError();
  };
  prof_begin(stream, "rotary_kernel");
  cudaError_t e;
  if (p.flags & KDA_ROTARY_INTERLEAVED) e = p.flags & KDA_ROTARY_INVERSE ? go(rotary_kernel<T, kE, true, true>) : go(rotary_kernel<T, kE, true, false>);
  else e = p.flags & KDA_ROTARY_INVERSE ? go(rotary_kernel<T, kE, false, true>) : go(rotary_kernel<T, kE, false, false>);
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
