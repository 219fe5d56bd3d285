// Writing tokens into the 4-bit cache and reading them back.
//
// For 32 channels of a token and head, a = max |x|:
//   e = least e >= -126 with a <= 6 * 2^e,  code = E2M1(x * 2^-e) to nearest even.
// In bits: a = m * 2^(E-127), m in [1, 2), is at most 1.5 * 2^(e+2) for e + 127 =
// E - 2 when m <= 1.5 and E - 1 when m > 1.5, so the scale byte is the exponent
// field of (bits(a) + 0x3fffff) minus 2.  x * 2^-e is exact, and the hardware's
// conversion rounds it once.
//
// Bound: HBM.  A warp takes eight tokens of a head, keys and values, with all its loads
// on their way at once.  Writing, a lane converts eight channels at a time (16 bytes of
// bf16, four lanes a scale group): a 32-bit word of a key row goes out as it is; value
// codes pass through shared memory, so that the lanes of eight tokens write the eight
// bytes that a unit keeps of each token next to one another.  Each token's place comes
// from its own slot; consecutive slots make whole lines of these stores.
// Measured for 65,536 tokens, 8 heads of 128 (replayed from a graph): bf16, 340 MB each way,
// write 67.9 us, 5.0 TB/s, read-back 52.3 us, 6.5 TB/s; fp32, 608 MB, write 98.2 us, 6.2 TB/s,
// read-back 93.7 us, 6.5 TB/s.  What keeps the bf16 write below the others has not been profiled.
#include "internal.cuh"

namespace kda {
namespace kv4 {
namespace {

constexpr int kThreads = 128;

// Eight channels as they lie in memory: the largest |x| by its bits (an inf or NaN stays
// above every finite value), and the values.
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void clear() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ uint32_t top() const {   // as fp32 bits
    const uint32_t m = 0x7fff7fffu, w = __vmaxu2(__vmaxu2(u.x & m, u.y & m), __vmaxu2(u.z & m, u.w & m));
    return max(w << 16, w & 0xffff0000u);
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ uint32_t top() const {
    float x[8];
    values(x);
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) t = max(t, __float_as_uint(x[i]) & 0x7fffffffu);
    return t;
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
};
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    __stcs(reinterpret_cast<float4*>(p) + i, make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]));
}

__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&x)[8]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
  __stcs(reinterpret_cast<uint2*>(p), make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b)));
}
__device__ __forceinline__ void store4(float* p, const float (&x)[8]) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
}

// E2M1 codes of eight scaled values, the first in the lowest bits
__device__ __forceinline__ uint32_t encode8(const float (&x)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}
__device__ __forceinline__ void decode8(uint32_t w, float (&x)[8]) {
  uint32_t r[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <int D>
__device__ __forceinline__ uint8_t* unit_of(uint8_t* cache, int32_t slot, int32_t page_size, int32_t Hkv, int head) {
  const int32_t page = slot / page_size, in = slot - page * page_size;
  const int32_t upp = page_size / kUnit;
  return cache + (((int64_t)page * Hkv + head) * upp + in / kUnit) * Unit<D>::kBytes;
}

constexpr int kTok = 8, kWarps = kThreads / 32;   // tokens of a warp

// The slot of token tok, or -1 when it has none; one beyond the cache is reported.
__device__ __forceinline__ int32_t slot_of(const CopyProblem& p, int64_t tok) {
  if (tok >= p.T) return -1;
  const int32_t s = p.slots[tok];
  if (s >= p.num_slots) report_bad(p.dev_err);
  return s < p.num_slots ? s : -1;
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) append_kernel(const CopyProblem p, int64_t n_items) {
  using U = Unit<D>;
  constexpr int LT = D / 8, TI = 32 / LT, NI = kTok / TI;   // lanes of a token; tokens of a load; loads
  __shared__ __align__(16) uint8_t stage[kWarps][kTok * (D / 2)];   // values [token][g][group] 16-bit words
  __shared__ __align__(16) uint8_t scales[kWarps][2][kTok][4];
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int sub = lane / LT, c8 = lane % LT, j = c8 >> 2, t = c8 & 3;   // this lane's token of a load, its channels 8 c8 ..
  for (int64_t item = (int64_t)blockIdx.x * kWarps + warp; item < n_items; item += (int64_t)gridDim.x * kWarps) {
    const int head = (int)(item % p.Hkv);
    const int64_t tok0 = item / p.Hkv * kTok;
    const int32_t mine = slot_of(p, tok0 + (lane & 7));   // lane i: token i % 8
    Eight<T> raw[2][NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int64_t tok = tok0 + i * TI + sub;
      raw[0][i].clear();
      raw[1][i].clear();
      if (tok < p.T) {
        raw[0][i].load(static_cast<const T*>(p.k) + tok * p.kt + head * p.kh + c8 * 8);
        raw[1][i].load(static_cast<const T*>(p.v) + tok * p.vt + head * p.vh + c8 * 8);
      }
    }
    __syncwarp();   // the last item's stage has been read
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        uint32_t top = raw[kv][i].top();
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        int32_t byte = max((int32_t)((top + 0x3fffffu) >> 23) - 2, 1);
        float y[8];
        raw[kv][i].values(y);
        const float inv = __uint_as_float((uint32_t)(254 - min(byte, 253)) << 23);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] *= inv;
        if (top >= 0x7f800000u) {   // not finite
          byte = 255;
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = 0.f;
        }
        const uint32_t code = encode8(y);
        const int tk = i * TI + sub;
        if (kv == 0) {
          const int32_t slot = __shfl_sync(0xffffffffu, mine, tk);
          if (slot >= 0)
            *reinterpret_cast<uint32_t*>(unit_of<D>(p.cache, slot, p.page_size, p.Hkv, head) + U::key_word(slot % kUnit, j, t)) = code;
        } else {
          uint16_t* w = reinterpret_cast<uint16_t*>(stage[warp] + tk * (D / 2));
          w[2 * t * U::kGroups + j] = (uint16_t)code;
          w[(2 * t + 1) * U::kGroups + j] = (uint16_t)(code >> 16);
        }
        if (t == 0) scales[warp][kv][tk][j] = (uint8_t)byte;
      }
    __syncwarp();
    if (mine >= 0) {   // lane: token lane % 8
      uint8_t* u = unit_of<D>(p.cache, mine, p.page_size, p.Hkv, head);
      const int r = mine % kUnit, tk = lane & 7;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int g = lane / 8 + 4 * i;
        const uint8_t* w = stage[warp] + tk * (D / 2) + g * (D / 16);
        if constexpr (D == 128) *reinterpret_cast<uint2*>(u + U::val_half(r, 0, g)) = *reinterpret_cast<const uint2*>(w);
        else *reinterpret_cast<uint32_t*>(u + U::val_half(r, 0, g)) = *reinterpret_cast<const uint32_t*>(w);
      }
      if (lane < 16) {   // lanes 0-7 the keys' scales, 8-15 the values'
        const int kv = lane / 8;
        uint8_t* dst = u + (kv ? U::kVs : U::kKs) + r * U::kGroups;
        if constexpr (D == 128) *reinterpret_cast<uint32_t*>(dst) = *reinterpret_cast<const uint32_t*>(scales[warp][kv][tk]);
        else *reinterpret_cast<uint16_t*>(dst) = *reinterpret_cast<const uint16_t*>(scales[warp][kv][tk]);
      }
    }
  }
}

__device__ __forceinline__ float scale_of(uint32_t byte) { return byte == 255 ? __uint_as_float(0x7fffffffu) : scale_f32(byte); }

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) gather_kernel(const CopyProblem p, int64_t n_items) {
  using U = Unit<D>;
  constexpr int GR = U::kGroups;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  for (int64_t item = (int64_t)blockIdx.x * kWarps + warp; item < n_items; item += (int64_t)gridDim.x * kWarps) {
    const int head = (int)(item % p.Hkv);
    const int64_t tok0 = item / p.Hkv * kTok;
    // keys: lane 4 i + t has words (j, t) of token i; values: lane 8 i + g has the four channels of every group at g
    // of tokens i and 4 + i
    const int t = lane & 3, g = lane & 7;
    const int tk[3] = {lane >> 2, lane >> 3, 4 + (lane >> 3)};
    uint32_t code[3][GR], sc[3];
    bool in[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int32_t slot = slot_of(p, tok0 + tk[i]);
      in[i] = tok0 + tk[i] < p.T;
#pragma unroll
      for (int j = 0; j < GR; ++j) code[i][j] = 0;
      sc[i] = 0;
      if (slot >= 0) {
        const uint8_t* u = unit_of<D>(p.cache, slot, p.page_size, p.Hkv, head);
        const int r = slot % kUnit;
        if (i == 0) {
          const uint8_t* w = u + U::key_word(r, 0, t);
          if constexpr (GR == 4) {
            const uint4 a = *reinterpret_cast<const uint4*>(w);
            code[0][0] = a.x; code[0][1] = a.y; code[0][2] = a.z; code[0][3] = a.w;
          } else {
            const uint2 a = *reinterpret_cast<const uint2*>(w);
            code[0][0] = a.x; code[0][1] = a.y;
          }
        } else {
          const uint8_t* w = u + U::val_half(r, 0, g);
          if constexpr (GR == 4) {
            const uint2 a = *reinterpret_cast<const uint2*>(w);
            code[i][0] = a.x & 0xffffu; code[i][1] = a.x >> 16; code[i][2] = a.y & 0xffffu; code[i][3] = a.y >> 16;
          } else {
            const uint32_t a = *reinterpret_cast<const uint32_t*>(w);
            code[i][0] = a & 0xffffu; code[i][1] = a >> 16;
          }
        }
        const uint8_t* f = u + (i ? U::kVs : U::kKs) + r * GR;
        sc[i] = GR == 4 ? *reinterpret_cast<const uint32_t*>(f) : *reinterpret_cast<const uint16_t*>(f);
      }
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      if (!in[i]) continue;
      T* out = static_cast<T*>(const_cast<void*>(i ? p.v : p.k)) + ((tok0 + tk[i]) * p.Hkv + head) * D;
#pragma unroll
      for (int j = 0; j < GR; ++j) {
        float x[8];
        decode8(code[i][j], x);
        const float s = scale_of(sc[i] >> (8 * j) & 0xffu);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= s;
        if (i == 0) store8(out + 32 * j + 8 * t, x);
        else store4(out + 32 * j + 4 * g, x);
      }
    }
  }
}

unsigned grid_for(int64_t n_items) {
  const int64_t n = (n_items + kWarps - 1) / kWarps;
  return (unsigned)(n > 1 << 20 ? 1 << 20 : n);
}

}  // namespace

cudaError_t launch_append(const CopyProblem& p, cudaStream_t stream) {
  const int64_t n = (p.T + kTok - 1) / kTok * p.Hkv;
  if (n == 0) return cudaSuccess;
  prof_begin(stream, "kv4_append_kernel");
  auto go = [&](auto kernel) { kernel<<<grid_for(n), kThreads, 0, stream>>>(p, n); };
  if (p.D == 128) p.dt == KDA_BF16 ? go(append_kernel<128, __nv_bfloat16>) : go(append_kernel<128, float>);
  else p.dt == KDA_BF16 ? go(append_kernel<64, __nv_bfloat16>) : go(append_kernel<64, float>);
  prof_end(stream);
  return cudaGetLastError();
}

cudaError_t launch_gather(const CopyProblem& p, cudaStream_t stream) {
  const int64_t n = (p.T + kTok - 1) / kTok * p.Hkv;
  if (n == 0) return cudaSuccess;
  prof_begin(stream, "kv4_gather_kernel");
  auto go = [&](auto kernel) { kernel<<<grid_for(n), kThreads, 0, stream>>>(p, n); };
  if (p.D == 128) p.dt == KDA_BF16 ? go(gather_kernel<128, __nv_bfloat16>) : go(gather_kernel<128, float>);
  else p.dt == KDA_BF16 ? go(gather_kernel<64, __nv_bfloat16>) : go(gather_kernel<64, float>);
  prof_end(stream);
  return cudaGetLastError();
}

}  // namespace kv4
}  // namespace kda
