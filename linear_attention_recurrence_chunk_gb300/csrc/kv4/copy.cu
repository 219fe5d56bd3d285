// Writing tokens into the 4-bit cache and reading them back.
//
// For 32 channels of a token and head, a = max |x|:
//   e = least e >= -126 with a <= 6 * 2^e,  code = E2M1(x * 2^-e) to nearest even.
// In bits: a = m * 2^(E-127), m in [1, 2), is at most 1.5 * 2^(e+2) for e + 127 =
// E - 2 when m <= 1.5 and E - 1 when m > 1.5, so the scale byte is the exponent
// field of (bits(a) + 0x3fffff) minus 2.  x * 2^-e is exact, and the hardware's
// conversion rounds it once.
//
// Bound: HBM.  A lane takes eight channels (16 bytes of bf16): one 32-bit key word
// or two 16-bit value words of the cache, four lanes a scale group.
#include "internal.cuh"

namespace kda {
namespace kv4 {
namespace {

constexpr int kThreads = 256;

// eight channels as fp32
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 u = __ldcs(reinterpret_cast<const float4*>(p) + i);
    x[4 * i] = u.x; x[4 * i + 1] = u.y; x[4 * i + 2] = u.z; x[4 * i + 3] = u.w;
  }
}
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

// Where a lane's eight channels of (token, head, keys or values) are: `item` counts
// groups of eight channels, keys of a token and head first, then its values.
template <int D>
struct Place {
  int64_t tok;
  int head, c8;   // c8: channel / 8
  bool val;
  __device__ __forceinline__ Place(int64_t item, int32_t Hkv) {
    constexpr int per = D / 8;
    c8 = (int)(item % per);
    const int64_t r = item / per;
    val = (r & 1) != 0;
    head = (int)((r >> 1) % Hkv);
    tok = (r >> 1) / Hkv;
  }
};

template <int D>
__device__ __forceinline__ uint8_t* unit_of(uint8_t* cache, int32_t slot, int32_t page_size, int32_t Hkv, int head) {
  const int32_t page = slot / page_size, in = slot - page * page_size;
  const int32_t upp = page_size / kUnit;
  return cache + (((int64_t)page * Hkv + head) * upp + in / kUnit) * Unit<D>::kBytes;
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) append_kernel(const CopyProblem p, int64_t n_items) {
  using U = Unit<D>;
  // whole warps run the loop: the scale is a maximum over four lanes
  for (int64_t item = (int64_t)blockIdx.x * kThreads + threadIdx.x; item - (threadIdx.x & 31) < n_items;
       item += (int64_t)gridDim.x * kThreads) {
    const bool in = item < n_items;
    const Place<D> at(in ? item : 0, p.Hkv);
    const int32_t slot = in ? p.slots[at.tok] : -1;
    const bool keep = slot >= 0 && slot < p.num_slots;
    if (slot >= 0 && !keep) report_bad(p.dev_err);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
    if (keep)
      load8(at.val ? static_cast<const T*>(p.v) + at.tok * p.vt + at.head * p.vh + at.c8 * 8
                   : static_cast<const T*>(p.k) + at.tok * p.kt + at.head * p.kh + at.c8 * 8,
            x);
    uint32_t top = 0;   // the largest |x| by its bits: an inf or NaN stays above every finite value
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const bool finite = top < 0x7f800000u;
    const int32_t byte = finite ? max((int32_t)((top + 0x3fffffu) >> 23) - 2, 1) : 255;
    const float inv = finite ? __uint_as_float((uint32_t)(254 - byte) << 23) : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = finite ? x[i] * inv : 0.f;
    const uint32_t code = encode8(x);
    if (!keep) continue;
    uint8_t* u = unit_of<D>(p.cache, slot, p.page_size, p.Hkv, at.head);
    const int r = slot % kUnit, j = at.c8 >> 2, t = at.c8 & 3;
    if (!at.val) {
      *reinterpret_cast<uint32_t*>(u + U::key_word(r, j, t)) = code;
    } else {
      *reinterpret_cast<uint16_t*>(u + U::val_half(r, j, 2 * t)) = (uint16_t)code;
      *reinterpret_cast<uint16_t*>(u + U::val_half(r, j, 2 * t + 1)) = (uint16_t)(code >> 16);
    }
    if (t == 0) u[(at.val ? U::kVs : U::kKs) + r * U::kGroups + j] = (uint8_t)byte;
  }
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) gather_kernel(const CopyProblem p, int64_t n_items) {
  using U = Unit<D>;
  for (int64_t item = (int64_t)blockIdx.x * kThreads + threadIdx.x; item < n_items;
       item += (int64_t)gridDim.x * kThreads) {
    const Place<D> at(item, p.Hkv);
    const int32_t slot = p.slots[at.tok];
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
    if (slot >= p.num_slots) report_bad(p.dev_err);
    if (slot >= 0 && slot < p.num_slots) {
      const uint8_t* u = unit_of<D>(p.cache, slot, p.page_size, p.Hkv, at.head);
      const int r = slot % kUnit, j = at.c8 >> 2, t = at.c8 & 3;
      const uint32_t code = at.val ? (uint32_t)*reinterpret_cast<const uint16_t*>(u + U::val_half(r, j, 2 * t)) |
                                         (uint32_t)*reinterpret_cast<const uint16_t*>(u + U::val_half(r, j, 2 * t + 1)) << 16
                                   : *reinterpret_cast<const uint32_t*>(u + U::key_word(r, j, t));
      const uint32_t byte = u[(at.val ? U::kVs : U::kKs) + r * U::kGroups + j];
      const float s = byte == 255 ? __uint_as_float(0x7fffffffu) : scale_f32(byte);
      decode8(code, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= s;
    }
    T* out = static_cast<T*>(const_cast<void*>(at.val ? p.v : p.k)) + (at.tok * p.Hkv + at.head) * D + at.c8 * 8;
    store8(out, x);
  }
}

unsigned grid_for(int64_t n_items) {
  const int64_t n = (n_items + kThreads - 1) / kThreads;
  return (unsigned)(n > 1 << 20 ? 1 << 20 : n);
}

}  // namespace

cudaError_t launch_append(const CopyProblem& p, cudaStream_t stream) {
  const int64_t n = p.T * p.Hkv * 2 * (p.D / 8);
  if (n == 0) return cudaSuccess;
  prof_begin(stream, "kv4_append_kernel");
  auto go = [&](auto kernel) { kernel<<<grid_for(n), kThreads, 0, stream>>>(p, n); };
  if (p.D == 128) p.dt == KDA_BF16 ? go(append_kernel<128, __nv_bfloat16>) : go(append_kernel<128, float>);
  else p.dt == KDA_BF16 ? go(append_kernel<64, __nv_bfloat16>) : go(append_kernel<64, float>);
  prof_end(stream);
  return cudaGetLastError();
}

cudaError_t launch_gather(const CopyProblem& p, cudaStream_t stream) {
  const int64_t n = p.T * p.Hkv * 2 * (p.D / 8);
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
