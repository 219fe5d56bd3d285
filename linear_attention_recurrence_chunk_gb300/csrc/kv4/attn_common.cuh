// Device helpers of the two attention kernels over the 4-bit cache.
#pragma once

#include <cuda_fp16.h>

#include "../tc_ptx.cuh"
#include "internal.cuh"

namespace kda {
namespace kv4 {

constexpr long long kWaitLimit = 2000000000LL;   // ~1 s of SM clocks per bounded wait
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The four bytes of w, each two E2M1 codes, as fp16 pairs.
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}

__device__ __forceinline__ uint32_t pack(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// A sequence's cached tokens and its query tokens; what is out of range is cut
// back (no access leaves the arrays) and said in *bad.
struct Seq {
  int32_t L, q0, qn;
};
__device__ __forceinline__ Seq seq_of(const AttnProblem& p, int n, bool* bad) {
  Seq s;
  const int64_t cap = p.num_pages > 0 ? (int64_t)p.max_pages * p.page_size : 0;
  s.L = p.lens[n];
  if (s.L < 0 || s.L > cap) {
    *bad = true;
    s.L = s.L < 0 ? 0 : (int32_t)cap;
  }
  s.q0 = n;
  s.qn = 1;
  if (p.cu) {
    s.q0 = p.cu[n];
    const int64_t qn = (int64_t)p.cu[n + 1] - s.q0;
    const bool ok = s.q0 >= 0 && qn >= 0 && qn <= p.max_q && (int64_t)s.q0 + qn <= p.T;
    if (!ok || (n == 0 && s.q0 != 0)) *bad = true;
    s.qn = ok ? (int32_t)qn : 0;
  }
  return s;
}

}  // namespace kv4
}  // namespace kda
