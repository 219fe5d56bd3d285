// The 4-bit key/value cache: its layout, the launchers behind include/kda_kv4.h
// and the device helpers that its kernels share.
#pragma once

#include "index.cuh"
#include "kda_internal.cuh"
#include "kda_kv4.h"

namespace kda {
namespace kv4 {

constexpr int kUnit = 16;   // tokens of a cache unit

// Byte offsets inside a unit of 16 tokens of one head (layout: include/kda_kv4.h).
template <int D>
struct Unit {
  static constexpr int kGroups = D / 32;            // scale groups of a token
  static constexpr int kBytes = 17 * D;
  static constexpr int kV = 8 * D, kKs = 16 * D, kVs = 16 * D + D / 2;
  static __host__ __device__ constexpr int key_word(int r, int j, int t) { return r * (D / 2) + 4 * (t * kGroups + j); }
  static __host__ __device__ constexpr int val_half(int r, int j, int g) {
    return kV + (r >> 3) * (4 * D) + ((g * 8 + (r & 7)) * kGroups + j) * 2;
  }
};

// A page, slot, length or prefix sum out of range: KDA_ERR_INVALID_ARG through
// kda_device_error(), as a malformed cu_seqlens of the recurrence.
__device__ __forceinline__ void report_bad(int32_t* dev_err) { atomicCAS(dev_err, 0, (int32_t)kDevErrBadSeqlens); }

// 2^(byte - 127); inf for byte 255 (0 for byte 0, which no written block has).
__device__ __forceinline__ float scale_f32(uint32_t byte) { return __uint_as_float(byte << 23); }

struct PageMapProblem {
  const int32_t *cached, *fresh;
  int32_t N;
  int32_t* table;
  int32_t max_pages;
  const int32_t* free_pages;
  int64_t num_free;
  const int32_t* free_start;
  int32_t page_size;
  int64_t num_tokens;
  int32_t *cu, *lens, *slots, *pos, *free_next;
  int32_t* dev_err;
};
constexpr int kMapMaxRequests = 28672;
cudaError_t launch_page_map(const PageMapProblem& p, cudaStream_t stream);

struct CopyProblem {   // append (k, v read) and gather (k, v written)
  const void *k, *v;
  const int32_t* slots;
  int64_t T;
  int32_t Hkv, D;
  int64_t kt, kh, vt, vh;   // strides in elements (append)
  kda_dtype dt;
  uint8_t* cache;
  int64_t num_slots;
  int32_t page_size;
  int32_t* dev_err;
};
cudaError_t launch_append(const CopyProblem& p, cudaStream_t stream);
cudaError_t launch_gather(const CopyProblem& p, cudaStream_t stream);

struct AttnProblem {
  const void* q;
  int64_t qt, qh;           // strides in elements
  const uint8_t* cache;
  int64_t num_pages;
  int32_t page_size;
  const int32_t* table;
  int32_t max_pages;
  const int32_t *lens, *cu; // cu: nullptr for one query token per sequence
  int64_t T;
  int32_t N, Hq, Hkv, D, max_q;
  float sm_scale;
  kda_dtype dt;
  void* o;
  float* lse;
  int32_t* dev_err;
  uint64_t upp_inv;         // page_inverse(units of a page)
};
size_t attention_workspace(int32_t Hq, int32_t Hkv, int32_t D, int32_t max_q, kda_dtype dt);
cudaError_t launch_extend(const AttnProblem& p, cudaStream_t stream);   // bf16 only
cudaError_t launch_attention(const AttnProblem& p, void* workspace, cudaStream_t stream);

}  // namespace kv4
}  // namespace kda
