// C ABI of the 4-bit key/value cache: argument validation and dispatch.
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "internal.cuh"

namespace {

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

struct Range {
  const void* p;
  size_t n;
};
bool overlaps(const Range& a, const Range& b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.n && y < x + a.n;
}

// Every output apart from every input and from the other outputs.
template <size_t NI, size_t NO>
bool apart(const Range (&in)[NI], const Range (&out)[NO]) {
  for (size_t i = 0; i < NO; ++i) {
    for (const Range& r : in)
      if (overlaps(out[i], r)) return false;
    for (size_t j = i + 1; j < NO; ++j)
      if (overlaps(out[i], out[j])) return false;
  }
  return true;
}

size_t elem(kda_dtype dt) { return dt == KDA_F32 ? 4 : 2; }

// Shape of a cache: status, and its bytes.
kda_status check_cache(int64_t num_pages, int32_t Hkv, int32_t page_size, int32_t D, size_t* bytes) {
  if (num_pages < 0 || Hkv <= 0 || Hkv > 65535) return KDA_ERR_INVALID_ARG;
  if (page_size <= 0 || page_size > 4096 || page_size % kda::kv4::kUnit != 0) return KDA_ERR_INVALID_ARG;
  if (num_pages > INT32_MAX / page_size) return KDA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return KDA_ERR_UNSUPPORTED;
  *bytes = (size_t)num_pages * (size_t)Hkv * (size_t)(page_size / kda::kv4::kUnit) * (size_t)(17 * D);
  return KDA_OK;
}

// A strided [T][H][D] tensor, T and H at least 1: strides in elements, 16-byte steps.
bool strides_ok(const void* p, int64_t T, int32_t H, int32_t D, int64_t ts, int64_t hs, size_t eb, Range* r) {
  const int64_t step = (int64_t)(16 / eb);
  if (!p || !aligned(p, 16) || ts % step != 0 || hs % step != 0) return false;
  constexpr int64_t kMost = (int64_t)1 << 31;
  if (ts < 0 || hs < 0 || ts > kMost || hs > kMost) return false;
  r->p = p;
  r->n = (size_t)((T - 1) * ts + (H - 1) * hs + D) * eb;
  return true;
}

}  // namespace

extern "C" {

size_t kda_kv4_cache_bytes(int64_t num_pages, int32_t Hkv, int32_t page_size, int32_t D) {
  size_t n = 0;
  return check_cache(num_pages, Hkv, page_size, D, &n) == KDA_OK ? n : SIZE_MAX;
}

kda_status kda_page_map(const int32_t* cached_lens, const int32_t* new_lens, int32_t N, int32_t* block_table,
                        int32_t max_pages, const int32_t* free_pages, int64_t num_free, const int32_t* free_start,
                        int32_t page_size, int64_t num_tokens, int32_t* cu_seqlens, int32_t* seq_lens,
                        int32_t* slot_map, int32_t* positions, int32_t* free_next, cudaStream_t stream) {
  if (N < 0 || max_pages < 0 || num_free < 0 || num_free > INT32_MAX || num_tokens < 0 ||
      num_tokens > INT32_MAX - 4096)
    return KDA_ERR_INVALID_ARG;
  if (page_size <= 0 || page_size > 4096 || page_size % kda::kv4::kUnit != 0) return KDA_ERR_INVALID_ARG;
  if (N > kda::kv4::kMapMaxRequests) return KDA_ERR_UNSUPPORTED;
  if (!free_start || !cu_seqlens || !free_next) return KDA_ERR_INVALID_ARG;
  if (N > 0 && (!cached_lens || !new_lens || !seq_lens)) return KDA_ERR_INVALID_ARG;
  if (N > 0 && max_pages > 0 && !block_table) return KDA_ERR_INVALID_ARG;
  if (num_free > 0 && !free_pages) return KDA_ERR_INVALID_ARG;
  if (num_tokens > 0 && (!slot_map || !positions)) return KDA_ERR_INVALID_ARG;
  const void* four[] = {cached_lens, new_lens, block_table, free_pages, free_start, cu_seqlens, seq_lens, free_next};
  for (const void* p : four)
    if (!aligned(p, 4)) return KDA_ERR_INVALID_ARG;
  if (!aligned(slot_map, 16) || !aligned(positions, 16)) return KDA_ERR_INVALID_ARG;
  const size_t n = (size_t)N * 4, t = (size_t)num_tokens * 4;
  const Range in[] = {{cached_lens, n}, {new_lens, n}, {free_pages, (size_t)num_free * 4}, {free_start, 4}};
  const Range out[] = {{block_table, n * (size_t)max_pages}, {cu_seqlens, n + 4}, {seq_lens, n},
                       {slot_map, t},  {positions, t},                           {free_next, 4}};
  if (!apart(in, out)) return KDA_ERR_INVALID_ARG;
  kda::kv4::PageMapProblem p{cached_lens, new_lens,   N,        block_table, max_pages, free_pages, num_free, free_start,
                             page_size,   num_tokens, cu_seqlens, seq_lens,  slot_map,  positions,  free_next, nullptr};
  if (kda::device_error_ptr(&p.dev_err) != cudaSuccess) return KDA_ERR_CUDA;
  return kda::kv4::launch_page_map(p, stream) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_kv4_append(const void* k, const void* v, const int32_t* slot_map, int64_t T, int32_t Hkv, int32_t D,
                          int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                          int64_t v_head_stride, kda_dtype dt, void* cache, int64_t num_pages, int32_t page_size,
                          cudaStream_t stream) {
  if (dt != KDA_F32 && dt != KDA_BF16) return KDA_ERR_INVALID_ARG;
  size_t bytes = 0;
  const kda_status st = check_cache(num_pages, Hkv, page_size, D, &bytes);
  if (st != KDA_OK) return st;
  if (T < 0 || T > INT32_MAX) return KDA_ERR_INVALID_ARG;
  if (T == 0) return KDA_OK;
  if (!slot_map || !aligned(slot_map, 4) || (bytes > 0 && !cache) || !aligned(cache, 16)) return KDA_ERR_INVALID_ARG;
  Range rk, rv;
  if (!strides_ok(k, T, Hkv, D, k_token_stride, k_head_stride, elem(dt), &rk) ||
      !strides_ok(v, T, Hkv, D, v_token_stride, v_head_stride, elem(dt), &rv))
    return KDA_ERR_INVALID_ARG;
  const Range in[] = {rk, rv, {slot_map, (size_t)T * 4}};
  const Range out[] = {{cache, bytes}};
  if (!apart(in, out)) return KDA_ERR_INVALID_ARG;
  kda::kv4::CopyProblem p{k, v, slot_map, T, Hkv, D, k_token_stride, k_head_stride, v_token_stride, v_head_stride, dt,
                          static_cast<uint8_t*>(cache), num_pages * page_size, page_size, nullptr};
  if (kda::device_error_ptr(&p.dev_err) != cudaSuccess) return KDA_ERR_CUDA;
  return kda::kv4::launch_append(p, stream) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_kv4_gather(const void* cache, int64_t num_pages, int32_t page_size, const int32_t* slot_map, int64_t T,
                          int32_t Hkv, int32_t D, kda_dtype dt, void* k, void* v, cudaStream_t stream) {
  if (dt != KDA_F32 && dt != KDA_BF16) return KDA_ERR_INVALID_ARG;
  size_t bytes = 0;
  const kda_status st = check_cache(num_pages, Hkv, page_size, D, &bytes);
  if (st != KDA_OK) return st;
  if (T < 0 || T > INT32_MAX) return KDA_ERR_INVALID_ARG;
  if (T == 0) return KDA_OK;
  if (!slot_map || !aligned(slot_map, 4) || (bytes > 0 && !cache) || !aligned(cache, 16)) return KDA_ERR_INVALID_ARG;
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16)) return KDA_ERR_INVALID_ARG;
  const size_t n = (size_t)T * Hkv * D * elem(dt);
  const Range in[] = {{cache, bytes}, {slot_map, (size_t)T * 4}};
  const Range out[] = {{k, n}, {v, n}};
  if (!apart(in, out)) return KDA_ERR_INVALID_ARG;
  kda::kv4::CopyProblem p{k, v, slot_map, T, Hkv, D, 0, 0, 0, 0, dt,
                          static_cast<uint8_t*>(const_cast<void*>(cache)), num_pages * page_size, page_size, nullptr};
  if (kda::device_error_ptr(&p.dev_err) != cudaSuccess) return KDA_ERR_CUDA;
  return kda::kv4::launch_gather(p, stream) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"

namespace {

kda_status check_attention(int64_t T, int32_t N, int32_t Hq, int32_t Hkv, int32_t D, int32_t max_q, kda_dtype dt) {
  if (dt != KDA_F32 && dt != KDA_BF16) return KDA_ERR_INVALID_ARG;
  if (T < 0 || N < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || max_q < 1) return KDA_ERR_INVALID_ARG;
  if (T > INT32_MAX || (int64_t)max_q * Hq > INT32_MAX || T * (int64_t)Hq > INT32_MAX) return KDA_ERR_INVALID_ARG;
  if (Hkv > 65535) return KDA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return KDA_ERR_UNSUPPORTED;
  if (N > 65535 || Hq / Hkv > 128) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

}  // namespace

extern "C" {

size_t kda_kv4_attention_workspace_size(int64_t T, int32_t N, int32_t Hq, int32_t Hkv, int32_t D, int32_t max_q_len,
                                        kda_dtype dt) {
  if (check_attention(T, N, Hq, Hkv, D, max_q_len, dt) != KDA_OK) return SIZE_MAX;
  return kda::kv4::attention_workspace(Hq, Hkv, D, max_q_len, dt);
}

kda_status kda_kv4_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* cache,
                             int64_t num_pages, int32_t page_size, const int32_t* block_table, int32_t max_pages,
                             const int32_t* seq_lens, const int32_t* cu_seqlens, int64_t T, int32_t N, int32_t Hq,
                             int32_t Hkv, int32_t D, int32_t max_q_len, float sm_scale, kda_dtype dt, void* o,
                             float* lse, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  kda_status st = check_attention(T, N, Hq, Hkv, D, max_q_len, dt);
  if (st != KDA_OK) return st;
  size_t bytes = 0;
  if ((st = check_cache(num_pages, Hkv, page_size, D, &bytes)) != KDA_OK) return st;
  if (max_pages < 0 || !isfinite(sm_scale)) return KDA_ERR_INVALID_ARG;
  if (!cu_seqlens && (T != N || max_q_len != 1)) return KDA_ERR_INVALID_ARG;
  if (T == 0 || N == 0) return KDA_OK;
  if (!o || !aligned(o, 16) || !aligned(lse, 4) || !seq_lens || !aligned(seq_lens, 4) || !aligned(cu_seqlens, 4))
    return KDA_ERR_INVALID_ARG;
  if ((max_pages > 0 && !block_table) || !aligned(block_table, 4) || (bytes > 0 && !cache) || !aligned(cache, 16))
    return KDA_ERR_INVALID_ARG;
  const size_t need = kda::kv4::attention_workspace(Hq, Hkv, D, max_q_len, dt);
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return KDA_ERR_INVALID_ARG;
  Range rq;
  if (!strides_ok(q, T, Hq, D, q_token_stride, q_head_stride, elem(dt), &rq)) return KDA_ERR_INVALID_ARG;
  const size_t rows = (size_t)T * Hq;
  const Range in[] = {rq, {cache, bytes}, {block_table, (size_t)N * max_pages * 4}, {seq_lens, (size_t)N * 4},
                      {cu_seqlens, ((size_t)N + 1) * 4}};
  const Range out[] = {{o, rows * D * elem(dt)}, {lse, rows * 4}, {workspace, need}};
  if (!apart(in, out)) return KDA_ERR_INVALID_ARG;
  kda::kv4::AttnProblem p{q, q_token_stride, q_head_stride, static_cast<const uint8_t*>(cache), num_pages, page_size,
                          block_table, max_pages, seq_lens, cu_seqlens, T, N, Hq, Hkv, D, max_q_len, sm_scale, dt, o,
                          lse, nullptr, 0};
  p.upp_inv = kda::kv4::page_inverse((uint32_t)(page_size / kda::kv4::kUnit));
  if (kda::device_error_ptr(&p.dev_err) != cudaSuccess) return KDA_ERR_CUDA;
  return kda::kv4::launch_attention(p, workspace, stream) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
