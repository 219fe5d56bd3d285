// Index arithmetic of the attention kernels over a paged cache, apart from the
// kernels so that it can be compiled and checked on the host over its whole range.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define KDA_INDEX_FN __host__ __device__ __forceinline__
#else
#define KDA_INDEX_FN inline
#endif

namespace kda {
namespace kv4 {

// unit / upp as a product, for unit < 2^27 (2^31 - 1 tokens) and upp <= 256 units of a page.
// The inverse is above 2^36 / upp by less than 1, so the quotient by less than
// 2^27 / 2^36 = 2^-9 <= 1 / (2 upp), which does not reach the next page; the product is at most 2^63.
KDA_INDEX_FN uint64_t page_inverse(uint32_t upp) { return (((uint64_t)1 << 36) + upp - 1) / upp; }
KDA_INDEX_FN uint32_t page_of_unit(uint32_t unit, uint64_t inverse) { return (uint32_t)(unit * inverse >> 36); }

// Token `at` of tile i, tiles of `tokens`.  What is loaded ahead lies up to two tiles behind the
// last, and a sequence may have 2^31 - 1 tokens: 64 bits.
KDA_INDEX_FN int64_t token_of_tile(int64_t i, int32_t tokens, int32_t at) { return i * tokens + at; }

// Units of 16 tokens, `most` at most, that tile i (tiles of `most` units) holds of a sequence of L.
// (L + 15 passes 31 bits.)
KDA_INDEX_FN int32_t units_of_tile(int32_t L, int32_t i, int32_t most) {
  const int32_t n = (int32_t)(((uint32_t)L + 15) / 16) - i * most;
  return n < most ? n : most;
}

// Blocks of R query rows that qn query tokens of G heads fill; qn G is at most 2^31 - 1.
KDA_INDEX_FN int32_t row_blocks(int32_t qn, int32_t G, int32_t R) { return (int32_t)(((uint32_t)(qn * G) + R - 1) / R); }

}  // namespace kv4
}  // namespace kda
