// The block-scaled 8-bit tensor-core instructions (tcgen05 kind::mxf8f6f4), what they need of
// shared memory and TMEM, and tensor maps over 8-bit matrices.
//
// D[m][n] += sum over 32 k of A[m][k] 2^(sa - 127) B[n][k] 2^(sb - 127), E4M3 values, E8M0 scale
// bytes, fp32 in TMEM.  The scales of 128 rows lie in four TMEM columns: the 32-bit word of row r
// in lane r % 32 (the same in each quarter of the lanes), column r / 32.  A word holds four bytes,
// and the instruction says which one it takes: here the byte of a K block of 128, so that one word
// serves four blocks and 16 instructions.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "tc_ptx.cuh"

namespace kda {
namespace dense {

constexpr long long kWaitLimit = 2000000000LL;   // ~1 s of SM clocks per bounded wait
constexpr int kStageK = 128;                     // bytes of K of a pipeline stage: one 128-byte swizzle row, one scale

// Instruction descriptor: E4M3 A and B, both K-major, E8M0 scales, shape M x N (x K = 32); the
// scale bytes that it takes are added by scale_ids.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
  return ((uint32_t)(N >> 3) << 17)     // N / 8
         | (1u << 23)                   // scale format: E8M0
         | ((uint32_t)(M >> 4) << 24);  // M / 16
}
__host__ __device__ constexpr uint32_t scale_ids(int byte) {
  return ((uint32_t)byte << 4) | ((uint32_t)byte << 29);   // of B, of A
}

// Descriptor of scale words in shared memory for tcgen05.cp: 32 rows of 16 bytes, no swizzle, 8-row
// groups 128 bytes apart.
__device__ __forceinline__ uint64_t desc_scales(uint32_t addr) {
  uint64_t d = 0;
  d |= (uint64_t)((addr >> 4) & 0x3FFFu);
  d |= (uint64_t)(128u >> 4) << 32;   // stride byte offset
  d |= (uint64_t)1u << 46;            // descriptor version 1
  return d;
}

// The products of a K block (four K = 32 steps, 32 bytes apart in both operands; the first adds to D when accumulate != 0,
// the others always), then an arrival on `bar` when they are done (kGroup 2: of both CTAs, mask: their ranks in the
// cluster).  Warp-level as in tc_ptx.cuh: all 32 lanes with uniform operands, one elected lane issues; one election for
// all five, since each costs about as much as an issue (a K block of 128 x 16, with the waits for it: 390 -> 310 cycles).
template <int kGroup>
__device__ __forceinline__ void mma_block_w(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t sa_tmem, uint32_t sb_tmem,
                                            uint32_t accumulate, uint64_t* bar, uint32_t mask) {
  if constexpr (kGroup == 1) {
    asm volatile(
        "{\n\t.reg .pred p, q, pe;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "setp.eq.u32 q, 0, 0;\n\t"
        "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
        "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
        "elect.sync _|pe, 0xffffffff;\n\t"
        "@pe tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t"
        "@pe tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a1, b1, %3, [%4], [%5], q;\n\t"
        "@pe tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a2, b2, %3, [%4], [%5], q;\n\t"
        "@pe tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a3, b3, %3, [%4], [%5], q;\n\t"
        "@pe tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%7];\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sa_tmem), "r"(sb_tmem), "r"(accumulate), "r"(tc::smem_u32(bar))
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p, q, pe;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t.reg .b16 m;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "setp.eq.u32 q, 0, 0;\n\t"
        "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
        "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
        "elect.sync _|pe, 0xffffffff;\n\t"
        "@pe tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t"
        "@pe tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a1, b1, %3, [%4], [%5], q;\n\t"
        "@pe tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a2, b2, %3, [%4], [%5], q;\n\t"
        "@pe tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a3, b3, %3, [%4], [%5], q;\n\t"
        "cvt.u16.u32 m, %8;\n\t"
        "@pe tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%7], m;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sa_tmem), "r"(sb_tmem), "r"(accumulate), "r"(tc::smem_u32(bar)), "r"(mask)
        : "memory");
  }
}

// 128 rows' scale words from shared memory to four TMEM columns; in order with the MMAs that the
// same thread issues after it.
template <int kGroup>
__device__ __forceinline__ void scales_to_tmem_w(uint32_t tmem, uint64_t desc) {
  if constexpr (kGroup == 1) {
    asm volatile(
        "{\n\t.reg .pred pe;\n\t"
        "elect.sync _|pe, 0xffffffff;\n\t"
        "@pe tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(tmem), "l"(desc)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred pe;\n\t"
        "elect.sync _|pe, 0xffffffff;\n\t"
        "@pe tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(tmem), "l"(desc)
        : "memory");
  }
}

// Wait of a warp whose next step brings it together again (an election): each lane asks and keeps its own answer.
// After a wait that ran out the next ones do not wait (`limit` is 0 then), so that the warp comes to its end.
__device__ __forceinline__ void wait_lane(uint64_t* bar, uint32_t parity, long long& limit) {
  if (!tc::mbar_wait(bar, parity, limit)) limit = 0;
}
// Wait of a whole warp; every lane asks (a branch for one lane costs some 500 cycles before the warp is together again).
__device__ __forceinline__ bool wait_w(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, kWaitLimit));
}

// A tile's load, and an arrival that expects its bytes, by the elected lane (kGroup 2: `bar` may be the other CTA's,
// an address of the cluster).
template <int kGroup>
__device__ __forceinline__ void tma_load_w(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, uint32_t bar) {
  if constexpr (kGroup == 1) {
    asm volatile(
        "{\n\t.reg .pred pe;\n\t"
        "elect.sync _|pe, 0xffffffff;\n\t"
        "@pe cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred pe;\n\t"
        "elect.sync _|pe, 0xffffffff;\n\t"
        "@pe cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
  }
}
__device__ __forceinline__ void expect_w(uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred pe;\n\t"
      "elect.sync _|pe, 0xffffffff;\n\t"
      "@pe mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
      "r"(bytes)
      : "memory");
}

// The CTAs of a cluster meet, with no order of memory (tc::cluster_sync_all's release costs up to 2,000 cycles while
// loads are on their way).
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// Arrival on an mbarrier of the cluster (address from mapa_shared), released at CTA scope: what it orders lies in
// this CTA's own shared memory (behind a proxy fence) or TMEM.  (A release at cluster scope costs about 1,000 cycles.)
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Arrive at this barrier of both CTAs (mask: their ranks in the cluster) once every MMA issued so far by the elected lane has completed.
__device__ __forceinline__ void commit_both_w(uint64_t* bar, uint32_t mask) {
  asm volatile(
      "{\n\t.reg .pred pe;\n\t.reg .b16 m;\n\t"
      "cvt.u16.u32 m, %1;\n\t"
      "elect.sync _|pe, 0xffffffff;\n\t"
      "@pe tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(tc::smem_u32(bar)),
      "r"(mask)
      : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::smem_u32(dst)), "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free_pair(uint32_t taddr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
}

constexpr int kScaleSlots = 4;   // groups of four K blocks whose scales are on their way (two of them in TMEM)

// Scale words of four K blocks, kb .. kb + 3 of `blocks` (bytes behind the last: 127, a factor 1), for kWords rows of a
// matrix's `size` scales: row(i) gives a row's number, negative for none (any word then).  No branch stands between the
// loads, so that all are on their way together, and nothing waits for them before word() takes them.  Rows of whole
// 32-bit words (`words`) take one load each.  Others take the two words around their four bytes (the same
// one twice where it holds all that are there), each with a byte of the row in it; and byte after byte where such a word reaches over
// the scales' ends.  (With bytes alone 4,813 x 1,920 x 10,304 took 66 us against 54, 331 x 2,688 x 4,992 12.1 against 9.5.)
constexpr uint32_t kOnes = 0x7f7f7f7fu;   // four factors of 1
template <int kWords>
struct Scales {
  uint32_t lo[kWords], hi[kWords], shift[kWords];
  uint32_t kept;   // the bytes of blocks that are there
  template <typename F>
  __device__ __forceinline__ void load(const uint8_t* scales, int64_t size, int32_t blocks, int32_t kb, bool words, F row) {
    const uint8_t* p[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const int64_t r = row(i);
      p[i] = scales + (r < 0 ? 0 : r) * blocks + kb;
      hi[i] = shift[i] = 0;   // (a copy of lo would wait for it)
    }
    const int n = min(blocks - kb, 4);
    kept = 0xffffffffu >> (32 - 8 * n);
    if (words) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) lo[i] = __ldcg(reinterpret_cast<const uint32_t*>(p[i]));
      return;
    }
    const uintptr_t from = reinterpret_cast<uintptr_t>(scales), to = from + size;
    uintptr_t a[kWords], b[kWords];
    bool inside = true;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      a[i] = reinterpret_cast<uintptr_t>(p[i]) & ~(uintptr_t)3, b[i] = (reinterpret_cast<uintptr_t>(p[i]) + n - 1) & ~(uintptr_t)3;
      inside = inside && a[i] >= from && b[i] + 4 <= to;
    }
    if (__all_sync(0xffffffffu, inside)) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        lo[i] = __ldcg(reinterpret_cast<const uint32_t*>(a[i]));
        hi[i] = __ldcg(reinterpret_cast<const uint32_t*>(b[i]));
        shift[i] = 8 * (uint32_t)(reinterpret_cast<uintptr_t>(p[i]) & 3);
      }
    } else {
      uint32_t c[kWords][4];
#pragma unroll
      for (int i = 0; i < kWords; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) c[i][j] = __ldcg(p[i] + min(j, n - 1));
#pragma unroll
      for (int i = 0; i < kWords; ++i) lo[i] = c[i][0] | c[i][1] << 8 | c[i][2] << 16 | c[i][3] << 24;
    }
  }
  __device__ __forceinline__ uint32_t word(int i) const { return (__funnelshift_r(lo[i], hi[i], shift[i]) & kept) | (kOnes & ~kept); }
};
inline bool scale_words(const void* a, const void* b, int64_t blocks) {
  return blocks % 4 == 0 && reinterpret_cast<uintptr_t>(a) % 4 == 0 && reinterpret_cast<uintptr_t>(b) % 4 == 0;
}

// ------------------------------------------------------------------------------ host
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encode() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// Boxes of 128 bytes of K (zeros behind K) by box_rows rows (zeros behind the last), 128-byte swizzle.  L2 takes 256 bytes
// at a time of rows that begin on 128-byte boundaries (128: 1 x 16,416 x 4,096 13.8 us against 13.6), else 128 (331 x 2,688 x
// 4,976 13.5 us against 14.7).
inline bool codes_map(CUtensorMap* m, const uint8_t* base, int64_t rows, int64_t K, int64_t stride, int box_rows) {
  const auto fn = tensor_map_encode();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)stride};
  const cuuint32_t box[2] = {kStageK, (cuuint32_t)box_rows};
  const cuuint32_t es[2] = {1, 1};
  const bool lines = stride % 128 == 0 && reinterpret_cast<uintptr_t>(base) % 128 == 0;
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, lines ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Boxes of box_cols x box_rows of an output of elements of eb bytes, for stores.
inline bool out_map(CUtensorMap* m, void* base, int64_t rows, int64_t cols, int64_t stride, size_t eb, int box_cols, int box_rows) {
  const auto fn = tensor_map_encode();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)stride * eb};
  const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
  const cuuint32_t es[2] = {1, 1};
  return fn(m, eb == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, base, dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace dense
}  // namespace kda
