// The product of 8-bit matrices for many rows of A (prompts).
//
//   out[m][n] = sum_k A[m][k] W[n][k]
//
// Bound: the tensor core.  Two CTAs of a cluster make one tile of 256 x 240 (cta_group::2: each holds half the
// rows of A and half the columns' weights, so that a byte of shared memory serves twice the products
// of a single CTA's tile).  240 columns, not 256, because the 512 columns of TMEM hold two accumulators, the one being
// filled and the one being stored, and the scales.  Persistent: a pair takes tile after tile, and loads, products and
// stores of neighbouring tiles overlap.
//
// Measured: 8,192 x 16,416 x 4,096 276 us of small whole numbers (4.0 PFLOP/s, 2.07 times the measured bf16 rate),
// 306 us of normally distributed values in single graphs and 361 in long runs, where the power limit holds the clock at
// 1.39 GHz; the tensor pipe is active 91 % of the cycles.  16,384 x 16,384 x 8,192 1.09 ms (4.0 PFLOP/s).
// 8,192 x 16,416 x 512 57 us: its output alone takes 41; with fp32 outputs 101 us (80), x 4,096 300 us.  Slower: five stages of six (298 us against 283, with
// eight storing warps); parts of K in clusters of four and six CTAs for few tiles (256 x 4,096 x 12,288: 21.7 us against the
// other kernel's 20.9); barriers arrived at with a release at cluster scope, 1,000 cycles each (780 us).  An output whose rows
// are not on 16-byte boundaries takes element stores: 8,192 x 16,417 x 512 106 us (by aligned windows of 64 bytes, more
// instructions each, 143).
//
// Warps of a CTA: 0 loads tiles, 1 issues products (of the leading CTA alone), 2 and 3 load scales, a group of four K
// blocks each in turn (of rows that are not whole words one warp's loads take longer than a group's products: 4,813 x
// 1,920 x 10,304 62 us with one, 54 with two), 4 to 7 store.
#include <limits.h>

#include <algorithm>

#include "internal.cuh"
#include "mma8.cuh"

namespace kda {
namespace dense {
namespace {

constexpr int kTM = 256, kTN = 240, kThreads = 256, kStages = 6;
constexpr uint32_t kA = 128 * kStageK, kB = kTN / 2 * kStageK, kStage = kA + kB;
constexpr uint32_t kScales = 3 * 512;   // one slot: 128 rows of A, twice 128 of W
constexpr uint32_t oScales = kStages * kStage, oOut = oScales + kScaleSlots * kScales;
// Per storing warp two pieces of 32 rows by 96 bytes of the output; or 32 rows of 32 sums (33 words apart).
constexpr uint32_t kPiece = 32 * 96, kTurnRow = 33;
constexpr uint32_t oBars = oOut + 4 * 2 * kPiece;
constexpr int kBars = 2 * kStages + 2 * kScaleSlots + 4;
constexpr uint32_t kAlloc = oBars + kBars * 8 + 8 + 1024;
constexpr uint32_t cScales = 2 * kTN;   // TMEM columns: two accumulators, two slots of scales
constexpr int kGroupM = 8;              // tiles are taken in bands of so many rows of tiles
static_assert(kAlloc <= 227 * 1024 && 32 * kTurnRow * 4 <= 2 * kPiece && oOut % 128 == 0, "shared memory");

// 8 columns of TMEM, not there before tmem_ld_end has waited for them.
__device__ __forceinline__ void tmem_ld8_begin(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
// The registers pass through the wait, so that nothing uses them before it.
template <int N>
__device__ __forceinline__ void tmem_ld_end(uint32_t (&r)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i])::"memory");
}
// Store of a piece by the elected lane, as a bulk group of its own; and a wait until at most kLeft of them still read shared memory.
__device__ __forceinline__ void tma_store_w(const CUtensorMap* map, int32_t x, int32_t y, uint32_t src) {
  asm volatile(
      "{\n\t.reg .pred pe;\n\t"
      "elect.sync _|pe, 0xffffffff;\n\t"
      "@pe cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];\n\t"
      "@pe cp.async.bulk.commit_group;\n\t}" ::"l"(reinterpret_cast<uint64_t>(map)),
      "r"(x), "r"(y), "r"(src)
      : "memory");
}
template <int kLeft>
__device__ __forceinline__ void stores_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kLeft) : "memory");
}

// Tile t of tm x tn: bands of kGroupM rows of tiles, column after column inside a band, so that the tiles in
// flight share both their rows of A and their weights in L2.
__device__ __forceinline__ void place(uint32_t t, uint32_t tm, uint32_t tn, uint32_t& im, uint32_t& in) {
  const uint32_t band = t / (kGroupM * tn), first = band * kGroupM, rows = min(tm - first, (uint32_t)kGroupM);
  const uint32_t rest = t - band * kGroupM * tn;
  in = rest / rows;
  im = first + rest - in * rows;
}

template <typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    fp8_matmul_pair_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB, const __grid_constant__ CUtensorMap mapO,
                           const uint8_t* sa, const uint8_t* sw, int64_t M, int64_t N, int32_t blocks, uint32_t tm, uint32_t tn, T* out, int64_t ldo,
                           int32_t wide, int32_t words, int32_t* dev_err) {
  extern __shared__ uint8_t raw[];
  uint8_t* sm = raw + ((1024u - (tc::smem_u32(raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + oBars);        // of the leading CTA: both CTAs' tiles are there
  uint64_t* empty = full + kStages;                                // of both: the stage has been used
  uint64_t *sfull = empty + kStages, *sempty = sfull + kScaleSlots;          // the same of the scales' slots
  uint64_t *tfull = sempty + kScaleSlots, *tempty = tfull + 2;               // accumulators: filled (both), stored (the leading CTA's)
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(tempty + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = tc::cluster_ctarank();
  const uint32_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1, tiles = tm * tn;
  const int groups = (blocks + 3) / 4;   // of four K blocks: a word of scales

  // Before the cluster meets: the first scales are read, and the leading CTA's own first loads go out.
  const uint32_t at = tc::smem_u32(sm), lead = tc::mapa_shared(full, 0);
  Scales<4> wa;
  Scales<8> wb;
  int left_a = 0, left_b = 0;   // rows of A, and of W, from this lane's first one on
  auto load_words = [&](uint32_t t, int gg) {   // of group gg of tile t
    uint32_t im, in;
    place(t, tm, tn, im, in);
    left_a = (int)min(M - (int64_t)im * kTM - 128 * rank - lane, (int64_t)128);
    left_b = (int)min(N - (int64_t)in * kTN - lane, (int64_t)256);
    wa.load(sa, M * blocks, blocks, 4 * gg, words, [&](int i) {
      const int64_t m = (int64_t)im * kTM + 128 * rank + 32 * i + lane;
      return m < M ? m : -1;
    });
    wb.load(sw, (N + kBlock - 1) / kBlock * blocks, blocks, 4 * gg, words, [&](int i) {
      const int64_t c = (int64_t)in * kTN + 32 * i + lane;
      return c < N ? c / kBlock : -1;
    });
  };
  auto load_tile = [&](int32_t kb, int st, int32_t ya, int32_t yb) {
    // the leading CTA expects both CTAs' bytes; the other's may come first, its arrival is what ends the phase
    if (rank == 0) expect_w(tc::smem_u32(full + st), 2 * kStage);
    tma_load_w<2>(at + st * kStage, &mapA, kb * kStageK, ya, lead + 8 * st);
    tma_load_w<2>(at + st * kStage + kA, &mapB, kb * kStageK, yb, lead + 8 * st);
  };
  const int early = rank == 0 ? min(blocks, kStages) : 0;   // of the first tile
  if (warp == 0) {
    if (lane < kBars) {   // in the order of their declaration: full, empty, sfull, sempty, tfull, tempty
      const int i = lane - 2 * kStages - kScaleSlots;
      tc::mbar_init(full + lane, i < -kScaleSlots ? 1 : i < 0 ? 2 : i < kScaleSlots + 2 ? 1 : 8);
    }
    tc::fence_mbar_init();
    tc::tma_prefetch_desc(&mapA);
    tc::tma_prefetch_desc(&mapB);
    __syncwarp();
  } else if (warp == 3) {
    tmem_alloc_pair(tmem_at, 512);
    let_next_start();   // not before: see there
  }
  wait_for_previous();
  if (warp == 0 && early > 0) {
    uint32_t im, in;
    place(pair, tm, tn, im, in);
    for (int kb = 0; kb < early; ++kb) load_tile(kb, kb, (int32_t)(im * kTM), (int32_t)(in * kTN));
  } else if (warp == 2 || warp == 3) {
    if (warp == 2 || groups > 1) load_words(pair, warp - 2);
    else if (pair + pairs < tiles) load_words(pair + pairs, 0);
  }
  tc::tc_fence_before();
  __syncthreads();
  cluster_meet();   // (the barriers' initialisation is released by its own fence)
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_at;
  bool ok = true;

  if (warp == 0) {
    int st = 0;
    uint32_t phase = 1;
    int64_t n = 0;   // stages so far
    for (uint32_t t = pair; t < tiles && ok; t += pairs) {
      uint32_t im, in;
      place(t, tm, tn, im, in);
      const int32_t ya = (int32_t)(im * kTM + 128 * rank), yb = (int32_t)(in * kTN + kTN / 2 * rank);
      for (int32_t kb = 0; kb < blocks; ++kb, ++n) {
        if (n >= kStages && !(ok = wait_w(empty + st, phase))) break;
        if (n >= early) load_tile(kb, st, ya, yb);
        if (++st == kStages) st = 0, phase ^= 1;
      }
    }
    // end with no copy and no arrival in flight
    for (int64_t i = n > kStages ? n - kStages : 0; i < n; ++i) ok = wait_w(empty + i % kStages, (uint32_t)(i / kStages) & 1) && ok;
  } else if (warp == 1) {
    if (rank == 0) {
      const uint64_t dA = tc::desc_kmajor_sw128(tc::smem_u32(sm)), dB = tc::desc_kmajor_sw128(tc::smem_u32(sm + kA));
      const uint64_t dS = desc_scales(tc::smem_u32(sm + oScales));
      int st = 0, it = 0;
      uint32_t phase = 0, g = 0;
      long long limit = kWaitLimit;
      for (uint32_t t = pair; t < tiles; t += pairs, ++it) {
        const uint32_t acc = tmem + (it & 1) * kTN;
        if (it >= 2) wait_lane(tempty + (it & 1), ((it >> 1) - 1) & 1, limit);
        for (int32_t k0 = 0; k0 < blocks; k0 += 4, ++g) {   // four K blocks, a word of scales
          const uint32_t slot = g % kScaleSlots, ca = tmem + cScales + (g & 1) * 12, cb = ca + 4;
          // the products that read these columns, two groups ago, are done
          if (g >= 2) wait_lane(sempty + (g - 2) % kScaleSlots, ((g - 2) / kScaleSlots) & 1, limit);
          wait_lane(sfull + slot, (g / kScaleSlots) & 1, limit);
          tc::tc_fence_after();
#pragma unroll
          for (int s = 0; s < 3; ++s) scales_to_tmem_w<2>(ca + 4 * s, dS + ((slot * kScales + 512 * s) >> 4));
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            if (k0 + b >= blocks) break;
            wait_lane(full + st, phase, limit);
            tc::tc_fence_after();
            mma_block_w<2>(acc, dA + (st * kStage >> 4), dB + (st * kStage >> 4), idesc_e4m3(kTM, kTN) | scale_ids(b), ca, cb,
                           b > 0 ? 1u : (uint32_t)k0, empty + st, 3u);
            if (++st == kStages) st = 0, phase ^= 1;
          }
          commit_both_w(sempty + slot, 3u);
        }
        commit_both_w(tfull + (it & 1), 3u);
      }
      ok = __all_sync(0xffffffffu, limit != 0);
      for (int i = it > 2 ? it - 2 : 0; i < it; ++i) ok = wait_w(tempty + (i & 1), (i >> 1) & 1) && ok;
    }
  } else if (warp < 4) {
    const uint32_t first = warp - 2;
    uint32_t g = first, t = pair;
    int gg = (int)first;
    if (gg == groups) gg = 0, t += pairs;
    while (t < tiles) {
      const uint32_t slot = g % kScaleSlots;
      if (g >= kScaleSlots && !(ok = wait_w(sempty + slot, (g / kScaleSlots - 1) & 1))) break;
      uint4* to = reinterpret_cast<uint4*>(sm + oScales + slot * kScales) + lane;
      const auto a_word = [&](int i) { return 32 * i < left_a ? wa.word(i) : kOnes; };   // rows behind the last: a factor 1
      const auto b_word = [&](int i) { return 32 * i < left_b ? wb.word(i) : kOnes; };
      to[0] = make_uint4(a_word(0), a_word(1), a_word(2), a_word(3));
      to[32] = make_uint4(b_word(0), b_word(1), b_word(2), b_word(3));
      to[64] = make_uint4(b_word(4), b_word(5), b_word(6), b_word(7));
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) arrive_cluster(tc::mapa_shared(sfull + slot, 0));
      for (int i = 0; i < 2; ++i)
        if (++gg == groups) gg = 0, t += pairs;
      if (t < tiles) load_words(t, gg);
      g += 2;
    }
    for (uint32_t i = 2; i <= kScaleSlots && g >= first + i; i += 2) ok = wait_w(sempty + (g - i) % kScaleSlots, ((g - i) / kScaleSlots) & 1) && ok;
  } else {
    const int q = warp - 4;
    uint8_t* mine = sm + oOut + q * 2 * kPiece;
    constexpr int kCols = 96 / sizeof(T);   // of a piece
    uint32_t piece = 0;
    int it = 0;
    for (uint32_t t = pair; t < tiles; t += pairs, ++it) {
      uint32_t im, in;
      place(t, tm, tn, im, in);
      if (!(ok = wait_w(tfull + (it & 1), (it >> 1) & 1))) break;
      tc::tc_fence_after();
      const uint32_t acc = tc::tmem_addr(tmem, 32 * q, (it & 1) * kTN);
      const int64_t m0 = (int64_t)im * kTM + 128 * rank + 32 * q, n0 = (int64_t)in * kTN;
      const int rows = (int)(M - m0 < 32 ? M - m0 : 32), cols = (int)(N - n0 < kTN ? N - n0 : kTN);
      auto freed = [&]() {   // the accumulator has been read
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(tc::mapa_shared(tempty + (it & 1), 0));
      };
      if (rows <= 0) {
        freed();
      } else if (wide) {
#pragma unroll 1
        for (int c = 0; c < cols; c += kCols, piece ^= 1) {   // a store for each, so that the last but one had this place
          uint32_t v[kCols];
#pragma unroll
          for (int i = 0; i < kCols; i += 8) tmem_ld8_begin(acc + c + i, v + i);
          stores_read<1>();   // that one has been read (a lane without stores does not wait)
          tmem_ld_end(v);
          if (c + kCols >= cols) freed();
          __syncwarp();
          uint4* to = reinterpret_cast<uint4*>(mine + piece * kPiece + 96 * lane);
#pragma unroll
          for (int i = 0; i < 6; ++i) {
            if constexpr (sizeof(T) == 2) {
              const float* f = reinterpret_cast<const float*>(v + 8 * i);
              to[i] = make_uint4(bf16x2(f[0], f[1]), bf16x2(f[2], f[3]), bf16x2(f[4], f[5]), bf16x2(f[6], f[7]));
            } else {
              to[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            }
          }
          tc::fence_proxy_async_smem();
          __syncwarp();
          tma_store_w(&mapO, (int32_t)n0 + c, (int32_t)m0, tc::smem_u32(mine + piece * kPiece));
        }
      } else {   // through shared memory: a row's columns next to one another
        float* turn = reinterpret_cast<float*>(mine);
#pragma unroll 1
        for (int c = 0; c < cols; c += 32) {   // (the last 32 of 240 reach into the next columns of TMEM: not stored)
          uint32_t v[32];
#pragma unroll
          for (int i = 0; i < 32; i += 8) tmem_ld8_begin(acc + c + i, v + i);
          tmem_ld_end(v);
          if (c + 32 >= cols) freed();
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 32; ++i) turn[lane * kTurnRow + i] = __uint_as_float(v[i]);
          __syncwarp();
          if (c + lane < cols) {
            T* o = out + m0 * ldo + n0 + c + lane;
            if (rows == 32) {
#pragma unroll
              for (int r = 0; r < 32; ++r, o += ldo) *o = from_f32<T>(turn[r * kTurnRow + lane]);
            } else {
#pragma unroll 4
              for (int r = 0; r < rows; ++r, o += ldo) *o = from_f32<T>(turn[r * kTurnRow + lane]);
            }
          }
        }
      }
    }
    stores_read<0>();
  }
  if (!__all_sync(0xffffffffu, ok) && lane == 0) atomicExch(dev_err, (int32_t)kDevErrTimeout);
  tc::tc_fence_before();
  __syncthreads();
  cluster_meet();   // both CTAs are done with one another's barriers and TMEM
  tc::tc_fence_after();
  if (warp == 3) tmem_free_pair(tmem, 512);
}

template <typename T>
cudaError_t launch(const MatmulProblem& p, int sms, cudaStream_t stream) {
  CUtensorMap ma, mb, mo;
  if (!codes_map(&ma, p.a, p.M, p.K, p.lda, 128) || !codes_map(&mb, p.w, p.N, p.K, p.ldw, kTN / 2)) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(fp8_matmul_pair_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kAlloc);
  if (e != cudaSuccess) return e;
  const int32_t blocks = (int32_t)((p.K + kStageK - 1) / kStageK);
  const int64_t tm = (p.M + kTM - 1) / kTM, tn = (p.N + kTN - 1) / kTN;
  // rows that begin on 16-byte boundaries leave by tensor stores
  const bool wide = reinterpret_cast<uintptr_t>(p.out) % 16 == 0 && (size_t)p.ldo * sizeof(T) % 16 == 0;
  if (!wide) mo = ma;
  else if (!out_map(&mo, p.out, p.M, p.N, p.ldo, sizeof(T), 96 / sizeof(T), 32)) return cudaErrorInvalidValue;
  if (tm * tn > INT32_MAX) return cudaErrorInvalidValue;   // (2^44 products of a K: no memory holds them)
  const unsigned grid = 2 * (unsigned)std::min<int64_t>(tm * tn, sms / 2);
  prof_begin(stream, "fp8_matmul_pair_kernel");
  e = launch_kernel(fp8_matmul_pair_kernel<T>, dim3(grid), kThreads, kAlloc, 0, stream, ma, mb, mo, p.sa, p.sw, p.M, p.N, blocks, tm, tn,
                    static_cast<T*>(p.out), p.ldo, wide, scale_words(p.sa, p.sw, blocks), p.dev_err);
  prof_end(stream);
  return e;
}

}  // namespace

cudaError_t launch_matmul_pair(const MatmulProblem& p, int sms, cudaStream_t stream) {
  return p.dt == KDA_F32 ? launch<float>(p, sms, stream) : launch<__nv_bfloat16>(p, sms, stream);
}

}  // namespace dense
}  // namespace kda
