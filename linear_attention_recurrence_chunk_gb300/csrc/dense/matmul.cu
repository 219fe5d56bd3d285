// The product of 8-bit matrices for few rows of A (decode steps).
//
//   out[m][n] = sum_k A[m][k] W[n][k]
//
// Bound: the weights' bytes from HBM.  So the weights are the 128-row operand of the tensor core and
// the tokens (kRows of them, 16 to 256) its columns: no row of the instruction is padding however
// few tokens there are.  A cluster of CTAs splits K of one tile, so that few tiles still
// fill the chip; each sends the others the sums that they join, through distributed shared memory, and adds its own
// share in a fixed order, with no scratch memory and one launch.
// Measured (replayed from a graph): 1 x 16,416 x 4,096 13.0 us (the bytes' floor 9.9; DRAM is busy 56 % of it, the first
// bytes come after 3 us), 8 x 2,052 x 512 2.4 us, 64 x 4,096 x 12,288 12.4 us (7.6), 256 x 4,096 x 12,288 16.7 us (8.2: a
// K block takes some 400 cycles, 256 of them products, and the join 2 us); with fp32 outputs as long.  In a loop of K blocks the issue counts
// as much as the products: see mma_block_w and wait_lane.  Not faster: pairs of CTAs on 256 rows of W (256 x
// 4,096 x 12,288 18.4 us against 18.5), eight-CTA clusters beyond 15 of them (two waves).  Joining by loads from the other
// CTAs took 14.9 us for 128 x 4,096 x 12,288, stores to them 13.4; stores of four tokens of a weight, whose
// lanes lie apart, 17.2; a CTA's own share stored by its own address 14.0.
#include <float.h>
#include <limits.h>

#include <algorithm>

#include "internal.cuh"
#include "mma8.cuh"

namespace kda {
namespace dense {
namespace {

constexpr int kThreads = 128;   // warp 0 loads tiles, 1 issues products, 2 and 3 load scales in turn; all store

// kDeep: one CTA an SM with all of its shared memory, else two.  (256 tokens: one.)
template <int kRows, bool kDeep>
struct Few {
  static constexpr int kStages = kRows == 16    ? (kDeep ? 11 : 5)
                                 : kRows == 32  ? (kDeep ? 10 : 5)
                                 : kRows == 64  ? (kDeep ? 8 : 4)
                                 : kRows == 128 ? (kDeep ? 6 : 3)
                                                : 4;
  static constexpr uint32_t kW = 128 * kStageK, kX = kRows * kStageK, kStage = kW + kX;
  static constexpr int kSets = (kRows + 127) / 128;               // of 128 tokens' scales
  static constexpr uint32_t kScales = 512 * (1 + kSets);          // one slot: weights', tokens'
  static constexpr uint32_t oScales = kStages * kStage, oBars = oScales + kScaleSlots * kScales;
  static constexpr int kBars = 2 * kStages + 2 * kScaleSlots + 1;   // at most 32: a lane initialises one each
  static constexpr uint32_t kBytes = oBars + kBars * 8 + 8, kAlloc = kBytes + 1024;   // + alignment
  static constexpr uint32_t cScales = kRows, kCols = kRows + 2 * 4 * (1 + kSets);      // TMEM columns
  static constexpr uint32_t kTmem = kCols <= 32 ? 32 : kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
  static_assert(kStages * kStage >= kRows * 512 && kBars <= 32 && kAlloc <= 227 * 1024, "shared memory; partial sums take the stages' place");
};

__device__ __forceinline__ void st_cluster(uint32_t addr, float x) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(x) : "memory");
}

__device__ __forceinline__ uint32_t cluster_address(uint32_t shared, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(shared), "r"(rank));
  return r;
}

template <int kRows, bool kDeep, typename T>
__global__ void __launch_bounds__(kThreads)
    fp8_matmul_few_kernel(const __grid_constant__ CUtensorMap mapW, const __grid_constant__ CUtensorMap mapX, const uint8_t* sw,
                          const uint8_t* sx, int64_t M, int64_t N, int32_t blocks, T* out, int64_t ldo, int32_t quads,
                          int32_t words, int32_t split, int32_t* dev_err) {
  using F = Few<kRows, kDeep>;
  extern __shared__ uint8_t raw[];
  uint8_t* sm = raw + ((1024u - (tc::smem_u32(raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + F::oBars);
  uint64_t *empty = full + F::kStages, *sfull = empty + F::kStages, *sempty = sfull + kScaleSlots, *done = sempty + kScaleSlots;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(done + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t tile = blockIdx.x / split, part = blockIdx.x - tile * split;   // a cluster a tile, a CTA a part of K
  const int64_t n0 = (int64_t)tile * 128, m0 = (int64_t)blockIdx.y * kRows;
  // this part's K blocks: whole groups of four, whose scales share a word
  const int32_t groups = (blocks + 3) / 4, kb0 = (int32_t)((int64_t)groups * part / split) * 4;
  const int32_t nb = (int32_t)min((int64_t)groups * (part + 1) / split * 4, (int64_t)blocks) - kb0;

  // Before the CTA meets: the first loads go out, and the first scales are read.
  const uint32_t at = tc::smem_u32(sm), bar = tc::smem_u32(full);
  const int first = min(nb, F::kStages);
  Scales<1> ww;
  Scales<4 * F::kSets> wx;
  auto load_tile = [&](int i, int st) {
    expect_w(bar + 8 * st, F::kStage);
    tma_load_w<1>(at + st * F::kStage, &mapW, (kb0 + i) * kStageK, (int32_t)n0, bar + 8 * st);
    tma_load_w<1>(at + st * F::kStage + F::kW, &mapX, (kb0 + i) * kStageK, (int32_t)m0, bar + 8 * st);
  };
  auto load_words = [&](int g) {
    ww.load(sw, (N + 127) / 128 * blocks, blocks, kb0 + 4 * g, words, [&](int) { return (int64_t)tile; });
    wx.load(sx, M * blocks, blocks, kb0 + 4 * g, words, [&](int i) {
      const int r = 32 * i + lane;
      return r < kRows && m0 + r < M ? m0 + r : (int64_t)-1;
    });
  };
  if (warp == 0) {
    if (lane < F::kBars) tc::mbar_init(full + lane, 1);
    tc::fence_mbar_init();
    tc::tma_prefetch_desc(&mapW);
    tc::tma_prefetch_desc(&mapX);
    __syncwarp();
  } else if (warp == 1) {
    tc::tmem_alloc(tmem_at, F::kTmem);
    tc::tmem_relinquish();
    let_next_start();   // not before: see there
  }
  wait_for_previous();
  if (warp == 0) {
    for (int i = 0; i < first; ++i) load_tile(i, i);
  } else if (warp >= 2 && 4 * (warp - 2) < nb) {
    load_words(warp - 2);
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_at;
  bool ok = true;

  if (warp == 0) {
    int st = 0, i = first;
    uint32_t phase = 0;
    for (; i < nb; ++i) {
      if (!(ok = wait_w(empty + st, phase))) break;
      load_tile(i, st);
      if (++st == F::kStages) st = 0, phase ^= 1;
    }
    if (!ok)   // end with no copy in flight
      for (int j = max(0, i - F::kStages); j < i; ++j) wait_w(full + j % F::kStages, (j / F::kStages) & 1);
  } else if (warp == 1) {
    const uint64_t dW = tc::desc_kmajor_sw128(tc::smem_u32(sm)), dX = tc::desc_kmajor_sw128(tc::smem_u32(sm + F::kW));
    const uint64_t dS = desc_scales(tc::smem_u32(sm + F::oScales));
    int st = 0;
    uint32_t phase = 0, cw = tmem + F::cScales;
    long long limit = kWaitLimit;
    for (int i = 0, g = 0; i < nb; i += 4, ++g) {   // four K blocks, a word of scales
      const int slot = g % kScaleSlots;
      // the products that read these columns, two groups ago, are done
      if (g >= 2) wait_lane(sempty + (g - 2) % kScaleSlots, ((g - 2) / kScaleSlots) & 1, limit);
      wait_lane(sfull + slot, (g / kScaleSlots) & 1, limit);
      tc::tc_fence_after();
#pragma unroll
      for (int s = 0; s < 1 + F::kSets; ++s) scales_to_tmem_w<1>(cw + 4 * s, dS + ((slot * F::kScales + 512 * s) >> 4));
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        if (i + b >= nb) break;
        wait_lane(full + st, phase, limit);
        tc::tc_fence_after();
        mma_block_w<1>(tmem, dW + (st * F::kStage >> 4), dX + (st * F::kStage >> 4), idesc_e4m3(128, kRows) | scale_ids(b), cw,
                               cw + 4, b > 0 ? 1u : (uint32_t)i, empty + st, 0);
        if (++st == F::kStages) st = 0, phase ^= 1;
      }
      tc::mma_commit_w(sempty + slot);
      cw = tmem + F::cScales + ((g + 1) & 1) * 4 * (1 + F::kSets);
    }
    ok = __all_sync(0xffffffffu, limit != 0);
    tc::mma_commit_w(done);
  } else {
    for (int g = warp - 2; 4 * g < nb; g += 2) {
      const int slot = g % kScaleSlots;
      if (g >= kScaleSlots) ok = wait_w(sempty + slot, (g / kScaleSlots - 1) & 1);
      if (!ok) break;
      uint4* to = reinterpret_cast<uint4*>(sm + F::oScales + slot * F::kScales) + lane;
      const uint32_t w = ww.word(0);
      to[0] = make_uint4(w, w, w, w);
      uint32_t x[4 * F::kSets];
#pragma unroll
      for (int i = 0; i < 4 * F::kSets; ++i) x[i] = 32 * i + lane < min((int64_t)kRows, M - m0) ? wx.word(i) : kOnes;
#pragma unroll
      for (int s = 0; s < F::kSets; ++s) to[32 * (1 + s)] = make_uint4(x[4 * s], x[4 * s + 1], x[4 * s + 2], x[4 * s + 3]);
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(sfull + slot);
      if (4 * (g + 2) < nb) load_words(g + 2);
    }
  }
  // every product done: the sums are in TMEM, and nothing reads or writes the stages any more
  ok = wait_w(done, 0) && ok;
  ok = __syncthreads_and(ok);
  tc::tc_fence_after();
  if (!ok && threadIdx.x == 0) atomicExch(dev_err, (int32_t)kDevErrTimeout);

  const int64_t n = n0 + threadIdx.x;
  const uint32_t td = tc::tmem_addr(tmem, 32 * warp, 0);
  const int rows = (int)(M - m0 < kRows ? M - m0 : kRows);
  T* o = out + m0 * ldo + n;
  if (split == 1) {
    if (ok) {
#pragma unroll 1
      for (int c = 0; c < rows; c += 16) {
        float v[16];
        tc::tmem_ld16(td + c, v);
        if (n < N) {
          if (c + 16 <= rows) {   // (a branch for each value costs 50 cycles)
#pragma unroll
            for (int e = 0; e < 16; ++e, o += ldo) *o = from_f32<T>(v[e]);
          } else {
#pragma unroll
            for (int e = 0; e < 15; ++e, o += ldo)
              if (c + e < rows) *o = from_f32<T>(v[e]);
          }
        }
      }
    }
  } else {
    // This CTA joins the tile's tokens part, part + split, ...: the others send it their sums of these, a token's 32 weights
    // of a warp side by side, to [part][token / split][128].
    const int R = kRows / split, down = __ffs(split) - 1;
    const uint32_t to = at + (part * R * 128 + threadIdx.x) * 4;
    cluster_meet();   // all products of the cluster are done: the sums take the stages' place
    if (ok) {
#pragma unroll 1
      for (int c = 0; c < rows; c += 16) {
        float v[16];
        tc::tmem_ld16(td + c, v);
#pragma unroll
        for (int e = 0; e < 16; ++e) st_cluster(cluster_address(to, e & (split - 1)) + ((c + e) >> down) * 512, v[e]);
      }
    }
    tc::cluster_sync_all();
    if (ok) {
      // a warp takes eight tokens at a time, a lane four columns of each
      constexpr int kAt = kRows < 64 ? 4 : 8;
      const int64_t nl = n0 + 4 * lane;
      const int left = (int)(N - nl < 4 ? N - nl : 4);   // columns of this lane
      const float4* sums = reinterpret_cast<const float4*>(sm) + lane;
      for (int i0 = kAt * warp; part + split * i0 < rows; i0 += kAt * (kThreads / 32)) {
        float4 x[kAt];
#pragma unroll
        for (int j = 0; j < kAt; ++j) x[j] = sums[min(i0 + j, R - 1) * 32];
#pragma unroll 1
        for (int s = 1; s < split; ++s) {   // in the order of K
          float4 y[kAt];
#pragma unroll
          for (int j = 0; j < kAt; ++j) y[j] = sums[(s * R + min(i0 + j, R - 1)) * 32];
#pragma unroll
          for (int j = 0; j < kAt; ++j) x[j].x += y[j].x, x[j].y += y[j].y, x[j].z += y[j].z, x[j].w += y[j].w;
        }
        T* y = out + (m0 + part + split * i0) * ldo + nl;
#pragma unroll
        for (int j = 0; j < kAt; ++j, y += split * ldo) {
          if (part + split * (i0 + j) >= rows) break;
          if (quads && left == 4) {
            if constexpr (sizeof(T) == 2) *reinterpret_cast<uint2*>(y) = make_uint2(bf16x2(x[j].x, x[j].y), bf16x2(x[j].z, x[j].w));
            else *reinterpret_cast<float4*>(y) = x[j];
          } else {
            if (left > 0) y[0] = from_f32<T>(x[j].x);
            if (left > 1) y[1] = from_f32<T>(x[j].y);
            if (left > 2) y[2] = from_f32<T>(x[j].z);
            if (left > 3) y[3] = from_f32<T>(x[j].w);
          }
        }
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) tc::tmem_dealloc(tmem, F::kTmem);
}

template <int kRows, bool kDeep, typename T>
cudaError_t launch_few(const MatmulProblem& p, int split, cudaStream_t stream) {
  using F = Few<kRows, kDeep>;
  CUtensorMap mw, mx;
  if (!codes_map(&mw, p.w, p.N, p.K, p.ldw, 128) || !codes_map(&mx, p.a, p.M, p.K, p.lda, kRows)) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(fp8_matmul_few_kernel<kRows, kDeep, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)F::kAlloc);
  if (e != cudaSuccess) return e;
  const int32_t blocks = (int32_t)((p.K + kStageK - 1) / kStageK);
  const bool quads = reinterpret_cast<uintptr_t>(p.out) % (4 * sizeof(T)) == 0 && p.ldo % 4 == 0;   // four columns a store
  prof_begin(stream, "fp8_matmul_few_kernel");
  e = launch_kernel(fp8_matmul_few_kernel<kRows, kDeep, T>,
                    dim3((unsigned)((p.N + 127) / 128 * split), (unsigned)((p.M + kRows - 1) / kRows)), kThreads, F::kAlloc, split, stream, mw, mx,
                    p.sw, p.sa, p.M, p.N, blocks, static_cast<T*>(p.out), p.ldo, quads, scale_words(p.sa, p.sw, blocks), split, p.dev_err);
  prof_end(stream);
  return e;
}

template <typename T>
cudaError_t launch(const MatmulProblem& p, const Cut& c, cudaStream_t stream) {
  switch (c.rows) {
    case 16: return c.deep ? launch_few<16, true, T>(p, c.split, stream) : launch_few<16, false, T>(p, c.split, stream);
    case 32: return c.deep ? launch_few<32, true, T>(p, c.split, stream) : launch_few<32, false, T>(p, c.split, stream);
    case 64: return c.deep ? launch_few<64, true, T>(p, c.split, stream) : launch_few<64, false, T>(p, c.split, stream);
    case 128: return c.deep ? launch_few<128, true, T>(p, c.split, stream) : launch_few<128, false, T>(p, c.split, stream);
    default: return launch_few<256, true, T>(p, c.split, stream);
  }
}

}  // namespace

bool cut_fits(const MatmulProblem& p, const Cut& c) {
  if (c.rows == 0) return true;
  const int64_t mt = (p.M + c.rows - 1) / c.rows;
  return mt <= 65535 && (p.N + 127) / 128 * mt * c.split <= INT32_MAX;
}

// How the product is cut, by the time in microseconds that it is expected to take.  The constants are fitted to 905 times
// of 160 sizes (1 to 2,048 rows, N 512 to 16,416, K 512 to 12,288).  On 919 times of the same sizes taken later, with
// every cut that they pick among them, they are within 7 % on average, and the cut that they pick is 0.4 % slower than
// the fastest on average, 12 % at most.
//   few rows:  a fixed part; waves of CTAs, a K block of each at so many KB through its SM, and its output; then the
//              join of the parts of K.
//   pairs:     a fixed part; waves of pairs, 0.236 us a K block.
// The waves and the bytes of HBM overlap but for a part of the shorter.
// `out` bytes an output value; only: the one number of parts of K to look at (0: any).
static Cut least_time(const MatmulProblem& p, int sms, float out, int only) {
  const int64_t groups = (p.K + 4 * kStageK - 1) / (4 * kStageK), tiles = (p.N + 127) / 128;
  const float blocks = (float)((p.K + kStageK - 1) / kStageK);
  const float hbm = (((float)p.M + (float)p.N) * (float)p.K + out * (float)p.M * (float)p.N) / 7.13e6f;
  const auto waves = [](int64_t n, int64_t room) { return (float)((n + room - 1) / room); };
  const auto both = [&](float work) { return std::max(hbm, work) + 0.501f * std::min(hbm, work); };
  const int64_t pairs = ((p.M + 255) / 256) * ((p.N + 239) / 240);
  Cut best{0, 1, true};
  float least = only > 1 ? FLT_MAX : 4.29f + both(waves(pairs, sms / 2) * 0.236f * blocks);
  for (int rows = 16; rows <= 256; rows *= 2) {
    const int64_t mt = (p.M + rows - 1) / rows;
    for (int split = 1; split <= 8 && split <= groups; split *= 2) {
      if ((only && split != only) || !cut_fits(p, {rows, split, true})) continue;
      const int64_t ctas = tiles * mt * split;
      // CTAs that run at once, one an SM or two, by clusters: 152, 152, 144, 120 and 304, 304, 296, 288 on GB300's 152 SMs
      // (cudaOccupancyMaxActiveClusters)
      const int room1 = split <= 2 ? sms : split == 4 ? sms * 18 / 19 : sms * 15 / 19;
      const int room2 = split <= 2 ? 2 * sms : split == 4 ? 2 * sms * 37 / 38 : 2 * sms * 18 / 19;
      const bool deep = ctas <= room1, one = deep || rows == 256;
      const float kb = (float)std::min<int64_t>((int64_t)blocks, 4 * ((groups + split - 1) / split)), stage = 16.f + (float)rows / 8.f;
      const float work = kb * (one ? 0.00535f * stage + 0.0211f : 0.0111f * stage + 0.0197f) + 0.594f + 0.0109f * (float)rows;
      const float join = split == 1 ? 0.f : 0.175f + 0.013f * (float)rows + 0.117f * (float)split;
      const float t = 1.38f + both(waves(ctas, one ? room1 : room2) * work) + join;
      if (t < least) least = t, best = Cut{rows, split, deep};
    }
  }
  return best;
}

// The order of a sum is that of its parts of K, whatever the tiles: fp32 outputs take as many parts as bf16 ones, which
// are then the same sums, rounded.  (One size in 10,000 would take others of its own: 39 x 6,169 x 7,184 with fp32 outputs 14.5
// us and 16.1 by its own, 61 x 4,955 x 9,888 16.8 and 14.3.)
Cut choose_cut(const MatmulProblem& p, int sms) {
  const Cut c = least_time(p, sms, 2.f, 0);
  return p.dt == KDA_F32 ? least_time(p, sms, 4.f, c.split) : c;
}

cudaError_t launch_matmul(const MatmulProblem& p, const Cut* cut, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  const Cut c = cut ? *cut : choose_cut(p, sms);
  if (c.rows == 0) return launch_matmul_pair(p, sms, stream);
  return p.dt == KDA_F32 ? launch<float>(p, c, stream) : launch<__nv_bfloat16>(p, c, stream);
}

}  // namespace dense
}  // namespace kda
