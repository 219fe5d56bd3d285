// Attention of many query rows per key/value head over the 4-bit cache (a chunk of
// a prompt over what is cached, itself included): bf16 queries, both products on
// tcgen05 with the scores and the output in TMEM.
//
//   S = Q K^T  [128 rows x 128 tokens],  P = 2^(S c - m + 9),  O += P V  [128 rows x D]
//
// A CTA takes 256 rows (query tokens times query heads of one key/value head) as
// two blocks of 128 and walks the tokens in tiles of 128.  Warps 0-3 and 4-7 turn a
// tile's codes into two fp16 operand tiles, keys [tokens][D] and values [D][tokens],
// both K-major with 128-byte swizzle, a tile ahead of the products; warps 8-11 and
// 12-15 are the softmax of the two blocks, a thread per row, and the first of each four
// issues its block's products.
// Nothing orders the blocks against each other, so that one's products may run under the
// other's softmax: per tile and block two products of 128 x 128 x D against 128
// exponentials per thread.
//
// Ranges.  A query row is scaled by a power of two to 2^14 <= max|q| < 2^15 (bf16 is exact
// in fp16 then, but for channels 2^28 below the largest).  A tile's keys are held relative
// to its largest key scale 2^EK, as code 2^(e - EK + 8), exact for groups down to
// 2^-21 of it and off by 2^-33 of it at most; S is multiplied back in fp32.  Values
// likewise relative to the largest value scale of their channel group so far, 2^EV (2^-95 at
// least); the group's output follows it when it grows.  The reference m of a row follows its maximum only when that has
// grown by more than 2^6 (few tiles do, and each costs a pass over O in TMEM), so
// weights reach 2^15 and lose bits below 2^-23 of the largest.
// Groups that are not finite: keys become NaN operands; for values, whose NaN would
// reach rows that do not see the token, each row notes the groups of the tokens
// that it sees, and its output becomes NaN there.
//
// Measured: 3 sequences, 3,394 tokens over 16,860 cached, 32 query on 8 key heads of 128,
// 398 us, 37 % of the bf16 matrix rate for the causal work.  Counters: tensor pipe 35 % of
// active cycles, ALU 39 %, issue 47 %, no unit full; the longest stall is the wait for
// memory and TMEM loads.  Against 402 us, with one part left out (results wrong, for timing
// only): the weights' arithmetic 288 us, most of the products 327, the conversions 360.
// Slower or equal: scores in two buffers of 64 tokens 452, blocks in strict turns 452, two threads
// per row on 24 warps 442, one pass with maxima by chunks 443, a row's scores kept in
// registers 402 to 406.
#include "attn_common.cuh"

namespace kda {
namespace kv4 {
namespace {

constexpr int kRows = 256, kTok = 128;
constexpr int kThreads = 16 * 32;
constexpr float kLazy = 6.f, kUp = 9.f;   // kUp + kLazy = 15: weights stay in fp16's range

template <int D>
struct L {
  static constexpr int kAtoms = D / 64;                       // 64-channel swizzle atoms of Q and K
  static constexpr uint32_t kQb = kAtoms * 16384;             // a block of 128 query rows
  static constexpr uint32_t kK = kAtoms * 16384, kV = 2 * D * 128;   // operand tiles
  static constexpr uint32_t oK = 2 * kQb, oV = oK + 2 * kK, oFlags = oV + 2 * kV;   // two stages each
  static constexpr uint32_t oMeta = oFlags + 2 * kTok, oBar = oMeta + 2 * 16;
  static constexpr uint32_t kBars = 12, oTmem = oBar + kBars * 8, kBytes = oTmem + 8, kAlloc = kBytes + 1024;
  static_assert(kAlloc <= 232448 && oK % 1024 == 0 && oV % 1024 == 0 && oBar % 8 == 0, "layout");
  static constexpr uint32_t kOnes = D == 128 ? 0x01010101u : 0x0101u, kLeastEV = 32 * kOnes;   // a byte per channel group
  static constexpr uint32_t cS = 0, cO = 256;                 // TMEM: S (and P over it) of block b at 128 b, O at 256 + 128 b
};

// fp16 bits of 2^f' with exponent field f (f <= 0: subnormal or 0)
__device__ __forceinline__ uint32_t pow2_h(int f) { return f >= 1 ? (uint32_t)f << 10 : f >= -9 ? 1u << (9 + f) : 0u; }
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ int byte_at(uint32_t w, int i) { return (int)(w >> (8 * i) & 0xffu); }

// 32 fp32 columns of this thread's TMEM lane: the load, and the wait that all loads
// before it (whose registers pass through it) have arrived.
__device__ __forceinline__ void tmem_ld32_begin(uint32_t a, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(a)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32_end(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                 "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
                 "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29])
               :
               : "memory");
  asm volatile("" : "+f"(v[30]), "+f"(v[31]));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv4_extend_kernel(const __grid_constant__ AttnProblem p, int32_t blocks) {
  using M = L<D>;
  using U = Unit<D>;
  constexpr int GR = D / 32;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // the longest rows first: the last row blocks of all sequences and heads
  const int per = p.N * p.Hkv;
  const int rb = blocks - 1 - (int)(blockIdx.x / per), n = (int)(blockIdx.x % per) / p.Hkv, h = (int)(blockIdx.x % per) % p.Hkv;
  bool bad = false;
  const Seq s = seq_of(p, n, &bad);
  if (bad && h == 0 && rb == 0 && tid == 0) report_bad(p.dev_err);
  const int G = p.Hq / p.Hkv;
  const int R0 = rb * kRows;
  const int rows = min((int64_t)kRows, (int64_t)s.qn * G - R0);
  if (rows <= 0) return;
  const bool two = rows > 128;
  const int lim0 = s.L - s.qn + R0 / G, lim1 = s.L - s.qn + (R0 + rows - 1) / G;   // last tokens seen, first and last row
  const int nt = lim1 < 0 ? 0 : lim1 / kTok + 1;

  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + M::oBar);
  uint64_t *kfull = bar, *vfull = bar + 2, *kvempty = bar + 4, *sfull = bar + 6, *drain = bar + 8, *ready = bar + 10;
  int4* meta = reinterpret_cast<int4*>(sm + M::oMeta);   // per stage: EK, -, EV (a byte per group), whether values are not finite
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + M::oTmem);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(kfull + i, 4);
      tc::mbar_init(vfull + i, 4);
      tc::mbar_init(kvempty + i, two ? 2 : 1);
      tc::mbar_init(sfull + i, 1);
      tc::mbar_init(drain + i, 1);
      tc::mbar_init(ready + i, 4);   // the four warps of block i: Q, then each tile's weights
    }
    tc::fence_mbar_init();
  }
  if (warp == 0) {
    tc::tmem_alloc(tslot, 512);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tslot;
  auto wait_all = [](uint64_t* b, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, tc::mbar_wait(b, parity, kWaitLimit));
  };
  bool ok = true;

  if (warp < 8) {
    // ---------------- codes to operands: keys in warps 0-3, values in warps 4-7
    // Loads run ahead of their use: page pointers two tiles, scales and codes one.  A
    // warp finds the tile's largest scale by itself, from all tokens' scales.
    const int upp = p.page_size / kUnit;
    auto unit_ptr = [&](int64_t tok) -> const uint8_t* {   // null behind the last token
      if (tok >= s.L) return nullptr;
      const int unit = (int)tok / kUnit;
      int64_t page = p.table[(int64_t)n * p.max_pages + unit / upp];
      if (page < 0 || page >= p.num_pages) {
        report_bad(p.dev_err);
        page = 0;
      }
      return p.cache + ((page * p.Hkv + h) * upp + unit % upp) * U::kBytes;
    };
    if (warp < 4) {
      // thread: token row tid; for the maximum, the scales of tokens 4 lane .. + 3
      uint4 kr[GR];
      uint32_t ks = 0, all[GR];
      const uint8_t *ku, *au;
      auto load = [&]() {
        const uint4* row = reinterpret_cast<const uint4*>(ku + U::key_word(tid % kUnit, 0, 0));
#pragma unroll
        for (int j = 0; j < GR; ++j) kr[j] = ku ? __ldg(row + j) : make_uint4(0, 0, 0, 0);
        ks = 0;
        if (ku)
          ks = GR == 4 ? *reinterpret_cast<const uint32_t*>(ku + U::kKs + (tid % kUnit) * 4)
                       : *reinterpret_cast<const uint16_t*>(ku + U::kKs + (tid % kUnit) * 2);
        const uint32_t* sc = reinterpret_cast<const uint32_t*>(au + U::kKs + (4 * lane % kUnit) * GR);
#pragma unroll
        for (int j = 0; j < GR; ++j) all[j] = au ? __ldg(sc + j) : 0u;
      };
      ku = unit_ptr(tid);
      au = unit_ptr(4 * lane);
      if (nt > 0) load();
      ku = unit_ptr(kTok + tid);
      au = unit_ptr(kTok + 4 * lane);
      for (int i = 0; i < nt; ++i) {
        const int st = i & 1, left = s.L - i * kTok;   // tokens from the tile's first on
        uint32_t top = 0;
        if (left >= kTok) {
#pragma unroll
          for (int j = 0; j < GR; ++j) top = __vmaxu4(top, all[j]);
          top = __vmaxu4(top, top >> 16);
          top = max(top & 0xffu, top >> 8 & 0xffu);
          top = __reduce_max_sync(0xffffffffu, top);
        }
        if (left < kTok || top == 255u) {   // only finite scales of tokens that are there
          top = 0;
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int j = 0; j < GR; ++j) {
              const int at = t * GR + j, b = byte_at(all[at >> 2], at & 3);
              top = max(top, 4 * lane + t >= left || b == 255 ? 0u : (uint32_t)b);
            }
          top = __reduce_max_sync(0xffffffffu, top);
        }
        const int EK = max(9, (int)top);
        if (i >= 2) ok = wait_all(kvempty + st, ((i >> 1) - 1) & 1);
        if (!ok) break;
        if (tid == 0) meta[st].x = EK;
        // row tid, chunk c = 4 j + t holds the word (j, t)
        uint8_t* dst = sm + M::oK + st * M::kK + tid * 128;
        uint32_t sc[GR];
#pragma unroll
        for (int j = 0; j < GR; ++j) {
          const int b = byte_at(ks, j);
          sc[j] = (b == 255 ? 0x7fffu : b == 0 ? 0u : pow2_h(b - EK + 23)) * 0x10001u;
        }
        const uint32_t* w = reinterpret_cast<const uint32_t*>(kr);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int j = 0; j < GR; ++j) {
            uint32_t r[4];
            e2m1x8(w[t * GR + j], r);
            const int c = 4 * j + t;
            *reinterpret_cast<uint4*>(dst + (c >> 3) * 16384 + (((c & 7) ^ (tid & 7)) << 4)) =
                make_uint4(mul2(r[0], sc[j]), mul2(r[1], sc[j]), mul2(r[2], sc[j]), mul2(r[3], sc[j]));
          }
        load();
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(kfull + st);
        ku = unit_ptr(token_of_tile(i + 2, kTok, tid));
        au = unit_ptr(token_of_tile(i + 2, kTok, 4 * lane));
      }
    } else {
      // thread: 8-token block vb of the tile, g
      const int vb = tid & 15, vg = (tid >> 4) & 7;
      constexpr int SW = GR / 2;   // 16-byte words of 8 tokens' scales
      uint4 vr[GR], vs4[SW];
      const uint8_t* vu;
      auto load = [&]() {
        const uint4* v = reinterpret_cast<const uint4*>(vu + U::val_half(8 * (vb & 1), 0, vg));
        const uint4* sc = reinterpret_cast<const uint4*>(vu + U::kVs + 8 * (vb & 1) * GR);
#pragma unroll
        for (int j = 0; j < GR; ++j) vr[j] = vu ? __ldg(v + j) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < SW; ++j) vs4[j] = vu ? __ldg(sc + j) : make_uint4(0, 0, 0, 0);
      };
      vu = unit_ptr(8 * vb);
      if (nt > 0) load();
      vu = unit_ptr(kTok + 8 * vb);
      uint32_t EV = M::kLeastEV;
      for (int i = 0; i < nt; ++i) {
        const int st = i & 1, tv = i * kTok + 8 * vb;
        // the tokens' scales, a byte per group, tokens behind the last: 0, whatever the cache holds there
        uint32_t vs[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          const uint32_t* w = reinterpret_cast<const uint32_t*>(vs4);
          vs[t] = GR == 4 ? w[t] : w[t >> 1] >> (16 * (t & 1)) & 0xffffu;
        }
        if (s.L - tv < 8) {
#pragma unroll
          for (int t = 0; t < 8; ++t)
            if (tv + t >= s.L) vs[t] = 0;
        }
        uint32_t hi = vs[0], lo = vs[0];
#pragma unroll
        for (int t = 1; t < 8; ++t) {
          hi = __vmaxu4(hi, vs[t]);
          lo = __vminu4(lo, vs[t]);
        }
        bool nan = false;
        if (__any_sync(0xffffffffu, __vmaxu4(hi, EV) != EV)) {   // a warp holds all 16 blocks
#pragma unroll
          for (int j = 0; j < GR; ++j) {
            uint32_t vm = __reduce_max_sync(0xffffffffu, (uint32_t)byte_at(hi, j));
            if (vm == 255u) {   // the largest of the others
              nan = true;
              vm = 0;
#pragma unroll
              for (int t = 0; t < 8; ++t) vm = max(vm, byte_at(vs[t], j) == 255 ? 0u : (uint32_t)byte_at(vs[t], j));
              vm = __reduce_max_sync(0xffffffffu, vm);
            }
            EV = (EV & ~(0xffu << (8 * j))) | max((uint32_t)byte_at(EV, j), vm) << (8 * j);
          }
        }
        uint32_t sp[4][GR];   // scale pairs of tokens 2 m, 2 m + 1
        const uint32_t low = EV - 22 * M::kOnes;
        if (!nan && !__any_sync(0xffffffffu, __vminu4(lo, low) != low)) {   // exponent fields by bytes: all between 1 and 23
          const uint32_t base = EV - 23 * M::kOnes;
#pragma unroll
          for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int j = 0; j < GR; ++j)
              sp[m][j] = (__byte_perm(vs[2 * m] - base, vs[2 * m + 1] - base, j | (4 + j) << 8) & 0x001f001fu) << 10;
        } else {
#pragma unroll
          for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int j = 0; j < GR; ++j) {
              const int a = byte_at(vs[2 * m], j), b = byte_at(vs[2 * m + 1], j), up = 23 - byte_at(EV, j);
              sp[m][j] = (a == 0 || a == 255 ? 0u : pow2_h(a + up)) | (b == 0 || b == 255 ? 0u : pow2_h(b + up)) << 16;
            }
        }
        if (i >= 2) ok = wait_all(kvempty + st, ((i >> 1) - 1) & 1);
        if (!ok) break;
        if (tid == 128) *reinterpret_cast<int2*>(&meta[st].z) = make_int2((int)EV, nan ? 1 : 0);
        if (nan && vg == 0) {   // which tokens have which groups
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            uint32_t f = 0;
#pragma unroll
            for (int j = 0; j < GR; ++j) f |= (byte_at(vs[t], j) == 255 ? 1u : 0u) << j;
            sm[M::oFlags + st * kTok + 8 * vb + t] = (uint8_t)f;
          }
        }
        // channel 32 j + 4 g + c, chunk of 8 tokens vb
        uint8_t* dst = sm + M::oV + st * M::kV + (vb >> 3) * (D * 128);
        const uint32_t* w = reinterpret_cast<const uint32_t*>(vr);   // token t: words t GR / 2 ..
#pragma unroll
        for (int i2 = 0; i2 < GR / 2; ++i2) {
          uint32_t e[4][4], o[4][4];   // [pair m][byte]: even and odd channels
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const uint32_t A = w[2 * m * (GR / 2) + i2], B = w[(2 * m + 1) * (GR / 2) + i2];
            e2m1x8((A & 0x0f0f0f0fu) | ((B << 4) & 0xf0f0f0f0u), e[m]);
            e2m1x8(((A >> 4) & 0x0f0f0f0fu) | (B & 0xf0f0f0f0u), o[m]);
          }
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const int j = 2 * i2 + (b >> 1), ch = 32 * j + 4 * vg + 2 * (b & 1);
            *reinterpret_cast<uint4*>(dst + ch * 128 + (((vb & 7) ^ (ch & 7)) << 4)) =
                make_uint4(mul2(e[0][b], sp[0][j]), mul2(e[1][b], sp[1][j]), mul2(e[2][b], sp[2][j]), mul2(e[3][b], sp[3][j]));
            *reinterpret_cast<uint4*>(dst + (ch + 1) * 128 + (((vb & 7) ^ ((ch + 1) & 7)) << 4)) =
                make_uint4(mul2(o[0][b], sp[0][j]), mul2(o[1][b], sp[1][j]), mul2(o[2][b], sp[2][j]), mul2(o[3][b], sp[3][j]));
          }
        }
        load();
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(vfull + st);
        vu = unit_ptr(token_of_tile(i + 2, kTok, 8 * vb));
      }
    }
  } else {
    // ---------------- softmax of block b, this thread's row; its first warp issues the block's products
    const int b = (warp - 8) >> 2, wq = warp & 3, r = 32 * wq + lane, row = 128 * b + r;
    const uint32_t tl = 32u * wq;
    const bool live = row < rows;
    const int rr = R0 + row;
    const int64_t orow = ((int64_t)s.q0 + rr / G) * p.Hq + h * G + rr % G;
    float down = 0.f;
    {
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) + ((int64_t)s.q0 + rr / G) * p.qt + (int64_t)(h * G + rr % G) * p.qh;
      uint4 x[D / 8];
      uint32_t top = 0;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        x[c] = live ? __ldg(reinterpret_cast<const uint4*>(src) + c) : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, max(w[e] << 16 & 0x7fffffffu, w[e] & 0x7fff0000u));
      }
      const uint32_t ex = min(max(top >> 23, 27u), 254u);
      const float up = copysignf(__uint_as_float((268u - ex) << 23), p.sm_scale);
      down = __uint_as_float((ex - 14u) << 23) * fabsf(p.sm_scale) * kLog2e;
      uint8_t* dst = sm + b * M::kQb + r * 128;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
        uint32_t y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = pack(__uint_as_float(w[e] << 16) * up, __uint_as_float(w[e] & 0xffff0000u) * up);
        *reinterpret_cast<uint4*>(dst + (c >> 3) * 16384 + (((c & 7) ^ (r & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
      }
    }
    constexpr uint32_t kIdS = tc::idesc_f16_f32(128, kTok), kIdO = tc::idesc_f16_f32(128, D);
    const uint64_t dQ = tc::desc_kmajor_sw128(tc::smem_u32(sm + b * M::kQb)),
                   dK = tc::desc_kmajor_sw128(tc::smem_u32(sm + M::oK)), dV = tc::desc_kmajor_sw128(tc::smem_u32(sm + M::oV));
    const int lim = live ? s.L - s.qn + rr / G : -1;
    const uint32_t cS = M::cS + 128 * b, cO = M::cO + 128 * b;
    float m = -INFINITY, l = 0.f;
    uint32_t EV = M::kLeastEV;
    uint32_t nans = 0;
    const bool run = b == 0 || two;
    const int steps = run ? nt : 0;
    // S of tile i, once its keys are there
    auto scores = [&](int i) -> bool {
      const int st = i & 1;
      if (!wait_all(kfull + st, (i >> 1) & 1)) return false;
      tc::tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
        tc::mma_16bit_w(tmem + cS, dQ + off, dK + ((st * M::kK) >> 4) + off, kIdS, kk > 0);
      }
      tc::mma_commit_w(sfull + b);
      return true;
    };
    bool issued = false;
    if (steps > 0) {
      tc::fence_proxy_async_smem();   // Q, written by the threads, read by the products
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(ready + b);
      if (wq == 0) {
        ok = wait_all(ready + b, 0) && scores(0);
        issued = ok;
      }
    }
    for (int i = 0; i < steps; ++i) {
      const int st = i & 1;
      // (the scales beside the operand tiles are read here, so that a stage's phases are never two ahead)
      if (ok) ok = wait_all(kfull + st, (i >> 1) & 1) && wait_all(vfull + st, (i >> 1) & 1) && wait_all(sfull + b, i & 1);
      if (!ok) break;
      tc::tc_fence_after();
      const int4 mt = meta[st];
      const float cf = fmaxf(down * __uint_as_float((uint32_t)(mt.x - 8) << 23), 1.17549435e-38f);
      const int t0 = i * kTok;
      const bool cut = t0 + kTok - 1 > lim0;
      // the maximum; 32 scores at a time, the next ones on their way.  (Rolled, as below:
      // the roles' code together overflows the instruction cache.)
      float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      float x[32], y[32];
      auto tops_of = [&](float (&v)[32], int c) {
        if (cut) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (t0 + 32 * c + e > lim) v[e] = -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < 32; e += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k) tops[k] = fmaxf(tops[k], fmaxf(v[e + k], v[e + k + 4]));
      };
      tmem_ld32_begin(tc::tmem_addr(tmem, tl, cS), x);
#pragma unroll 1
      for (int c = 0; c < 4; c += 2) {
        tmem_ld32_end(x);
        tmem_ld32_begin(tc::tmem_addr(tmem, tl, cS + 32 * (c + 1)), y);
        tops_of(x, c);
        tmem_ld32_end(y);
        tmem_ld32_begin(tc::tmem_addr(tmem, tl, cS + (c < 2 ? 64 : 0)), x);   // at the end the first ones again, for the weights
        tops_of(y, c + 1);
      }
      float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
      top *= cf;
      // the reference and the output's scales; all only move up
      float f = 1.f;
      if (top > m + kLazy || m == -INFINITY) {
        if (m != -INFINITY) f = ex2(m - top);
        m = top;
      }
      l *= f;
      const uint32_t was = EV;
      EV = (uint32_t)mt.z;
      if (i > 0 && __any_sync(0xffffffffu, f != 1.f || EV != was)) {   // the products into O so far have completed (before S was committed)
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          float v[16];
          uint32_t w[16];
          const float fo = f * __uint_as_float((uint32_t)max(127 + byte_at(was, c >> 1) - byte_at(EV, c >> 1), 0) << 23);
          tc::tmem_ld16(tc::tmem_addr(tmem, tl, cO + 16 * c), v);
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(v[e] * fo);
          tc::tmem_st16(tc::tmem_addr(tmem, tl, cO + 16 * c), w);
        }
      }
      const float ref = (m == -INFINITY ? 0.f : m) - kUp;
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      auto weights_of = [&](float (&v)[32], int c) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 z = __ffma2_rn(make_float2(v[2 * e], v[2 * e + 1]), make_float2(cf, cf), make_float2(-ref, -ref));
          v[2 * e] = ex2(z.x);
          v[2 * e + 1] = ex2(z.y);
        }
        if (cut) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (t0 + 32 * c + e > lim) v[e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          w[e] = pack(v[2 * e], v[2 * e + 1]);
          sum[e & 1] = __fadd2_rn(sum[e & 1], make_float2(v[2 * e], v[2 * e + 1]));
        }
        tc::tmem_st16(tc::tmem_addr(tmem, tl, cS + 16 * c), w);   // over scores that have been read
        if (mt.w) {   // groups that are not finite, of the tokens that this row sees (with a weight of 0 too)
#pragma unroll 1
          for (int e = 0; e < 32; ++e) nans |= t0 + 32 * c + e <= lim ? sm[M::oFlags + st * kTok + 32 * c + e] : 0u;
        }
      };
#pragma unroll 1
      for (int c = 0; c < 4; c += 2) {
        tmem_ld32_end(x);
        tmem_ld32_begin(tc::tmem_addr(tmem, tl, cS + 32 * (c + 1)), y);
        weights_of(x, c);
        tmem_ld32_end(y);
        if (c < 2) tmem_ld32_begin(tc::tmem_addr(tmem, tl, cS + 64), x);
        weights_of(y, c + 1);
      }
      l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      tc::tmem_st_wait();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(ready + b);
      if (wq == 0) {
        ok = wait_all(ready + b, (i + 1) & 1);
        if (!ok) break;
        tc::tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kTok / 16; ++kk)
          tc::mma_16bit_tw(tmem + cO, tmem + cS + 8 * kk, dV + ((st * M::kV + (kk >> 2) * (D * 128) + (kk & 3) * 32) >> 4), kIdO,
                           (i > 0 || kk > 0) ? 1u : 0u);
        tc::mma_commit_w(kvempty + st);
        if (i + 1 < nt) ok = scores(i + 1);
        else tc::mma_commit_w(sfull + b);
      }
    }
    if (issued && !ok) {   // end with no product in flight
      tc::mma_commit_w(drain + b);
      wait_all(drain + b, 0);
    }
    if (run && ok) {
      if (nt > 0) {
        ok = wait_all(sfull + b, nt & 1);   // the last product into O
        tc::tc_fence_after();
      }
      if (ok) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o) + orow * D;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          float v[16];
          if (nt > 0) tc::tmem_ld16(tc::tmem_addr(tmem, tl, cO + 16 * c), v);
          uint32_t w[8];
          const float back = __uint_as_float((uint32_t)(byte_at(EV, c >> 1) - 8) << 23);   // 2^(EV - 135)
          const bool none = nt == 0 || l == 0.f, gone = (nans >> (c >> 1) & 1u) != 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float x = none ? 0.f : v[2 * e] * inv * back, y = none ? 0.f : v[2 * e + 1] * inv * back;
            const __nv_bfloat162 z = __floats2bfloat162_rn(x, y);
            w[e] = gone ? 0x7fff7fffu : *reinterpret_cast<const uint32_t*>(&z);
          }
          if (live) {
            reinterpret_cast<uint4*>(o)[2 * c] = make_uint4(w[0], w[1], w[2], w[3]);
            reinterpret_cast<uint4*>(o)[2 * c + 1] = make_uint4(w[4], w[5], w[6], w[7]);
          }
        }
        if (live && p.lse) p.lse[orow] = l == 0.f ? -INFINITY : (log2f(l) + m - kUp) * kLn2;
      }
    }
  }
  if (!ok && lane == 0) atomicExch(p.dev_err, (int32_t)kDevErrTimeout);
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 0) tc::tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t launch(const AttnProblem& p, cudaStream_t stream) {
  cudaError_t e = cudaFuncSetAttribute(kv4_extend_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L<D>::kAlloc);
  if (e != cudaSuccess) return e;
  const int64_t blocks = ((int64_t)p.max_q * (p.Hq / p.Hkv) + kRows - 1) / kRows;
  prof_begin(stream, "kv4_extend_kernel");
  kv4_extend_kernel<D><<<(unsigned)(blocks * p.N * p.Hkv), kThreads, L<D>::kAlloc, stream>>>(p, (int32_t)blocks);
  prof_end(stream);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_extend(const AttnProblem& p, cudaStream_t stream) {
  return p.D == 128 ? launch<128>(p, stream) : launch<64>(p, stream);
}

}  // namespace kv4
}  // namespace kda
