// Attention of a few query rows per key/value head over the 4-bit cache: decode
// steps, verification of draft tokens, and every other query count and type that
// the tiled kernel for long query chunks does not take.
//
//   s_pr = sm_scale q_r . k_p,  o_r = sum_p e^{s_pr - m_r} v_p / sum_p e^{s_pr - m_r}
//
// in one pass over the cached tokens with a running maximum m_r.  The rows r of a
// key/value head are its query heads times the sequence's query tokens.
//
// Products.  On m16n8k16 fp16 instructions with the tokens (for the scores) and
// the channels (for the output) as the 16 rows and eight query rows as the
// columns, so that eight query heads on a key/value head fill the instruction:
//   S^T [16 tokens x 8 rows] = K [16 x D] q^T,   O^T [16 channels x 8 rows] += V^T [16 x 16 tokens] P^T.
// E2M1 codes convert to fp16 exactly, one instruction for two of them.  A unit's
// bytes are laid out so that a lane's four 32-bit words of a key row are its
// operands of all eight k steps, two steps per scale group: the group's sum is
// multiplied by its power of two in fp32 when it joins the score.  A lane's value
// bytes are two tokens of four channels; interleaving their nibbles makes each
// byte the pair of tokens that an operand register holds.  The softmax weights,
// accumulators with a token per row, are the transposed operand: one 8 x 8
// transposing move each (movmatrix), after a multiplication by the token's value
// scale of the channel group.
// Ranges.  A query row is scaled by a power of two to 2^14 <= max|q| < 2^15, which
// is exact in fp16 but for channels 2^28 below the largest.  Weights are taken
// relative to m_r and to the largest value scale 2^E seen: p 2^(15 - E) 2^e <= 2^15,
// so a weight loses bits only when p 2^(e - E) is below 2^-29.  E below 2^-27 counts
// as that.
// fp32 inputs: q and the weights each as the sum of two fp16 numbers, two products
// for one.
//
// Split.  The tiles of all (sequence, head, row block) segments form one line that
// is cut into equal parts, one per worker, whatever the lengths; a worker is a
// warp, or for few segments a whole CTA (its warps take the tiles of a segment in
// turn and join in shared memory).  At most the first and the last piece of a
// worker's part is not a whole segment: it goes to the workspace, and a second
// kernel joins the pieces of a segment in their order.  Lengths are read on the
// device; the cut needs one sum over the sequences, which every CTA takes itself.
// Each warp feeds itself through a ring of tiles filled by bulk copies.
#include "attn_common.cuh"

namespace kda {
namespace kv4 {
namespace {

constexpr int kCtas = 152;                       // one persistent CTA per SM
constexpr int kFewSegments = 64;                 // up to so many segments, a CTA is one worker

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// what pack() left of (a, b), packed
__device__ __forceinline__ uint32_t pack_rest(float a, float b, uint32_t hi) {
  const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return pack(a - h.x, b - h.y);
}

__device__ __forceinline__ void bulk_g2s(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(tc::smem_u32(bar))
               : "memory");
}

// Byte i of a scale word as 2^(byte - 127); with kCheck byte 255 is NaN.
template <bool kCheck>
__device__ __forceinline__ float scale_at(uint32_t w, int i) {
  const uint32_t b = (i < 3 ? w << (23 - 8 * i) : w >> 1) & 0x7f800000u;
  return __uint_as_float(kCheck && b == 0x7f800000u ? 0x7fffffffu : b);
}

// Sizes of one instance: head size, blocks of eight rows, fp16 parts of q and the weights.
template <int D_, int NT_, int PARTS_>
struct Cfg {
  static constexpr int D = D_, NT = NT_, PARTS = PARTS_;
  static constexpr int R = 8 * NT;                  // query rows of a segment
  static constexpr int MT = NT == 1 ? 4 : 2;        // units of a tile
  static constexpr int TILE = kUnit * MT;
  static constexpr int STAGES = NT == 1 ? 2 : 4;
  static constexpr bool QREG = NT <= 2 && PARTS == 1;   // q operands in registers
  static constexpr int W = QREG ? 12 : 8;           // warps of a CTA
  static constexpr int GR = D / 32, KS = D / 16;
  static constexpr int kStage = MT * Unit<D>::kBytes, kRing = STAGES * kStage;
  static constexpr int kQ = QREG ? 0 : KS * NT * PARTS * 256;
  static constexpr int kPart = R * (D + 2) * 4;     // a warp's result in shared memory: O, then (m, l)
  static constexpr int oQ = W * kRing, oBar = oQ + W * kQ, oSum = oBar + W * STAGES * 8, kSmem = oSum + (W + 1) * 8;
  static_assert(kPart <= kRing, "a warp's result fits its ring");
  static_assert(kSmem <= 232448, "shared memory");
  static_assert(kStage % 16 == 0 && kRing % 128 == 0, "alignment");
};

// Pieces in the workspace: slot 2 w is the first piece of worker w, 2 w + 1 its last.
struct Parts {
  int4* owner;   // [workers] (sequence, head, row block, pieces that follow in workers w + 1 ..); .w = 0: none
  float2* ml;    // [2 workers][R] reference exponent and sum
  float* o;      // [2 workers][R][D]
};

// A sequence's tiles and row blocks.
struct Work : Seq {
  int32_t tiles, rts;
};

template <class C>
__device__ __forceinline__ Work work_of(const AttnProblem& p, int n, bool* bad) {
  Work s;
  static_cast<Seq&>(s) = seq_of(p, n, bad);
  s.tiles = s.L > 0 ? (s.L - 1) / C::TILE + 1 : 1;   // no token: one empty tile writes the zeros
  s.rts = (s.qn * (p.Hq / p.Hkv) + C::R - 1) / C::R;
  return s;
}

// A worker's place on the line of tiles.
template <class C>
struct Cursor {
  int n, seg, tile;   // sequence, its (head, row block) segment, first tile of the piece
  int64_t left;       // tiles of the worker's part from here on
  Work s;

  __device__ __forceinline__ int count() const { return (int)min((int64_t)(s.tiles - tile), left); }
  __device__ __forceinline__ void next(const AttnProblem& p) {
    left -= count();
    tile = 0;
    if (left <= 0) return;
    bool bad = false;
    if (++seg == p.Hkv * s.rts) {
      seg = 0;
      do s = work_of<C>(p, ++n, &bad);
      while (s.rts == 0);   // tiles are left, so such a sequence follows
    }
  }
};

template <class C>
struct Acc {
  float O[2 * C::GR][C::NT][4];
  float m[C::NT][2], ref[C::NT][2], l[C::NT][2];   // running maximum (log2), reference m + E - 142, sum relative to it
};

// One tile.  kSlow: rows see only a part of it, or it holds a group that is not finite.
template <class C, bool kSlow>
__device__ __forceinline__ void tile_step(uint8_t* st, const uint32_t (&qr)[C::QREG ? C::NT : 1][C::QREG ? C::KS : 1][2],
                                          const uint8_t* qs, const float (&cf)[C::NT][2], const int (&lim)[C::NT][2],
                                          int tok0, int E, Acc<C>& a) {
  using U = Unit<C::D>;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  float S[C::MT][C::NT][4];
#pragma unroll
  for (int mt = 0; mt < C::MT; ++mt) {
    const uint8_t* u = st + mt * U::kBytes;
    uint32_t kw[2][C::GR], ks[2];
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const uint8_t* row = u + U::key_word(g + 8 * hf, 0, t);
      if constexpr (C::GR == 4) {
        const uint4 x = *reinterpret_cast<const uint4*>(row);
        kw[hf][0] = x.x; kw[hf][1] = x.y; kw[hf][2] = x.z; kw[hf][3] = x.w;
        ks[hf] = *reinterpret_cast<const uint32_t*>(u + U::kKs + (g + 8 * hf) * 4);
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(row);
        kw[hf][0] = x.x; kw[hf][1] = x.y;
        ks[hf] = *reinterpret_cast<const uint16_t*>(u + U::kKs + (g + 8 * hf) * 2);
      }
    }
#pragma unroll
    for (int j = 0; j < C::GR; ++j) {
      uint32_t r0[4], r1[4];
      e2m1x8(kw[0][j], r0);
      e2m1x8(kw[1][j], r1);
      const float s0 = scale_at<kSlow>(ks[0], j), s1 = scale_at<kSlow>(ks[1], j);
#pragma unroll
      for (int nt = 0; nt < C::NT; ++nt) {
        float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if constexpr (C::QREG) {
            mma16816(c, r0[2 * h], r1[2 * h], r0[2 * h + 1], r1[2 * h + 1], qr[nt][2 * j + h][0], qr[nt][2 * j + h][1]);
          } else {
#pragma unroll
            for (int part = 0; part < C::PARTS; ++part) {
              const uint2 b = *reinterpret_cast<const uint2*>(qs + ((part * C::KS + 2 * j + h) * C::NT + nt) * 256 + lane * 8);
              mma16816(c, r0[2 * h], r1[2 * h], r0[2 * h + 1], r1[2 * h + 1], b.x, b.y);
            }
          }
        }
        float(&s)[4] = S[mt][nt];
        s[0] = j ? fmaf(s0, c[0], s[0]) : s0 * c[0];
        s[1] = j ? fmaf(s0, c[1], s[1]) : s0 * c[1];
        s[2] = j ? fmaf(s1, c[2], s[2]) : s1 * c[2];
        s[3] = j ? fmaf(s1, c[3], s[3]) : s1 * c[3];
      }
    }
    if constexpr (kSlow) {
#pragma unroll
      for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (tok0 + mt * kUnit + g + 8 * (e >> 1) > lim[nt][e & 1]) S[mt][nt][e] = -INFINITY;
    }
  }

  // running maximum and reference of each column; the accumulators follow them
  bool move = false;
  float f[C::NT][2];
#pragma unroll
  for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = fmaxf(S[0][nt][e], S[0][nt][e + 2]);
#pragma unroll
      for (int mt = 1; mt < C::MT; ++mt) x = fmaxf(x, fmaxf(S[mt][nt][e], S[mt][nt][e + 2]));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
      const float m = fmaxf(a.m[nt][e], x * cf[nt][e]);
      const float ref = (m == -INFINITY ? 0.f : m) + (float)(E - 142);
      // a row that has seen nothing has nothing to follow
      f[nt][e] = a.m[nt][e] == -INFINITY ? 1.f : ex2(a.ref[nt][e] - ref);
      move |= f[nt][e] != 1.f;
      a.m[nt][e] = m;
      a.ref[nt][e] = ref;
    }
  if (__any_sync(0xffffffffu, move)) {
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt) {
      a.l[nt][0] *= f[nt][0];
      a.l[nt][1] *= f[nt][1];
#pragma unroll
      for (int i = 0; i < 2 * C::GR; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) a.O[i][nt][e] *= f[nt][e & 1];
    }
  }
#pragma unroll
  for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 4; ++e) S[mt][nt][e] = ex2(fmaf(S[mt][nt][e], cf[nt][e & 1], -a.ref[nt][e & 1]));
      a.l[nt][0] += S[mt][nt][0] + S[mt][nt][2];
      a.l[nt][1] += S[mt][nt][1] + S[mt][nt][3];
    }

#pragma unroll
  for (int mt = 0; mt < C::MT; ++mt) {
    const uint8_t* u = st + mt * U::kBytes;
    uint32_t xy[2][2][C::GR / 2];   // [8-token block][even or odd channel]: bytes of token pairs
    uint32_t vs[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const uint8_t* at = u + U::val_half(8 * b + 2 * t, 0, g);
      uint32_t w[C::GR];
      if constexpr (C::GR == 4) {
        const uint4 x = *reinterpret_cast<const uint4*>(at);
        w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
        vs[b] = *reinterpret_cast<const uint32_t*>(u + U::kVs + (g + 8 * b) * 4);
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(at);
        w[0] = x.x; w[1] = x.y;
        vs[b] = *reinterpret_cast<const uint16_t*>(u + U::kVs + (g + 8 * b) * 2);
      }
#pragma unroll
      for (int i = 0; i < C::GR / 2; ++i) {
        const uint32_t A = w[i], B = w[C::GR / 2 + i];
        xy[b][0][i] = (A & 0x0f0f0f0fu) | ((B << 4) & 0xf0f0f0f0u);
        xy[b][1][i] = ((A >> 4) & 0x0f0f0f0fu) | (B & 0xf0f0f0f0u);
      }
    }
#pragma unroll
    for (int i = 0; i < C::GR / 2; ++i) {
      uint32_t x0[4], y0[4], x1[4], y1[4];
      e2m1x8(xy[0][0][i], x0);
      e2m1x8(xy[0][1][i], y0);
      e2m1x8(xy[1][0][i], x1);
      e2m1x8(xy[1][1][i], y1);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int j = 2 * i + k;
        const float s0 = scale_at<kSlow>(vs[0], j), s1 = scale_at<kSlow>(vs[1], j);
#pragma unroll
        for (int nt = 0; nt < C::NT; ++nt) {
          float(&s)[4] = S[mt][nt];
          float w[4] = {s[0] * s0, s[1] * s0, s[2] * s1, s[3] * s1};
          if constexpr (kSlow) {   // a token that a row does not see adds nothing to it, whatever its values are
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (s[e] == 0.f) w[e] = 0.f;
          }
          const uint32_t h0 = pack(w[0], w[1]), h1 = pack(w[2], w[3]);
          const uint32_t b0 = transpose8x8(h0), b1 = transpose8x8(h1);
          mma16816(a.O[2 * j][nt], x0[2 * k], y0[2 * k], x1[2 * k], y1[2 * k], b0, b1);
          mma16816(a.O[2 * j + 1][nt], x0[2 * k + 1], y0[2 * k + 1], x1[2 * k + 1], y1[2 * k + 1], b0, b1);
          if constexpr (C::PARTS == 2) {
            const uint32_t c0 = transpose8x8(pack_rest(w[0], w[1], h0)), c1 = transpose8x8(pack_rest(w[2], w[3], h1));
            mma16816(a.O[2 * j][nt], x0[2 * k], y0[2 * k], x1[2 * k], y1[2 * k], c0, c1);
            mma16816(a.O[2 * j + 1][nt], x0[2 * k + 1], y0[2 * k + 1], x1[2 * k + 1], y1[2 * k + 1], c0, c1);
          }
        }
      }
    }
  }
}

// The largest finite value-scale byte of a tile, and whether a key or value scale in it is 255.
template <class C>
__device__ __forceinline__ int tile_scales(const uint8_t* st, bool* special) {
  using U = Unit<C::D>;
  const int lane = threadIdx.x & 31;
  constexpr int kWords = C::D / 8;   // 32-bit words of value scales per unit (as many of key scales)
  uint32_t k4 = 0, v4 = 0;
#pragma unroll
  for (int i = 0; i < (C::MT * kWords + 31) / 32; ++i) {
    const int w = lane + 32 * i;
    if (w < C::MT * kWords) {
      const uint8_t* u = st + (w / kWords) * U::kBytes + U::kKs + (w % kWords) * 4;
      k4 = __vmaxu4(k4, *reinterpret_cast<const uint32_t*>(u));
      v4 = __vmaxu4(v4, *reinterpret_cast<const uint32_t*>(u + C::D / 2));
    }
  }
  uint32_t both = __vmaxu4(k4, v4);
  both = __vmaxu4(both, both >> 16);
  *special = __any_sync(0xffffffffu, (both & 0xffu) == 255u || (both >> 8 & 0xffu) == 255u);
  if (*special) {
    v4 = 0;
    for (int w = lane; w < C::MT * kWords; w += 32) {
      const uint32_t x = *reinterpret_cast<const uint32_t*>(st + (w / kWords) * U::kBytes + U::kVs + (w % kWords) * 4);
      v4 = __vmaxu4(v4, x & ~__vcmpeq4(x, 0xffffffffu));
    }
  }
  v4 = __vmaxu4(v4, v4 >> 16);
  const uint32_t top = max(v4 & 0xffu, v4 >> 8 & 0xffu);
  return (int)__reduce_max_sync(0xffffffffu, top);
}

// Result rows: o (of the type) and lse, or a piece for the join.
template <class C, typename T>
__device__ __forceinline__ void write_row4(const AttnProblem& p, int64_t row, int ch, float l, const float (&x)[4]) {
  const float inv = l == 0.f ? 0.f : 1.f / l;
  T* o = static_cast<T*>(p.o) + row * C::D + ch;
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(o) = make_float4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0] * inv, x[1] * inv), b = __floats2bfloat162_rn(x[2] * inv, x[3] * inv);
    *reinterpret_cast<uint2*>(o) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
}
__device__ __forceinline__ float lse_of(float ref, float l) { return l == 0.f ? -INFINITY : (log2f(l) + ref) * kLn2; }

template <class C, typename T>
__global__ void __launch_bounds__(C::W * 32, 1) kv4_attention_kernel(const __grid_constant__ AttnProblem p,
                                                                     const Parts parts) {
  using U = Unit<C::D>;
  extern __shared__ __align__(128) uint8_t sm[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint8_t* ring = sm + warp * C::kRing;
  uint8_t* qs = sm + C::oQ + warp * C::kQ;
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::oBar) + warp * C::STAGES;
  int64_t* sums = reinterpret_cast<int64_t*>(sm + C::oSum);
  const int G = p.Hq / p.Hkv;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- the line: tiles and segments of every sequence, a range of sequences per warp
  const int per = (p.N + C::W - 1) / C::W;
  const int na = min(warp * per, p.N), nb = min(na + per, p.N);
  bool bad = false;
  int64_t mine = 0, segs = 0;
  for (int n = na + lane; n < nb; n += 32) {
    const Work s = work_of<C>(p, n, &bad);
    mine += (int64_t)s.tiles * s.rts;
    segs += s.rts;
  }
  if (bad && blockIdx.x == 0) report_bad(p.dev_err);
#pragma unroll
  for (int off = 16; off; off >>= 1) {
    mine += __shfl_xor_sync(0xffffffffu, mine, off);
    segs += __shfl_xor_sync(0xffffffffu, segs, off);
  }
  if (threadIdx.x == 0) sums[C::W] = 0;
  if (lane == 0) {
    sums[warp] = mine * p.Hkv;
    for (int i = 0; i < C::STAGES; ++i) tc::mbar_init(full + i, 1);
    tc::fence_mbar_init();
  }
  __syncthreads();
  if (lane == 0) atomicAdd(reinterpret_cast<unsigned long long*>(sums + C::W), (unsigned long long)(segs * p.Hkv));
  __syncthreads();
  int64_t total = 0;
  for (int w = 0; w < C::W; ++w) total += sums[w];
  const bool wide = sums[C::W] <= kFewSegments;   // a CTA is one worker
  const int64_t most = wide ? gridDim.x : (int64_t)gridDim.x * C::W;
  const int64_t workers = min(most, total);
  const int64_t me = wide ? blockIdx.x : (int64_t)blockIdx.x * C::W + warp;
  // every entry of the owner table is written: a wide grid's workers have the first ones
  int4* own_at = parts.owner + (wide ? (int64_t)warp * gridDim.x + blockIdx.x : me);
  if (me >= workers) {   // nothing to do (in a wide grid, for the whole CTA)
    if (lane == 0) *own_at = make_int4(0, 0, 0, 0);
    return;
  }
  const int64_t x0 = me * total / workers, x1 = (me + 1) * total / workers;

  Cursor<C> cur;   // find x0: the warp's range, then the sequence
  {
    int64_t at = 0;
    int w = 0;
    while (at + sums[w] <= x0) at += sums[w++];
    int n0 = min(w * per, p.N);
    for (;; n0 += 32) {
      const int n = n0 + lane;
      bool b = false;
      int64_t c = 0;
      if (n < p.N) {
        const Work s = work_of<C>(p, n, &b);
        c = (int64_t)s.tiles * s.rts * p.Hkv;
      }
      int64_t inc = c;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += y;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, at + inc > x0);
      if (past) {
        const int src = __ffs(past) - 1;
        const int64_t before = at + __shfl_sync(0xffffffffu, inc - c, src);
        cur.n = n0 + src;
        bool dummy = false;
        cur.s = work_of<C>(p, cur.n, &dummy);
        cur.seg = (int)((x0 - before) / cur.s.tiles);
        cur.tile = (int)((x0 - before) % cur.s.tiles);
        break;
      }
      at += __shfl_sync(0xffffffffu, inc, 31);
    }
    cur.left = x1 - x0;
  }
  const int wi = wide ? warp : 0, step = wide ? C::W : 1;

  // ---- the ring
  Cursor<C> pc = cur;   // what to fetch next
  int pk = wi;          // tile of its piece
  uint32_t issued = 0, used = 0;
  bool ok = true;
  const int upp = p.page_size / kUnit;
  auto produce = [&]() {
    while (pc.left > 0 && pk >= pc.count()) {
      if (wide) return;   // the next piece's tiles follow once this one's result is joined
      pc.next(p);
      pk = wi;
    }
    if (pc.left <= 0) return;
    const int tile = pc.tile + pk;
    pk += step;
    const int slot = issued % C::STAGES;
    ++issued;
    const int units = min(C::MT, (pc.s.L + kUnit - 1) / kUnit - tile * C::MT);   // 0 for an empty sequence
    if (lane == 0) tc::mbar_arrive_expect_tx(full + slot, units * U::kBytes);
    __syncwarp();
    const bool whole = upp % C::MT == 0;   // a tile lies in one page
    if (lane < (whole ? min(units, 1) : units)) {
      const int unit = tile * C::MT + lane;
      int64_t page = p.table[(int64_t)pc.n * p.max_pages + unit / upp];
      if (page < 0 || page >= p.num_pages) {
        report_bad(p.dev_err);
        page = 0;
      }
      const int h = pc.seg / pc.s.rts;
      bulk_g2s(tc::smem_u32(ring + slot * C::kStage + lane * U::kBytes),
               p.cache + ((page * p.Hkv + h) * upp + unit % upp) * U::kBytes, (whole ? units : 1) * U::kBytes, full + slot);
    }
  };
  for (int i = 0; i < C::STAGES; ++i) produce();

  int4 owner = make_int4(0, 0, 0, 0);
  for (; cur.left > 0; cur.next(p)) {
    const int cnt = cur.count(), rt = cur.seg % cur.s.rts, h = cur.seg / cur.s.rts;
    const int rows = min(C::R, cur.s.qn * G - rt * C::R);
    if (wide && cur.left != x1 - x0) {   // the ring was used to join the last piece
      pc = cur;
      pk = wi;
      for (int i = 0; i < C::STAGES; ++i) produce();
    }

    // q rows as operands, each scaled by a power of two
    uint32_t qr[C::QREG ? C::NT : 1][C::QREG ? C::KS : 1][2];
    float cf[C::NT][2];
    int lim[C::NT][2];
    __syncwarp();   // the last piece's operands have been read
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt) {
      const int r = nt * 8 + g;
      float x[C::GR][8];
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < C::GR; ++j) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[j][i] = 0.f;
        if (r < rows) {
          const int rr = rt * C::R + r;
          const T* src = static_cast<const T*>(p.q) + ((int64_t)cur.s.q0 + rr / G) * p.qt + (int64_t)(h * G + rr % G) * p.qh +
                         32 * j + 8 * t;
          if constexpr (sizeof(T) == 4) {
            const float4 a = reinterpret_cast<const float4*>(src)[0], b = reinterpret_cast<const float4*>(src)[1];
            x[j][0] = a.x; x[j][1] = a.y; x[j][2] = a.z; x[j][3] = a.w;
            x[j][4] = b.x; x[j][5] = b.y; x[j][6] = b.z; x[j][7] = b.w;
          } else {
            const uint4 a = *reinterpret_cast<const uint4*>(src);
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              x[j][2 * i] = __uint_as_float(w[i] << 16);
              x[j][2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[j][i]) & 0x7fffffffu);
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const uint32_t ex = min(max(top >> 23, 27u), 254u);
      // the sign of sm_scale goes with q, so that the factor of a score is positive
      const float up = copysignf(__uint_as_float((268u - ex) << 23), p.sm_scale);
      const float down = fmaxf(__uint_as_float((ex - 14u) << 23) * fabsf(p.sm_scale) * kLog2e, 1.17549435e-38f);
      cf[nt][0] = __shfl_sync(0xffffffffu, down, 8 * t);
      cf[nt][1] = __shfl_sync(0xffffffffu, down, 8 * t + 4);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int c = nt * 8 + 2 * t + e;
        lim[nt][e] = c < rows ? cur.s.L - cur.s.qn + (rt * C::R + c) / G : -1;
      }
#pragma unroll
      for (int ks = 0; ks < C::KS; ++ks) {
        const float* y = &x[ks >> 1][4 * (ks & 1)];
        const uint32_t b0 = pack(y[0] * up, y[1] * up), b1 = pack(y[2] * up, y[3] * up);
        if constexpr (C::QREG) {
          qr[nt][ks][0] = b0;
          qr[nt][ks][1] = b1;
        } else {
          *reinterpret_cast<uint2*>(qs + (ks * C::NT + nt) * 256 + lane * 8) = make_uint2(b0, b1);
          if constexpr (C::PARTS == 2)
            *reinterpret_cast<uint2*>(qs + ((C::KS + ks) * C::NT + nt) * 256 + lane * 8) =
                make_uint2(pack_rest(y[0] * up, y[1] * up, b0), pack_rest(y[2] * up, y[3] * up, b1));
        }
      }
    }
    __syncwarp();
    // the last token that every row of the segment sees
    const int lim_all = cur.s.L - cur.s.qn + (rt * C::R) / G;

    Acc<C> a;
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        a.m[nt][e] = -INFINITY;
        a.ref[nt][e] = a.l[nt][e] = 0.f;
#pragma unroll
        for (int i = 0; i < 2 * C::GR; ++i) a.O[i][nt][e] = a.O[i][nt][e + 2] = 0.f;
      }
    int E = 100;
    for (int k = wi; k < cnt; k += step) {
      const int tile = cur.tile + k, slot = used % C::STAGES, tok0 = tile * C::TILE;
      uint8_t* st = ring + slot * C::kStage;
      if (ok) ok = __all_sync(0xffffffffu, tc::mbar_wait(full + slot, (used / C::STAGES) & 1, kWaitLimit));
      ++used;
      if (ok) {
        const bool cut = tok0 + C::TILE - 1 > lim_all;
        if (tok0 + C::TILE > cur.s.L) {   // scales behind the last token: 0, whatever the cache holds there
          for (int i = lane; i < C::TILE; i += 32)
            if (tok0 + i >= cur.s.L) {
              uint8_t* u = st + (i / kUnit) * U::kBytes + (i % kUnit) * C::GR;
              if constexpr (C::GR == 4) {
                *reinterpret_cast<uint32_t*>(u + U::kKs) = 0;
                *reinterpret_cast<uint32_t*>(u + U::kVs) = 0;
              } else {
                *reinterpret_cast<uint16_t*>(u + U::kKs) = 0;
                *reinterpret_cast<uint16_t*>(u + U::kVs) = 0;
              }
            }
          tc::fence_proxy_async_smem();   // before the ring's next copy into these bytes
          __syncwarp();
        }
        bool special;
        E = max(E, tile_scales<C>(st, &special));
        if (cut || special) tile_step<C, true>(st, qr, qs, cf, lim, tok0, E, a);
        else tile_step<C, false>(st, qr, qs, cf, lim, tok0, E, a);
      }
      __syncwarp();
      if (ok) produce();
    }
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float& l = a.l[nt][e];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
      }

    // ---- the piece's result
    const bool starts = cur.tile == 0, whole = starts && cnt == cur.s.tiles;
    const int64_t slot = 2 * me + (starts ? 1 : 0);
    if (starts && !whole) {   // this worker's last piece; who has the rest of the segment?
      const int64_t y = x1 + (cur.s.tiles - cnt) - 1;
      owner = make_int4(cur.n, h, rt, (int)(((y + 1) * workers - 1) / total - me));
    }
    const int64_t row0 = (int64_t)cur.s.q0 * p.Hq;   // row r: token r / G, head h G + r % G
    if (!wide) {
#pragma unroll
      for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = nt * 8 + 2 * t + e, rr = rt * C::R + c;
          if (c >= rows) continue;
          const int64_t row = row0 + (int64_t)(rr / G) * p.Hq + h * G + rr % G;
          if (g == 0) {
            if (!whole) parts.ml[slot * C::R + c] = make_float2(a.ref[nt][e], a.l[nt][e]);
            else if (p.lse) p.lse[row] = lse_of(a.ref[nt][e], a.l[nt][e]);
          }
#pragma unroll
          for (int j = 0; j < C::GR; ++j) {
            const float x[4] = {a.O[2 * j][nt][e], a.O[2 * j][nt][e + 2], a.O[2 * j + 1][nt][e], a.O[2 * j + 1][nt][e + 2]};
            if (whole) write_row4<C, T>(p, row, 32 * j + 4 * g, a.l[nt][e], x);
            else
              *reinterpret_cast<float4*>(parts.o + (slot * C::R + c) * C::D + 32 * j + 4 * g) =
                  make_float4(x[0], x[1], x[2], x[3]);
          }
        }
    } else {   // the warps' results through shared memory
      float* mo = reinterpret_cast<float*>(ring);
      float2* mml = reinterpret_cast<float2*>(mo + C::R * C::D);
#pragma unroll
      for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = nt * 8 + 2 * t + e;
          if (g == 0) mml[c] = make_float2(a.ref[nt][e], a.l[nt][e]);
#pragma unroll
          for (int j = 0; j < C::GR; ++j)
            *reinterpret_cast<float4*>(mo + c * C::D + 32 * j + 4 * g) =
                make_float4(a.O[2 * j][nt][e], a.O[2 * j][nt][e + 2], a.O[2 * j + 1][nt][e], a.O[2 * j + 1][nt][e + 2]);
        }
      __syncthreads();
      for (int i = threadIdx.x; i < rows * (C::D / 4); i += C::W * 32) {
        const int c = i / (C::D / 4), ch = (i % (C::D / 4)) * 4, rr = rt * C::R + c;
        auto ml_of = [&](int w) {
          return reinterpret_cast<const float2*>(sm + w * C::kRing + C::R * C::D * 4)[c];
        };
        float ref = -INFINITY;   // over the warps that saw a token (or a NaN) for this row
        for (int w = 0; w < C::W; ++w) {
          const float2 x = ml_of(w);
          if (x.y != 0.f) ref = fmaxf(ref, x.x);
        }
        float l = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
        for (int w = 0; w < C::W; ++w) {
          const float2 y = ml_of(w);
          if (y.y == 0.f) continue;
          const float f = ex2(y.x - ref);
          const float4 v = *reinterpret_cast<const float4*>(sm + w * C::kRing + (c * C::D + ch) * 4);
          l = fmaf(y.y, f, l);
          x[0] = fmaf(v.x, f, x[0]); x[1] = fmaf(v.y, f, x[1]); x[2] = fmaf(v.z, f, x[2]); x[3] = fmaf(v.w, f, x[3]);
        }
        if (l == 0.f) ref = 0.f;
        const int64_t row = row0 + (int64_t)(rr / G) * p.Hq + h * G + rr % G;
        if (ch == 0) {
          if (!whole) parts.ml[slot * C::R + c] = make_float2(ref, l);
          else if (p.lse) p.lse[row] = lse_of(ref, l);
        }
        if (whole) write_row4<C, T>(p, row, ch, l, x);
        else *reinterpret_cast<float4*>(parts.o + (slot * C::R + c) * C::D + ch) = make_float4(x[0], x[1], x[2], x[3]);
      }
      tc::fence_proxy_async_smem();   // before the next piece's copies into the rings
      __syncthreads();
    }
  }
  if (lane == 0) *own_at = wide && warp != 0 ? make_int4(0, 0, 0, 0) : owner;
  if (!ok) {   // never leave copies in flight: wait (bounded) for the last ones
    for (uint32_t i = issued > C::STAGES ? issued - C::STAGES : 0; i < issued; ++i)
      tc::mbar_wait(full + i % C::STAGES, (i / C::STAGES) & 1, kWaitLimit);
    if (lane == 0) atomicExch(p.dev_err, (int32_t)kDevErrTimeout);
  }
}

// Joins the pieces of the segments that a worker boundary cuts: block w those of the
// segment that begins in worker w and goes on in the next ones, a thread per row and
// four channels, in the order of the pieces.
template <class C, typename T>
__global__ void __launch_bounds__(C::R * C::D / 4) kv4_join_kernel(const __grid_constant__ AttnProblem p, const Parts parts) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t w = blockIdx.x;
  const int4 own = parts.owner[w];
  if (own.w == 0) return;
  const int c = threadIdx.x / (C::D / 4), ch = (threadIdx.x % (C::D / 4)) * 4;
  const int G = p.Hq / p.Hkv, rr = own.z * C::R + c;
  const int q0 = p.cu ? p.cu[own.x] : own.x, qn = p.cu ? p.cu[own.x + 1] - q0 : 1;
  if (rr >= qn * G) return;
  auto slot = [&](int i) { return i == 0 ? 2 * w + 1 : 2 * (w + i); };
  float ref = -INFINITY;
#pragma unroll 4
  for (int i = 0; i <= own.w; ++i) {
    const float2 x = parts.ml[slot(i) * C::R + c];
    if (x.y != 0.f) ref = fmaxf(ref, x.x);
  }
  float l = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int i = 0; i <= own.w; ++i) {
    const float2 y = parts.ml[slot(i) * C::R + c];
    const float4 v = *reinterpret_cast<const float4*>(parts.o + (slot(i) * C::R + c) * C::D + ch);
    const float f = y.y != 0.f ? ex2(y.x - ref) : 0.f;
    if (f == 0.f) continue;
    l = fmaf(y.y, f, l);
    x[0] = fmaf(v.x, f, x[0]); x[1] = fmaf(v.y, f, x[1]); x[2] = fmaf(v.z, f, x[2]); x[3] = fmaf(v.w, f, x[3]);
  }
  const int64_t row = ((int64_t)q0 + rr / G) * p.Hq + own.y * G + rr % G;
  if (ch == 0 && p.lse) p.lse[row] = lse_of(ref, l);
  write_row4<C, T>(p, row, ch, l, x);
}

template <class C>
size_t parts_bytes() {
  const size_t w = (size_t)kCtas * C::W;
  return w * sizeof(int4) + 2 * w * C::R * (sizeof(float2) + C::D * sizeof(float));
}

template <class C, typename T>
cudaError_t launch(const AttnProblem& p, void* workspace, cudaStream_t stream) {
  cudaError_t e;
  int dev = 0, sms = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(kv4_attention_kernel<C, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem)) !=
      cudaSuccess)
    return e;
  const size_t w = (size_t)kCtas * C::W;
  Parts parts;
  parts.owner = static_cast<int4*>(workspace);
  parts.o = reinterpret_cast<float*>(parts.owner + w);
  parts.ml = reinterpret_cast<float2*>(parts.o + 2 * w * C::R * C::D);
  const unsigned grid = (unsigned)(sms < kCtas ? sms : kCtas);
  prof_begin(stream, "kv4_attention_kernel");
  kv4_attention_kernel<C, T><<<grid, C::W * 32, C::kSmem, stream>>>(p, parts);
  prof_end(stream);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid * C::W, 1, 1);
  cfg.blockDim = dim3(C::R * C::D / 4, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];   // its blocks may come up while the first kernel ends; they wait for its results
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  prof_begin(stream, "kv4_join_kernel");
  e = cudaLaunchKernelEx(&cfg, kv4_join_kernel<C, T>, p, parts);
  prof_end(stream);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

// Calls f with the instance for these sizes: as many blocks of eight rows as a
// sequence's rows fill, up to four (two for fp32).
template <typename F>
auto with_cfg(int32_t Hq, int32_t Hkv, int32_t D, int32_t max_q, kda_dtype dt, F f) {
  const int64_t rows = (int64_t)max_q * (Hq / Hkv);
  if (dt == KDA_F32) {
    if (D == 128) return rows <= 8 ? f(Cfg<128, 1, 2>{}, float{}) : f(Cfg<128, 2, 2>{}, float{});
    return rows <= 8 ? f(Cfg<64, 1, 2>{}, float{}) : f(Cfg<64, 2, 2>{}, float{});
  }
  const __nv_bfloat16 z{};
  if (D == 128) return rows <= 8 ? f(Cfg<128, 1, 1>{}, z) : rows <= 16 ? f(Cfg<128, 2, 1>{}, z) : f(Cfg<128, 4, 1>{}, z);
  return rows <= 8 ? f(Cfg<64, 1, 1>{}, z) : rows <= 16 ? f(Cfg<64, 2, 1>{}, z) : f(Cfg<64, 4, 1>{}, z);
}

// Whether the tiled kernel takes the call: bf16, and a sequence's rows fill at least one of
// its blocks of 128 rows.
bool extend_rows(const AttnProblem& p) {
  const int64_t rows = (int64_t)p.max_q * (p.Hq / p.Hkv);
  return p.dt == KDA_BF16 && rows >= 128 && (rows + 255) / 256 * p.N * p.Hkv <= INT32_MAX;
}
}  // namespace

size_t attention_workspace(int32_t Hq, int32_t Hkv, int32_t D, int32_t max_q, kda_dtype dt) {
  return with_cfg(Hq, Hkv, D, max_q, dt, [](auto c, auto) { return parts_bytes<decltype(c)>(); });
}

cudaError_t launch_attention(const AttnProblem& p, void* workspace, cudaStream_t stream) {
  if (extend_rows(p)) return launch_extend(p, stream);
  return with_cfg(p.Hq, p.Hkv, p.D, p.max_q, p.dt,
                  [&](auto c, auto z) { return launch<decltype(c), decltype(z)>(p, workspace, stream); });
}

}  // namespace kv4
}  // namespace kda
