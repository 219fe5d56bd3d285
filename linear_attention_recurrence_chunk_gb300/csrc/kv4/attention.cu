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
// is exact in fp16 but for channels 2^28 below the largest.  Weights are 2^14 at
// most and multiplied, transposed, by the value scales relative to a reference of
// their channel group, 2^(e - E) <= 2, in fp16: exact where e - E >= -14 and a product is
// normal; a tile with smaller ones multiplies in fp32 first.  E is the largest e seen in
// the group, or one below it, and at least 2^-107; the group's output follows it.  So a
// weight loses bits only when p 2^(e - E) is below 2^-28.  The sum l takes the weights
// before they are rounded.
// fp32 inputs: q and the weights each as the sum of two fp16 numbers, two products
// for one.
//
// Split.  The tiles of all (sequence, head, row block) segments form one line, each
// segment with a little room for its beginning and end, that is cut into equal
// parts, one per worker, whatever the lengths; a worker is a warp, or for few
// segments a whole CTA (its warps take the tiles of a segment in turn and join in
// shared memory).  At most the first and the last piece of a worker's part is not a
// whole segment: it goes to the workspace, and a second kernel joins the pieces of a
// segment in their order.  Lengths are read on the device; the cut needs one sum over
// the sequences, which every CTA takes itself.  Each warp feeds itself through a ring
// of tiles filled by bulk copies.
//
// Measured: one token of 48 sequences up to 32,000, 64 query on 8 key heads of 128: 107 us
// with the join, 563 MB at 5.2 TB/s (fp32: 150 us for 497 K tokens).  Counters: issue 57 %
// and ALU pipe 56 % of active cycles, DRAM 68 %, 260 warp instructions for 16 tokens of a
// head.  Before later steps, which took 111 to 107 us, 16 warps of 32-token tiles took 136 us
// and 8 warps with three stages 119.
#include <algorithm>
#include <cstdlib>

#include "attn_common.cuh"

namespace kda {
namespace kv4 {
namespace {

constexpr int kCtas = 152;                       // one persistent CTA per SM
// Up to so many segments a CTA is one worker: one token over 131,072, 4 key heads, 27.6 us
// against 87.6 with a warp as the worker.  Between 16 and 160 the bound made no difference
// to the sizes timed.
constexpr int kFewSegments = 64;

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// c = a b
__device__ __forceinline__ void mma16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
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

__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
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
  static constexpr int MT = 4, TILE = kUnit * MT;   // units and tokens of a tile
  static constexpr int MH = NT == 1 ? 4 : 2;        // units of a softmax step: as many as the registers hold scores of
  static constexpr int STAGES = 2;
  static constexpr bool QREG = NT <= 2 && PARTS == 1;   // q operands in registers
  static constexpr int W = NT == 1 && PARTS == 1 ? 12 : 8;   // warps of a CTA
  // room of a segment's beginning and end on the line, in tiles.  With 1, 2, 3, 4 (us): 256 sequences up to 2,048 tokens,
  // 96 query on 8 key heads 108.6, 97.3, 91.7, 95.5; 48 up to 32,000, 64 on 8, 108.4, 108.2, 107.4, 108.8; 32 up to 8,191 with
  // 5 tokens, 32 on 8, 67.9, 65.9, 67.2, 67.9; 256 up to 500, 8 on 8, 26.3, 26.5, 27.9, 29.8; 128 up to 1,000 with heads of
  // 64, 16 on 4, 15.0, 15.8, 16.2, 16.4; 40 fp32 up to 3,000, 32 on 8, 24.4, 25.9, 25.5, 26.3.
  static constexpr int HEAD = 3;
  static constexpr int GR = D / 32, KS = D / 16;
  static constexpr int kStage = MT * Unit<D>::kBytes, kRing = STAGES * kStage;
  static constexpr int kQ = QREG ? 0 : KS * NT * PARTS * 256;
  // a warp's tables: a tile's scales, of keys as fp32 [token][group], of values as fp16
  // [token pair][group][2]; the rows' score factors, last tokens and places in the output
  static constexpr int tV = TILE * GR * 4, tRow = tV + TILE * 8, kTab = tRow + R * 16;
  static constexpr int kPart = R * (D + 2) * 4;     // a warp's result in shared memory: O, then (m, l)
  static constexpr int oQ = W * kRing, oTab = oQ + W * kQ, oBar = oTab + W * kTab, oSum = oBar + W * STAGES * 8,
                       kSmem = oSum + (W + 1) * 8;
  static_assert(kPart <= kRing, "a warp's result fits its ring");
  static_assert(kSmem <= 232448, "shared memory");
  static_assert(kStage % 16 == 0 && kRing % 128 == 0 && kTab % 16 == 0, "alignment");
};

// Pieces in the workspace: slot 2 w is the first piece of worker w, 2 w + 1 its last.
struct Parts {
  int4* owner;   // [workers] (first query token, head * 64 + rows, first row, pieces that follow in workers w + 1 ..); .w = 0: none
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
  s.rts = row_blocks(s.qn, p.Hq / p.Hkv, C::R);
  return s;
}

// A worker's place on the line: a segment takes HEAD + tiles of it.
template <class C>
struct Cursor {
  int n, seg, pos;    // sequence, its (head, row block) segment, place in the segment
  int64_t left;       // what is left of the worker's part
  Work s;

  __device__ __forceinline__ int span() const { return (int)min((int64_t)(C::HEAD + s.tiles - pos), left); }
  __device__ __forceinline__ int first() const { return max(pos - C::HEAD, 0); }             // tiles of the piece
  __device__ __forceinline__ int last() const { return max(pos + span() - C::HEAD, 0); }     // (one behind)
  __device__ __forceinline__ void next(const AttnProblem& p) {
    left -= span();
    pos = 0;
    if (left <= 0) return;
    bool bad = false;
    if (++seg == p.Hkv * s.rts) {
      seg = 0;
      do s = work_of<C>(p, ++n, &bad);
      while (s.rts == 0);   // something is left, so such a sequence follows
    }
  }
};

template <class C>
struct Acc {
  float O[2 * C::GR][C::NT][4];
  float m[C::NT][2], l[C::NT][2];   // running maximum (log2) and sum of 2^(s - m + 14) of each column
};

// 2^x, 0 below the smallest normal number; x <= 127
__device__ __forceinline__ float pow2(int x) { return __uint_as_float((uint32_t)max(127 + x, 0) << 23); }
__device__ __forceinline__ int byte_of(uint32_t w, int i) { return (int)(w >> (8 * i) & 0xffu); }

template <class C>
constexpr uint32_t kOnes = C::GR == 4 ? 0x01010101u : 0x0101u;   // a byte per group
constexpr uint32_t kLeastE = 20;                                  // 2^-107

// A tile's scales into the warp's tables.  E, a byte per channel group, the reference of its value scales, is the
// largest of a piece's first tile (fresh), raised when one is above 2^(E + 1) later.  Returns whether the tile
// needs the careful step: a group that is not finite, a key scale of 2^97 or more (the scores'
// sums, up to 2^24.6 of it before the rows' factors, might pass fp32), or a value scale outside
// 2^(E - 14) .. 2^(E + 1), whose fp16 relative to E is not a normal number.
template <class C>
__device__ __forceinline__ bool load_scales(const uint8_t* st, uint8_t* tab, int left, bool fresh, uint32_t& E) {
  using U = Unit<C::D>;
  const int lane = threadIdx.x & 31;
  uint32_t k[2] = {0, 0}, v[2] = {0, 0};   // of tokens 2 lane, 2 lane + 1; a byte per group
  const bool in = lane < C::TILE / 2;
  if (in) {
    const uint8_t* u = st + (lane / 8) * U::kBytes + U::kKs + (lane % 8) * 2 * C::GR;
    if constexpr (C::GR == 4) {
      const uint2 a = *reinterpret_cast<const uint2*>(u), b = *reinterpret_cast<const uint2*>(u + C::D / 2);
      k[0] = a.x; k[1] = a.y; v[0] = b.x; v[1] = b.y;
    } else {
      const uint32_t a = *reinterpret_cast<const uint32_t*>(u), b = *reinterpret_cast<const uint32_t*>(u + C::D / 2);
      k[0] = a & 0xffffu; k[1] = a >> 16; v[0] = b & 0xffffu; v[1] = b >> 16;
    }
  }
  const int have = min(left - 2 * lane, in ? 2 : 0);   // of the two tokens; the cache may hold anything behind the last
  auto raise = [&](uint32_t room) {                    // E to a group's largest value scale but 255 where that is more than E + room
#pragma unroll
    for (int j = 0; j < C::GR; ++j) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) m = max(m, i < have ? (v[i] >> (8 * j) & 0xffu) % 255u : 0u);
      m = __reduce_max_sync(0xffffffffu, m);
      if (m > (E >> (8 * j) & 0xffu) + room) E = (E & ~(0xffu << (8 * j))) | m << (8 * j);
    }
  };
  if (fresh) {
    E = kLeastE * kOnes<C>;
    raise(0);
  }
  if (have < 2) {   // tokens that are not there: nothing that a weight of 0 would not cancel
    if (have < 1) k[0] = 0, v[0] = E;
    k[1] = 0;
    v[1] = E;
  }
  // exponent fields of the value scales less one: a byte outside 0 .. 15 (or a borrow, which leaves one) shows in
  // the high nibbles, for E <= 239; a key byte of 224 or more by a carry
  uint32_t d0 = v[0] - (E - 14 * kOnes<C>), d1 = v[1] - (E - 14 * kOnes<C>);
  uint32_t odd = (d0 | d1) & (C::GR == 4 ? 0xf0f0f0f0u : 0xfffff0f0u);
#pragma unroll
  for (int i = 0; i < 2; ++i) odd |= ((k[i] & 0x7f7f7f7fu) + 0x20202020u) & k[i] & 0x80808080u;
  odd |= E & E << 1 & E << 2 & E << 3 & 0x80808080u;   // E > 239
  const bool careful = __any_sync(0xffffffffu, odd != 0);
  if (careful) raise(1);
  if (in) {
    float* kf = reinterpret_cast<float*>(tab) + 2 * lane * C::GR;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float f[C::GR];
#pragma unroll
      for (int j = 0; j < C::GR; ++j) f[j] = scale_f32(k[i] >> (8 * j) & 0xffu);
      if (careful) {
#pragma unroll
        for (int j = 0; j < C::GR; ++j) f[j] = f[j] == INFINITY ? __uint_as_float(0x7fffffffu) : f[j];
      }
      if constexpr (C::GR == 4) reinterpret_cast<float4*>(kf)[i] = make_float4(f[0], f[1], f[2], f[3]);
      else reinterpret_cast<float2*>(kf)[i] = make_float2(f[0], f[1]);
    }
    if (!careful) {
      d0 += kOnes<C>;   // exponent fields 1 .. 16
      d1 += kOnes<C>;
      uint32_t h[C::GR];
#pragma unroll
      for (int j = 0; j < C::GR; ++j) h[j] = (__byte_perm(d0, d1, j | (4 + j) << 8) & 0x001f001fu) << 10;
      uint8_t* vf = tab + C::tV + lane * C::GR * 4;
      if constexpr (C::GR == 4) *reinterpret_cast<uint4*>(vf) = make_uint4(h[0], h[1], h[2], h[3]);
      else *reinterpret_cast<uint2*>(vf) = make_uint2(h[0], h[1]);
    } else {          // the careful step takes the bytes
      uint32_t* vw = reinterpret_cast<uint32_t*>(tab + C::tV) + 2 * lane;
      vw[0] = v[0];
      vw[1] = v[1];
    }
  }
  __syncwarp();
  return careful;
}

// One step of MH units.  cut: rows see only a part of it (a flag and not another instance, which would
// crowd the instruction cache).  was: E before this tile.  kCareful: see load_scales.
template <class C, bool kCareful>
__device__ __forceinline__ void tile_step(const uint8_t* st, const float* ktab, const uint8_t* vtab, const uint8_t* rowtab,
                                          const uint32_t (&qr)[C::QREG ? C::NT : 1][C::QREG ? C::KS : 1][2],
                                          const uint8_t* qs, int tok0, bool cut, uint32_t E, uint32_t was, Acc<C>& a) {
  using U = Unit<C::D>;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const float2* cfs = reinterpret_cast<const float2*>(rowtab) + t;                 // of columns 2 t, 2 t + 1
  const int2* lims = reinterpret_cast<const int2*>(rowtab + C::R * 4) + t;
  float S[C::MH][C::NT][4];
#pragma unroll
  for (int mt = 0; mt < C::MH; ++mt) {
    const uint8_t* u = st + mt * U::kBytes;
    uint32_t kw[2][C::GR];
    float ks[2][C::GR];
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const uint8_t* row = u + U::key_word(g + 8 * hf, 0, t);
      const float* sc = ktab + (mt * kUnit + g + 8 * hf) * C::GR;
      if constexpr (C::GR == 4) {
        const uint4 x = *reinterpret_cast<const uint4*>(row);
        kw[hf][0] = x.x; kw[hf][1] = x.y; kw[hf][2] = x.z; kw[hf][3] = x.w;
        const float4 f = *reinterpret_cast<const float4*>(sc);
        ks[hf][0] = f.x; ks[hf][1] = f.y; ks[hf][2] = f.z; ks[hf][3] = f.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(row);
        kw[hf][0] = x.x; kw[hf][1] = x.y;
        const float2 f = *reinterpret_cast<const float2*>(sc);
        ks[hf][0] = f.x; ks[hf][1] = f.y;
      }
    }
#pragma unroll
    for (int j = 0; j < C::GR; ++j) {
      uint32_t r0[4], r1[4];
      e2m1x8(kw[0][j], r0);
      e2m1x8(kw[1][j], r1);
#pragma unroll
      for (int nt = 0; nt < C::NT; ++nt) {
        float c[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int part = 0; part < C::PARTS; ++part) {
            uint32_t b0, b1;
            if constexpr (C::QREG) {
              b0 = qr[nt][2 * j + h][0];
              b1 = qr[nt][2 * j + h][1];
            } else {
              const uint2 b = *reinterpret_cast<const uint2*>(qs + ((part * C::KS + 2 * j + h) * C::NT + nt) * 256 + lane * 8);
              b0 = b.x;
              b1 = b.y;
            }
            if (h == 0 && part == 0) mma16816_first(c, r0[2 * h], r1[2 * h], r0[2 * h + 1], r1[2 * h + 1], b0, b1);
            else mma16816(c, r0[2 * h], r1[2 * h], r0[2 * h + 1], r1[2 * h + 1], b0, b1);
          }
        }
        float(&s)[4] = S[mt][nt];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float f = ks[e >> 1][j];
          if constexpr (kCareful) {   // the row's factor joins the scale before the sum; a product beyond fp32 only meets sums near 0
            f *= e & 1 ? cfs[4 * nt].y : cfs[4 * nt].x;
            if (f > 0x1p127f) f = 0x1p127f;   // (a NaN stays)
          }
          s[e] = j ? fmaf(f, c[e], s[e]) : f * c[e];
        }
      }
    }
    if (cut) {
#pragma unroll
      for (int nt = 0; nt < C::NT; ++nt) {
        const int2 lim = lims[4 * nt];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (tok0 + mt * kUnit + g + 8 * (e >> 1) > (e & 1 ? lim.y : lim.x)) S[mt][nt][e] = -INFINITY;
      }
    }
  }

  // running maximum of each column; the accumulators follow it, and E
  bool move = was != E;
  float f[C::NT][2], ref[C::NT][2], cf[C::NT][2];
#pragma unroll
  for (int nt = 0; nt < C::NT; ++nt) {
    const float2 x = kCareful ? make_float2(1.f, 1.f) : cfs[4 * nt];
    cf[nt][0] = fmaxf(x.x, 0x1p-149f);   // above 0, so that -inf keeps its sign
    cf[nt][1] = fmaxf(x.y, 0x1p-149f);
  }
#pragma unroll
  for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = fmaxf(S[0][nt][e], S[0][nt][e + 2]);
#pragma unroll
      for (int mt = 1; mt < C::MH; ++mt) x = fmaxf(x, fmaxf(S[mt][nt][e], S[mt][nt][e + 2]));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
      const float m = fmaxf(a.m[nt][e], x * cf[nt][e]);
      // a row that has seen nothing has nothing to follow
      f[nt][e] = a.m[nt][e] == -INFINITY ? 1.f : ex2(a.m[nt][e] - m);
      move |= f[nt][e] != 1.f;
      a.m[nt][e] = m;
      ref[nt][e] = (m == -INFINITY ? 0.f : m) - 14.f;
    }
  if (__any_sync(0xffffffffu, move)) {
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt) {
      a.l[nt][0] *= f[nt][0];
      a.l[nt][1] *= f[nt][1];
#pragma unroll
      for (int i = 0; i < 2 * C::GR; ++i) {
        const float moved = pow2(byte_of(was, i / 2) - byte_of(E, i / 2));
#pragma unroll
        for (int e = 0; e < 4; ++e) a.O[i][nt][e] *= f[nt][e & 1] * moved;
      }
    }
  }
#pragma unroll
  for (int mt = 0; mt < C::MH; ++mt)
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 4; ++e) S[mt][nt][e] = ex2(fmaf(S[mt][nt][e], cf[nt][e & 1], -ref[nt][e & 1]));
      a.l[nt][0] += S[mt][nt][0] + S[mt][nt][2];
      a.l[nt][1] += S[mt][nt][1] + S[mt][nt][3];
    }

#pragma unroll
  for (int mt = 0; mt < C::MH; ++mt) {
    const uint8_t* u = st + mt * U::kBytes;
    uint32_t xy[2][2][C::GR / 2];   // [8-token block][even or odd channel]: bytes of token pairs
    uint32_t vs[2][C::GR];          // [8-token block]: scales of the tokens 2 t, 2 t + 1
    uint32_t pk[2][C::NT][C::PARTS];   // transposed weights of a block
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const uint8_t* at = u + U::val_half(8 * b + 2 * t, 0, g);
      uint32_t w[C::GR];
      const uint8_t* sc = vtab + (mt * 8 + 4 * b + t) * C::GR * 4;
      if constexpr (C::GR == 4) {
        const uint4 x = *reinterpret_cast<const uint4*>(at);
        w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
        if constexpr (!kCareful) {
          const uint4 f = *reinterpret_cast<const uint4*>(sc);
          vs[b][0] = f.x; vs[b][1] = f.y; vs[b][2] = f.z; vs[b][3] = f.w;
        }
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(at);
        w[0] = x.x; w[1] = x.y;
        if constexpr (!kCareful) {
          const uint2 f = *reinterpret_cast<const uint2*>(sc);
          vs[b][0] = f.x; vs[b][1] = f.y;
        }
      }
#pragma unroll
      for (int i = 0; i < C::GR / 2; ++i) {
        const uint32_t A = w[i], B = w[C::GR / 2 + i];
        xy[b][0][i] = (A & 0x0f0f0f0fu) | ((B << 4) & 0xf0f0f0f0u);
        xy[b][1][i] = ((A >> 4) & 0x0f0f0f0fu) | (B & 0xf0f0f0f0u);
      }
      if constexpr (!kCareful) {
#pragma unroll
        for (int nt = 0; nt < C::NT; ++nt) {
          const float p0 = S[mt][nt][2 * b], p1 = S[mt][nt][2 * b + 1];
          const uint32_t hi = pack(p0, p1);
          pk[b][nt][0] = transpose8x8(hi);
          if constexpr (C::PARTS == 2) pk[b][nt][C::PARTS - 1] = transpose8x8(pack_rest(p0, p1, hi));
        }
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
#pragma unroll
        for (int nt = 0; nt < C::NT; ++nt) {
          uint32_t b[2][C::PARTS];
          if constexpr (!kCareful) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
              for (int part = 0; part < C::PARTS; ++part) b[hf][part] = mul2(pk[hf][nt][part], vs[hf][j]);
          } else {
            const uint32_t* vw = reinterpret_cast<const uint32_t*>(vtab) + mt * kUnit;
            const int ej = byte_of(E, j);
            const float to_e = __uint_as_float(ej < 254 ? (uint32_t)(254 - ej) << 23 : 0x00400000u);   // 2^(127 - E)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {   // the token of this lane's two weights
              const float sc = scale_at<true>(vw[g + 8 * hf], j) * to_e;
              const float p0 = S[mt][nt][2 * hf], p1 = S[mt][nt][2 * hf + 1];
              // a token that a row does not see adds nothing to it, whatever its values are; one that it sees makes it NaN
              // where they are, also with a weight of 0
              const int2 lim = lims[4 * nt];
              const int tok = tok0 + mt * kUnit + g + 8 * hf;
              const float w0 = tok > lim.x ? 0.f : p0 * sc, w1 = tok > lim.y ? 0.f : p1 * sc;
              const uint32_t hi = pack(w0, w1);
              b[hf][0] = transpose8x8(hi);
              if constexpr (C::PARTS == 2) b[hf][C::PARTS - 1] = transpose8x8(pack_rest(w0, w1, hi));
            }
          }
#pragma unroll
          for (int d = 0; d < 2; ++d) {
            const uint32_t a0 = x0[2 * k + d], a1 = y0[2 * k + d], a2 = x1[2 * k + d], a3 = y1[2 * k + d];
            float(&o)[4] = a.O[2 * j + d][nt];
            if constexpr (C::PARTS == 1) {
              mma16816(o, a0, a1, a2, a3, b[0][0], b[1][0]);
            } else {   // the instruction's sum cuts off: over thousands of units that would show in fp32
              float c[4];
              mma16816_first(c, a0, a1, a2, a3, b[0][C::PARTS - 1], b[1][C::PARTS - 1]);
              mma16816(c, a0, a1, a2, a3, b[0][0], b[1][0]);
#pragma unroll
              for (int e = 0; e < 4; ++e) o[e] += c[e];
            }
          }
        }
      }
    }
  }
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
  uint8_t* tab = sm + C::oTab + warp * C::kTab;
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::oBar) + warp * C::STAGES;
  int64_t* sums = reinterpret_cast<int64_t*>(sm + C::oSum);
  const int G = p.Hq / p.Hkv;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- the line: the room of every sequence's segments, a range of sequences per warp
  const int per = (p.N + C::W - 1) / C::W;
  const int na = min(warp * per, p.N), nb = min(na + per, p.N);
  bool bad = false;
  int64_t mine = 0, segs = 0;
  for (int n = na + lane; n < nb; n += 32) {
    const Work s = work_of<C>(p, n, &bad);
    mine += (int64_t)(C::HEAD + s.tiles) * s.rts;
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
  const bool wide = sums[C::W] <= kFewSegments;   // a CTA is one worker
  // The line's length and its workers, from sums that no warp writes any more.  Called again where a segment outlasts
  // the worker's part (hence volatile): fewer registers in the loop.
  auto whole_line = [&](int64_t& total, int64_t& workers) {
    const volatile int64_t* v = sums;
    total = 0;
    for (int w = 0; w < C::W; ++w) total += v[w];
    workers = min(wide ? (int64_t)gridDim.x : (int64_t)gridDim.x * C::W, total);
  };
  int64_t total, workers;
  whole_line(total, workers);
  const int64_t me = wide ? blockIdx.x : (int64_t)blockIdx.x * C::W + warp;
  // every entry of the owner table is written: a wide grid's workers have the first ones
  int4* own_at = parts.owner + (wide ? (int64_t)warp * gridDim.x + blockIdx.x : me);
  if (me >= workers) {   // nothing to do (in a wide grid, for the whole CTA)
    if (lane == 0) *own_at = make_int4(0, 0, 0, 0);
    return;
  }
  const int64_t x0 = me * total / workers;

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
        c = (int64_t)(C::HEAD + s.tiles) * s.rts * p.Hkv;
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
        cur.seg = (int)((x0 - before) / (C::HEAD + cur.s.tiles));
        cur.pos = (int)((x0 - before) % (C::HEAD + cur.s.tiles));
        break;
      }
      at += __shfl_sync(0xffffffffu, inc, 31);
    }
    cur.left = (me + 1) * total / workers - x0;
  }
  const int wi = wide ? warp : 0, step = wide ? C::W : 1;

  // ---- the ring
  Cursor<C> pc = cur;   // what to fetch next
  int pk = wi;          // tile of its piece
  uint32_t issued = 0, used = 0;
  bool ok = true;
  const uint32_t upp = p.page_size / kUnit;
  const bool in_page = upp % C::MT == 0;                    // a tile lies in one page
  auto produce = [&]() {
    while (pc.left > 0 && pc.first() + pk >= pc.last()) {
      if (wide) return;   // the next piece's tiles follow once this one's result is joined
      pc.next(p);
      pk = wi;
    }
    if (pc.left <= 0) return;
    const int tile = pc.first() + pk;
    pk += step;
    const int slot = issued % C::STAGES;
    ++issued;
    const int units = units_of_tile(pc.s.L, tile, C::MT);   // 0 for an empty sequence
    if (lane == 0) tc::mbar_arrive_expect_tx(full + slot, units * U::kBytes);
    __syncwarp();
    if (lane < (in_page ? min(units, 1) : units)) {
      const uint32_t unit = tile * C::MT + lane, at = page_of_unit(unit, p.upp_inv);
      int64_t page = p.table[(int64_t)pc.n * p.max_pages + at];
      if (page < 0 || page >= p.num_pages) {
        report_bad(p.dev_err);
        page = 0;
      }
      const int h = pc.seg / pc.s.rts;
      bulk_g2s(tc::smem_u32(ring + slot * C::kStage + lane * U::kBytes),
               p.cache + ((page * p.Hkv + h) * upp + (unit - at * upp)) * U::kBytes, (in_page ? units : 1) * U::kBytes, full + slot);
    }
  };
  for (int i = 0; i < C::STAGES; ++i) produce();

  int4 owner = make_int4(0, 0, 0, 0);
  bool joined = false;
  for (; cur.left > 0; cur.next(p)) {
    const int first = cur.first(), last = cur.last(), rt = cur.seg % cur.s.rts, h = cur.seg / cur.s.rts;
    if (first == last) continue;   // the part ends in the room before the segment's first tile
    const int rows = min(C::R, cur.s.qn * G - rt * C::R);
    if (wide && joined) {   // the ring was used to join the last piece
      pc = cur;
      pk = wi;
      for (int i = 0; i < C::STAGES; ++i) produce();
    }

    // q rows as operands, each scaled by a power of two
    uint32_t qr[C::QREG ? C::NT : 1][C::QREG ? C::KS : 1][2];
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
        if (r < rows && cur.s.L > 0) {
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
      const float down = __uint_as_float((ex - 14u) << 23) * fabsf(p.sm_scale) * kLog2e;
      if (t == 0) {
        reinterpret_cast<float*>(tab + C::tRow)[r] = down;
        const int rr = rt * C::R + r, tok = rr / G;
        reinterpret_cast<int*>(tab + C::tRow + C::R * 4)[r] = r < rows ? cur.s.L - cur.s.qn + tok : -1;
        reinterpret_cast<int*>(tab + C::tRow + C::R * 8)[r] = (cur.s.q0 + tok) * p.Hq + h * G + (rr - tok * G);   // below T Hq
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
        a.l[nt][e] = 0.f;
#pragma unroll
        for (int i = 0; i < 2 * C::GR; ++i) a.O[i][nt][e] = a.O[i][nt][e + 2] = 0.f;
      }
    uint32_t E = kLeastE * kOnes<C>;
    for (int tile = first + wi; tile < last; tile += step) {
      const int slot = used % C::STAGES, tok0 = tile * C::TILE;
      const uint8_t* st = ring + slot * C::kStage;
      if (ok) ok = __all_sync(0xffffffffu, tc::mbar_wait(full + slot, (used / C::STAGES) & 1, kWaitLimit));
      ++used;
      if (ok && cur.s.L > 0) {
        uint32_t was = E;
        const bool fresh = tile == first + wi;
        const bool careful = load_scales<C>(st, tab, cur.s.L - tok0, fresh, E);
        if (fresh) was = E;
#pragma unroll 1
        for (int u = 0; u < C::MT && tok0 + u * kUnit < cur.s.L; u += C::MH) {
          const uint8_t* su = st + u * U::kBytes;
          const float* ktab = reinterpret_cast<const float*>(tab) + u * kUnit * C::GR;
          // (bytes of two tokens as one word each in the careful step, a pair of fp16 per group else)
          const uint8_t* vtab = tab + C::tV + u * (careful ? kUnit * 4 : 8 * C::GR * 4);
          const int tok = tok0 + u * kUnit;
          const bool cut = tok + C::MH * kUnit - 1 > lim_all;
          if (careful) tile_step<C, true>(su, ktab, vtab, tab + C::tRow, qr, qs, tok, cut, E, was, a);
          else tile_step<C, false>(su, ktab, vtab, tab + C::tRow, qr, qs, tok, cut, E, was, a);
          was = E;
        }
      }
      __syncwarp();
      if (ok) produce();
    }
    // The groups' outputs, and each column's sum and reference, on one scale 2^Eo: O / l is the output.  The largest
    // group's, but at least 2^-27, where l 2^-Eo fits, and at most 2^63, where groups of 2^-63 keep their bits (the largest's
    // sums, 2^49 at most, fit all the same).
    int Eo = 0;
#pragma unroll
    for (int j = 0; j < C::GR; ++j) Eo = max(Eo, byte_of(E, j));
    Eo = min(max(Eo, 100), 190);
    if (E != Eo * kOnes<C>) {
#pragma unroll
      for (int i = 0; i < 2 * C::GR; ++i) {
        const float to = pow2(byte_of(E, i / 2) - Eo);
#pragma unroll
        for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) a.O[i][nt][e] *= to;
      }
    }
    float ref[C::NT][2];
    const float to_o = pow2(127 - Eo);
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float& l = a.l[nt][e];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        l *= to_o;
        ref[nt][e] = (a.m[nt][e] == -INFINITY ? 0.f : a.m[nt][e]) + (float)(Eo - 141);
      }

    // ---- the piece's result
    const bool starts = first == 0, whole = starts && last == cur.s.tiles;
    const int64_t slot = 2 * me + (starts ? 1 : 0);
    if (starts && !whole) {   // this worker's last piece; who has the rest of the segment?
      int64_t all, cut;
      whole_line(all, cut);
      const int64_t y = (me + 1) * all / cut - cur.left - cur.pos + C::HEAD + cur.s.tiles - 1;   // its last tile on the line
      owner = make_int4(cur.s.q0, h * 64 + rows, rt * C::R, (int)(((y + 1) * cut - 1) / all - me));
    }
    if (!wide) {
#pragma unroll
      for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = nt * 8 + 2 * t + e;
          if (c >= rows) continue;
          const int64_t row = reinterpret_cast<const int*>(tab + C::tRow + C::R * 8)[c];
          if (g == 0) {
            if (!whole) parts.ml[slot * C::R + c] = make_float2(ref[nt][e], a.l[nt][e]);
            else if (p.lse) p.lse[row] = lse_of(ref[nt][e], a.l[nt][e]);
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
          if (g == 0) mml[c] = make_float2(ref[nt][e], a.l[nt][e]);
#pragma unroll
          for (int j = 0; j < C::GR; ++j)
            *reinterpret_cast<float4*>(mo + c * C::D + 32 * j + 4 * g) =
                make_float4(a.O[2 * j][nt][e], a.O[2 * j][nt][e + 2], a.O[2 * j + 1][nt][e], a.O[2 * j + 1][nt][e + 2]);
        }
      __syncthreads();
      for (int i = threadIdx.x; i < rows * (C::D / 4); i += C::W * 32) {
        const int c = i / (C::D / 4), ch = (i % (C::D / 4)) * 4;
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
        const int64_t row = reinterpret_cast<const int*>(tab + C::tRow + C::R * 8)[c];   // (every warp's table has them)
        if (ch == 0) {
          if (!whole) parts.ml[slot * C::R + c] = make_float2(ref, l);
          else if (p.lse) p.lse[row] = lse_of(ref, l);
        }
        if (whole) write_row4<C, T>(p, row, ch, l, x);
        else *reinterpret_cast<float4*>(parts.o + (slot * C::R + c) * C::D + ch) = make_float4(x[0], x[1], x[2], x[3]);
      }
      tc::fence_proxy_async_smem();   // before the next piece's copies into the rings
      __syncthreads();
      joined = true;
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
// segment that begins in worker w and goes on in the next ones, a warp per row (half
// a warp for D = 64), in the order of the pieces, eight of them on their way at once.
constexpr int kJoinWarps = 8;
template <class C, typename T>
__global__ void __launch_bounds__(kJoinWarps * 32) kv4_join_kernel(const __grid_constant__ AttnProblem p, const Parts parts) {
  constexpr int kLanes = C::D / 4, kAtOnce = 8;   // lanes of a row; pieces
  const int64_t w = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 own = parts.owner[w];
  if (own.w == 0) return;
  const int G = p.Hq / p.Hkv, h = own.y >> 6, rows = own.y & 63, ch = (threadIdx.x % kLanes) * 4;
  for (int c = threadIdx.x / kLanes; c < rows; c += kJoinWarps * 32 / kLanes) {
    float ref = -INFINITY, l = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
    for (int i0 = 0; i0 <= own.w; i0 += kAtOnce) {
      float2 y[kAtOnce];
      float4 v[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int64_t slot = (i0 + i == 0 ? 2 * w + 1 : 2 * (w + i0 + i)) * C::R + c;
        const bool in = i0 + i <= own.w;
        y[i] = in ? __ldcg(parts.ml + slot) : make_float2(0.f, 0.f);
        v[i] = in ? __ldcg(reinterpret_cast<const float4*>(parts.o + slot * C::D + ch)) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float top = ref;
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i)
        if (y[i].y != 0.f) top = fmaxf(top, y[i].x);
      const float back = ref == -INFINITY ? 1.f : ex2(ref - top);   // nothing to bring along from before the first weight
      ref = top;
      l *= back;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] *= back;
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        if (y[i].y == 0.f) continue;   // (a NaN is not)
        const float f = ex2(y[i].x - ref);
        l = fmaf(y[i].y, f, l);
        x[0] = fmaf(v[i].x, f, x[0]); x[1] = fmaf(v[i].y, f, x[1]); x[2] = fmaf(v[i].z, f, x[2]); x[3] = fmaf(v[i].w, f, x[3]);
      }
    }
    const int rr = own.z + c;
    const int64_t row = ((int64_t)own.x + rr / G) * p.Hq + h * G + rr % G;
    if (ch == 0 && p.lse) p.lse[row] = lse_of(ref, l);
    write_row4<C, T>(p, row, ch, l, x);
  }
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
  cfg.blockDim = dim3(kJoinWarps * 32, 1, 1);
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

// Calls f with the instance for these sizes: one block of eight rows, or two, of which a
// segment with more rows takes several.  (Three and four blocks at once were built: their
// accumulators leave too few registers, 20 rows over 8,191 tokens 66 us against 50.)
template <typename F>
auto with_cfg(int32_t Hq, int32_t Hkv, int32_t D, int32_t max_q, kda_dtype dt, F f) {
  const bool one = (int64_t)max_q * (Hq / Hkv) <= 8;
  if (dt == KDA_F32) {
    if (D == 128) return one ? f(Cfg<128, 1, 2>{}, float{}) : f(Cfg<128, 2, 2>{}, float{});
    return one ? f(Cfg<64, 1, 2>{}, float{}) : f(Cfg<64, 2, 2>{}, float{});
  }
  const __nv_bfloat16 z{};
  if (D == 128) return one ? f(Cfg<128, 1, 1>{}, z) : f(Cfg<128, 2, 1>{}, z);
  return one ? f(Cfg<64, 1, 1>{}, z) : f(Cfg<64, 2, 1>{}, z);
}

// Whether the tiled kernel takes the call (bf16).  The host does not know the lengths, so the
// rule takes the sequences to be alike in cached and in query tokens: both kernels' times then
// grow with the cached tokens alike.  Per 1,024 cached tokens the cut line takes about
// 0.074 us for each 32 rows of a key/value head, on the whole GPU; the tiled kernel 18 us
// a wave of 152 CTAs of up to 128 rows, 22 us of up to 256.  Measured over 16,384 cached tokens
// (line / tiled, us): 8 sequences of 8 heads with 64 rows 171 / 285, 128 rows 319 / 288,
// 512 rows 1,216 / 360; one sequence of 8 heads with 256 rows 99 / 346; 8 of 2 heads with
// 512 rows 316 / 353, 1,024 rows 616 / 354.  Up to 24 rows the line is far ahead (16 rows:
// 66 / 279).  Where the sequences are not alike it may choose the slower one, and either kernel
// may be slower than two calls (32 query on 8 key heads, line / tiled): 2,048 tokens over 4,096 beside
// 31 single ones over up to 32,000 729 / 709, chosen tiled, and apart 152 (tiled) + 76 (line); beside
// 255 single ones 1,425 / 3,471, chosen line, and apart 152 + 488; 64 sequences of 16 tokens of
// 64 on 8 heads, one over 131,072 and the others over 2,048, 639 / 2,175, chosen tiled (all over 4,064:
// 634 / 320).  KDA_KV4_TILED=0 or =1 forces a kernel for bf16 calls.
bool extend_rows(const AttnProblem& p) {
  const int64_t G = p.Hq / p.Hkv, rows = (int64_t)p.max_q * G;
  if (p.dt != KDA_BF16 || (rows + 255) / 256 * p.N * p.Hkv > INT32_MAX) return false;
  const int64_t work = p.Hkv * std::max<int64_t>(p.N, (p.T * G + 31) / 32);
  const int64_t waves = (p.Hkv * std::max<int64_t>(p.N, (p.T * G + 255) / 256) + kCtas - 1) / kCtas;
  bool tiled = rows > 24 && work > (rows > 128 ? 297 : 243) * waves;
  if (const char* env = std::getenv("KDA_KV4_TILED")) tiled = std::atoi(env) != 0;
  return tiled;
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
