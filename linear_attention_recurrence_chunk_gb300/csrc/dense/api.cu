// C ABI of the dense half of a decoder layer: argument validation and dispatch.
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "internal.cuh"

namespace {

using kda::dense::kBlock;

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
bool dtype_ok(kda_dtype dt) { return dt == KDA_F32 || dt == KDA_BF16; }
int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }

constexpr int64_t kMost = (int64_t)INT32_MAX - 511;   // rows or columns
constexpr int64_t kMostK = (int64_t)1 << 27;           // (a tile's 2^20 K blocks end well inside a bounded wait)
constexpr int64_t kMostStride = (int64_t)1 << 37;     // elements (a tensor map's strides are below 2^40 bytes)

// Rows of a strided [rows][C] matrix (rows, C at least 1), its bytes from first to last.
Range span(const void* p, int64_t rows, int64_t C, int64_t stride, size_t eb) {
  return {p, (size_t)((rows - 1) * stride + C) * eb};
}
bool shape_ok(int64_t rows, int64_t C) {
  return rows >= 0 && C >= 0 && rows <= kMost && C <= kMost && (rows == 0 || C <= ((int64_t)1 << 42) / rows);
}
bool stride_ok(int64_t stride, int64_t C) { return stride >= C && stride <= kMostStride; }

// Heads of D values, T tokens of them: what a rotation reads of a part, or writes of it.
struct Heads {
  const void* p;
  int64_t t, h;   // strides in elements from token to token (T = 1: 0) and head to head (H = 1: 0)
  int32_t H;
  int64_t token(int32_t D) const { return (H - 1) * h + D; }
  Range bytes(int64_t T, int32_t D, size_t eb) const { return {p, H > 0 ? (size_t)((T - 1) * t + token(D)) * eb : 0}; }
};
// Whether two of these may have a value in common.  Parts whose bytes lie over one another are told apart as parts of one
// projection are: between one another's tokens (the same token stride), or heads (the same head stride, which divides the
// tokens').
bool share(const Heads& a, const Heads& b, int64_t T, int32_t D, size_t eb) {
  if (!overlaps(a.bytes(T, D, eb), b.bytes(T, D, eb))) return false;
  if (T > 1 && a.t != b.t) return true;
  const int64_t d = (int64_t)(reinterpret_cast<intptr_t>(b.p) - reinterpret_cast<intptr_t>(a.p)) / (int64_t)eb;
  const auto beside = [d](int64_t step, int64_t na, int64_t nb) {   // na and nb values of each `step`, d apart
    const int64_t r = step > 0 ? (d % step + step) % step : 0;
    return step > 0 && r >= na && r + nb <= step;
  };
  if (T > 1 && beside(a.t, a.token(D), b.token(D))) return false;
  const int64_t h = std::max(a.h, b.h);   // of one head: 0
  return !((a.H == 1 || a.h == h) && (b.H == 1 || b.h == h) && h > 0 && (T == 1 || a.t % h == 0) && beside(h, D, D));
}

kda_status done(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

// kda_fp8_matmul, by the cut that the sizes ask for or by a given one.
kda_status matmul(kda::dense::MatmulProblem p, const kda::dense::Cut* cut, cudaStream_t stream) {
  const int64_t M = p.M, N = p.N, K = p.K;
  if (!dtype_ok(p.dt) || M < 0 || N < 0 || K < 1) return KDA_ERR_INVALID_ARG;
  if (K % 16 != 0 || M > kMost || N > kMost || K > kMostK) return KDA_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return KDA_OK;
  const auto up16 = [](int64_t v) { return (v + 15) / 16 * 16; };
  if (M == 1) p.lda = K, p.ldo = N;   // a stride over one row has no meaning
  if (N == 1) p.ldw = up16(K);
  if (!p.a || !p.w || !p.sa || !p.sw || !p.out) return KDA_ERR_INVALID_ARG;
  if (!aligned(p.a, 16) || !aligned(p.w, 16) || !aligned(p.out, elem(p.dt)) || p.lda % 16 != 0 || p.ldw % 16 != 0) return KDA_ERR_INVALID_ARG;
  if (!stride_ok(p.lda, K) || !stride_ok(p.ldw, K) || !stride_ok(p.ldo, N)) return KDA_ERR_INVALID_ARG;
  const Range in[] = {span(p.a, M, K, p.lda, 1), span(p.w, N, K, p.ldw, 1), {p.sa, (size_t)(M * blocks_of(K))},
                      {p.sw, (size_t)(blocks_of(N) * blocks_of(K))}};
  const Range res[] = {span(p.out, M, N, p.ldo, elem(p.dt))};
  if (!apart(in, res)) return KDA_ERR_INVALID_ARG;
  if (cut) {
    const int r = cut->rows, s = cut->split;
    const bool is_few = (r == 16 || r == 32 || r == 64 || r == 128 || r == 256) && (s == 1 || s == 2 || s == 4 || s == 8);
    if (!(r == 0 && s == 1) && !(is_few && s <= (blocks_of(K) + 3) / 4)) return KDA_ERR_INVALID_ARG;
    if (!kda::dense::cut_fits(p, *cut)) return KDA_ERR_UNSUPPORTED;
  }
  if (kda::device_error_ptr(&p.dev_err) != cudaSuccess) return KDA_ERR_CUDA;
  return done(kda::dense::launch_matmul(p, cut, stream));
}

}  // namespace

extern "C" {

kda_status kda_fp8_quant(const void* x, int64_t x_stride, int64_t T, int64_t C, int32_t block_rows, kda_dtype dt, uint8_t* codes,
                         uint8_t* scales, cudaStream_t stream) {
  if (!dtype_ok(dt) || !shape_ok(T, C) || (block_rows != 1 && block_rows != kBlock)) return KDA_ERR_INVALID_ARG;
  if (T == 0 || C == 0) return KDA_OK;
  if (T == 1) x_stride = C;   // a stride over one row has no meaning
  if (!x || !codes || !scales || !aligned(x, elem(dt)) || !stride_ok(x_stride, C)) return KDA_ERR_INVALID_ARG;
  const int64_t srows = block_rows == 1 ? T : blocks_of(T);
  const Range in[] = {span(x, T, C, x_stride, elem(dt))};
  const Range out[] = {{codes, (size_t)(T * C)}, {scales, (size_t)(srows * blocks_of(C))}};
  if (!apart(in, out)) return KDA_ERR_INVALID_ARG;
  return done(kda::dense::launch_quant({x, x_stride, T, C, block_rows, dt, codes, scales}, stream));
}

kda_status kda_fp8_values(const uint8_t* codes, const uint8_t* scales, int64_t T, int64_t C, int32_t block_rows, kda_dtype dt, void* y,
                          cudaStream_t stream) {
  if (!dtype_ok(dt) || !shape_ok(T, C) || (block_rows != 1 && block_rows != kBlock)) return KDA_ERR_INVALID_ARG;
  if (T == 0 || C == 0) return KDA_OK;
  if (!codes || !scales || !y || !aligned(y, elem(dt))) return KDA_ERR_INVALID_ARG;
  const int64_t srows = block_rows == 1 ? T : blocks_of(T);
  const Range in[] = {{codes, (size_t)(T * C)}, {scales, (size_t)(srows * blocks_of(C))}};
  const Range out[] = {{y, (size_t)(T * C) * elem(dt)}};
  if (!apart(in, out)) return KDA_ERR_INVALID_ARG;
  return done(kda::dense::launch_values({codes, scales, T, C, block_rows, dt, y}, stream));
}

kda_status kda_add_rmsnorm(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride, const float* weight, float eps,
                           int64_t T, int64_t C, kda_dtype dt, void* h, void* y, uint8_t* codes, uint8_t* scales, cudaStream_t stream) {
  if (!dtype_ok(dt) || !shape_ok(T, C) || !(eps >= 0.f) || isinf(eps)) return KDA_ERR_INVALID_ARG;
  if (C > kda::dense::kNormMost) return KDA_ERR_UNSUPPORTED;
  if (T == 0 || C == 0) return KDA_OK;
  if (T == 1) x_stride = residual_stride = C;
  const size_t eb = elem(dt);
  if (!x || !aligned(x, eb) || !stride_ok(x_stride, C) || !aligned(weight, 4)) return KDA_ERR_INVALID_ARG;
  if (residual && (!aligned(residual, eb) || !stride_ok(residual_stride, C))) return KDA_ERR_INVALID_ARG;
  if ((residual != nullptr) != (h != nullptr) || !aligned(h, eb)) return KDA_ERR_INVALID_ARG;
  if ((y != nullptr) == (codes != nullptr) || (codes != nullptr) != (scales != nullptr) || !aligned(y, eb)) return KDA_ERR_INVALID_ARG;
  const size_t n = (size_t)(T * C);
  const Range rx = span(x, T, C, x_stride, eb), rr = span(residual, T, C, residual_stride, eb), rw = {weight, (size_t)C * 4};
  const Range rh = {h, n * eb}, ry = {y, n * eb}, rc = {codes, n}, rs = {scales, (size_t)(T * blocks_of(C))};
  // h over x or the residual, y over x, row for row; else apart
  const bool x_dense = x_stride == C, r_dense = residual_stride == C;
  if (overlaps(rh, rx) && !(h == x && x_dense)) return KDA_ERR_INVALID_ARG;
  if (residual && overlaps(rh, rr) && !(h == residual && r_dense)) return KDA_ERR_INVALID_ARG;
  if (overlaps(ry, rx) && !(y == x && x_dense)) return KDA_ERR_INVALID_ARG;
  if (overlaps(rh, ry) || (residual && overlaps(ry, rr)) || overlaps(rh, rw) || overlaps(ry, rw)) return KDA_ERR_INVALID_ARG;
  const Range in[] = {rx, residual ? rr : Range{nullptr, 0}, rw, rh};
  const Range out[] = {rc, rs};
  if (!apart(in, out)) return KDA_ERR_INVALID_ARG;
  return done(kda::dense::launch_norm({x, x_stride, residual, residual_stride, weight, eps, T, C, dt, h, y, codes, scales}, stream));
}

kda_status kda_fp8_matmul(const uint8_t* a, int64_t a_stride, const uint8_t* a_scales, const uint8_t* w, int64_t w_stride,
                          const uint8_t* w_scales, int64_t M, int64_t N, int64_t K, kda_dtype dt, void* out, int64_t out_stride,
                          cudaStream_t stream) {
  return matmul({a, a_scales, w, w_scales, a_stride, w_stride, M, N, K, dt, out, out_stride, nullptr}, nullptr, stream);
}

kda_status kda_fp8_matmul_cut(const uint8_t* a, int64_t a_stride, const uint8_t* a_scales, const uint8_t* w, int64_t w_stride,
                              const uint8_t* w_scales, int64_t M, int64_t N, int64_t K, kda_dtype dt, void* out, int64_t out_stride,
                              int32_t rows, int32_t split, int32_t deep, cudaStream_t stream) {
  const kda::dense::Cut cut{rows, split, deep != 0};
  return matmul({a, a_scales, w, w_scales, a_stride, w_stride, M, N, K, dt, out, out_stride, nullptr}, &cut, stream);
}

kda_status kda_fp8_matmul_choice(int64_t M, int64_t N, int64_t K, kda_dtype dt, int32_t sms, int32_t* cut) {
  if (!dtype_ok(dt) || M < 1 || N < 1 || K < 16 || M > kMost || N > kMost || K > kMostK || sms < 2 || !cut) return KDA_ERR_INVALID_ARG;
  const kda::dense::Cut c = kda::dense::choose_cut({nullptr, nullptr, nullptr, nullptr, K, K, M, N, K, dt, nullptr, N, nullptr}, sms);
  cut[0] = c.rows, cut[1] = c.split, cut[2] = c.deep;
  return KDA_OK;
}

kda_status kda_rotary(const void* q, int64_t q_token_stride, int64_t q_head_stride, int32_t Hq, const void* k, int64_t k_token_stride,
                      int64_t k_head_stride, int32_t Hk, const int32_t* positions, int64_t T, int32_t D, int32_t rot, const double* freqs,
                      float amplitude, int32_t flags, kda_dtype dt, void* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
                      void* k_out, int64_t k_out_token_stride, int64_t k_out_head_stride, cudaStream_t stream) {
  if (!dtype_ok(dt) || T < 0 || T > kMost || Hq < 0 || Hk < 0 || D < 1 || rot < 0 || rot > D || rot % 2 != 0 || !isfinite(amplitude) ||
      (flags & ~(KDA_ROTARY_INTERLEAVED | KDA_ROTARY_INVERSE)) != 0)
    return KDA_ERR_INVALID_ARG;
  if (D > 1024 || Hq > 1024 || Hk > 1024 || Hq + Hk > 1024) return KDA_ERR_UNSUPPORTED;
  if (T == 0 || Hq + Hk == 0) return KDA_OK;
  if (!positions || !aligned(positions, 4) || (rot > 0 && (!freqs || !aligned(freqs, 8)))) return KDA_ERR_INVALID_ARG;
  const size_t eb = elem(dt);
  kda::dense::RotaryPart part[2] = {{q, q_out, q_token_stride, q_head_stride, q_out_token_stride, q_out_head_stride, Hq},
                                    {k, k_out, k_token_stride, k_head_stride, k_out_token_stride, k_out_head_stride, Hk}};
  Heads in[2] = {}, out[2] = {};
  bool place[2] = {false, false};
  for (int i = 0; i < 2; ++i) {
    kda::dense::RotaryPart& p = part[i];
    if (p.H == 0) continue;
    if (T == 1) p.xt = p.yt = 0;
    if (p.H == 1) p.xh = p.yh = 0;
    if (!p.x || !p.y || !aligned(p.x, eb) || !aligned(p.y, eb)) return KDA_ERR_INVALID_ARG;
    const int64_t st[] = {p.xt, p.xh, p.yt, p.yh};
    for (int64_t s : st)
      if (s < 0 || s > kMostStride) return KDA_ERR_INVALID_ARG;
    // an output's heads and tokens do not lie over one another: the heads of a token side by side, or the tokens of a head
    if ((p.H > 1 && p.yh < D) || (T > 1 && p.yt < D)) return KDA_ERR_INVALID_ARG;
    if (p.H > 1 && T > 1 && p.yt < (p.H - 1) * p.yh + D && p.yh < (T - 1) * p.yt + D) return KDA_ERR_INVALID_ARG;
    in[i] = {p.x, p.xt, p.xh, p.H};
    out[i] = {p.y, p.yt, p.yh, p.H};
    place[i] = p.x == p.y && p.xt == p.yt && p.xh == p.yh;
  }
  const Range tables[] = {{positions, (size_t)T * 4}, {freqs, (size_t)rot / 2 * 8}};
  for (int i = 0; i < 2; ++i) {
    for (const Range& r : tables)
      if (overlaps(out[i].bytes(T, D, eb), r)) return KDA_ERR_INVALID_ARG;
    for (int j = 0; j < 2; ++j)
      if (!(i == j && place[i]) && share(out[i], in[j], T, D, eb)) return KDA_ERR_INVALID_ARG;
  }
  if (share(out[0], out[1], T, D, eb)) return KDA_ERR_INVALID_ARG;
  return done(kda::dense::launch_rotary({part[0], part[1], positions, freqs, T, D, rot, amplitude, flags, dt}, stream));
}

}  // extern "C"
