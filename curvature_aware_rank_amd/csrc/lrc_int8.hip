// Matrix products in 8-bit integers: the per-token quantiser, the linear layer and the gated projections.
//
// A token is held as x_k = s q_k with s = fl32(max|x| / 127), a weight's output channel likewise, so
//   z = s_t w_n sum_k q_tk p_nk:  the integer sum is exact (below 2^31 for fewer than 2^17 input channels),
// and scales, bias, activation, residual or the gate's product are applied to it in the epilogue.
#include "lrc_pair.h"

namespace lrc {
namespace {

constexpr int QT = 256;

// ---- the quantiser --------------------------------------------------------------------
// A token in registers, read once (wider ones: two passes).  Bound by memory: 65536 x 4096 bf16 161 us (5.0 TB/s), what a
// copy reaches; 8192 x 4096 22.5 in a row of its own calls, 24.1 on inputs that no cache holds (4.2 TB/s, the launch's
// start and end are 4 of it), 28 to 34 traced behind a product; 32 tokens 4.0, a launch.  `dq`: columns written,
// zeros behind the d that exist.
template <class T, int WPR, int V>
__global__ __launch_bounds__(row_threads(WPR)) void quantize_tokens_kernel(const T* __restrict__ x, int64_t ldx,
                                                                           int64_t n, int d, int8_t* __restrict__ q,
                                                                           int64_t ldq, int dq,
                                                                           float* __restrict__ scale,
                                                                           int32_t* __restrict__ info) {
  using S = RowShape<T, WPR, V>;
  __shared__ uint32_t red[2][WPR > 1 ? S::GROUPS * WPR : 1];
  const int lane = threadIdx.x & 63, group = threadIdx.x / S::LANES, l = threadIdx.x % S::LANES;
  const int64_t step = int64_t(gridDim.x) * S::GROUPS;
  int64_t t = int64_t(blockIdx.x) * S::GROUPS + group;
  RawRow<T, WPR, V> raw;
  raw.load(x + t * ldx, d, l, t < n);
  bool bad = false;
  int slot = 0;
  for (int64_t t0 = int64_t(blockIdx.x) * S::GROUPS; t0 < n; t0 += step, t += step, slot ^= 1) {
    float v[V][8];
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < V; ++k) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[k][e] = raw.at(8 * k + e);
      m = mag8(v[k], m, bad);
    }
    raw.load(x + (t + step) * ldx, d, l, t + step < n);
    const float s = token_step(row_max<WPR>(m, red[slot], l >> 6, lane, group));
    if (t >= n) continue;
    if (l == 0) scale[t] = s;
    const float inv = token_inverse(s);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c = (k * S::LANES + l) * 8;
      if (c < dq) st8_token_codes(q + t * ldq + c, dq - c, v[k], s, inv, bad);
    }
  }
  if (info != nullptr && bad) *info = LRC_ENONFINITE;
}
template <class T>
__global__ __launch_bounds__(QT) void quantize_wide_kernel(const T* __restrict__ x, int64_t ldx, int d,
                                                           int8_t* __restrict__ q, int64_t ldq, int dq,
                                                           float* __restrict__ scale, int32_t* __restrict__ info) {
  __shared__ uint32_t red[4];
  const int64_t t = blockIdx.x;
  uint32_t m = 0;
  bool bad = false;
  float v[8];
  for (int c = 8 * threadIdx.x; c < d; c += 8 * QT) {
    ld8(x + t * ldx + c, d - c, v);
    m = mag8(v, m, bad);
  }
  const float s = token_step(row_max<4>(m, red, threadIdx.x >> 6, threadIdx.x & 63, 0));
  const float inv = token_inverse(s);
  if (threadIdx.x == 0) scale[t] = s;
  for (int c = 8 * threadIdx.x; c < dq; c += 8 * QT) {
    ld8(x + t * ldx + c, d - c, v);
    st8_token_codes(q + t * ldq + c, dq - c, v, s, inv, bad);
  }
  if (info != nullptr && bad) *info = LRC_ENONFINITE;
}

template <class T>
lrc_status quantize(hipStream_t st, const T* x, int64_t n, int64_t d, int64_t ldx, int8_t* q, int64_t ldq, int64_t dq,
                    float* scale, int32_t* info) {
  ProfScope scope("quantize_tokens_kernel", st, 3.0 * double(n) * double(d), double(n) * double(d) * (sizeof(T) + 1));
  if (d > ROW_MAX) {
    quantize_wide_kernel<T><<<unsigned(n), QT, 0, st>>>(x, ldx, int(d), q, ldq, int(dq), scale, info);
    LRC_LAUNCHED();
    return LRC_OK;
  }
  return with_any_row_shape(d, [&](auto w, auto v) -> lrc_status {
    constexpr int WPR = decltype(w)::value, V = decltype(v)::value;
    using S = RowShape<T, WPR, V>;
    const unsigned grid = unsigned(std::min<int64_t>(cdiv(n, S::GROUPS), 2048 / std::max(1, WPR / 4)));
    quantize_tokens_kernel<T, WPR, V><<<grid, S::THREADS, 0, st>>>(x, ldx, n, int(d), q, ldq, int(dq), scale, info);
    LRC_LAUNCHED();
    return LRC_OK;
  });
}

// ---- operands ---------------------------------------------------------------------------
// Rows of int8 with a pitch of whole 16-byte pieces, zeros behind the columns.  16 bytes per thread.
struct PitchJob {
  const int8_t* p = nullptr;
  int8_t* out = nullptr;
  int64_t ld = 0, rows = 0, blocks = 0;
};
__global__ __launch_bounds__(QT) void pitch_kernel(PitchJob a, PitchJob b, PitchJob c, int cols, int pieces) {
  int64_t block = blockIdx.x;
  PitchJob j = a;
  if (block >= a.blocks) {
    block -= a.blocks;
    j = b;
    if (block >= b.blocks) {
      block -= b.blocks;
      j = c;
    }
  }
  const int64_t i = block * QT + threadIdx.x, r = i / pieces;
  const int g = int(i % pieces) * 16;
  if (r >= j.rows) return;
  const gemm::u32x4 v = gemm::row_piece(reinterpret_cast<const uint8_t*>(j.p) + r * j.ld + g, cols - g);
  *reinterpret_cast<gemm::u32x4*>(j.out + r * int64_t(pieces) * 16 + g) = v;
}

constexpr int64_t KMAX = int64_t(1) << 17;    // input channels stay below: |sum| < 2^31 for codes of any value
constexpr int64_t NMAX = int64_t(1) << 24;
int64_t round16(int64_t v) { return (v + 15) & ~int64_t(15); }

bool sizes_ok(int64_t n, int64_t i, int64_t o) {
  return n >= 0 && n < (int64_t(1) << 31) && i >= 1 && i < KMAX && o >= 1 && o <= NMAX;
}

struct Int8Room {
  int8_t *x = nullptr, *w0 = nullptr, *w1 = nullptr;
  float *scale = nullptr, *partial = nullptr;
  size_t bytes = 0;
};
Int8Room int8_room(void* ws, int64_t n, int64_t di, int64_t dn, bool pair) {
  Int8Room r;
  Carve cv(ws);
  const int64_t k = round16(di);
  r.x = cv.take<int8_t>(size_t(n) * k);
  r.scale = cv.take<float>(size_t(n));
  if (!gemm::stream_int8(n, dn, di, pair)) {
    if (di % 16 != 0) {
      r.w0 = cv.take<int8_t>(size_t(dn) * k);
      if (pair) r.w1 = cv.take<int8_t>(size_t(dn) * k);
    }
    r.partial = cv.take<float>(gemm::rows_workspace(n, dn, k / 2, pair) / 4);
  }
  r.bytes = cv.bytes();
  return r;
}

struct Int8Args {
  const void* x;
  int64_t ldx;
  const int8_t* xq;
  int64_t ldxq;
  const float* xs;
  int64_t n, di, dn;
  const int8_t* w[2];
  int64_t ldw[2];
  const float* ws[2];
  Epilogue ep;
};

// A row that the tiles read where it lies: whole 16-byte pieces, a pitch their offsets hold.
bool in_place(const int8_t* p, int64_t ld) { return rows_vec16(p, ld, 1) && ld <= 2 * GEMM_MAX_LD; }

template <class T, bool PAIR>
lrc_status int8_product(hipStream_t st, const Int8Args& a, void* ws, int32_t* info) {
  const Int8Room room = int8_room(ws, a.n, a.di, a.dn, PAIR);
  const int64_t k = round16(a.di);
  const int8_t* xq = a.xq;
  int64_t ldx = a.ldxq;
  gemm::Companion co;
  co.row_scale = a.xs;
  co.col_scale = a.ws[0];
  co.col_scale2 = a.ws[1];
  constexpr int W = PAIR ? 2 : 1;
  const double flops = 2.0 * W * double(a.n) * double(a.dn) * double(a.di);
  const double bytes = double(a.n) * a.di + W * double(a.dn) * a.di + double(sizeof(T)) * double(a.n) * a.dn;
  auto few = [&](const void* x, int64_t ld, bool own) {
    Epilogue ep = a.ep;
    ep.info = own ? info : nullptr;
    return gemm::few_rows<T, INT8, W>(st, "int8_rows_kernel", x, ld, own, a.w[0], a.ldw[0], a.w[1], a.ldw[1], a.n,
                                      a.dn, a.di, ep, co, flops, bytes);
  };
  const bool rows = gemm::stream_int8(a.n, a.dn, a.di, PAIR);
  if (rows && a.x != nullptr && gemm::own_tokens(a.n, a.dn, a.di)) return few(a.x, a.ldx, true);
  if (a.x != nullptr) {
    LRC_TRY(quantize(st, static_cast<const T*>(a.x), a.n, a.di, a.ldx, room.x, k, k, room.scale, info));
    xq = room.x;
    ldx = k;
    co.row_scale = room.scale;
  }
  if (rows) return few(xq, ldx, false);
  const int8_t* w[2] = {a.w[0], a.w[1]};
  int64_t ldw[2] = {a.ldw[0], a.ldw[1]};
  if (a.di % 16 != 0) {   // rows of no whole pieces are laid out anew
    const int64_t pieces = k / 16;
    PitchJob j[3];
    int count = 0;
    auto add = [&](const int8_t*& p, int64_t& ld, int64_t rows, int8_t* out) {
      j[count++] = {p, out, ld, rows, cdiv(rows * pieces, QT)};
      p = out;
      ld = k;
    };
    if (a.x == nullptr) add(xq, ldx, a.n, room.x);
    for (int i = 0; i < W; ++i) add(w[i], ldw[i], a.dn, i ? room.w1 : room.w0);
    const int64_t grid = j[0].blocks + j[1].blocks + j[2].blocks;
    if (grid >= (int64_t(1) << 31)) return LRC_EINVAL;
    ProfScope scope("int8_pitch_kernel", st, 0.0, 2.0 * double(a.di) * double(W * a.dn + (a.x ? 0 : a.n)));
    pitch_kernel<<<unsigned(grid), QT, 0, st>>>(j[0], j[1], j[2], int(a.di), int(pieces));
    LRC_LAUNCHED();
  }
  auto operand = [](const int8_t* p, int64_t ld) {
    return GemmOperand{reinterpret_cast<const uint16_t*>(p), ld / 2, 0};
  };
  if (PAIR) co.B = operand(w[1], ldw[1]);
  return gemm::rows_product<T, INT8, PAIR>(st, PAIR ? "int8_gated_kernel" : "int8_kernel", operand(xq, ldx),
                                           operand(w[0], ldw[0]), a.n, a.dn, k / 2, a.ep, co, room.partial, flops,
                                           bytes);
}

// what both calls check of x and the weights
template <class A>
lrc_status check(const A& a, int dt, int act, int weights, size_t need, void* ws, size_t ws_bytes) {
  if ((dt != LRC_F32 && dt != LRC_BF16) || act < LRC_ACT_NONE || act > LRC_ACT_SILU) return LRC_EDTYPE;
  if (!sizes_ok(a.n, a.di, a.dn) || a.ep.ldy < a.dn) return LRC_EINVAL;
  if ((a.x != nullptr && (a.ldx < a.di || a.xq != nullptr || a.xs != nullptr)) || (a.xq != nullptr && a.ldxq < a.di))
    return LRC_EINVAL;
  if ((a.xq == nullptr) != (a.xs == nullptr)) return LRC_EINVAL;
  for (int i = 0; i < weights; ++i)
    if (a.ldw[i] < a.di) return LRC_EINVAL;
  if (a.n == 0) return LRC_OK;
  if ((a.x == nullptr && a.xq == nullptr) || a.ep.y == nullptr) return LRC_EINVAL;
  for (int i = 0; i < weights; ++i)
    if (a.w[i] == nullptr || a.ws[i] == nullptr) return LRC_EINVAL;
  if (a.di % 16 == 0) {   // the tiles read these where they lie
    if (a.xq != nullptr && !in_place(a.xq, a.ldxq)) return LRC_EINVAL;
    for (int i = 0; i < weights; ++i)
      if (!in_place(a.w[i], a.ldw[i])) return LRC_EINVAL;
  }
  return ws_bytes < need || (need > 0 && ws == nullptr) ? LRC_EWORKSPACE : LRC_OK;
}

}  // namespace
}  // namespace lrc

using namespace lrc;

extern "C" lrc_status lrc_quantize_tokens(const void* x, lrc_dtype dt, int64_t n_tokens, int64_t d, int64_t ldx,
                                          int8_t* q, int64_t ldq, float* scale, int32_t* info, void* stream) {
  if (dt != LRC_F32 && dt != LRC_BF16) return LRC_EDTYPE;
  if (!sizes_ok(n_tokens, 1, d) || ldx < d || ldq < d) return LRC_EINVAL;
  if (n_tokens == 0) return LRC_OK;
  if (x == nullptr || q == nullptr || scale == nullptr) return LRC_EINVAL;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (dt == LRC_BF16) return quantize(st, static_cast<const uint16_t*>(x), n_tokens, d, ldx, q, ldq, d, scale, info);
  return quantize(st, static_cast<const float*>(x), n_tokens, d, ldx, q, ldq, d, scale, info);
}

extern "C" size_t lrc_int8_linear_workspace(int64_t n_tokens, int64_t d_in, int64_t d_out) {
  return sizes_ok(n_tokens, d_in, d_out) ? int8_room(nullptr, n_tokens, d_in, d_out, false).bytes : 0;
}

extern "C" lrc_status lrc_int8_linear(const void* x, lrc_dtype dt, int64_t n_tokens, int64_t d_in, int64_t d_out,
                                      int64_t ldx, const int8_t* xcodes, int64_t ldxc, const float* xscale,
                                      const int8_t* W, int64_t ldw, const float* wscale, const float* bias,
                                      lrc_act act, const void* residual, int64_t ldr, void* y, int64_t ldy,
                                      int32_t* info, void* ws, size_t ws_bytes, void* stream) {
  Int8Args a = {x, ldx, xcodes, ldxc, xscale, n_tokens, d_in, d_out, {W, nullptr}, {ldw, 0}, {wscale, nullptr}, {}};
  a.ep.bias = bias;
  a.ep.act = act;
  a.ep.res = residual;
  a.ep.ldr = ldr;
  a.ep.y = y;
  a.ep.ldy = ldy;
  if (residual != nullptr && ldr < d_out) return LRC_EINVAL;
  const size_t need = lrc_int8_linear_workspace(n_tokens, d_in, d_out);
  LRC_TRY(check(a, dt, act, 1, need, ws, ws_bytes));
  if (n_tokens == 0) return LRC_OK;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return dt == LRC_BF16 ? int8_product<uint16_t, false>(st, a, ws, info) : int8_product<float, false>(st, a, ws, info);
}

extern "C" size_t lrc_int8_gated_linear_workspace(int64_t n_tokens, int64_t d_in, int64_t d_ff) {
  return sizes_ok(n_tokens, d_in, d_ff) ? int8_room(nullptr, n_tokens, d_in, d_ff, true).bytes : 0;
}

extern "C" lrc_status lrc_int8_gated_linear(const void* x, lrc_dtype dt, int64_t n_tokens, int64_t d_in, int64_t d_ff,
                                            int64_t ldx, const int8_t* xcodes, int64_t ldxc, const float* xscale,
                                            const int8_t* Wg, int64_t ldwg, const float* gscale, const int8_t* Wu,
                                            int64_t ldwu, const float* uscale, lrc_act act, void* h, int64_t ldh,
                                            int32_t* info, void* ws, size_t ws_bytes, void* stream) {
  Int8Args a = {x, ldx, xcodes, ldxc, xscale, n_tokens, d_in, d_ff, {Wg, Wu}, {ldwg, ldwu}, {gscale, uscale}, {}};
  a.ep.act = act;
  a.ep.y = h;
  a.ep.ldy = ldh;
  const size_t need = lrc_int8_gated_linear_workspace(n_tokens, d_in, d_ff);
  LRC_TRY(check(a, dt, act, 2, need, ws, ws_bytes));
  if (n_tokens == 0) return LRC_OK;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return dt == LRC_BF16 ? int8_product<uint16_t, true>(st, a, ws, info) : int8_product<float, true>(st, a, ws, info);
}
