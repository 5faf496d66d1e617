// Gated feed-forward block: g = x Wg^T, u = x Wu^T, h = act(g) u, and its gradients from g and u kept in full or
// in 8 bits:
//   dg = dh u act'(g),  du = dh act(g),  dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x
//
// bf16 forward: one product whose tiles hold as many channels of Wg as of Wu (lrc_gemm_tile.h), so x is staged once
// for both and act(g) u is formed from the accumulators; g and u reach memory only where they are kept.
// (8192 x 4096 x 11008: forward 1180 us; backward dz 199 us, memory, 5.4 TB/s; dx, dWg and dWu 3650, 1220 TFLOP/s:
// the matrix pipes, busy 65 % of the cycles at 1.79 GHz.)
// bf16 backward: one pass writes dg and du (the output-gradient streams of the two projections) and what their
// rounding to bf16 left out; dx is one product whose k runs over dg Wg and then du Wu, dWg and dWu one each whose k
// runs over the tokens twice, the left-out piece first (a gradient so carries 16 bits of dz and no more than its own
// rounding); all three in one launch where their tiles are of one kind.  Sums fp32 throughout.  dx takes the streams
// as they are returned, as the linear layer's does: it is the gradient that belongs to them, and the left-out pieces
// would add a third to the products' time.  Its error is 1.4 times that of one rounding.
// Few tokens, both types: the weights are streamed once (lrc_pair.h).
// fp32 otherwise: the products are those of the linear layer (fp32 instructions, or six of bf16 pieces), each laying
// out x for itself, the gate an elementwise pass.  1024 x 4096 x 2 x 11008: forward 1450 us (products 2 x 604 of it,
// operands 2 x 76, gate 25), 128 TFLOP/s; backward 2500 (products 2 x 1107, operands 2 x 103, dz 46), 148 TFLOP/s; the
// library's fp32 product reaches 154 at 8192^3.
#include "lrc_operand.h"
#include "lrc_pair.h"

namespace lrc {
namespace {

constexpr int ET = 256;
constexpr int64_t WIDE = int64_t(1) << 20;       // channels (a tile's offsets hold their rows)

bool sizes_ok(int64_t n, int64_t i, int64_t f) {
  return n >= 0 && n < GEMM_MAX_K && i >= 1 && i <= WIDE && f >= 1 && f <= WIDE;
}

// ---- elementwise passes -------------------------------------------------------------------
// One 8-channel piece of one token per lane, eight lanes to a block of 64; bound by memory.
template <class T>
__global__ __launch_bounds__(ET) void gate_kernel(const T* __restrict__ g, const T* __restrict__ u, int64_t ldz,
                                                  int64_t n, int64_t d, int64_t blocks, Epilogue ep,
                                                  gemm::Companion co) {
  const int64_t i = (int64_t(blockIdx.x) * ET + threadIdx.x) >> 3;
  const int lane = threadIdx.x & 63;
  const int64_t row = i / blocks, col = i % blocks * CKB + 8 * (lane & 7);
  const int64_t left = row < n ? d - col : 0;
  const int cnt = int(left < 0 ? 0 : left > 8 ? 8 : left);
  float a[8], b[8];
  ld8(g + row * ldz + col, cnt, a);
  ld8(u + row * ldz + col, cnt, b);
  bool bad = false;
  gemm::finish_pair8<T>(ep, co, row, col, cnt, a, b, lane, bad);
  if (ep.info != nullptr && bad) *ep.info = LRC_ENONFINITE;
}

// a = act(z), s = act'(z) of eight values, z -> a
__device__ __forceinline__ void act_and_slope(int act, float (&z)[8], float (&s)[8]) {
  if (act == LRC_ACT_RELU) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      s[e] = relu_slope(z[e]);
      z[e] = relu(z[e]);
    }
  } else if (act == LRC_ACT_GELU) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float w;
      const float q = normal_tail(fabsf(z[e]), w), p = z[e] >= 0.f ? 1.f - q : q;
      s[e] = fmaf(z[e] * w, 0.39894228040143268f, p);
      z[e] *= p;
    }
  } else if (act == LRC_ACT_SILU) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float p = logistic(z[e]);
      s[e] = p * (1.f + z[e] * (1.f - p));
      z[e] *= p;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = 1.f;
  }
}

template <class T>
struct GatePass {
  const T *dh, *g, *u;
  int64_t lddh, ldz, n, d, nb, w8;
  const int8_t *gcodes, *gexps, *ucodes, *uexps;
  int act;
  T *dg, *du;              // packed
  uint16_t *pg, *pu;       // bf16 with rows of no whole pieces: copies of w8 columns, zeros behind the last
  uint16_t *lg, *lu;       // what the rounding left out, w8 columns
};
template <class T>
__device__ __forceinline__ void put_grad(T* o, uint16_t* copy, uint16_t* low, int64_t at, int64_t at8, int cnt,
                                         const float (&v)[8]) {
  st8(o + at, cnt, v);
  if (copy != nullptr) st8(copy + at8, 8, v);
  if (low != nullptr) {   // zeros where the stream is not finite
    float r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float h = round_to(v[e], static_cast<const uint16_t*>(nullptr));
      r[e] = finite_f(h) ? v[e] - h : 0.f;
    }
    st8(low + at8, 8, r);
  }
}
// The workgroups behind `blocks` lay out the products' other operands, so that those cost no launch of their own.
template <class T, bool CK>
__global__ __launch_bounds__(ET) void gated_dz_kernel(GatePass<T> p, int64_t blocks, OperandJobs jobs) {
  if (blockIdx.x >= blocks) {
    if constexpr (std::is_same<T, uint16_t>::value) lay_operand<T>(jobs, blockIdx.x - blocks, nullptr);
    return;
  }
  const int64_t i = int64_t(blockIdx.x) * ET + threadIdx.x, per = p.w8 / 8;
  const int64_t t = i / per, c = i % per * 8;
  if (t >= p.n) return;
  const int64_t left = p.d - c;
  const int cnt = int(left > 8 ? 8 : left);
  float dh[8], z[8], u[8], s[8];
  ld8(p.dh + t * p.lddh + c, cnt, dh);
  if (CK) {
    ld8_codes(p.gcodes + t * p.d + c, cnt, pow2f(p.gexps[t * p.nb + (c >> 6)]), z);
    ld8_codes(p.ucodes + t * p.d + c, cnt, pow2f(p.uexps[t * p.nb + (c >> 6)]), u);
  } else {
    ld8(p.g + t * p.ldz + c, cnt, z);
    ld8(p.u + t * p.ldz + c, cnt, u);
  }
  act_and_slope(p.act, z, s);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    u[e] = dh[e] * u[e] * s[e];
    z[e] = dh[e] * z[e];
  }
  const int64_t at = t * p.d + c, at8 = t * p.w8 + c;
  put_grad(p.dg, p.pg, p.lg, at, at8, cnt, u);
  put_grad(p.du, p.pu, p.lu, at, at8, cnt, z);
}

// ---- forward ------------------------------------------------------------------------------
struct GatedRoom {
  float *g = nullptr, *u = nullptr, *partial = nullptr;
  uint16_t *x = nullptr, *wg = nullptr, *wu = nullptr, *low = nullptr, *dz = nullptr;
  void* inner = nullptr;   // workspace of the fp32 products
  size_t bytes = 0;
};
GatedRoom forward_room(void* ws, int dt, int64_t n, int64_t di, int64_t df) {
  GatedRoom r;
  Carve cv(ws);
  if (dt == LRC_F32) {
    r.g = cv.take<float>(size_t(n) * df);
    r.u = cv.take<float>(size_t(n) * df);
    r.inner = cv.take<char>(lrc_linear_workspace(LRC_F32, n, di, df));
  } else {
    if (di % 8 != 0) {
      r.x = cv.take<uint16_t>(size_t(n) * round8(di));
      r.wg = cv.take<uint16_t>(size_t(df) * round8(di));
      r.wu = cv.take<uint16_t>(size_t(df) * round8(di));
    }
    r.partial = cv.take<float>(gemm::rows_workspace(n, df, di, true) / 4);
  }
  r.bytes = cv.bytes();
  return r;
}

struct GatedArgs {
  int64_t n, di, df;
  const void* x;
  int64_t ldx;
  const void *Wg, *Wu;
  int64_t ldw;
  Epilogue ep;
  gemm::Companion co;
};

lrc_status gated_bf16(hipStream_t st, GatedArgs& a, const GatedRoom& room) {
  const double flops = 4.0 * double(a.n) * double(a.df) * double(a.di);
  const double bytes = 2.0 * (double(a.n) * a.di + 2.0 * double(a.df) * a.di + double(a.n) * a.df);
  if (gemm::stream_bf16_pair(a.n, a.df, a.di) && a.ep.codes == nullptr)
    return gemm::few_rows<uint16_t, BF16, 2>(st, "gated_rows_kernel", a.x, a.ldx, false, a.Wg, a.ldw, a.Wu, a.ldw, a.n,
                                             a.df, a.di, a.ep, a.co, flops, bytes);
  GemmOperand x = {static_cast<const uint16_t*>(a.x), a.ldx, 0}, g = {static_cast<const uint16_t*>(a.Wg), a.ldw, 0},
              u = {static_cast<const uint16_t*>(a.Wu), a.ldw, 0};
  if (a.di % 8 != 0) {
    const OperandJobs jobs = {{bf16_job(a.x, nullptr, a.ldx, a.n, a.di, room.x),
                               bf16_job(a.Wg, nullptr, a.ldw, a.df, a.di, room.wg),
                               bf16_job(a.Wu, nullptr, a.ldw, a.df, a.di, room.wu)}};
    LRC_TRY(lay_out_bf16(st, jobs, 3));
    const int64_t w8 = round8(a.di);
    x = {room.x, w8, 0};
    g = {room.wg, w8, 0};
    u = {room.wu, w8, 0};
  }
  a.co.B = u;
  return gemm::rows_product<uint16_t, BF16, true>(st, "gated_kernel", x, g, a.n, a.df, a.di, a.ep, a.co, room.partial,
                                                  flops, bytes);
}

lrc_status gated_f32(hipStream_t st, GatedArgs& a, const GatedRoom& room) {
  if (gemm::stream_f32_pair(a.n, a.df, a.di) && a.ep.codes == nullptr)
    return gemm::few_rows<float, FP32, 2>(st, "gated_rows_kernel", a.x, a.ldx, false, a.Wg, a.ldw, a.Wu, a.ldw, a.n,
                                          a.df, a.di, a.ep, a.co, 4.0 * double(a.n) * double(a.df) * double(a.di),
                                          4.0 * (double(a.n) * a.di + 2.0 * double(a.df) * a.di + double(a.n) * a.df));
  const size_t inner = lrc_linear_workspace(LRC_F32, a.n, a.di, a.df);
  // g and u go where they are kept, else to the workspace
  float *g = static_cast<float*>(a.ep.z), *u = static_cast<float*>(a.co.z);
  const int64_t ldz = g != nullptr ? a.ep.ldz : a.df;
  if (g == nullptr) g = room.g, u = room.u;
  auto product = [&](const void* W, float* z) {
    return lrc_linear(a.x, LRC_F32, a.n, a.di, a.df, a.ldx, W, a.ldw, nullptr, LRC_ACT_NONE, nullptr, 0, z, ldz,
                      nullptr, 0, nullptr, nullptr, nullptr, room.inner, inner, st);
  };
  LRC_TRY(product(a.Wg, g));
  LRC_TRY(product(a.Wu, u));
  const int64_t blocks = cdiv(a.df, CKB), grid = cdiv(a.n * blocks * 8, ET);
  if (grid >= (int64_t(1) << 31)) return LRC_EINVAL;
  ProfScope scope("gate_kernel", st, 0.0, 12.0 * double(a.n) * double(a.df));
  Epilogue ep = a.ep;
  ep.z = nullptr;   // kept already
  gate_kernel<float><<<unsigned(grid), ET, 0, st>>>(g, u, ldz, a.n, a.df, blocks, ep, a.co);
  LRC_LAUNCHED();
  return LRC_OK;
}

// ---- backward -----------------------------------------------------------------------------
GatedRoom backward_room(void* ws, int dt, int64_t n, int64_t di, int64_t df) {
  GatedRoom r;
  Carve cv(ws);
  if (dt == LRC_F32) {
    r.inner = cv.take<char>(lrc_linear_backward_workspace(LRC_F32, n, di, df));
  } else {
    const int64_t f8 = round8(df), i8 = round8(di);
    r.low = cv.take<uint16_t>(size_t(2) * n * f8);
    if (df % 8 != 0) r.dz = cv.take<uint16_t>(size_t(2) * n * f8);
    r.x = cv.take<uint16_t>(size_t(n) * i8);
    if (di % 8 != 0) r.wg = cv.take<uint16_t>(size_t(2) * df * i8);
    r.partial = cv.take<float>(gemm_gradients_workspace(n, di, df) / 4);
  }
  r.bytes = cv.bytes();
  return r;
}

struct GatedBack {
  int64_t n, di, df;
  const void* dh;
  int64_t lddh;
  const void *Wg, *Wu;
  int64_t ldw;
  const void* x;
  int64_t ldx;
  const int8_t *xcodes, *xexps;
  int act;
  const void *g, *u;
  int64_t ldz;
  const int8_t *gcodes, *gexps, *ucodes, *uexps;
  void *dg, *du, *dx;
  int64_t lddx;
  void *dWg, *dWu;
  int dw_dt;
  int64_t lddw;
};

template <class T>
lrc_status gate_backward(hipStream_t st, const GatedBack& a, const GatedRoom& room, bool low,
                         const OperandJobs& jobs) {
  GatePass<T> p = {};
  p.dh = static_cast<const T*>(a.dh);
  p.g = static_cast<const T*>(a.g);
  p.u = static_cast<const T*>(a.u);
  p.lddh = a.lddh;
  p.ldz = a.ldz;
  p.n = a.n;
  p.d = a.df;
  p.nb = cdiv(a.df, CKB);
  p.w8 = round8(a.df);
  p.gcodes = a.gcodes;
  p.gexps = a.gexps;
  p.ucodes = a.ucodes;
  p.uexps = a.uexps;
  p.act = a.act;
  p.dg = static_cast<T*>(a.dg);
  p.du = static_cast<T*>(a.du);
  const int64_t plane = a.n * p.w8;
  if (room.dz != nullptr) {
    p.pg = room.dz;
    p.pu = room.dz + plane;
  }
  if (low) {
    p.lg = room.low;
    p.lu = room.low + plane;
  }
  const int64_t blocks = cdiv(a.n * (p.w8 / 8), ET);
  const int64_t grid = blocks + jobs.job[0].blocks + jobs.job[1].blocks + jobs.job[2].blocks;
  if (grid >= (int64_t(1) << 31)) return LRC_EINVAL;
  const double e = sizeof(T), kept = a.g == nullptr ? 1 : e;
  ProfScope scope("gated_dz_kernel", st, 0.0, double(a.n) * double(a.df) * (3 * e + 2 * kept + (low ? 4 : 0)));
  if (a.g == nullptr)
    gated_dz_kernel<T, true><<<unsigned(grid), ET, 0, st>>>(p, blocks, jobs);
  else
    gated_dz_kernel<T, false><<<unsigned(grid), ET, 0, st>>>(p, blocks, jobs);
  LRC_LAUNCHED();
  return LRC_OK;
}

lrc_status gated_back_f32(hipStream_t st, const GatedBack& a, const GatedRoom& room) {
  LRC_TRY(gate_backward<float>(st, a, room, false, OperandJobs{}));
  auto grads = [&](const void* dz, const void* W, void* dW, bool add) -> lrc_status {
    if (a.dx == nullptr && dW == nullptr) return LRC_OK;
    return linear_grads_f32(st, a.n, a.di, a.df, static_cast<const float*>(dz), a.df, static_cast<const float*>(W),
                            a.ldw, static_cast<const float*>(a.x), a.ldx, a.xcodes, a.xexps,
                            static_cast<float*>(a.dx), a.lddx, add, static_cast<float*>(dW), a.lddw, room.inner);
  };
  LRC_TRY(grads(a.dg, a.Wg, a.dWg, false));
  return grads(a.du, a.Wu, a.dWu, true);
}

// distance of two bf16 operands as the planes of one
int64_t apart(const uint16_t* from, const uint16_t* to) {
  return (reinterpret_cast<intptr_t>(to) - reinterpret_cast<intptr_t>(from)) / 2;
}

lrc_status gated_back_bf16(hipStream_t st, const GatedBack& a, const GatedRoom& room) {
  const bool dw = a.dWg != nullptr, held = a.x == nullptr;
  const int64_t f8 = round8(a.df), i8 = round8(a.di), plane = a.n * f8;
  const uint16_t *dg = static_cast<const uint16_t*>(a.dg), *du = static_cast<const uint16_t*>(a.du);
  if (room.dz != nullptr) {
    dg = room.dz;
    du = room.dz + plane;
  }
  const uint16_t *wg = static_cast<const uint16_t*>(a.Wg), *wu = static_cast<const uint16_t*>(a.Wu);
  const uint16_t* x = static_cast<const uint16_t*>(a.x);
  int64_t ldw = a.ldw, ldx = a.ldx;
  OperandJobs jobs;
  if (dw && (held || a.di % 8 != 0)) {
    jobs.job[0] = bf16_job(held ? static_cast<const void*>(a.xcodes) : a.x, held ? a.xexps : nullptr,
                           held ? a.di : a.ldx, a.n, a.di, room.x);
    x = room.x;
    ldx = i8;
  }
  if (a.dx != nullptr && room.wg != nullptr) {
    uint16_t* second = room.wg + a.df * i8;
    jobs.job[1] = bf16_job(a.Wg, nullptr, a.ldw, a.df, a.di, room.wg);
    jobs.job[2] = bf16_job(a.Wu, nullptr, a.ldw, a.df, a.di, second);
    wg = room.wg;
    wu = second;
    ldw = i8;
  }
  LRC_TRY(gate_backward<uint16_t>(st, a, room, dw, jobs));
  const double product = 2.0 * double(a.n) * double(a.df) * double(a.di);
  const double xbytes = 2.0 * (2.0 * double(a.n) * a.df + 2.0 * double(a.df) * a.di + double(a.n) * a.di);
  const double wbytes = 2.0 * (4.0 * double(a.n) * a.df + double(a.n) * a.di + 2.0 * double(a.df) * a.di);
  // dx: the second segment takes the second planes
  const GemmOperand G = {dg, f8, apart(dg, du)}, W = {wg, ldw, apart(wg, wu)};
  Epilogue epx, epw;
  epx.y = a.dx;
  epx.ldy = a.lddx;
  const GemmOperand A1 = {dg, f8, apart(dg, room.low)}, A2 = {du, f8, apart(du, room.low + plane)}, B = {x, ldx, 0};
  epw.y = a.dWg;
  epw.y2 = a.dWu;
  epw.ldy = a.lddw;
  if (a.dx == nullptr && !dw) return LRC_OK;
  auto go = [&](auto tag) {
    return gemm_gradients<decltype(tag)>(st, "gated_grads_kernel", G, W, A1, A2, B, a.n, a.di, a.df, epx, epw,
                                         room.partial, (a.dx ? 2 * product : 0) + (dw ? 4 * product : 0),
                                         (a.dx ? xbytes : 0) + (dw ? wbytes : 0));
  };
  return dw && a.dw_dt == LRC_F32 ? go(float{}) : go(uint16_t{});
}

bool act_ok(int a) { return a >= LRC_ACT_NONE && a <= LRC_ACT_SILU; }
// bf16 operands that are read where they lie start on 16 bytes and keep to pitches of whole pieces
bool in_place(const void* p, int64_t ld, int64_t cols, int dt) {
  return dt != LRC_BF16 || cols % 8 != 0 || (rows_vec16(p, ld, 2) && ld <= GEMM_MAX_LD);
}

}  // namespace
}  // namespace lrc

using namespace lrc;

extern "C" size_t lrc_gated_linear_workspace(lrc_dtype dt, int64_t n_tokens, int64_t d_in, int64_t d_ff) {
  if (!sizes_ok(n_tokens, d_in, d_ff)) return 0;
  return forward_room(nullptr, dt, n_tokens, d_in, d_ff).bytes;
}

extern "C" lrc_status lrc_gated_linear(const void* x, lrc_dtype dt, int64_t n_tokens, int64_t d_in, int64_t d_ff,
                                       int64_t ldx, const void* Wg, const void* Wu, int64_t ldw, lrc_act act, void* h,
                                       int64_t ldh, void* g, void* u, int64_t ldz, int8_t* gcodes, int8_t* gexps,
                                       int8_t* ucodes, int8_t* uexps, int32_t* info, void* ws, size_t ws_bytes,
                                       void* stream) {
  if ((dt != LRC_F32 && dt != LRC_BF16) || !act_ok(act)) return LRC_EDTYPE;
  if (!sizes_ok(n_tokens, d_in, d_ff) || ldx < d_in || ldw < d_in || ldh < d_ff) return LRC_EINVAL;
  if ((g == nullptr) != (u == nullptr) || (g != nullptr && (ldz < d_ff || gcodes != nullptr))) return LRC_EINVAL;
  const bool codes = gcodes != nullptr;
  if ((gexps != nullptr) != codes || (ucodes != nullptr) != codes || (uexps != nullptr) != codes) return LRC_EINVAL;
  if (n_tokens == 0) return LRC_OK;
  if (x == nullptr || Wg == nullptr || Wu == nullptr || h == nullptr) return LRC_EINVAL;
  if (!in_place(x, ldx, d_in, dt) || !in_place(Wg, ldw, d_in, dt) || !in_place(Wu, ldw, d_in, dt)) return LRC_EINVAL;
  const GatedRoom room = forward_room(ws, dt, n_tokens, d_in, d_ff);
  if (ws_bytes < room.bytes || (room.bytes > 0 && ws == nullptr)) return LRC_EWORKSPACE;
  GatedArgs a = {n_tokens, d_in, d_ff, x, ldx, Wg, Wu, ldw, {}, {}};
  a.ep.act = act;
  a.ep.y = h;
  a.ep.ldy = ldh;
  a.ep.z = g;
  a.co.z = u;
  a.ep.ldz = codes ? d_ff : ldz;
  a.ep.codes = gcodes;
  a.ep.exps = gexps;
  a.co.codes = ucodes;
  a.co.exps = uexps;
  a.ep.nb = cdiv(d_ff, CKB);
  a.ep.info = info;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return dt == LRC_BF16 ? gated_bf16(st, a, room) : gated_f32(st, a, room);
}

extern "C" size_t lrc_gated_linear_backward_workspace(lrc_dtype dt, int64_t n_tokens, int64_t d_in, int64_t d_ff) {
  if (!sizes_ok(n_tokens, d_in, d_ff)) return 0;
  return backward_room(nullptr, dt, n_tokens, d_in, d_ff).bytes;
}

extern "C" lrc_status lrc_gated_linear_backward(const void* dh, lrc_dtype dt, int64_t n_tokens, int64_t d_in,
                                                int64_t d_ff, int64_t lddh, const void* Wg, const void* Wu,
                                                int64_t ldw, const void* x, int64_t ldx, const int8_t* xcodes,
                                                const int8_t* xexps, lrc_act act, const void* g, const void* u,
                                                int64_t ldz, const int8_t* gcodes, const int8_t* gexps,
                                                const int8_t* ucodes, const int8_t* uexps, void* dg, void* du,
                                                void* dx, int64_t lddx, void* dWg, void* dWu, lrc_dtype dw_dt,
                                                int64_t lddw, void* ws, size_t ws_bytes, void* stream) {
  const bool dw = dWg != nullptr;
  if ((dt != LRC_F32 && dt != LRC_BF16) || !act_ok(act)) return LRC_EDTYPE;
  if (dw && dw_dt != LRC_F32 && dw_dt != dt) return LRC_EDTYPE;
  if (!sizes_ok(n_tokens, d_in, d_ff) || lddh < d_ff || (g != nullptr && ldz < d_ff) || (dWu != nullptr) != dw)
    return LRC_EINVAL;
  if ((dx != nullptr && (lddx < d_in || ldw < d_in)) || (dw && (lddw < d_in || (x != nullptr && ldx < d_in))))
    return LRC_EINVAL;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (n_tokens == 0) {   // sums over nothing
    const int size = dw_dt == LRC_F32 ? 4 : 2;
    if (dWg != nullptr) LRC_TRY(zero_rows(st, dWg, d_ff, d_in, lddw, size));
    if (dWu != nullptr) LRC_TRY(zero_rows(st, dWu, d_ff, d_in, lddw, size));
    return LRC_OK;
  }
  if (dh == nullptr || dg == nullptr || du == nullptr || (g == nullptr) != (u == nullptr)) return LRC_EINVAL;
  if (g == nullptr && (gcodes == nullptr || gexps == nullptr || ucodes == nullptr || uexps == nullptr))
    return LRC_EINVAL;
  if (dx != nullptr && (Wg == nullptr || Wu == nullptr)) return LRC_EINVAL;
  if (dw && x == nullptr && (xcodes == nullptr || xexps == nullptr)) return LRC_EINVAL;
  if (!in_place(dg, d_ff, d_ff, dt) || !in_place(du, d_ff, d_ff, dt)) return LRC_EINVAL;
  if (dx != nullptr && (!in_place(Wg, ldw, d_in, dt) || !in_place(Wu, ldw, d_in, dt))) return LRC_EINVAL;
  if (dw && x != nullptr && !in_place(x, ldx, d_in, dt)) return LRC_EINVAL;
  const GatedRoom room = backward_room(ws, dt, n_tokens, d_in, d_ff);
  if (ws_bytes < room.bytes || (room.bytes > 0 && ws == nullptr)) return LRC_EWORKSPACE;
  const GatedBack a = {n_tokens, d_in, d_ff, dh, lddh, Wg, Wu, ldw, x, ldx, xcodes, xexps, act, g, u, ldz, gcodes,
                       gexps, ucodes, uexps, dg, du, dx, lddx, dWg, dWu, int(dw_dt), lddw};
  return dt == LRC_BF16 ? gated_back_bf16(st, a, room) : gated_back_f32(st, a, room);
}
