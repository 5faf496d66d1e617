// Matrix products on the matrix cores with a fused epilogue: the linear layer's forward, dx and dW
// products of bf16 or fp32 operands, sums in fp32.
//
// An output tile of BM x BN belongs to one workgroup; its waves hold blocks of MF x MF
// accumulators (16 x 16 x 32, 32 x 32 x 16 or, in fp32, 16 x 16 x 4 matrix instructions).  Both
// operands travel from memory straight into LDS (16 bytes per lane, no staging registers) in stages
// of 64 or 128 bytes of a row, two or four stage buffers, all but one in flight while one is
// multiplied.  A buffer resource bounds each operand, so rows past the matrix and k past its end
// read as zeros without any masking of data.
//   K_ROWS: a tile row's k steps lie together; its 16-byte granules change places by the row's
//     number, so that the 16 rows of a fragment read cover every bank once.
//   K_COLS: a k step's channels lie together; fragments come from transposing LDS reads
//     (ds_read_b64_tr_b16), in fp32 from four reads of 4 bytes, granules changing places by the
//     step's number.
// What bounds it: the matrix pipes, busy 64 % of the cycles of dx at 8192 x 4096 x 11008 (at 1.8 GHz) and
// 63 % of dW's (1.9), and what leaves them idle: 47 % forward (2.1 GHz), where the sixth round of tiles
// is 38 % full and nothing hides the epilogue.  8192 x 4096 x 11008 forward 680 us in a
// row of its own calls (1090 TFLOP/s; the vendor's library on the same box 690), 730 between other
// kernels; dx 590-640, dW 590-650 (twice where dz has two pieces); 4096^3 103 us (library 90).  fp32 split in
// three: 8192 x 1024 x 4096 315-345 us (200 TFLOP/s of fp32 products, fp32 instructions reach 140).
// fp32 tiles: 2048 x 2048 x 1024 68 us (126 TFLOP/s; library 65).  24 tokens x 11008 x 4096: 21 us
// and 4 for the splits' sums, 4.3 TB/s of weight.
// Few tiles leave compute units idle, so k may be split: every split writes its fp32 tile and
// a second kernel adds them in split order and runs the epilogue (bit-reproducible).
#include "lrc_gemm_tile.h"

#include <cmath>

namespace lrc {
namespace gemm {

template <class TO, int KA, int KB, int MF, int WM, int WN, int FM, int FN, int KS, int NST, int SEG, Element EL>
__global__ __launch_bounds__(64 * WM * WN, 2) void gemm_bf16_kernel(GemmOperand A, GemmOperand B, int64_t M, int64_t N,
                                                                    int64_t K, GemmSegments seg, TileGrid tg,
                                                                    Epilogue ep, float* __restrict__ partial,
                                                                    const int32_t* __restrict__ skip) {
  gemm_tile<TO, KA, KB, MF, WM, WN, FM, FN, KS, NST, SEG, EL>(A, B, M, N, K, seg, tg, ep, partial, skip, Companion{},
                                                           blockIdx.x);
}
// f(matrix instruction's edge, waves, a wave's fragments, stage, stages) of a tile whose B runs along columns
template <int V>
using I = std::integral_constant<int, V>;
template <int TILE, class F>
__device__ __forceinline__ void with_cols_tile(F f) {
  if constexpr (TILE == LARGE)
    f(I<32>{}, I<4>{}, I<2>{}, I<2>{}, I<4>{}, I<32>{}, I<4>{});
  else if constexpr (TILE == SMALL)
    f(I<16>{}, I<2>{}, I<2>{}, I<4>{}, I<4>{}, I<64>{}, I<2>{});
  else
    f(I<16>{}, I<4>{}, I<1>{}, I<1>{}, I<4>{}, I<64>{}, I<4>{});
}
// Both in one launch: dx does not wait for the weight gradients, and neither often fills the chip to its end.  The
// product with the longer tiles goes first.  One launch / two, us a call: 300 x 136 -> 264 12.6 / 20.8, 1000 x 521 -> 303
// 22.9 / 31.2, 1813 x 11016 -> 144 78 / 129, 8192 x 1024 -> 4096 475 / 509, 2048 x 4096 -> 11008 985 / 1116,
// 8192 x 4096 -> 11008 3998 / 3989.
struct Product {
  GemmOperand A, B;
  int64_t M, N, K;
  TileGrid tg;
  Epilogue ep;
  float* partial;
  int64_t groups() const { return int64_t(NXCD) * tg.per_xcd * tg.splits; }
};
template <class TO, int TILE>
__global__ __launch_bounds__(TILE == LARGE ? 512 : 256, 2) void gemm_gradients_kernel(Product w, GemmOperand A2,
                                                                                      Product x, int x0, int w0) {
  const int block = blockIdx.x;
  GemmSegments seg;
  seg.count = 2;
  if (w0 < x0 ? block < x0 : block >= w0) {
    seg.pa = 1u;
    Companion co;
    co.B = A2;
    auto go = [&](auto mf, auto wm, auto wn, auto fm, auto fn, auto ks, auto nst) {
      gemm_tile<TO, K_COLS, K_COLS, mf, wm, wn, fm, fn, ks, nst, 2, BF16>(w.A, w.B, w.M, w.N, w.K, seg, w.tg, w.ep,
                                                                          w.partial, nullptr, co, block - w0);
    };
    with_cols_tile<TILE>(go);
  } else {
    seg.pa = seg.pb = 1u << 2;
    auto go = [&](auto mf, auto wm, auto wn, auto fm, auto fn, auto ks, auto nst) {
      gemm_tile<uint16_t, K_ROWS, K_COLS, mf, wm, wn, fm, fn, ks, nst, 1, BF16>(
          x.A, x.B, x.M, x.N, x.K, seg, x.tg, x.ep, x.partial, nullptr, Companion{}, block - x0);
    };
    with_cols_tile<TILE>(go);
  }
}

// Sum of the splits' tiles in split order, then the epilogue.  One lane per eight columns, the
// eight lanes of a 64-column block together.
template <class TO>
__global__ __launch_bounds__(256) void gemm_finish_kernel(const float* __restrict__ partial, int splits, int64_t M,
                                                          int64_t N, int64_t np, int64_t blocks, Epilogue ep,
                                                          const int32_t* __restrict__ skip) {
  if (skip != nullptr && *skip != 0) return;
  const int64_t g = (int64_t(blockIdx.x) * 256 + threadIdx.x) >> 3;
  const int lane = threadIdx.x & 63;
  int64_t row = g / blocks;
  const int64_t col = g % blocks * CKB + 8 * (lane & 7);
  const int64_t left = row < M ? N - col : 0;
  const int cnt = int(left < 0 ? 0 : left > 8 ? 8 : left);
  float v[8] = {};
  if (cnt > 0) {
    const float* p = partial + row * np + col;
    const int64_t plane = M * np;
    for (int s0 = 0; s0 < splits; s0 += 8) {   // eight splits' loads in flight, added in order
      f32x4 lo[8], hi[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float* q = p + min(s0 + u, splits - 1) * plane;
        lo[u] = *reinterpret_cast<const f32x4*>(q);
        hi[u] = *reinterpret_cast<const f32x4*>(q + 4);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] += s0 + u < splits ? lo[u][e] : 0.f;
          v[4 + e] += s0 + u < splits ? hi[u][e] : 0.f;
        }
    }
  }
  bool bad = false;
  float bias[8];
  bias8(ep, col, cnt, bias);
  if (ep.y2 != nullptr && 2 * row >= M) {   // the second of two products
    row -= M / 2;
    ep.y = ep.y2;
  }
  finish8<TO>(ep, row, col, cnt, bias, v, lane, bad);
  if (ep.info != nullptr && bad) *ep.info = LRC_ENONFINITE;
}

}  // namespace gemm

using namespace gemm;

size_t gemm_bf16_workspace(int64_t M, int64_t N, int64_t K, int KA, int KB, bool f32) {
  double c;
  size_t most = f32 ? plan_bytes(plan_f32(M, N, K, c), M, N) : 0;
  for (int count : {1, 3, 6})
    most = std::max(most, plan_bytes(plan_gemm(M, N, K, count, large_stage(KA, KB), c), M, N));
  return most;
}
double gemm_f32_time(int64_t M, int64_t N, int64_t K) {
  double c;
  plan_f32(M, N, K, c);
  return c;
}
double gemm_split_time(int64_t M, int64_t N, int64_t K, int KA, int KB) {
  double c;
  plan_gemm(M, N, K, 6, large_stage(KA, KB), c);
  return c;
}

template <class TO>
lrc_status gemm_finish(hipStream_t st, const float* partial, int splits, int64_t M, int64_t N, const Epilogue& ep,
                       const int32_t* skip) {
  const int64_t np = (N + 7) & ~int64_t(7), blocks = cdiv(N, CKB), threads = M * blocks * 8;
  if (cdiv(threads, 256) >= (int64_t(1) << 31)) return LRC_EINVAL;
  gemm_finish_kernel<TO><<<unsigned(cdiv(threads, 256)), 256, 0, st>>>(partial, splits, M, N, np, blocks, ep, skip);
  LRC_LAUNCHED();
  return LRC_OK;
}
template lrc_status gemm_finish<float>(hipStream_t, const float*, int, int64_t, int64_t, const Epilogue&, const int32_t*);
template lrc_status gemm_finish<uint16_t>(hipStream_t, const float*, int, int64_t, int64_t, const Epilogue&,
                                          const int32_t*);

template <class TO, int KA, int KB>
lrc_status gemm_bf16(hipStream_t st, const char* name, GemmOperand A, GemmOperand B, int64_t M, int64_t N, int64_t K,
                     const GemmSegments& seg, const Epilogue& ep, float* partial, const int32_t* skip, double flops,
                     double bytes) {
  // Stages of a large tile: 64 k steps in two buffers where both operands' rows run along k (a
  // row's piece is then a whole 128-byte line: 8192 x 4096 x 11008 678 us against 712), else 32
  // in four (dx 560 against 579, dW 581 against 610).  Small tiles: 64 in two (785 against 954).
  // The 16 x 16 x 32 matrix instruction is the faster one (8192 x 4096 x 4096 199 us against 215 with
  // 32 x 32 x 16, 2048 x 4096 x 4096 on small tiles 62 against 69).  Large tiles with K_COLS operands
  // keep the larger one: their transposing reads need more address registers, and the smaller one's
  // two full fragment sets then spill (dx 272 against 225, dW 445 against 213).
  constexpr int KL = large_stage(KA, KB), NL = KL == 64 ? 2 : 4, ML = KL == 64 ? 16 : 32;
  double cost;
  const Plan p = seg.type == FP32 ? plan_f32(M, N, K, cost) : plan_gemm(M, N, K, seg.count, KL, cost);
  ProfScope scope(name, st, flops, bytes);
  const TileGrid& tg = p.tg;
  const int64_t grid = int64_t(NXCD) * tg.per_xcd * tg.splits;
  if (grid >= (int64_t(1) << 31)) return LRC_EINVAL;
  constexpr bool BITS = std::is_same<TO, uint16_t>::value;
  auto launch = [&](auto many, auto type) {
    constexpr int SEG = decltype(many)::value;
    constexpr Element EL = decltype(type)::value;
    if constexpr (EL == FP32)
      gemm_bf16_kernel<TO, KA, KB, 16, 4, 1, 1, 4, 64, 2, SEG, EL><<<unsigned(grid), 256, 0, st>>>(
          A, B, M, N, K, seg, tg, ep, partial, skip);
    else if (p.tile == LARGE)
      gemm_bf16_kernel<TO, KA, KB, ML, 4, 2, 64 / ML, 128 / ML, KL, NL, SEG, EL><<<unsigned(grid), 512, 0, st>>>(
          A, B, M, N, K, seg, tg, ep, partial, skip);
    else if (p.tile == SMALL)
      gemm_bf16_kernel<TO, KA, KB, 16, 2, 2, 4, 4, 64, 2, SEG, EL><<<unsigned(grid), 256, 0, st>>>(
          A, B, M, N, K, seg, tg, ep, partial, skip);
    else if constexpr (SEG == 0)
      gemm_bf16_kernel<TO, KA, KB, 16, 4, 1, 1, 4, 64, 4, SEG, EL><<<unsigned(grid), 256, 0, st>>>(
          A, B, M, N, K, seg, tg, ep, partial, skip);
    else
      return false;
    return true;
  };
  using std::integral_constant;
  // bf16 layers have one plane; an fp32 result may come of one (dW of a bf16 layer) or more.  What no caller asks for
  // has no kernel, and is refused.
  bool launched = false;
  if (seg.type == FP32) {
    if constexpr (!BITS) launched = launch(integral_constant<int, 0>{}, integral_constant<Element, FP32>{});
  } else if (seg.count == 1) {
    if constexpr (BITS || KA == K_COLS) launched = launch(integral_constant<int, 0>{}, integral_constant<Element, BF16>{});
  } else if constexpr (!BITS) {
    if (seg.count == 3 || seg.count == 6)   // the counts that the workspace is sized for
      launched = launch(integral_constant<int, 1>{}, integral_constant<Element, BF16>{});
  }
  if (!launched) return LRC_EINVAL;
  LRC_LAUNCHED();
  if (tg.splits == 1) return LRC_OK;
  const int splits = tg.splits;
  return gemm_finish<TO>(st, partial, splits, M, N, ep, skip);
}

// The plans of dx and of both weight gradients.  One kind of tile for all, in one launch, unless two launches cost
// less; whichever gradients are asked for, so that their bits do not depend on it.  A second launch costs SECOND_LAUNCH
// or more (8 us at 300 x 136 -> 264).  Two it is where a product's split of k saves more: 7546 x 128 -> 9320 487 us
// against 498 in one (4147 x 80 -> 8464 230 against 226).  The estimate is wrong where the weight gradients have few
// tokens to sum: 288 x 4384 -> 768 44 in one, 37 in two, 512 x 4096 -> 11008 367 and 359.
struct GradPlan {
  Plan x, w;
  bool joined;
};
// Workgroups of two lengths on `slots`, the longer ones first.
static double joint_cost(double slots, int64_t ga, double ta, int64_t gb, double tb) {
  if (ta < tb) std::swap(ga, gb), std::swap(ta, tb);
  const double rounds = std::floor(double(ga) / slots), rest = double(ga) - rounds * slots;
  // b starts on the free slots of a's last round: `ahead` of its tiles each before the others end
  const double start = rounds * ta, ahead = rest > 0 ? std::floor(ta / tb) : 0, early = (slots - rest) * ahead;
  if (rest > 0 && double(gb) <= early) return start + ta;
  const double left = double(gb) - early;
  return start + ahead * tb + std::ceil(std::max(left, 1.0) / slots) * tb;
}
constexpr double SECOND_LAUNCH = 5.0;
static GradPlan plan_gradients(int64_t n, int64_t di, int64_t df) {
  GradPlan best;
  double apart_x = 1e30, apart_w = 1e30, joint = 1e30;
  Plan ax, aw;
  const double unique = 4.0 * (double(df) * double(n + di) + double(n) * double(2 * df + di));
  constexpr double CACHE = 24e6;
  for (Tile tile : {LARGE, SMALL, TINY}) {
    double cx, cw;
    const Plan x = plan_tiles(tile, n, di, df, 2, 32, cx);
    Plan w = plan_tiles(tile, 2 * df, di, n, 2, 32, cw);
    const int edge = tile == LARGE ? 256 : tile == SMALL ? 128 : 64;
    w.tg.nm = cdiv(df, edge);   // each product's own edge
    w.tg.half = w.tg.nm * w.tg.nn;
    w.tg.tiles = 2 * w.tg.half;
    w.tg.per_xcd = int(cdiv(w.tg.tiles, NXCD));
    if (cx < apart_x) apart_x = cx, ax = x;
    if (cw < apart_w) apart_w = cw, aw = w;
    const double round = tile == LARGE ? LARGE_ROUND : tile == SMALL ? SMALL_ROUND : TINY_ROUND;
    for (int mx = 0; mx < (x.tg.splits > 1 ? 2 : 1); ++mx)
      for (int mw = 0; mw < (w.tg.splits > 1 ? 2 : 1); ++mw) {
        Plan px = x, pw = w;
        if (mx) px.tg.splits = 1, px.tg.steps_per_split = 2 * px.tg.steps;
        if (mw) pw.tg.splits = 1, pw.tg.steps_per_split = 2 * pw.tg.steps;
        const int64_t gx = px.tg.tiles * px.tg.splits, gw = pw.tg.tiles * pw.tg.splits;
        const double step = tile == LARGE ? 0.5 * LARGE_STEP
                            : tile == SMALL ? (gx + gw > 256 ? SMALL_STEP_FULL : SMALL_STEP_HALF)
                                            : (gx + gw > 256 ? TINY_STEP_FULL : TINY_STEP_HALF);
        double c = joint_cost(tile == LARGE ? 256 : 512, gx, px.tg.steps_per_split * step + round, gw,
                              pw.tg.steps_per_split * step + round);
        // every tile reads its rows: from memory the first time, and from the caches (7546 x 128 -> 9320 on the
        // smallest tiles 576 us against 488)
        const double reads = 8.0 * edge * (double(px.tg.tiles) * double(df) + double(pw.tg.tiles) * double(n));
        c = std::max(c, unique / MEMORY + std::max(0.0, reads - unique) / CACHE);
        if (px.tg.splits > 1) c += 4.0 + 8.0 * px.tg.splits * double(n) * double(di) / MEMORY;
        if (pw.tg.splits > 1) c += 4.0 + 16.0 * pw.tg.splits * double(df) * double(di) / MEMORY;
        if (c < joint) joint = c, best.x = px, best.w = pw;
      }
  }
  best.joined = joint <= apart_x + apart_w + SECOND_LAUNCH;
  if (!best.joined) best.x = ax, best.w = aw;
  return best;
}
size_t gemm_gradients_workspace(int64_t n, int64_t di, int64_t df) {
  const GradPlan p = plan_gradients(n, di, df);
  return plan_bytes(p.x, n, di) + plan_bytes(p.w, 2 * df, di);
}
template <class TO>
lrc_status gemm_gradients(hipStream_t st, const char* name, GemmOperand Ax, GemmOperand Bx, GemmOperand A1,
                          GemmOperand A2, GemmOperand B, int64_t n, int64_t di, int64_t df, const Epilogue& epx,
                          const Epilogue& epw, float* partial, double flops, double bytes) {
  const GradPlan p = plan_gradients(n, di, df);
  const Product x = {Ax, Bx, n, di, df, p.x.tg, epx, partial};
  const Product w = {A1, B, df, di, n, p.w.tg, epw, partial + plan_bytes(p.x, n, di) / 4};
  const bool dx = epx.y != nullptr, dw = epw.y != nullptr;
  if (x.groups() + w.groups() >= (int64_t(1) << 31)) return LRC_EINVAL;
  ProfScope scope(name, st, flops, bytes);
  auto launch = [&](Tile tile, int gx, int gw) {   // workgroups of dx and of dWg and dWu
    const bool x_first = gw == 0 || (gx > 0 && p.x.tg.steps_per_split > p.w.tg.steps_per_split);
    const int x0 = x_first ? 0 : gw, w0 = x_first ? gx : 0;
    auto go = [&](auto t) {
      constexpr int TILE = decltype(t)::value;
      gemm_gradients_kernel<TO, TILE><<<unsigned(gx + gw), TILE == LARGE ? 512 : 256, 0, st>>>(w, A2, x, x0, w0);
    };
    if (tile == LARGE)
      go(I<LARGE>{});
    else if (tile == SMALL)
      go(I<SMALL>{});
    else
      go(I<TINY>{});
  };
  const int gx = dx ? int(x.groups()) : 0, gw = dw ? int(w.groups()) : 0;
  if (p.joined || !dx || !dw) {
    launch(dx ? p.x.tile : p.w.tile, gx, gw);
  } else {
    launch(p.x.tile, gx, 0);
    LRC_LAUNCHED();
    launch(p.w.tile, 0, gw);
  }
  LRC_LAUNCHED();
  if (dx && p.x.tg.splits > 1) LRC_TRY(gemm_finish<uint16_t>(st, x.partial, p.x.tg.splits, n, di, epx, nullptr));
  return dw && p.w.tg.splits > 1 ? gemm_finish<TO>(st, w.partial, p.w.tg.splits, 2 * df, di, epw, nullptr) : LRC_OK;
}
template lrc_status gemm_gradients<float>(hipStream_t, const char*, GemmOperand, GemmOperand, GemmOperand, GemmOperand,
                                          GemmOperand, int64_t, int64_t, int64_t, const Epilogue&, const Epilogue&,
                                          float*, double, double);
template lrc_status gemm_gradients<uint16_t>(hipStream_t, const char*, GemmOperand, GemmOperand, GemmOperand, GemmOperand,
                                             GemmOperand, int64_t, int64_t, int64_t, const Epilogue&, const Epilogue&,
                                             float*, double, double);

#define LRC_GEMM(TO, KA, KB)                                                                                   \
  template lrc_status gemm_bf16<TO, KA, KB>(hipStream_t, const char*, GemmOperand, GemmOperand, int64_t, int64_t, \
                                            int64_t, const GemmSegments&, const Epilogue&, float*, const int32_t*, double,      \
                                            double);
LRC_GEMM(uint16_t, K_ROWS, K_ROWS)
LRC_GEMM(uint16_t, K_ROWS, K_COLS)
LRC_GEMM(uint16_t, K_COLS, K_COLS)
LRC_GEMM(float, K_ROWS, K_ROWS)
LRC_GEMM(float, K_ROWS, K_COLS)
LRC_GEMM(float, K_COLS, K_COLS)
#undef LRC_GEMM

}  // namespace lrc
