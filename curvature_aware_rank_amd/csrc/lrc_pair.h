// Products of a token block with weights whose rows run along k, beside those of lrc_gemm.hip: 8-bit
// integers, and two weights that share x (g = x Wg^T, u = x Wu^T, h = act(g) u).
//
// Integers take the tiles, stages and fragments of bf16 with 16 bytes holding twice the k
// (16 x 16 x 64 matrix instructions): 8192 x 4096 x 8192 230 us, 2390 TOP/s (the vendor's library 2050),
// 8192 x 4096 x 11008 with GELU 380.  A pair's tile holds as many channels of each weight, so x is staged
// once for both: 8192 x 4096 x 2 x 11008 bf16 with SiLU and checkpoints 1180 us (1250 TFLOP/s).
// What bounds them: matrix pipes busy 45 % (integers) and 58 % of the cycles at 2.0 GHz; 73 % inside the
// k loop, whose LDS reads take as many cycles as its products; the rest is the epilogue, 16 to 19 us a
// round of tiles (GELU alone 12), and a last round that is part full.  One workgroup going on to its next
// tile, whose first loads land under the epilogue, lost in the loop (registers) what it gained outside.
#pragma once

#include "lrc_gemm_tile.h"
#include "lrc_rows.h"

namespace lrc {
namespace gemm {

template <class TO, int WM, int WN, int FM, int FN, int NST, Element EL, bool PAIR>
__global__ __launch_bounds__(64 * WM * WN, 2) void rows_product_kernel(GemmOperand A, GemmOperand B, int64_t M,
                                                                       int64_t N, int64_t K, TileGrid tg, Epilogue ep,
                                                                       Companion co, float* __restrict__ partial) {
  gemm_tile<TO, K_ROWS, K_ROWS, 16, WM, WN, FM, FN, 64, NST, false, EL, PAIR>(A, B, M, N, K, GemmSegments{}, tg, ep,
                                                                              partial, nullptr, co, blockIdx.x);
}

// Sum of the splits' tiles in split order (integers: exact in any), then the epilogue.  One lane per
// eight channels, the eight lanes of a 64-channel block together.
template <class TO, Element EL, bool PAIR>
__global__ __launch_bounds__(256) void rows_finish_kernel(const float* __restrict__ partial, int splits, int64_t M,
                                                          int64_t N, int64_t np, int64_t blocks, Epilogue ep,
                                                          Companion co) {
  const int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) >> 3;
  const int lane = threadIdx.x & 63;
  const int64_t row = i / blocks, col = i % blocks * CKB + 8 * (lane & 7);
  const int64_t left = row < M ? N - col : 0;
  const int cnt = int(left < 0 ? 0 : left > 8 ? 8 : left);
  constexpr int W = PAIR ? 2 : 1;
  using V4 = std::conditional_t<EL == INT8, i32x4, f32x4>;
  V4 acc[W][2] = {};
  if (cnt > 0) {
    const float* p = partial + row * W * np + col;
    const int64_t plane = M * W * np;
    constexpr int U = 8 / W;
    for (int s0 = 0; s0 < splits; s0 += U) {   // eight loads of 32 bytes in flight, added in order
      V4 t[U][W][2];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const V4* q = reinterpret_cast<const V4*>(p + min(s0 + u, splits - 1) * plane + w * np);
          t[u][w][0] = q[0];
          t[u][w][1] = q[1];
        }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int w = 0; w < W; ++w)
          if (s0 + u < splits) {
            acc[w][0] += t[u][w][0];
            acc[w][1] += t[u][w][1];
          }
    }
  }
  float v[W][8];
#pragma unroll
  for (int w = 0; w < W; ++w) __builtin_memcpy(v[w], acc[w], 32);
  if constexpr (EL == INT8) {
    const float s = cnt > 0 ? co.row_scale[row] : 0.f;
    float sc[8];
    col8(co.col_scale + col, cnt, sc);
    scale8(s, sc, v[0]);
    if constexpr (PAIR) {
      col8(co.col_scale2 + col, cnt, sc);
      scale8(s, sc, v[1]);
    }
  }
  bool bad = false;
  if constexpr (PAIR) {
    finish_pair8<TO>(ep, co, row, col, cnt, v[0], v[1], lane, bad);
  } else {
    float bias[8];
    bias8(ep, col, cnt, bias);
    finish8<TO>(ep, row, col, cnt, bias, v[0], lane, bad);
  }
  if (ep.info != nullptr && bad) *ep.info = LRC_ENONFINITE;
}

// K: k steps in 16-bit halves
inline Plan plan_rows(int64_t M, int64_t N, int64_t K, bool pair) {
  double cost;
  return plan_gemm(M, pair ? 2 * N : N, K, 1, 64, cost);
}
// bytes of the tiles in the workspace; those of a pair's checkpoint pass through it where tiles are tiny
inline size_t rows_workspace(int64_t M, int64_t N, int64_t K, bool pair) {
  const Plan p = plan_rows(M, N, K, pair);
  if (!pair) return plan_bytes(p, M, N);
  return p.tg.splits > 1 || p.tile == TINY ? 2 * size_t(p.tg.splits) * M * ((N + 7) & ~int64_t(7)) * 4 : 0;
}

template <class TO, Element EL, bool PAIR>
lrc_status rows_product(hipStream_t st, const char* name, GemmOperand A, GemmOperand B, int64_t M, int64_t N,
                        int64_t K, const Epilogue& ep, const Companion& co, float* partial, double flops,
                        double bytes) {
  Plan p = plan_rows(M, N, K, PAIR);
  TileGrid& tg = p.tg;
  tg.hold = PAIR && ep.codes != nullptr && p.tile == TINY;
  const int64_t grid = int64_t(NXCD) * tg.per_xcd * tg.splits;
  if (grid >= (int64_t(1) << 31)) return LRC_EINVAL;
  ProfScope scope(name, st, flops, bytes);
  const unsigned g = unsigned(grid);
  if (p.tile == LARGE)
    rows_product_kernel<TO, 4, 2, 4, 8, 2, EL, PAIR><<<g, 512, 0, st>>>(A, B, M, N, K, tg, ep, co, partial);
  else if (p.tile == SMALL) {
    // A checkpoint's blocks need waves with 64 channels of each weight (4051 x 832 -> 2816 57 us; through the workspace
    // and a second launch 82); otherwise square ones read fewer fragments.
    if constexpr (PAIR && EL == BF16) {
      if (ep.codes != nullptr && tg.splits == 1)
        rows_product_kernel<TO, 4, 1, 2, 8, 2, EL, PAIR><<<g, 256, 0, st>>>(A, B, M, N, K, tg, ep, co, partial);
      else
        rows_product_kernel<TO, 2, 2, 4, 4, 2, EL, PAIR><<<g, 256, 0, st>>>(A, B, M, N, K, tg, ep, co, partial);
    } else {
      rows_product_kernel<TO, 2, 2, 4, 4, 2, EL, PAIR><<<g, 256, 0, st>>>(A, B, M, N, K, tg, ep, co, partial);
    }
  }
  else
    rows_product_kernel<TO, 4, 1, 1, 4, 4, EL, PAIR><<<g, 256, 0, st>>>(A, B, M, N, K, tg, ep, co, partial);
  LRC_LAUNCHED();
  if (tg.splits == 1 && !tg.hold) return LRC_OK;
  const int64_t np = (N + 7) & ~int64_t(7), blocks = cdiv(N, CKB), threads = M * blocks * 8;
  if (cdiv(threads, 256) >= (int64_t(1) << 31)) return LRC_EINVAL;
  rows_finish_kernel<TO, EL, PAIR><<<unsigned(cdiv(threads, 256)), 256, 0, st>>>(partial, tg.splits, M, N, np, blocks,
                                                                                 ep, co);
  LRC_LAUNCHED();
  return LRC_OK;
}

// ---- few tokens: the weights streamed once ------------------------------------------------
// A wave holds 16 channels (of each weight) x 16 G tokens and takes a share of k; its weight fragments
// come straight from memory (a lane reads 16 bytes of one weight row, the four lanes of a row 64 bytes),
// x from the caches.  The waves' sums are added in order in LDS, then the epilogue.  PIECE: k steps of 64
// bytes of a row.
template <Element EL>
struct RowPiece;
template <>
struct RowPiece<BF16> {
  using T = uint16_t;
  using Acc = f32x4;
  static constexpr int K = 32;
  static __device__ __forceinline__ Acc mma(const u32x4& w, const u32x4& x, Acc c) {
    return Block<16>::mma(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x), c);
  }
};
template <>
struct RowPiece<FP32> {   // an instruction takes one of a lane's four k steps; any order of k serves both operands
  using T = uint32_t;
  using Acc = f32x4;
  static constexpr int K = 16;
  static __device__ __forceinline__ Acc mma(const u32x4& w, const u32x4& x, Acc c) {
    return Block<16>::mma_f32(__builtin_bit_cast(f32x4, w), __builtin_bit_cast(f32x4, x), c);
  }
};
template <>
struct RowPiece<INT8> {
  using T = uint8_t;
  using Acc = i32x4;
  static constexpr int K = 64;
  static __device__ __forceinline__ Acc mma(const u32x4& w, const u32x4& x, Acc c) {
    return Block<16>::mma_i8(__builtin_bit_cast(i32x4, w), __builtin_bit_cast(i32x4, x), c);
  }
};

// 16 bytes of a row at any alignment, zeros behind the `left` elements that exist
template <class T>
__device__ __forceinline__ u32x4 row_piece(const T* p, int left) {
  constexpr int EL = 16 / int(sizeof(T)), BITS = 8 * int(sizeof(T)), PER = 4 / int(sizeof(T));
  u32x4 v = {0u, 0u, 0u, 0u};
  if (left >= EL) {
    __builtin_memcpy(&v, p, 16);
  } else if (left > 0) {   // as ld_short
    T t[EL - 1];
#pragma unroll
    for (int e = 0; e < EL - 1; ++e) t[e] = p[min(e, left - 1)];
#pragma unroll
    for (int e = 0; e < EL - 1; ++e) v[e / PER] |= e < left ? uint32_t(t[e]) << (BITS * (e % PER)) : 0u;
  }
  return v;
}

// OWN (integers, at most OWN_TOKENS): x is the tokens themselves, in the type of y, and every workgroup quantises them
// into LDS while its first weights are on the way: a launch less, but each token's codes delay the workgroup.  One
// launch / two, us a call: one token 1024 -> 4096 5.6 / 8.5, 4096 -> 4096 6.9 / 9.4, 4096 -> 11008 11.4 / 15.2,
// 8192 -> 4096 10.1 / 12.2; four 1024 -> 4096 6.8 / 8.5, 4096 -> 4096 9.8 / 10.0, 4096 -> 11008 17 / 16.
constexpr int OWN_TOKENS = 4, OWN_ROOM = 16384;

template <class TO, int NW>
__device__ __forceinline__ void quantize_own(const TO* x, int64_t ldx, int n, int K, int pitch, int8_t* xq, float* xs,
                                             uint32_t (*red)[NW], bool& bad) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int t = 0; t < n; ++t) {
    const int c = 8 * threadIdx.x;   // K <= 512 NW
    float v[8];
    ld8(x + t * ldx + c, K - c, v);
    uint32_t m = wave_max(mag8(v, 0, bad));
    if (lane == 0) red[t & 1][wave] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW; ++w) m = max(m, red[t & 1][w]);
    const float s = token_step(m);
    if (threadIdx.x == 0) xs[t] = s;
    if (c < pitch) st8_token_codes(xq + t * pitch + c, 8, v, s, token_inverse(s), bad);
  }
  __syncthreads();
}

template <class TO, Element EL, int W, int G, int NW, bool OWN>
__global__ __launch_bounds__(64 * NW) void few_rows_kernel(const void* __restrict__ x, int64_t ldx,
                                                           const typename RowPiece<EL>::T* __restrict__ W0, int64_t ld0,
                                                           const typename RowPiece<EL>::T* __restrict__ W1, int64_t ld1,
                                                           int n, int64_t N, int K, Epilogue ep, Companion co) {
  using P = RowPiece<EL>;
  using T = typename P::T;
  // pieces in flight (of both weights; registers for more would leave a compute unit too few waves), elements of a
  // lane's 16 bytes
  constexpr int U = 4 / W, E = 16 / int(sizeof(T));
  __shared__ __attribute__((aligned(16))) typename P::Acc part[NW * W * G * 64];
  __shared__ __attribute__((aligned(16))) int8_t xq[OWN ? OWN_ROOM : 16];
  __shared__ float xs[OWN ? OWN_TOKENS : 1];
  __shared__ uint32_t red[2][NW];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t n0 = int64_t(blockIdx.x) * 16;
  // rows past the end repeat the last one, their results are not written
  const int64_t ch = min(n0 + (lane & 15), N - 1);
  const T* w[W];
  w[0] = W0 + ch * ld0;
  if constexpr (W == 2) w[1] = W1 + ch * ld1;
  const int pieces = (K + P::K - 1) / P::K, per = (pieces + NW - 1) / NW;
  const int p0 = wave * per, p1 = min(pieces, p0 + per), k0 = E * (lane >> 4);
  auto whole = [&](int p) { return (p + U) * P::K <= K && p + U <= p1; };
  u32x4 wv[U][W];
  auto load = [&](int p, u32x4 (&to)[U][W]) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < W; ++j) to[u][j] = row_piece<T>(w[j] + (p + u) * P::K + k0, E);
  };
  if (whole(p0)) load(p0, wv);
  const int pitch = (K + 63) & ~63;
  if constexpr (OWN) {
    bool bad = false;
    quantize_own<TO, NW>(static_cast<const TO*>(x), ldx, n, K, pitch, xq, xs, red, bad);
    if (ep.info != nullptr && bad) *ep.info = LRC_ENONFINITE;
  }
  const T* xr[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int t = min(16 * g + (lane & 15), n - 1);
    xr[g] = OWN ? reinterpret_cast<const T*>(xq) + t * pitch : static_cast<const T*>(x) + t * ldx;
  }
  typename P::Acc acc[W][G] = {};
  int p = p0;
  for (; whole(p); p += U) {   // the next pieces of the weights are loaded before these are used
    u32x4 next[U][W], xv[U][G];
    const bool more = whole(p + U);
    if (more) load(p + U, next);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int g = 0; g < G; ++g) xv[u][g] = row_piece<T>(xr[g] + (p + u) * P::K + k0, E);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int j = 0; j < W; ++j) acc[j][g] = P::mma(wv[u][j], xv[u][g], acc[j][g]);
    if (more) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < W; ++j) wv[u][j] = next[u][j];
    }
  }
  for (; p < p1; ++p) {   // k past the end reads as zero on both sides
    const int k = p * P::K + k0;
    u32x4 wt[W];
#pragma unroll
    for (int j = 0; j < W; ++j) wt[j] = row_piece<T>(w[j] + k, K - k);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const u32x4 xv = row_piece<T>(xr[g] + k, OWN ? E : K - k);
#pragma unroll
      for (int j = 0; j < W; ++j) acc[j][g] = P::mma(wt[j], xv, acc[j][g]);
    }
  }
#pragma unroll
  for (int j = 0; j < W; ++j)
#pragma unroll
    for (int g = 0; g < G; ++g) part[((wave * W + j) * G + g) * 64 + lane] = acc[j][g];
  __syncthreads();
  // accumulator element e of lane l: channel 4 (l / 16) + e, token l % 16
  using S = std::conditional_t<EL == INT8, int, float>;
  const S* sums = reinterpret_cast<const S*>(part);
  for (int i = threadIdx.x; i < G * 256; i += 64 * NW) {
    const int t = i >> 4, c = i & 15;
    const int64_t col = n0 + c;
    if (t >= n || col >= N) continue;
    const int at = (t >> 4) * 256 + ((c >> 2) * 16 + (t & 15)) * 4 + (c & 3);
    float v[W];
#pragma unroll
    for (int j = 0; j < W; ++j) {
      S s = 0;
#pragma unroll
      for (int q = 0; q < NW; ++q) s += sums[(q * W + j) * G * 256 + at];
      v[j] = float(s);
      if (EL == INT8) v[j] = v[j] * (j ? co.col_scale2 : co.col_scale)[col] * (OWN ? xs[t] : co.row_scale[t]);
    }
    if constexpr (W == 1) {
      if (ep.bias != nullptr) v[0] += ep.bias[col];
    }
    if (W == 2 && ep.z != nullptr) {
      st_elem(static_cast<TO*>(ep.z) + t * ep.ldz + col, v[0]);
      st_elem(static_cast<TO*>(co.z) + t * ep.ldz + col, v[W - 1]);
    }
    float a[1] = {v[0]};
    act_apply(ep.act, a);
    if (W == 2) a[0] *= v[W - 1];
    if (ep.res != nullptr) a[0] += ld_elem(static_cast<const TO*>(ep.res) + t * ep.ldr + col);
    st_elem(static_cast<TO*>(ep.y) + t * ep.ldy + col, a[0]);
  }
}

// waves of a workgroup of up to 16 tokens: with few channels more waves share the k of each
inline int few_waves(int64_t N) { return cdiv(N, 16) <= 256 ? 16 : 8; }
// Whether the few tokens are quantised by the product itself: where their codes fit the LDS room and a thread has at
// most eight channels of a token (quantize_own loads a token in one go).  Wider rows take the quantiser's launch: one
// token 11008 -> 4096 17.5 us, 8192 -> 28672 45.
inline bool own_tokens(int64_t n, int64_t N, int64_t K) {
  return n <= OWN_TOKENS && n * ((K + 63) & ~int64_t(63)) <= OWN_ROOM && K <= 512 * few_waves(N);
}

// Whether up to 64 tokens stream the weights.  Every 16 channels read x again (from the caches, about 9.5 TB/s), tiles
// read it once but where k is split end in a second launch of 4 to 5 us.  Integers, rows / tiles in us: 4096 -> 11008
// 10.8 / 11.3 at 4 tokens, 11.7 / 11.2 at 8, 19 / 11.7 at 32; split, 11008 -> 4096 15.9 / 16.5 at 24, 17.7 / 16.6 at 32,
// 4096 -> 4096 11.7 / 12.6 at 64; two weights 4096 -> 4096 9.9 / 10.1 at 32, 11.6 / 10.4 at 33.  Rows of no whole
// pieces, which tiles would first lay out anew, always do.
inline bool stream_int8(int64_t n, int64_t N, int64_t K, bool pair) {
  if (n > 64 || K % 16 != 0) return n <= 64;
  if (pair && n > 32) return false;
  const double x = double(cdiv(N, 16)) * double(n) * double(K);
  return x <= (plan_rows(n, N, K / 2, pair).tg.splits > 1 ? 75e6 : pair ? 16e6 : 24e6);
}
// bf16, two weights, rows / tiles (weights not in the caches).  Up to 8 tokens rows lose little where many channels fill
// the chip with tiles and gain more elsewhere: at 8 4096 -> 11008 39.7 / 38.9, 2048 -> 5632 14.8 / 14.0, 8192 -> 28672
// 169 / 165, 11008 -> 4096 39.3 / 43.1, 4096 -> 4096 16.1 / 19.4; at one 36.0 / 38.6, 14.1 / 13.8, 156 / 165, 37.5 / 42.8,
// 15.0 / 19.5.  More tokens: 4096 -> 11008 43.2 / 39.3 at 16, 11008 -> 4096 42.5 / 43.6 at 16 and 52 / 44 at 24,
// 1024 -> 4096 7.6 / 7.5 at 32.
inline bool stream_bf16_pair(int64_t n, int64_t N, int64_t K) {
  if (n > 64 || K % 8 != 0) return n <= 64;
  return n <= 8 || (n <= 32 && N * K <= (int64_t(1) << 22));
}

// fp32, two weights, rows / the linear layer's two products: 4096 -> 1024 35 / 33 at 17 tokens, 52 / 34 at 33; with more
// channels, whose waves fill the chip, 11008 -> 4096 90 / 114 at 16, 117 / 115 at 24, 4096 -> 4096 38 / 51 at 32,
// 55 / 52 at 33; rows that the products would lay out anew, 2999 -> 5001 76 / 112 at 64, 3957 -> 19 43 / 59.
inline bool stream_f32_pair(int64_t n, int64_t N, int64_t K) {
  const int64_t x = n * K;
  if (n > 64) return false;
  if (n <= 8 || x <= (int64_t(1) << 16) || (K % 4 != 0 && x <= (int64_t(1) << 18))) return true;
  return N >= 2048 && (n <= 16 || (n <= 32 && x <= (int64_t(1) << 17)));
}

// n <= 64; own: x is the tokens themselves (own_tokens)
template <class TO, Element EL, int W>
lrc_status few_rows(hipStream_t st, const char* name, const void* x, int64_t ldx, bool own, const void* W0, int64_t ld0,
                    const void* W1, int64_t ld1, int64_t n, int64_t N, int64_t K, const Epilogue& ep,
                    const Companion& co, double flops, double bytes) {
  using T = typename RowPiece<EL>::T;
  ProfScope scope(name, st, flops, bytes);
  const unsigned grid = unsigned(cdiv(N, 16));
  auto go = [&](auto groups, auto waves, auto quantise) {
    constexpr int G = decltype(groups)::value, NW = decltype(waves)::value;
    few_rows_kernel<TO, EL, W, G, NW, decltype(quantise)::value><<<grid, 64 * NW, 0, st>>>(
        x, ldx, static_cast<const T*>(W0), ld0, static_cast<const T*>(W1), ld1, int(n), N, int(K), ep, co);
  };
  using std::false_type;
  using std::integral_constant;
  if (own) {
    if constexpr (EL == INT8) {
      if (few_waves(N) == 16)
        go(integral_constant<int, 1>{}, integral_constant<int, 16>{}, std::true_type{});
      else
        go(integral_constant<int, 1>{}, integral_constant<int, 8>{}, std::true_type{});
    }
  } else if (n > 32) {
    go(integral_constant<int, 4>{}, integral_constant<int, 8>{}, false_type{});
  } else if (n > 16) {
    go(integral_constant<int, 2>{}, integral_constant<int, 8>{}, false_type{});
  } else if (few_waves(N) == 16) {
    go(integral_constant<int, 1>{}, integral_constant<int, 16>{}, false_type{});
  } else {
    go(integral_constant<int, 1>{}, integral_constant<int, 8>{}, false_type{});
  }
  LRC_LAUNCHED();
  return LRC_OK;
}

}  // namespace gemm
}  // namespace lrc
