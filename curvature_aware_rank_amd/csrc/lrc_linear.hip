// Linear layer of a token block: y = act(x W^T + b) + residual, and its gradients from
// activations kept in full or in 8 bits.
//
// All three products are D[m][n] = sum_k A(m, k) B(n, k):
//   forward  m = token, n = output channel, k = input channel;   A = x, B = W: rows along k
//   dx       m = token, n = input channel,  k = output channel;  A = dz rows, B = W's columns
//   dW       m = output channel, n = input channel, k = token;   A, B = columns of dz and x
// An operand is therefore a row-major matrix whose rows run along k (K_ROWS) or whose rows
// are the k steps (K_COLS), or a checkpoint of the latter kind (K_CODES).
#include "lrc_train.h"

#include <algorithm>
#include <type_traits>

namespace lrc {
namespace {

constexpr int LT = 256;

__device__ __forceinline__ int64_t cdiv_dev(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Operand {
  const void* p;        // elements, or int8 codes (leading dim ld)
  int64_t ld;
  const int8_t* exps;   // K_CODES: block exponents, nb per row
  int64_t nb;
  bool vec;             // rows are whole aligned 16-byte pieces
};

// ---- any size, stride and alignment: 64 x 64 tiles, four waves of 32 x 32 ---------------
// Operands pass through registers into LDS as [row][k], a step ahead of the products; two LDS
// buffers, one barrier a step (2048 x 2048 x 1024: fp32 93 us, 92 TFLOP/s; bf16 60).  Bound by the
// latency of a step's loads where tiles are few, so k
// is then split over workgroups and the splits' tiles are added in order by a second kernel.
constexpr int GT = 64;    // tile edge

template <class T>
struct GTile {
  static constexpr int K = sizeof(T) == 2 ? 64 : 32;   // k per step: 128 bytes of a row
  static constexpr int PITCH = sizeof(T) == 2 ? K + 8 : K + 4;
  static constexpr int PIECES = GT * K / 8 / LT;       // pieces of eight of a thread and step
};

// Eight values of an operand as T bits: for K_ROWS along k at (row, k), for the others along
// the rows at step k.
template <class T, int KIND>
__device__ __forceinline__ void operand8(const Operand& o, int64_t row, int64_t k, int64_t rows, int64_t kk,
                                         float (&v)[8]) {
  if (KIND == K_ROWS) {
    const int64_t left = row < rows ? kk - k : 0;
    ld8(static_cast<const T*>(o.p) + row * o.ld + k, int(left < 0 ? 0 : left > 8 ? 8 : left), v);
    return;
  }
  const int64_t left = k < kk ? rows - row : 0;
  const int cnt = int(left < 0 ? 0 : left > 8 ? 8 : left);
  if (KIND == K_COLS) {
    ld8(static_cast<const T*>(o.p) + k * o.ld + row, cnt, v);
  } else {   // eight channels from a multiple of eight: one block
    const float step = cnt > 0 ? pow2f(o.exps[k * o.nb + (row >> 6)]) : 0.f;
    ld8_codes(static_cast<const int8_t*>(o.p) + k * o.ld + row, cnt, step, v);
  }
}

__device__ __forceinline__ void lds_put8(float* p, const float (&v)[8]) {
  *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
  *reinterpret_cast<f32x4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ void lds_put8(uint16_t* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                            pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// Piece i of a thread: its tile row and k (K_ROWS: along k, else along the rows).
template <class T, int KIND>
__device__ __forceinline__ void piece_at(int i, int& row, int& k) {
  const int p = threadIdx.x + LT * i;
  if (KIND == K_ROWS) {
    row = p / (GTile<T>::K / 8);
    k = p % (GTile<T>::K / 8) * 8;
  } else {
    k = p >> 3;
    row = (p & 7) * 8;
  }
}
template <class T, int KIND>
__device__ __forceinline__ void fetch_any(const Operand& o, int64_t row0, int64_t k0, int64_t rows, int64_t kk,
                                          float (&v)[GTile<T>::PIECES][8]) {
#pragma unroll
  for (int i = 0; i < GTile<T>::PIECES; ++i) {
    int row, k;
    piece_at<T, KIND>(i, row, k);
    operand8<T, KIND>(o, row0 + row, k0 + k, rows, kk, v[i]);
  }
}
template <class T, int KIND>
__device__ __forceinline__ void store_any(T* lds, const float (&v)[GTile<T>::PIECES][8]) {
  constexpr int P = GTile<T>::PITCH;
#pragma unroll
  for (int i = 0; i < GTile<T>::PIECES; ++i) {
    int row, k;
    piece_at<T, KIND>(i, row, k);
    if (KIND == K_ROWS) {
      lds_put8(lds + row * P + k, v[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) st_elem(lds + (row + e) * P + k, v[i][e]);
    }
  }
}

__device__ __forceinline__ void mma_any(const uint16_t* a, const uint16_t* b, int lane, f32x4& acc) {
  const int off = (lane & 15) * GTile<uint16_t>::PITCH + 8 * (lane >> 4);
#pragma unroll
  for (int s = 0; s < GTile<uint16_t>::K; s += 32)
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(*reinterpret_cast<const bf16x8*>(a + off + s),
                                                  *reinterpret_cast<const bf16x8*>(b + off + s), acc, 0, 0, 0);
}
__device__ __forceinline__ void mma_any(const float* a, const float* b, int lane, f32x4& acc) {
  const int off = (lane & 15) * GTile<float>::PITCH + (lane >> 4);
#pragma unroll
  for (int s = 0; s < GTile<float>::K; s += 4)
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[off + s], b[off + s], acc, 0, 0, 0);
}

struct AnyPlan {
  int64_t tiles_n, tiles;
  int splits;
  int64_t k_per_split;
};
template <class T>
AnyPlan plan_any(int64_t M, int64_t N, int64_t K) {
  AnyPlan p;
  p.tiles_n = cdiv(N, GT);
  p.tiles = cdiv(M, GT) * p.tiles_n;
  const int64_t steps = std::max<int64_t>(1, cdiv(K, GTile<T>::K));
  // up to four workgroups per compute unit (their steps' loads hide each other), eight steps at
  // least in each split (a second launch and the partial tiles cost about as much as eight steps)
  const int64_t s = std::max<int64_t>(1, std::min<int64_t>({1024 / std::max<int64_t>(1, p.tiles), steps / 8, 32}));
  const int64_t per = cdiv(steps, s);
  p.splits = int(cdiv(steps, per));
  p.k_per_split = per * GTile<T>::K;
  return p;
}

// `only`: NULL, or a device word without which the product is not wanted.  The workgroups take
// tiles in turn, so that a product that is not wanted costs few of them.
template <class T, class TO, int KA, int KB>
__global__ __launch_bounds__(LT) void linear_any_kernel(Operand A, Operand B, int64_t M, int64_t N, int64_t K,
                                                        AnyPlan plan, Epilogue ep, float* __restrict__ partial,
                                                        const int32_t* __restrict__ only) {
  if (only != nullptr && *only == 0) return;
  constexpr int P = GTile<T>::PITCH, PC = GTile<T>::PIECES, BK = GTile<T>::K;
  constexpr int EP = GT + 4;   // epilogue tile pitch
  constexpr int STAGE = 2 * GT * P * int(sizeof(T));
  __shared__ __attribute__((aligned(16))) uint8_t lds[GT * EP * 4 > 2 * STAGE ? GT * EP * 4 : 2 * STAGE];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wr = (wave >> 1) * 32, wc = (wave & 1) * 32;
  const int split = blockIdx.y;
  const int64_t k_begin = int64_t(split) * plan.k_per_split, k_end = min(K, k_begin + plan.k_per_split);
  bool bad = false;
  for (int64_t tile_i = blockIdx.x; tile_i < plan.tiles; tile_i += gridDim.x) {
    const int64_t m0 = tile_i / plan.tiles_n * GT, n0 = tile_i % plan.tiles_n * GT;
    f32x4 acc[2][2] = {};
    float va[PC][8], vb[PC][8];
    fetch_any<T, KA>(A, m0, k_begin, M, k_end, va);
    fetch_any<T, KB>(B, n0, k_begin, N, k_end, vb);
    int buf = 0;
    for (int64_t k0 = k_begin; k0 < k_end; k0 += BK, buf ^= 1) {
      T* la = reinterpret_cast<T*>(lds + buf * STAGE);
      T* lb = la + GT * P;
      store_any<T, KA>(la, va);
      store_any<T, KB>(lb, vb);
      if (k0 + BK < k_end) {
        fetch_any<T, KA>(A, m0, k0 + BK, M, k_end, va);
        fetch_any<T, KB>(B, n0, k0 + BK, N, k_end, vb);
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) mma_any(la + (wr + 16 * i) * P, lb + (wc + 16 * j) * P, lane, acc[i][j]);
    }
    __syncthreads();
    float* tile = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          tile[(wr + 16 * i + 4 * (lane >> 4) + e) * EP + wc + 16 * j + (lane & 15)] = acc[i][j][e];
    __syncthreads();
    const int64_t col = n0 + 8 * (lane & 7), np = (N + 7) & ~int64_t(7);
    float bias[8];
    bias8(ep, col, int(min(N - col, int64_t(8))), bias);
    for (int r = threadIdx.x >> 3; r < GT; r += LT / 8) {
      const int64_t row = m0 + r;
      const int64_t left = row < M ? N - col : 0;
      const int cnt = int(left < 0 ? 0 : left > 8 ? 8 : left);
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = tile[r * EP + 8 * (lane & 7) + e];
      if (plan.splits > 1) {
        if (cnt > 0) st8(partial + (int64_t(split) * M + row) * np + col, 8, v);
      } else {
        finish8<TO>(ep, row, col, cnt, bias, v, lane, bad);
      }
    }
    __syncthreads();   // the tile is read before the next one's steps
  }
  if (ep.info != nullptr && bad) *ep.info = LRC_ENONFINITE;
}

// ---- few tokens: the weight streamed once ------------------------------------------------
// Up to 64 tokens.  Bound by reading W (4096 to 11008 bf16, one token: 17 us, 5.3 TB/s): a wave holds 16 output channels x 16 G tokens and takes
// a share of k; its W fragments come straight from memory (a lane reads 16 bytes of one weight
// row, the four lanes of a row 64 bytes, four such pieces in flight), x comes from the caches.
// The waves' sums are added in order in LDS, then the epilogue.  fp32: a 16-byte piece holds
// four k steps, one matrix instruction takes one of them from every lane (any order of k serves
// as long as both operands agree on it).
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <class T>
struct RowsPiece;
template <>
struct RowsPiece<uint16_t> {
  static constexpr int K = 32;
  static __device__ __forceinline__ void mma(const u32x4& w, const u32x4& x, f32x4& acc) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x), acc, 0,
                                                  0, 0);
  }
};
template <>
struct RowsPiece<float> {
  static constexpr int K = 16;
  static __device__ __forceinline__ void mma(const u32x4& w, const u32x4& x, f32x4& acc) {
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w[0]), __uint_as_float(x[0]), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w[1]), __uint_as_float(x[1]), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w[2]), __uint_as_float(x[2]), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w[3]), __uint_as_float(x[3]), acc, 0, 0, 0);
  }
};

// 16 bytes of a row at any alignment, zeros behind the `left` elements that exist
template <class T>
__device__ __forceinline__ u32x4 piece(const T* p, int left) {
  constexpr int EL = 16 / int(sizeof(T));
  u32x4 v = {0u, 0u, 0u, 0u};
  if (left >= EL) {
    __builtin_memcpy(&v, p, 16);
  } else if (left > 0) {   // as ld_short
    T t[EL - 1];
#pragma unroll
    for (int e = 0; e < EL - 1; ++e) t[e] = p[min(e, left - 1)];
#pragma unroll
    for (int e = 0; e < EL - 1; ++e) {
      const uint32_t u = sizeof(T) == 4 ? __float_as_uint(float(t[e])) : uint32_t(t[e]) << (16 * (e & 1));
      v[sizeof(T) == 4 ? e : e >> 1] |= e < left ? u : 0u;
    }
  }
  return v;
}

template <class T, int G, int NW>
__global__ __launch_bounds__(64 * NW) void linear_rows_kernel(const T* __restrict__ x, int64_t ldx,
                                                              const T* __restrict__ W, int64_t ldw, int n, int64_t N,
                                                              int K, Epilogue ep) {
  using P = RowsPiece<T>;
  constexpr int U = 4, EL = 16 / int(sizeof(T));   // pieces in flight, elements of a piece
  __shared__ __attribute__((aligned(16))) float part[NW * G * 256];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t n0 = int64_t(blockIdx.x) * 16;
  // rows past the end repeat the last one, their results are not written
  const T* w = W + min(n0 + (lane & 15), N - 1) * ldw;
  const T* xr[G];
#pragma unroll
  for (int g = 0; g < G; ++g) xr[g] = x + int64_t(min(16 * g + (lane & 15), n - 1)) * ldx;
  const int pieces = (K + P::K - 1) / P::K, per = (pieces + NW - 1) / NW;
  const int p0 = wave * per, p1 = min(pieces, p0 + per), k0 = EL * (lane >> 4);
  f32x4 acc[G] = {};
  int p = p0;
  for (; (p + U) * P::K <= K && p + U <= p1; p += U) {
    u32x4 wv[U], xv[U][G];
#pragma unroll
    for (int u = 0; u < U; ++u) wv[u] = piece<T>(w + (p + u) * P::K + k0, EL);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int g = 0; g < G; ++g) xv[u][g] = piece<T>(xr[g] + (p + u) * P::K + k0, EL);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int g = 0; g < G; ++g) P::mma(wv[u], xv[u][g], acc[g]);
  }
  for (; p < p1; ++p) {   // k past the end reads as zero on both sides
    const int k = p * P::K + k0;
    const u32x4 wv = piece<T>(w + k, K - k);
#pragma unroll
    for (int g = 0; g < G; ++g) P::mma(wv, piece<T>(xr[g] + k, K - k), acc[g]);
  }
#pragma unroll
  for (int g = 0; g < G; ++g) *reinterpret_cast<f32x4*>(part + ((wave * G + g) * 64 + lane) * 4) = acc[g];
  __syncthreads();
  // accumulator element e of lane l: channel 4 (l / 16) + e, token l % 16
  for (int i = threadIdx.x; i < G * 256; i += 64 * NW) {
    const int t = i >> 4, c = i & 15;
    const int64_t col = n0 + c;
    if (t >= n || col >= N) continue;
    const int at = (t >> 4) * 256 + ((c >> 2) * 16 + (t & 15)) * 4 + (c & 3);
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < NW; ++q) v += part[q * G * 256 + at];
    if (ep.bias != nullptr) v += ep.bias[col];
    if (ep.z != nullptr) st_elem(static_cast<T*>(ep.z) + t * ep.ldz + col, v);
    float a[1] = {v};
    act_apply(ep.act, a);
    v = a[0];
    if (ep.res != nullptr) v += ld_elem(static_cast<const T*>(ep.res) + t * ep.ldr + col);
    st_elem(static_cast<T*>(ep.y) + t * ep.ldy + col, v);
  }
}

// Up to 8 tokens always.  Up to 64 where x, which every 16 channels read again, is small beside a
// launch (bf16 rows / tiles with split k, us: 4096 x 4096 at 16 tokens 10.0 / 13.4, at 32 13.8 / 13.0;
// 2048 x 2048 at 48 10.5 / 11.0, at 64 12.0 / 11.8; 8192 x 1024 at 8 13.9 / 14.3, at 24 21 / 12; fp32
// 4096 x 4096 at 16 23 / 27, at 32 31 / 29) and W, in bf16, too (4096 x 11008 at 16 29 / 24); and
// where tiles would first lay W out anew (whole rows of no whole pieces: as much again as reading
// it twice).
bool few_tokens(int64_t n, int64_t di, int64_t dn, size_t size) {
  if (n <= 8 || n > 64) return n <= 8;
  if (di % int64_t(16 / size) != 0) return true;
  return size == 2 ? n * di <= (int64_t(3) << 15) && di * dn <= (int64_t(1) << 24) : n * di <= (int64_t(1) << 16);
}

template <class T>
lrc_status linear_rows(hipStream_t st, const Operand& x, const Operand& W, int64_t n, int64_t dn, int64_t di,
                       const Epilogue& ep, double bytes) {
  ProfScope scope("linear_rows_kernel", st, 2.0 * double(n) * double(dn) * double(di), bytes);
  const unsigned grid = unsigned(cdiv(dn, 16));
  auto go = [&](auto groups) {
    constexpr int G = decltype(groups)::value;
    const T *xp = static_cast<const T*>(x.p), *wp = static_cast<const T*>(W.p);
    // few channels: more waves share the k of each
    if (grid <= 256)
      linear_rows_kernel<T, G, 16><<<grid, 1024, 0, st>>>(xp, x.ld, wp, W.ld, int(n), dn, int(di), ep);
    else
      linear_rows_kernel<T, G, 8><<<grid, 512, 0, st>>>(xp, x.ld, wp, W.ld, int(n), dn, int(di), ep);
  };
  if (n <= 16)
    go(std::integral_constant<int, 1>{});
  else if (n <= 32)
    go(std::integral_constant<int, 2>{});
  else
    go(std::integral_constant<int, 4>{});
  LRC_LAUNCHED();
  return LRC_OK;
}

// ---- chunks of tokens ---------------------------------------------------------------------
struct ColPlan {
  int64_t rows, chunks;   // tokens per chunk
};
// Chunks of 8 to 32 tokens, enough of them to spread a short or narrow stream over the chip (dz of
// 3588 x 22: 32 tokens a chunk 21 us, 8 tokens 8 us); up to 32 tokens are one chunk of sixteen waves
// (25 x 866: 12 us against 20 on four), whose sums need no second pass.
ColPlan col_plan(int64_t n, int64_t d) {
  ColPlan p;
  const int64_t spread = (n * cdiv(d, 512) / 1024 + 3) & ~int64_t(3);
  p.rows = n <= 32 ? 32 : std::max(std::min<int64_t>(32, std::max<int64_t>(8, spread)), cdiv(n, 1024));
  p.chunks = cdiv(n, p.rows);
  return p;
}

// ---- dz = dy act'(z), and the chunk sums of db ------------------------------------------
// Bound by memory: dy and z read, dz written, and its lower piece (8192 x 11008 from codes 139 us,
// 4.5 TB/s).  A lane takes eight consecutive channels, the workgroup's waves take the chunk's tokens
// in turn; db's share of the chunk is the waves' sums added in order.
//
// The dW of a bf16 layer whose activation has a smooth slope takes dz in two bf16 pieces, the stream
// and `low`, what the stream's rounding left out (rows of w8): 16 bits, so that dW carries no more
// than its own rounding (with the stream alone its error was 1.3 to 1.55 times that), for a second
// product (650 us at 8192 x 4096 x 11008).  Both pieces have the range of fp32, so a token that counts
// for nothing may hold any finite value on the side that meets zeros.
template <class T, bool CK, int NW>
__global__ __launch_bounds__(64 * NW) void dz_kernel(const T* __restrict__ dy, int64_t lddy, int64_t n, int64_t d,
                                                const T* __restrict__ z, int64_t ldz,
                                                const int8_t* __restrict__ codes, const int8_t* __restrict__ exps,
                                                int64_t nb, int act, T* __restrict__ dz, int64_t lddz, int64_t rows,
                                                float* __restrict__ partial,
                                                int32_t* __restrict__ clear, uint16_t* __restrict__ low,
                                                int64_t w8) {
  __shared__ float sums[NW - 1][64][9];
  if (clear != nullptr && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) clear[0] = clear[1] = 0;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t(blockIdx.x) * 64 + lane) * 8;
  const int64_t left = d - c;
  const int cnt = int(left < 0 ? 0 : left > 8 ? 8 : left);
  const int64_t t0 = int64_t(blockIdx.y) * rows, t1 = min(n, t0 + rows);
  float s[8] = {};
  auto run = [&](auto whole) {   // whole pieces: no branches between the loads, which overlap
    const int len = decltype(whole)::value ? 8 : cnt;
#pragma unroll 2
    for (int64_t t = t0 + wave; t < t1; t += NW) {
      float g[8];
      ld8(dy + t * lddy + c, len, g);
      if (act != LRC_ACT_NONE) {
        float zv[8];
        if (CK)
          ld8_codes(codes + t * d + c, len, pow2f(exps[t * nb + (c >> 6)]), zv);
        else
          ld8(z + t * ldz + c, len, zv);
        slope_apply(act, zv, g);
        st8(dz + t * lddz + c, len, g);
        if (low != nullptr) {   // zeros behind the last channel, and where the stream is not finite
          float r[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float h = round_to(g[e], static_cast<const uint16_t*>(nullptr));
            r[e] = finite_f(h) ? g[e] - h : 0.f;
          }
          st8(low + t * w8 + c, 8, r);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] += g[e];
    }
  };
  if (cnt >= 8)
    run(std::true_type{});
  else if (cnt > 0)
    run(std::false_type{});
  if (partial == nullptr) return;
  if (wave > 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[wave - 1][lane][e] = s[e];
  }
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
#pragma unroll
    for (int w = 0; w < NW - 1; ++w) s[e] += sums[w][lane][e];
    if (e < cnt) partial[int64_t(blockIdx.y) * d + c + e] = s[e];
  }
}

// rows of `halves` 16-bit words, pitch `ld`, set to zero
__global__ __launch_bounds__(LT) void zero_rows_kernel(uint16_t* p, int64_t rows, int64_t halves, int64_t ld) {
  const int64_t step = int64_t(gridDim.x) * LT;
  for (int64_t i = int64_t(blockIdx.x) * LT + threadIdx.x; i < rows * halves; i += step)
    p[i / halves * ld + i % halves] = 0;
}

constexpr int64_t DMAX = int64_t(1) << 24;
bool sizes_ok(int64_t n, int64_t i, int64_t o) {
  return n >= 0 && n < (int64_t(1) << 31) && i >= 1 && i <= DMAX && o >= 1 && o <= DMAX;
}
bool act_ok(int a) { return a >= LRC_ACT_NONE && a <= LRC_ACT_SILU; }

// ---- operands for the matrix cores ------------------------------------------------------
// An operand the bf16 product cannot read where it lies is first written to the workspace as
// rows of `planes` pieces of w8 = 8 ceil(cols / 8) bf16 (zeros behind the columns):
//   bf16 whose rows are not whole 16-byte pieces, and checkpoints (exact in bf16): one piece;
//   fp32 on fp32 tiles: one piece of fp32, where its rows are not whole 16-byte pieces;
//   fp32 otherwise: three pieces with x = h + m + l exactly (8 + 8 + 8 significant bits).  A product of
//   two such operands is h h + h m + m h + h l + m m + l h, the terms left out are below
//   2^-24 of it: six bf16 products give fp32 accuracy at more than the fp32 matrix rate.  An
//   infinity would meet one of the other sign from the lower pieces.  So an entry that is not finite
//   or passes SPLIT_MAX raises `flag`, and the product is done on fp32 tiles instead; without one no
//   sum of up to GEMM_MAX_K terms passes 2^127.
constexpr float SPLIT_MAX = 0x1p50f;
template <class T>
__device__ __forceinline__ void split_store(uint16_t* o, int64_t w8, float (&v)[8], bool& bad);
template <>
__device__ __forceinline__ void split_store<uint16_t>(uint16_t* o, int64_t, float (&v)[8], bool&) {
  st8(o, 8, v);
}
template <>
__device__ __forceinline__ void split_store<float>(uint16_t* o, int64_t w8, float (&v)[8], bool& bad) {
  float h[8], m[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    bad |= !(fabsf(v[e]) <= SPLIT_MAX);
    h[e] = round_to(v[e], static_cast<const uint16_t*>(nullptr));
    const float r = v[e] - h[e];
    m[e] = round_to(r, static_cast<const uint16_t*>(nullptr));
    v[e] = r - m[e];
  }
  st8(o, 8, h);
  st8(o + w8, 8, m);
  st8(o + 2 * w8, 8, v);
}
// Up to three operands in one launch: a workgroup belongs to the job its index falls into.
struct OperandJob {
  const void* p = nullptr;
  const int8_t* exps = nullptr;   // codes if not NULL
  uint16_t* out = nullptr;
  int64_t ld = 0, nb = 0, rows = 0, cols = 0, w8 = 0, blocks = 0;
  int planes = 1;                      // of bf16; 0: one of fp32
  unsigned raises = 0;                 // the products that read it, bit i the one that flag[i] moves
};
constexpr int JOB_ROWS = 4;   // rows of a thread
struct OperandJobs {
  OperandJob job[3];
};
template <class T>
__global__ __launch_bounds__(LT) void operand_kernel(OperandJobs jobs, int32_t* __restrict__ flag) {
  int64_t block = blockIdx.x;
  int q = 0;
  while (q < 2 && block >= jobs.job[q].blocks) block -= jobs.job[q++].blocks;
  const OperandJob& j = jobs.job[q];
  // four rows of one piece of columns
  const int64_t i = block * LT + threadIdx.x, per = j.w8 / 8;
  const int64_t r0 = i / per * JOB_ROWS, c = i % per * 8;
  if (r0 >= j.rows) return;
  const int cnt = int(j.cols - c > 8 ? 8 : j.cols - c);
  float v[JOB_ROWS][8];
  bool bad = false;
  auto load = [&](auto whole) {   // whole pieces: no branches between the loads, which overlap
    const int len = decltype(whole)::value ? 8 : cnt;
#pragma unroll
    for (int q4 = 0; q4 < JOB_ROWS; ++q4) {
      const int64_t r = min(r0 + q4, j.rows - 1);
      if (j.exps != nullptr)
        ld8_codes(static_cast<const int8_t*>(j.p) + r * j.ld + c, len, pow2f(j.exps[r * j.nb + (c >> 6)]), v[q4]);
      else
        ld8(static_cast<const T*>(j.p) + r * j.ld + c, len, v[q4]);
    }
  };
  if (cnt >= 8)
    load(std::true_type{});
  else
    load(std::false_type{});
#pragma unroll
  for (int q4 = 0; q4 < JOB_ROWS; ++q4) {
    const int64_t r = r0 + q4;
    if (r >= j.rows) break;
    uint16_t* o = j.out + r * j.planes * j.w8 + c;
    if (j.planes == 0)
      st8(reinterpret_cast<float*>(j.out) + r * j.w8 + c, 8, v[q4]);
    else if (j.exps != nullptr) {
      split_store<uint16_t>(o, j.w8, v[q4], bad);
      if (sizeof(T) == 4) {   // one exact piece, which meets three
#pragma unroll
        for (int e = 0; e < 8; ++e) bad |= fabsf(v[q4][e]) > SPLIT_MAX;
      }
    } else {
      split_store<T>(o, j.w8, v[q4], bad);
    }
  }
  if (sizeof(T) == 4 && bad) {
    if (j.raises & 1) flag[0] = 1;
    if (j.raises & 2) flag[1] = 1;
  }
}
__global__ void clear_flag_kernel(int32_t* flag) { flag[0] = flag[1] = 0; }

int64_t round8(int64_t v) { return (v + 7) & ~int64_t(7); }

// Room in the workspace for one such operand, in bf16.
template <class T>
size_t operand_room(int64_t rows, int64_t cols) {
  return size_t(rows) * (sizeof(T) == 4 ? 3 : 1) * round8(cols);
}

struct Prepared {
  GemmOperand op;
  int planes;
};

// Adds the operand to the jobs if it cannot be read where it lies.
template <class T>
Prepared want_operand(OperandJobs& jobs, int& count, const Operand& o, int64_t rows, int64_t cols, uint16_t* room,
                      bool native, unsigned raises) {
  const bool codes = o.exps != nullptr, there = !codes && o.vec && o.ld <= GEMM_MAX_LD;
  if (native && there && cols % 4 == 0) return {{static_cast<const uint16_t*>(o.p), 2 * o.ld, 0}, 1};
  if (sizeof(T) == 2 && there && cols % 8 == 0)
    return {{static_cast<const uint16_t*>(o.p), o.ld, 0}, 1};
  OperandJob& j = jobs.job[count++];
  j.p = o.p;
  j.exps = o.exps;
  j.out = room;
  j.ld = o.ld;
  j.nb = o.nb;
  j.rows = rows;
  j.cols = cols;
  j.w8 = round8(cols);
  j.planes = native ? 0 : sizeof(T) == 4 && !codes ? 3 : 1;
  j.raises = raises;
  j.blocks = cdiv(cdiv(rows, JOB_ROWS) * (j.w8 / 8), LT);
  if (native) return {{room, 2 * j.w8, 0}, 1};
  return {{room, j.planes * j.w8, j.w8}, j.planes};
}
template <class T>
lrc_status prepare_operands(hipStream_t st, const OperandJobs& jobs, int count, int32_t* flag) {
  if (count == 0) return LRC_OK;
  int64_t grid = 0;
  double bytes = 0;
  for (int i = 0; i < count; ++i) {
    const OperandJob& j = jobs.job[i];
    grid += j.blocks;
    bytes += double(j.rows) * double(j.cols) * ((j.exps ? 1.0 : double(sizeof(T))) + (j.planes ? 2.0 * j.planes : 4.0));
  }
  if (grid >= (int64_t(1) << 31)) return LRC_EINVAL;
  ProfScope scope("linear_operand_kernel", st, 0.0, bytes);
  operand_kernel<T><<<unsigned(grid), LT, 0, st>>>(jobs, flag);
  LRC_LAUNCHED();
  return LRC_OK;
}

// segments of a product of operands with so many planes (h, m, l), smallest terms first
GemmSegments segments(int pa, int pb) {
  GemmSegments s;
  auto add = [&](int i, uint32_t a, uint32_t b) {
    s.pa |= a << (2 * i);
    s.pb |= b << (2 * i);
    s.count = i + 1;
  };
  if (pa == 3 && pb == 3) {
    add(0, 2, 0), add(1, 0, 2), add(2, 1, 1), add(3, 1, 0), add(4, 0, 1), add(5, 0, 0);
  } else if (pa == 3) {
    add(0, 2, 0), add(1, 1, 0), add(2, 0, 0);
  } else if (pb == 3) {
    add(0, 0, 2), add(1, 0, 1), add(2, 0, 0);
  }
  return s;
}

// Whether the products may go to the pipelined tiles (lrc_gemm.hip) or all to the ones that take
// any operand.  bf16, forward / dx / dW in us, pipelined against any: in place 65 x 16 x 16 3.9 / 5.3 /
// 4.3 against 4.5 / 5.0 / 6.6, 1000 x 16 x 16 4 / 4 / 8 against 5 / 5 / 20, 2048 x 2048 x 1024 18 / 18
// / 19 against 68 / 66 / 89; laid out first 1000 x 17 x 17 8 / 8 / 12 against 6 / 6 / 27, 300 x 65 x 65
// 9 / 9 / 10 against 6 / 7 / 15, 1000 x 521 x 303 12 / 12 / 14 against 14 / 14 / 28: whole pieces
// always, others from 2^18 multiplications.  fp32 from 2^24, where F32Times chooses.
template <class T>
bool large_product(int64_t n, int64_t di, int64_t dn) {
  const double work = double(n) * double(di) * double(dn);
  if (n > GEMM_MAX_K) return false;
  if (sizeof(T) == 2 && di % 8 == 0 && dn % 8 == 0) return true;
  return work >= double(sizeof(T) == 2 ? 1 << 18 : 1 << 24);
}
// How the large fp32 products of a call run: on the tiles that take any operand (ANY), on pipelined
// fp32 tiles (NATIVE), or in three bf16 pieces (SPLIT), by the shortest estimate in microseconds.
// Measured forward, all three: 301 x 1928 x 768 22 / 19 / 39, 1024^3 33 / 23 / 42, 123 x 7725 x 1049
// (rows laid out anew) 36 / 50 / 70, 2048 x 2048 x 1024 93 / 68 / 83, 6913 x 1075 x 1981 299 / 257 /
// 191, 7547 x 3581 x 640 365 / 334 / 269.
enum F32Way { ANY, NATIVE, SPLIT };
struct F32Times {
  double any = 0, native = 0, split = 14;   // (the split's launches before and behind its products)
  void product(int64_t M, int64_t N, int64_t K, int KA, int KB) {
    // 32 k steps of a 64 x 64 tile: 1.3 us alone on a compute unit (the latency of its loads), less
    // by far with others there, more where operands run along columns
    const AnyPlan p = plan_any<float>(M, N, K);
    const double each = double(cdiv(p.tiles * p.splits, 256)), step = KA == K_COLS ? 0.9 : KB == K_COLS ? 0.72 : 0.65;
    any += 6.0 + double(cdiv(p.k_per_split, 32)) * std::max(1.3, each * step);
    if (p.splits > 1) any += 6.0 + 8.0 * p.splits * double(M) * double(N) / 4.5e6;
    native += gemm_f32_time(M, N, K);
    split += gemm_split_time(M, N, K, KA, KB);
  }
  // (by the sizes alone, so that rows of another alignment give the same bits)
  void operand(int64_t rows, int64_t cols) {
    const double cells = double(rows) * double(cols);
    split += cells * 10.0 / 4.5e6;
    if (cols % 4 != 0) native += (native_copies++ ? 0.0 : 5.0) + cells * 8.0 / 4.5e6;
  }
  int native_copies = 0;
  F32Way way() const { return any <= std::min(native, split) ? ANY : native <= split ? NATIVE : SPLIT; }
};
template <class T>
bool gemm_fits(int64_t rows_a, int64_t rows_b) {   // row lengths of the two operands
  return std::max(round8(rows_a), round8(rows_b)) * (sizeof(T) == 4 ? 3 : 1) <= GEMM_MAX_LD;
}

template <class T, class TO, int KA, int KB>
lrc_status product_any(hipStream_t st, const char* name, const Operand& A, const Operand& B, int64_t M, int64_t N,
                       int64_t K, const Epilogue& ep, float* partial, const int32_t* only, double bytes) {
  AnyPlan p = plan_any<T>(M, N, K);
  if (only) p.splits = 1, p.k_per_split = K;
  ProfScope scope(name, st, only ? 0.0 : 2.0 * double(M) * double(N) * double(K), only ? 0.0 : bytes);
  const dim3 grid(unsigned(std::min<int64_t>(p.tiles, only ? 1024 : int64_t(1) << 20)), unsigned(p.splits));
  linear_any_kernel<T, TO, KA, KB><<<grid, LT, 0, st>>>(A, B, M, N, K, p, ep, partial, only);
  LRC_LAUNCHED();
  return p.splits > 1 ? gemm_finish<TO>(st, partial, p.splits, M, N, ep, nullptr) : LRC_OK;
}
template <class T>
size_t any_room(int64_t M, int64_t N, int64_t K) {
  const AnyPlan p = plan_any<T>(M, N, K);
  return p.splits > 1 ? size_t(p.splits) * M * round8(N) : 0;
}

template <class T>
Operand plain(const void* p, int64_t ld) {
  return {p, ld, nullptr, 0, rows_vec16(p, ld, sizeof(T))};
}
template <class T>
void set_out(Epilogue& ep, void* y, int64_t ldy) {
  ep.y = y;
  ep.ldy = ldy;
}

// Workspace of the three products.
struct LinearRoom {
  int32_t* flag = nullptr;      // an fp32 operand of y or dx, or of dW, holds an entry that must not be split
  float* partial = nullptr;     // split products
  float* sums = nullptr;        // db chunks
  uint16_t *a = nullptr, *b = nullptr, *c = nullptr;   // operands
  uint16_t* low = nullptr;      // lower piece of a bf16 dz
  size_t bytes = 0;
};
template <class T>
LinearRoom forward_room(void* ws, int64_t n, int64_t di, int64_t dn) {
  LinearRoom r;
  Carve cv(ws);
  size_t part = any_room<T>(n, dn, di);
  const bool large = large_product<T>(n, di, dn) && gemm_fits<T>(di, di);
  if (large) part = std::max(part, gemm_bf16_workspace(n, dn, di, K_ROWS, K_ROWS, sizeof(T) == 4) / 4);
  r.partial = cv.take<float>(part);
  if (large) {
    r.flag = cv.take<int32_t>(2);
    if (sizeof(T) == 4 || di % 8 != 0) {
      r.a = cv.take<uint16_t>(operand_room<T>(n, di));
      r.b = cv.take<uint16_t>(operand_room<T>(dn, di));
    }
  }
  r.bytes = cv.bytes();
  return r;
}
template <class T>
LinearRoom backward_room(void* ws, int64_t n, int64_t di, int64_t dn) {
  LinearRoom r;
  Carve cv(ws);
  r.sums = cv.take<float>(size_t(col_plan(n, dn).chunks) * dn);
  size_t part = std::max(any_room<T>(n, di, dn), any_room<T>(dn, di, n));
  const bool large = large_product<T>(n, di, dn) && gemm_fits<T>(di, dn);
  if (large)
    part = std::max({part, gemm_bf16_workspace(n, di, dn, K_ROWS, K_COLS, sizeof(T) == 4) / 4,
                     gemm_bf16_workspace(dn, di, n, K_COLS, K_COLS, sizeof(T) == 4) / 4});
  if (sizeof(T) == 2) r.low = cv.take<uint16_t>(operand_room<T>(n, dn));
  r.partial = cv.take<float>(part);
  if (large) r.c = cv.take<uint16_t>(operand_room<T>(n, di));   // x
  if (large) {
    r.flag = cv.take<int32_t>(2);
    if (sizeof(T) == 4 || dn % 8 != 0) r.a = cv.take<uint16_t>(operand_room<T>(n, dn));
    if (sizeof(T) == 4 || di % 8 != 0) r.b = cv.take<uint16_t>(operand_room<T>(dn, di));
  }
  r.bytes = cv.bytes();
  return r;
}
// whether an operand is read in place or has its room
template <class T>
bool has_room(const Operand& o, int64_t cols) {
  return sizeof(T) == 4 || cols % 8 != 0 || o.vec;   // (rooms depend on sizes alone)
}

template <class T>
lrc_status linear_forward(hipStream_t st, const void* x, int64_t n, int64_t di, int64_t dn, int64_t ldx, const void* W,
                          int64_t ldw, const float* bias, int act, const void* res, int64_t ldr, void* y, int64_t ldy,
                          void* z, int64_t ldz, int8_t* zcodes, int8_t* zexps, int32_t* info, void* ws) {
  Epilogue ep;
  ep.bias = bias;
  ep.act = act;
  ep.res = res;
  ep.ldr = ldr;
  set_out<T>(ep, y, ldy);
  ep.z = z;
  ep.ldz = zcodes != nullptr ? dn : ldz;
  ep.codes = zcodes;
  ep.exps = zexps;
  ep.nb = cdiv(dn, CKB);
  ep.info = info;
  const double bytes = double(sizeof(T)) * (double(n) * di + double(dn) * di + double(n) * dn * (res ? 2 : 1));
  const Operand ox = plain<T>(x, ldx), ow = plain<T>(W, ldw);
  // the kept pre-activation's blocks of 64 channels need a tile that holds them
  if (few_tokens(n, di, dn, sizeof(T)) && zcodes == nullptr)
    return linear_rows<T>(st, ox, ow, n, dn, di, ep, bytes);
  const LinearRoom room = forward_room<T>(ws, n, di, dn);
  F32Way way = SPLIT;
  if (sizeof(T) == 4 && room.flag != nullptr) {
    F32Times t;
    t.product(n, dn, di, K_ROWS, K_ROWS);
    t.operand(n, di);
    t.operand(dn, di);
    way = t.way();
  }
  const bool native = way == NATIVE;
  if (room.flag == nullptr || way == ANY || !has_room<T>(ox, di) || !has_room<T>(ow, di) ||
      std::max(ldx, ldw) > GEMM_MAX_LD)
    return product_any<T, T, K_ROWS, K_ROWS>(st, "linear_any_kernel", ox, ow, n, dn, di, ep, room.partial, nullptr, bytes);
  const int32_t* flag = sizeof(T) == 4 && !native ? room.flag : nullptr;
  if (flag) {
    clear_flag_kernel<<<1, 1, 0, st>>>(room.flag);
    LRC_LAUNCHED();
  }
  OperandJobs jobs;
  int count = 0;
  const Prepared a = want_operand<T>(jobs, count, ox, n, di, room.a, native, 1);
  const Prepared b = want_operand<T>(jobs, count, ow, dn, di, room.b, native, 1);
  LRC_TRY(prepare_operands<T>(st, jobs, count, room.flag));
  GemmSegments seg = segments(a.planes, b.planes);
  if (native) seg.type = FP32;
  LRC_TRY((gemm_bf16<T, K_ROWS, K_ROWS>(st, "linear_kernel", a.op, b.op, n, dn, di, seg, ep, room.partial, flag,
                                        2.0 * double(n) * double(dn) * double(di), bytes)));
  if (!flag) return LRC_OK;
  return product_any<T, T, K_ROWS, K_ROWS>(st, "linear_any_kernel", ox, ow, n, dn, di, ep, room.partial, flag, bytes);
}

}  // namespace
}  // namespace lrc

using namespace lrc;

extern "C" size_t lrc_linear_workspace(lrc_dtype dt, int64_t n_tokens, int64_t d_in, int64_t d_out) {
  if (!sizes_ok(n_tokens, d_in, d_out)) return 0;
  return dt == LRC_BF16 ? forward_room<uint16_t>(nullptr, n_tokens, d_in, d_out).bytes
                        : forward_room<float>(nullptr, n_tokens, d_in, d_out).bytes;
}

extern "C" lrc_status lrc_linear(const void* x, lrc_dtype dt, int64_t n_tokens, int64_t d_in, int64_t d_out,
                                 int64_t ldx, const void* W, int64_t ldw, const float* bias, lrc_act act,
                                 const void* residual, int64_t ldr, void* y, int64_t ldy, void* z, int64_t ldz,
                                 int8_t* zcodes, int8_t* zexps, int32_t* info, void* ws, size_t ws_bytes,
                                 void* stream) {
  if ((dt != LRC_F32 && dt != LRC_BF16) || !act_ok(act)) return LRC_EDTYPE;
  if (!sizes_ok(n_tokens, d_in, d_out) || ldx < d_in || ldw < d_in || ldy < d_out) return LRC_EINVAL;
  if ((residual != nullptr && ldr < d_out) || (z != nullptr && ldz < d_out)) return LRC_EINVAL;
  if ((zcodes == nullptr) != (zexps == nullptr) || (z != nullptr && zcodes != nullptr)) return LRC_EINVAL;
  if (n_tokens == 0) return LRC_OK;
  if (x == nullptr || W == nullptr || y == nullptr) return LRC_EINVAL;
  const size_t need = lrc_linear_workspace(dt, n_tokens, d_in, d_out);
  if (ws_bytes < need || (need > 0 && ws == nullptr)) return LRC_EWORKSPACE;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (dt == LRC_BF16)
    return linear_forward<uint16_t>(st, x, n_tokens, d_in, d_out, ldx, W, ldw, bias, act, residual, ldr, y, ldy, z,
                                    ldz, zcodes, zexps, info, ws);
  return linear_forward<float>(st, x, n_tokens, d_in, d_out, ldx, W, ldw, bias, act, residual, ldr, y, ldy, z, ldz,
                               zcodes, zexps, info, ws);
}

extern "C" size_t lrc_linear_backward_workspace(lrc_dtype dt, int64_t n_tokens, int64_t d_in, int64_t d_out) {
  if (!sizes_ok(n_tokens, d_in, d_out)) return 0;
  return dt == LRC_BF16 ? backward_room<uint16_t>(nullptr, n_tokens, d_in, d_out).bytes
                        : backward_room<float>(nullptr, n_tokens, d_in, d_out).bytes;
}

namespace lrc {
namespace {
struct BackArgs {
  int64_t n, di, dn;
  const void* dy;
  int64_t lddy;
  const void* W;
  int64_t ldw;
  const void* x;
  int64_t ldx;
  const int8_t *xcodes, *xexps;
  int act;
  const void* z;
  int64_t ldz;
  const int8_t *zcodes, *zexps;
  void* dz;
  int64_t lddz;
  void* dx;
  int64_t lddx;
  void* dW;
  int dw_dt;
  int64_t lddw;
  float* db;
};

template <class T>
lrc_status linear_back(hipStream_t st, const BackArgs& a, void* ws) {
  const LinearRoom room = backward_room<T>(ws, a.n, a.di, a.dn);
  const int64_t n = a.n, di = a.di, dn = a.dn;
  const bool with_dz = a.act != LRC_ACT_NONE;
  const void* g = with_dz ? a.dz : a.dy;
  const int64_t ldg = with_dz ? a.lddz : a.lddy;
  const Operand og = plain<T>(g, ldg), ow = plain<T>(a.W, a.ldw);
  const bool held = a.x == nullptr;
  const Operand ox = held ? Operand{a.xcodes, di, a.xexps, cdiv(di, CKB), false}
                          : plain<T>(a.x, a.ldx);
  const bool fast_g = room.flag != nullptr && has_room<T>(og, dn) && ldg <= GEMM_MAX_LD;
  // few tokens read W once on either kind of tile: a large one is not laid out anew for them (in fp32
  // the estimates count that)
  const bool w_in_place = sizeof(T) == 4 || ((ow.vec && di % 8 == 0) || di * dn <= (int64_t(1) << 21));
  bool fast_dx = fast_g && a.dx != nullptr && has_room<T>(ow, di) && a.ldw <= GEMM_MAX_LD &&
                       (w_in_place || n > 64);
  // a slope that is neither 0 nor 1 leaves bits in dz that the stream's bf16 does not hold
  const bool low = sizeof(T) == 2 && with_dz && a.act != LRC_ACT_RELU && a.dW != nullptr;
  bool fast_dw = fast_g && a.dW != nullptr && (held || low || (has_room<T>(ox, di) && a.ldx <= GEMM_MAX_LD));
  F32Way way = SPLIT;
  if (sizeof(T) == 4 && (fast_dx || fast_dw)) {
    // one way for both products, whether both are wanted or not: a gradient's bits do not depend on
    // the other's being asked for (one alone may so take a kernel that is not its fastest: dx of 512
    // tokens, 4096 -> 4096 141 us against 133, the call included)
    F32Times t;
    t.operand(n, dn);
    t.product(n, di, dn, K_ROWS, K_COLS), t.operand(dn, di);
    t.product(dn, di, n, K_COLS, K_COLS), t.operand(n, di);
    way = t.way();
    if (way == ANY) fast_dx = fast_dw = false;
  }
  const bool native = way == NATIVE;
  int32_t* flag = sizeof(T) == 4 && !native && (fast_dx || fast_dw) ? room.flag : nullptr;
  if (with_dz || a.db != nullptr) {
    const ColPlan p = col_plan(n, dn);
    {
      ProfScope scope("dz_kernel", st, 0.0, double(n) * dn * sizeof(T) * (a.act != LRC_ACT_NONE ? 3 : 1));
      const dim3 grid(unsigned(cdiv(dn, 512)), unsigned(p.chunks));
      float* part = a.db != nullptr && p.chunks > 1 ? room.sums : a.db;   // one chunk's sums are db
      const T *dy = static_cast<const T*>(a.dy), *z = static_cast<const T*>(a.z);
      T* dz = static_cast<T*>(a.dz);
      const bool codes = a.z == nullptr && a.act != LRC_ACT_NONE;
      const int64_t nb = cdiv(dn, CKB), w8 = round8(dn);
      auto go = [&](auto held_z, auto waves) {
        constexpr bool CK = decltype(held_z)::value;
        constexpr int NW = decltype(waves)::value;
        dz_kernel<T, CK, NW><<<grid, 64 * NW, 0, st>>>(dy, a.lddy, n, dn, z, a.ldz, a.zcodes, a.zexps, nb, a.act, dz,
                                                       a.lddz, p.rows, part, flag, low ? room.low : nullptr, w8);
      };
      using std::integral_constant;
      if (codes && p.chunks == 1)
        go(std::true_type{}, integral_constant<int, 16>{});
      else if (codes)
        go(std::true_type{}, integral_constant<int, 4>{});
      else if (p.chunks == 1)
        go(std::false_type{}, integral_constant<int, 16>{});
      else
        go(std::false_type{}, integral_constant<int, 4>{});
      LRC_LAUNCHED();
    }
    if (a.db != nullptr && p.chunks > 1) LRC_TRY(reduce_partials(st, room.sums, p.chunks, dn, dn, a.db, nullptr));
  } else if (flag) {
    clear_flag_kernel<<<1, 1, 0, st>>>(flag);
    LRC_LAUNCHED();
  }
  if (a.dx == nullptr && a.dW == nullptr) return LRC_OK;
  const double e = sizeof(T);
  OperandJobs jobs;
  int count = 0;
  Prepared pg, pw, px;
  if (fast_dx || fast_dw) pg = want_operand<T>(jobs, count, og, n, dn, room.a, native, 3);
  if (fast_dx) pw = want_operand<T>(jobs, count, ow, dn, di, room.b, native, 1);
  if (fast_dw) px = want_operand<T>(jobs, count, ox, n, di, room.c, native, 2);
  LRC_TRY(prepare_operands<T>(st, jobs, count, room.flag));
  if (a.dx != nullptr) {
    Epilogue ep;
    set_out<T>(ep, a.dx, a.lddx);
    const double bytes = e * (double(n) * dn + double(dn) * di + double(n) * di);
    if (fast_dx) {
      GemmSegments seg = segments(pg.planes, pw.planes);
      if (native) seg.type = FP32;
      LRC_TRY((gemm_bf16<T, K_ROWS, K_COLS>(st, "linear_dx_kernel", pg.op, pw.op, n, di, dn, seg, ep, room.partial, flag,
                                            2.0 * double(n) * double(dn) * double(di), bytes)));
    }
    if (!fast_dx || flag)
      LRC_TRY((product_any<T, T, K_ROWS, K_COLS>(st, "linear_dx_any_kernel", og, ow, n, di, dn, ep,
                                                 room.partial, fast_dx ? flag : nullptr, bytes)));
  }
  if (a.dW == nullptr) return LRC_OK;
  const double bytes = e * (double(n) * dn + double(dn) * di) + double(n) * di * (held ? 1.0 : e);
  auto go = [&](auto tag) -> lrc_status {
    using TO = decltype(tag);
    const int32_t* moved = flag ? flag + 1 : nullptr;
    Epilogue ep;
    set_out<TO>(ep, a.dW, a.lddw);
    auto any = [&](const Operand& g8, const Epilogue& e8, const int32_t* only) -> lrc_status {
      if (held)
        return product_any<T, TO, K_COLS, K_CODES>(st, "linear_dw_any_kernel", g8, ox, dn, di, n, e8, room.partial, only,
                                                   bytes);
      return product_any<T, TO, K_COLS, K_COLS>(st, "linear_dw_any_kernel", g8, ox, dn, di, n, e8, room.partial, only,
                                                bytes);
    };
    auto fast = [&](const GemmOperand& g8, const GemmSegments& seg, const Epilogue& e8) -> lrc_status {
      return gemm_bf16<TO, K_COLS, K_COLS>(st, "linear_dw_kernel", g8, px.op, dn, di, n, seg, e8, room.partial, moved,
                                           2.0 * double(n) * double(dn) * double(di), bytes);
    };
    // dW = low^T x first, then dz^T x on top of it.  Where the first is not finite, an entry of x is
    // not, or the second overflows by itself: its infinity or NaN is the result.
    if (low) {
      const int64_t w8 = round8(dn);
      Epilogue first = ep;
      first.finite = true;
      if (fast_dw)
        LRC_TRY(fast({room.low, w8, 0}, GemmSegments{}, first));
      else
        LRC_TRY(any(plain<T>(room.low, w8), first, nullptr));
      ep.res = a.dW;
      ep.ldr = a.lddw;
    }
    if (fast_dw) {
      GemmSegments seg = segments(pg.planes, px.planes);
      if (native) seg.type = FP32;
      LRC_TRY(fast(pg.op, seg, ep));
      if (!moved) return LRC_OK;
    }
    return any(og, ep, fast_dw ? moved : nullptr);
  };
  if (a.dw_dt == LRC_F32) return go(float{});
  return go(uint16_t{});
}
}  // namespace
}  // namespace lrc

extern "C" lrc_status lrc_linear_backward(const void* dy, lrc_dtype dt, int64_t n_tokens, int64_t d_in, int64_t d_out,
                                          int64_t lddy, const void* W, int64_t ldw, const void* x, int64_t ldx,
                                          const int8_t* xcodes, const int8_t* xexps, lrc_act act, const void* z,
                                          int64_t ldz, const int8_t* zcodes, const int8_t* zexps, void* dz,
                                          int64_t lddz, void* dx, int64_t lddx, void* dW, lrc_dtype dw_dt,
                                          int64_t lddw, float* db, void* ws, size_t ws_bytes, void* stream) {
  if ((dt != LRC_F32 && dt != LRC_BF16) || !act_ok(act)) return LRC_EDTYPE;
  if (dW != nullptr && dw_dt != LRC_F32 && dw_dt != dt) return LRC_EDTYPE;
  if (!sizes_ok(n_tokens, d_in, d_out) || lddy < d_out) return LRC_EINVAL;
  if ((dx != nullptr && (lddx < d_in || ldw < d_in)) || (dW != nullptr && lddw < d_in)) return LRC_EINVAL;
  if (x != nullptr && ldx < d_in) return LRC_EINVAL;
  if (act != LRC_ACT_NONE && ((z != nullptr && ldz < d_out) || lddz < d_out)) return LRC_EINVAL;
  if (n_tokens > 0) {
    if (dy == nullptr || (dx != nullptr && W == nullptr)) return LRC_EINVAL;
    if (dW != nullptr && x == nullptr && (xcodes == nullptr || xexps == nullptr)) return LRC_EINVAL;
    if (act != LRC_ACT_NONE && (dz == nullptr || (z == nullptr && (zcodes == nullptr || zexps == nullptr))))
      return LRC_EINVAL;
  }
  const size_t need = lrc_linear_backward_workspace(dt, n_tokens, d_in, d_out);
  if (ws_bytes < need || (need > 0 && ws == nullptr)) return LRC_EWORKSPACE;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (n_tokens == 0) {   // sums over nothing
    if (dW != nullptr) {
      const int64_t half = dw_dt == LRC_F32 ? 2 : 1;
      const int64_t grid = std::min<int64_t>(cdiv(d_out * d_in * half, LT), 16384);
      zero_rows_kernel<<<unsigned(grid), LT, 0, st>>>(static_cast<uint16_t*>(dW), d_out, d_in * half, lddw * half);
      LRC_LAUNCHED();
    }
    if (db != nullptr) LRC_TRY(reduce_partials(st, nullptr, 0, d_out, d_out, db, nullptr));
    return LRC_OK;
  }
  const BackArgs a = {n_tokens, d_in, d_out, dy,  lddy,  W,     ldw, x,    ldx, xcodes, xexps, act,
                      z,        ldz,  zcodes, zexps, dz, lddz, dx,  lddx, dW,  int(dw_dt), lddw, db};
  return dt == LRC_BF16 ? linear_back<uint16_t>(st, a, ws) : linear_back<float>(st, a, ws);
}
