// Layer norm of token rows: forward (with the input's 8-bit checkpoint) and backward.
#include "lrc_rows.h"

#include <algorithm>
#include <type_traits>

namespace lrc {
namespace {

constexpr int NT = 256;
constexpr int ROWS_PER_CHUNK = 64;   // tokens per partial of a column sum

// sum over the 256 threads, the same value in every one (fixed order)
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

// ---- any width: one workgroup per token, three passes over the row --------------------
template <class T>
__global__ __launch_bounds__(NT) void ln_fwd_rows_kernel(const T* __restrict__ x, int64_t ldx, int d,
                                                         const float* __restrict__ gamma,
                                                         const float* __restrict__ beta, float eps,
                                                         T* __restrict__ y, int64_t ldy, float* __restrict__ mean,
                                                         float* __restrict__ rstd, int8_t* __restrict__ codes,
                                                         int8_t* __restrict__ exps, int64_t nb,
                                                         int32_t* __restrict__ info) {
  __shared__ float red[4];
  const int64_t t = blockIdx.x;
  const T* row = x + t * ldx;
  float s = 0.f;
  const float half = 0.5f / float(d);
  for (int j = threadIdx.x; j < d; j += NT) s = fmaf(ld_elem(row + j), half, s);
  const float mu = mean_of(block_sum(s, red));
  float q = 0.f;
  for (int j = threadIdx.x; j < d; j += NT) {
    const float c = ld_elem(row + j) - mu;
    q = fmaf(c, c, q);
  }
  const float rs = 1.f / sqrtf(block_sum(q, red) / float(d) + eps);
  if (threadIdx.x == 0) {
    mean[t] = mu;
    rstd[t] = rs;
  }
  for (int j = threadIdx.x; j < d; j += NT) {
    const float xh = (ld_elem(row + j) - mu) * rs;
    st_elem(y + t * ldy + j, fmaf(xh, gamma ? gamma[j] : 1.f, beta ? beta[j] : 0.f));
  }
  if (codes == nullptr) return;
  const int lane = threadIdx.x & 63;
  bool bad = false;
  for (int64_t b = threadIdx.x >> 6; b < nb; b += NT / 64) {   // one wave per block of 64 channels
    const int c = int(b) * CKB + lane;
    const float v = c < d ? ld_elem(row + c) : 0.f;
    bad |= !finite_f(v);
    float m = finite_mag(v);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    const int e = ckpt_exponent(m);
    if (c < d) codes[t * d + c] = int8_t(ckpt_code(v, pow2f(-e)));
    if (lane == 0) exps[t * nb + b] = int8_t(e);
  }
  if (info != nullptr && bad) *info = LRC_ENONFINITE;
}

template <class T, bool CK>
__device__ __forceinline__ float input_at(const T* x, int64_t ldx, const int8_t* codes, const int8_t* exps, int64_t nb,
                                          int64_t t, int j, int d) {
  if (CK) return float(codes[t * d + j]) * pow2f(exps[t * nb + (j >> 6)]);
  return ld_elem(x + t * ldx + j);
}

// xh of the backward pass.  A held value may lie a step away from the token's: where a mask filled the
// token with the lowest value, centred and divided by a spread of zero it passes the largest number,
// and must not turn the token's dy of zeros into NaN.
template <bool CK>
__device__ __forceinline__ float normalised(float x, float mu, float r) {
  const float t = (x - mu) * r;
  return CK && fabsf(t) == __builtin_inff() ? copysignf(3.402823466e38f, t) : t;
}

template <class T, bool CK>
__global__ __launch_bounds__(NT) void ln_bwd_rows_kernel(const T* __restrict__ dy, int64_t lddy, int d,
                                                         const T* __restrict__ x, int64_t ldx,
                                                         const int8_t* __restrict__ codes,
                                                         const int8_t* __restrict__ exps, int64_t nb,
                                                         const float* __restrict__ mean,
                                                         const float* __restrict__ rstd,
                                                         const float* __restrict__ gamma, T* __restrict__ dx,
                                                         int64_t lddx) {
  __shared__ float red[4];
  const int64_t t = blockIdx.x;
  const float mu = mean[t], rs = rstd[t];
  float s1 = 0.f, s2 = 0.f;
  for (int j = threadIdx.x; j < d; j += NT) {
    const float xh = normalised<CK>(input_at<T, CK>(x, ldx, codes, exps, nb, t, j, d), mu, rs);
    const float g = ld_elem(dy + t * lddy + j) * (gamma ? gamma[j] : 1.f);
    s1 += g;
    s2 = fmaf(g, xh, s2);
  }
  const float c1 = block_sum(s1, red) / float(d), c2 = block_sum(s2, red) / float(d);
  for (int j = threadIdx.x; j < d; j += NT) {
    const float xh = normalised<CK>(input_at<T, CK>(x, ldx, codes, exps, nb, t, j, d), mu, rs);
    const float g = ld_elem(dy + t * lddy + j) * (gamma ? gamma[j] : 1.f);
    st_elem(dx + t * lddx + j, rs * (g - c1 - xh * c2));
  }
}

// dgamma, dbeta of one chunk of tokens: one thread per channel
template <class T, bool CK>
__global__ __launch_bounds__(NT) void ln_bwd_cols_kernel(const T* __restrict__ dy, int64_t lddy, int64_t n, int d,
                                                         const T* __restrict__ x, int64_t ldx,
                                                         const int8_t* __restrict__ codes,
                                                         const int8_t* __restrict__ exps, int64_t nb,
                                                         const float* __restrict__ mean,
                                                         const float* __restrict__ rstd, int64_t rows,
                                                         float* __restrict__ partial) {
  const int j = blockIdx.x * NT + threadIdx.x;
  if (j >= d) return;
  const int64_t t0 = int64_t(blockIdx.y) * rows, t1 = min(n, t0 + rows);
  float a = 0.f, b = 0.f;
  for (int64_t t = t0; t < t1; ++t) {
    const float xh = normalised<CK>(input_at<T, CK>(x, ldx, codes, exps, nb, t, j, d), mean[t], rstd[t]);
    const float g = ld_elem(dy + t * lddy + j);
    a = fmaf(g, xh, a);
    b += g;
  }
  partial[(int64_t(blockIdx.y) * 2 + 0) * d + j] = a;
  partial[(int64_t(blockIdx.y) * 2 + 1) * d + j] = b;
}

// ---- rows of at most 16384 channels, held in registers ---------------------------------
// WPR waves share a token, each lane holds 8 V of its channels: the token is read from memory
// once, the statistics are taken from the registers (values centred before they are squared),
// and gamma, beta and the running sums of dgamma and dbeta stay in registers over all tokens of
// the workgroup.  The next token's loads are in flight while the present one is worked on.
// Lane l holds channels 8 (k LANES + l) .. + 7 of piece k, so eight lanes hold one checkpoint
// block; pieces are 16-byte accesses at any alignment, the last one of a ragged row is short.
// Bound by memory: forward with its checkpoint 65536 x 4096 bf16 250 us (1.35 GB, 5.4 TB/s), backward
// from a checkpoint 32768 x 4096 bf16 117 us (0.67 GB, 5.7 TB/s), the partials' sum 5 us more; one
// token of 4096 3 us, a launch.
template <class T, int WPR, int V>
__global__ __launch_bounds__(row_threads(WPR)) void ln_fwd_kernel(
    const T* __restrict__ x, int64_t ldx, int64_t n, int d, const float* __restrict__ gamma,
    const float* __restrict__ beta, float eps, T* __restrict__ y, int64_t ldy, float* __restrict__ mean,
    float* __restrict__ rstd, int8_t* __restrict__ codes, int8_t* __restrict__ exps, int64_t nb,
    int32_t* __restrict__ info) {
  using S = RowShape<T, WPR, V>;
  constexpr int E = S::E;
  __shared__ float red[2][WPR > 1 ? S::GROUPS * WPR : 1][1];
  const int lane = threadIdx.x & 63, group = threadIdx.x / S::LANES, l = threadIdx.x % S::LANES;
  const int wave = l >> 6;
  float ga[E], be[E];
  row_params<S, V>(gamma, 1.f, d, l, ga);
  row_params<S, V>(beta, 0.f, d, l, be);
  const float inv_d = 1.f / float(d);
  const int64_t step = int64_t(gridDim.x) * S::GROUPS;
  int64_t t = int64_t(blockIdx.x) * S::GROUPS + group;
  RawRow<T, WPR, V> raw;
  raw.load(x + t * ldx, d, l, t < n);
  bool bad = false;
  for (int64_t t0 = int64_t(blockIdx.x) * S::GROUPS; t0 < n; t0 += step, t += step) {
    float v[E];
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = raw.at(i);
    raw.load(x + (t + step) * ldx, d, l, t + step < n);
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < E; ++i) s[0] = fmaf(v[i], 0.5f * inv_d, s[0]);
    row_sums<WPR, 1>(s, red[0], wave, lane, group);
    const float mu = mean_of(s[0]);
    if (codes != nullptr) {   // before v is centred
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int c = (k * S::LANES + l) * 8;
        float p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = v[8 * k + e];
        st8_codes(codes + t * d + c, exps + t * nb + (c >> 6), t < n ? min(8, d - c) : 0, p, lane, bad);
      }
    }
    float q[1] = {0.f};
#pragma unroll
    for (int i = 0; i < E; ++i) {
      v[i] -= mu;
      q[0] = S::col(i, l) < d ? fmaf(v[i], v[i], q[0]) : q[0];
    }
    row_sums<WPR, 1>(q, red[1], wave, lane, group);
    const float rs = 1.f / sqrtf(q[0] * inv_d + eps);
    if (t >= n) continue;
    if (l == 0) {
      mean[t] = mu;
      rstd[t] = rs;
    }
    T* o = y + t * ldy;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c = (k * S::LANES + l) * 8;
      float p[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) p[e] = fmaf(v[8 * k + e] * rs, ga[8 * k + e], be[8 * k + e]);
      if (c < d) st8(o + c, d - c, p);
    }
  }
  if (info != nullptr && bad) *info = LRC_ENONFINITE;
}

// dx of every token and the workgroup's share of dgamma and dbeta (partial[2 b], partial[2 b + 1]
// of workgroup b; not written when NULL, and no dx when that is NULL).
template <class T, int WPR, int V, bool CK>
__global__ __launch_bounds__(row_threads(WPR)) void ln_bwd_kernel(
    const T* __restrict__ dy, int64_t lddy, int64_t n, int d, const T* __restrict__ x, int64_t ldx,
    const int8_t* __restrict__ codes, const int8_t* __restrict__ exps, int64_t nb, const float* __restrict__ mean,
    const float* __restrict__ rstd, const float* __restrict__ gamma, T* __restrict__ dx, int64_t lddx,
    float* __restrict__ partial) {
  using S = RowShape<T, WPR, V>;
  constexpr int E = S::E;
  __shared__ float red[2][WPR > 1 ? S::GROUPS * WPR : 1][2];
  __shared__ float sums[S::GROUPS > 1 ? (S::GROUPS - 1) * 2 * E * S::LANES : 1];
  const int lane = threadIdx.x & 63, group = threadIdx.x / S::LANES, l = threadIdx.x % S::LANES;
  const int wave = l >> 6;
  float ga[E], dg[E], db[E];
  row_params<S, V>(gamma, 1.f, d, l, ga);
#pragma unroll
  for (int i = 0; i < E; ++i) dg[i] = db[i] = 0.f;
  const float inv_d = 1.f / float(d);
  const int64_t step = int64_t(gridDim.x) * S::GROUPS;
  int64_t t = int64_t(blockIdx.x) * S::GROUPS + group;
  RawRow<T, WPR, V> rg, rx;
  RawCodes<WPR, V> rc;
  float mu = 0.f, rs = 0.f;
  auto load = [&](int64_t u) {
    const bool live = u < n;
    rg.load(dy + u * lddy, d, l, live);
    if (CK)
      rc.load(codes + u * d, exps + u * nb, d, l, live);
    else
      rx.load(x + u * ldx, d, l, live);
    mu = live ? mean[u] : 0.f;
    rs = live ? rstd[u] : 0.f;
  };
  load(t);
  int odd = 0;
  for (int64_t t0 = int64_t(blockIdx.x) * S::GROUPS; t0 < n; t0 += step, t += step, odd ^= 1) {
    float g[E], xh[E];
    const float r = rs;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      g[i] = rg.at(i);
      const float xv = CK ? rc.at(i) : rx.at(i);
      xh[i] = S::col(i, l) < d ? (xv - mu) * r : 0.f;
    }
    // as `normalised`; a wave's lanes share the token, and only a spread far below the mean gets there
    // (a test of every value took 145 us against 122 at 32768 x 4096)
    if (CK && __builtin_amdgcn_readfirstlane(fabsf(mu) * r > 0x1p120f)) {
#pragma unroll
      for (int i = 0; i < E; ++i) xh[i] = normalised<CK>(xh[i], 0.f, 1.f);
    }
    load(t + step);
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < E; ++i) {
      dg[i] = fmaf(g[i], xh[i], dg[i]);
      db[i] += g[i];
      g[i] *= ga[i];
      s[0] += g[i];
      s[1] = fmaf(g[i], xh[i], s[1]);
    }
    if (dx == nullptr) continue;
    row_sums<WPR, 2>(s, red[odd], wave, lane, group);
    if (t >= n) continue;
    const float c1 = s[0] * inv_d, c2 = s[1] * inv_d;
    T* o = dx + t * lddx;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c = (k * S::LANES + l) * 8;
      float p[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) p[e] = r * (g[8 * k + e] - c1 - xh[8 * k + e] * c2);
      if (c < d) st8(o + c, d - c, p);
    }
  }
  if (partial == nullptr) return;
  if (S::GROUPS > 1) {   // the workgroup's tokens of one pass, added in order
    if (group > 0) {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        sums[((group - 1) * 2 * E + i) * S::LANES + l] = dg[i];
        sums[((group - 1) * 2 * E + E + i) * S::LANES + l] = db[i];
      }
    }
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int k = 0; k < S::GROUPS - 1; ++k)
#pragma unroll
      for (int i = 0; i < E; ++i) {
        dg[i] += sums[(k * 2 * E + i) * S::LANES + l];
        db[i] += sums[(k * 2 * E + E + i) * S::LANES + l];
      }
  }
  float* p = partial + int64_t(blockIdx.x) * 2 * d;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = (k * S::LANES + l) * 8;
    float a[8], b[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      a[e] = dg[8 * k + e];
      b[e] = db[8 * k + e];
    }
    if (c < d) {
      st8(p + c, d - c, a);
      st8(p + d + c, d - c, b);
    }
  }
}

constexpr int MAX_PARTS = 1024;       // partials of dgamma and dbeta

// chunks of tokens of a column sum of wider rows
struct ColPlan {
  int64_t rows, chunks;
};
ColPlan col_plan(int64_t n) {
  ColPlan p;
  p.rows = std::max<int64_t>(ROWS_PER_CHUNK, cdiv(n, MAX_PARTS));
  p.chunks = cdiv(n, p.rows);
  return p;
}

// Workgroups of the backward kernel: each takes at least four tokens per group, so that the
// partials stay a small part of the traffic; 512 (two per compute unit, each with a token's loads
// ahead) carry wide rows, narrow ones take as many as are resident.
int64_t bwd_groups(int64_t n, int64_t d) {
  const int64_t at_once = d <= 1024 ? 4 : d <= 2048 ? 2 : 1, most = d <= 512 ? 1280 : d <= 2048 ? 768 : 512;
  return std::max<int64_t>(1, std::min<int64_t>(most, cdiv(n, 4 * at_once)));
}
int64_t bwd_parts(int64_t n, int64_t d) { return d <= ROW_MAX ? bwd_groups(n, d) : col_plan(n).chunks; }

// 32 columns x 8 slices of the parts per workgroup, the slices added in order
__global__ __launch_bounds__(NT) void reduce_partials_kernel(const float* __restrict__ partial, int64_t parts,
                                                             int64_t cols, int64_t split, float* __restrict__ out0,
                                                             float* __restrict__ out1) {
  __shared__ float acc[8][33];
  const int cx = threadIdx.x & 31, sl = threadIdx.x >> 5;
  const int64_t c = int64_t(blockIdx.x) * 32 + cx;
  float s = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int64_t p = sl; p < parts; p += 8) s += partial[p * cols + c];
  }
  acc[sl][cx] = s;
  __syncthreads();
  if (sl == 0 && c < cols) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += acc[i][cx];
    float* out = c < split ? out0 : out1;
    if (out != nullptr) out[c < split ? c : c - split] = v;
  }
}

template <class T>
lrc_status norm_forward(hipStream_t st, const T* x, int64_t n, int64_t d, int64_t ldx, const float* gamma,
                        const float* beta, float eps, T* y, int64_t ldy, float* mean, float* rstd, int8_t* codes,
                        int8_t* exps, int32_t* info) {
  const int64_t nb = cdiv(d, CKB);
  ProfScope scope("ln_fwd_kernel", st, 8.0 * double(n) * double(d),
                  double(n) * double(d) * (2 * sizeof(T) + (codes ? 1 : 0)) + 8.0 * double(n + d));
  if (d > ROW_MAX) {
    ln_fwd_rows_kernel<T><<<unsigned(n), NT, 0, st>>>(x, ldx, int(d), gamma, beta, eps, y, ldy, mean, rstd, codes,
                                                      exps, nb, info);
    LRC_LAUNCHED();
    return LRC_OK;
  }
  return with_row_shape(d, [&](auto w, auto v) -> lrc_status {
    constexpr int WPR = decltype(w)::value, V = decltype(v)::value;
    using S = RowShape<T, WPR, V>;
    const unsigned grid = unsigned(std::min<int64_t>(cdiv(n, S::GROUPS), 2048 / std::max(1, WPR / 4)));
    ln_fwd_kernel<T, WPR, V><<<grid, S::THREADS, 0, st>>>(x, ldx, n, int(d), gamma, beta, eps, y, ldy, mean, rstd,
                                                          codes, exps, nb, info);
    LRC_LAUNCHED();
    return LRC_OK;
  });
}

template <class T, bool CK>
lrc_status norm_backward(hipStream_t st, const T* dy, int64_t n, int64_t d, int64_t lddy, const T* x, int64_t ldx,
                         const int8_t* codes, const int8_t* exps, const float* mean, const float* rstd,
                         const float* gamma, T* dx, int64_t lddx, float* dgamma, float* dbeta, float* partial) {
  const int64_t nb = cdiv(d, CKB);
  const bool params = dgamma != nullptr || dbeta != nullptr;
  if (dx == nullptr && !params) return LRC_OK;
  {
    ProfScope scope("ln_bwd_kernel", st, 14.0 * double(n) * double(d),
                    double(n) * double(d) * (2 * sizeof(T) + (CK ? 1 : sizeof(T))) + 8.0 * double(n) + 12.0 * d);
    if (d <= ROW_MAX) {
      const unsigned grid = unsigned(bwd_groups(n, d));
      float* part = params ? partial : nullptr;
      LRC_TRY(with_row_shape(d, [&](auto w, auto v) -> lrc_status {
        constexpr int WPR = decltype(w)::value, V = decltype(v)::value;
        using S = RowShape<T, WPR, V>;
        ln_bwd_kernel<T, WPR, V, CK><<<grid, S::THREADS, 0, st>>>(dy, lddy, n, int(d), x, ldx, codes, exps, nb, mean,
                                                                  rstd, gamma, dx, lddx, part);
        LRC_LAUNCHED();
        return LRC_OK;
      }));
    } else {
      if (dx != nullptr) {
        ln_bwd_rows_kernel<T, CK><<<unsigned(n), NT, 0, st>>>(dy, lddy, int(d), x, ldx, codes, exps, nb, mean, rstd,
                                                              gamma, dx, lddx);
        LRC_LAUNCHED();
      }
      if (params) {
        const ColPlan p = col_plan(n);
        ln_bwd_cols_kernel<T, CK><<<dim3(unsigned(cdiv(d, NT)), unsigned(p.chunks)), NT, 0, st>>>(
            dy, lddy, n, int(d), x, ldx, codes, exps, nb, mean, rstd, p.rows, partial);
        LRC_LAUNCHED();
      }
    }
  }
  return params ? reduce_partials(st, partial, bwd_parts(n, d), 2 * d, d, dgamma, dbeta) : LRC_OK;
}

bool sizes_ok(int64_t n, int64_t d) { return n >= 0 && n < (int64_t(1) << 31) && d >= 1 && d <= (int64_t(1) << 24); }

}  // namespace

lrc_status reduce_partials(hipStream_t st, const float* partial, int64_t parts, int64_t cols, int64_t split,
                           float* out0, float* out1) {
  reduce_partials_kernel<<<unsigned(cdiv(cols, 32)), NT, 0, st>>>(partial, parts, cols, split, out0, out1);
  LRC_LAUNCHED();
  return LRC_OK;
}

}  // namespace lrc

using namespace lrc;

extern "C" lrc_status lrc_layer_norm(const void* x, lrc_dtype dt, int64_t n_tokens, int64_t d, int64_t ldx,
                                     const float* gamma, const float* beta, float eps, void* y, int64_t ldy,
                                     float* mean, float* rstd, int8_t* codes, int8_t* exps, int32_t* info,
                                     void* stream) {
  if (dt != LRC_F32 && dt != LRC_BF16) return LRC_EDTYPE;
  if (!sizes_ok(n_tokens, d) || ldx < d || ldy < d || !(eps >= 0.f)) return LRC_EINVAL;
  if ((codes == nullptr) != (exps == nullptr)) return LRC_EINVAL;
  if (n_tokens == 0) return LRC_OK;
  if (x == nullptr || y == nullptr || mean == nullptr || rstd == nullptr) return LRC_EINVAL;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (dt == LRC_BF16)
    return norm_forward(st, static_cast<const uint16_t*>(x), n_tokens, d, ldx, gamma, beta, eps,
                        static_cast<uint16_t*>(y), ldy, mean, rstd, codes, exps, info);
  return norm_forward(st, static_cast<const float*>(x), n_tokens, d, ldx, gamma, beta, eps, static_cast<float*>(y),
                      ldy, mean, rstd, codes, exps, info);
}

extern "C" size_t lrc_layer_norm_backward_workspace(int64_t n_tokens, int64_t d) {
  if (!sizes_ok(n_tokens, d)) return 0;
  Carve cv(nullptr);
  cv.take<float>(size_t(bwd_parts(n_tokens, d)) * 2 * d);
  return cv.bytes();
}

extern "C" lrc_status lrc_layer_norm_backward(const void* dy, lrc_dtype dt, int64_t n_tokens, int64_t d, int64_t lddy,
                                              const void* x, int64_t ldx, const int8_t* codes, const int8_t* exps,
                                              const float* mean, const float* rstd, const float* gamma, void* dx,
                                              int64_t lddx, float* dgamma, float* dbeta, void* ws, size_t ws_bytes,
                                              void* stream) {
  if (dt != LRC_F32 && dt != LRC_BF16) return LRC_EDTYPE;
  if (!sizes_ok(n_tokens, d) || lddy < d || (x != nullptr && ldx < d) || (dx != nullptr && lddx < d)) return LRC_EINVAL;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (n_tokens > 0) {
    if (dy == nullptr || mean == nullptr || rstd == nullptr) return LRC_EINVAL;
    if (x == nullptr && (codes == nullptr || exps == nullptr)) return LRC_EINVAL;
  }
  const size_t need = lrc_layer_norm_backward_workspace(n_tokens, d);
  if (ws_bytes < need || (need > 0 && ws == nullptr)) return LRC_EWORKSPACE;
  if (n_tokens == 0) {   // sums over nothing
    return reduce_partials(st, nullptr, 0, 2 * d, d, dgamma, dbeta);
  }
  float* partial = static_cast<float*>(ws);
  auto go = [&](auto tag) -> lrc_status {
    using T = decltype(tag);
    const T* g = static_cast<const T*>(dy);
    const T* xi = static_cast<const T*>(x);
    T* o = static_cast<T*>(dx);
    if (x != nullptr)
      return norm_backward<T, false>(st, g, n_tokens, d, lddy, xi, ldx, nullptr, nullptr, mean, rstd, gamma, o, lddx,
                                     dgamma, dbeta, partial);
    return norm_backward<T, true>(st, g, n_tokens, d, lddy, nullptr, 0, codes, exps, mean, rstd, gamma, o, lddx,
                                  dgamma, dbeta, partial);
  };
  return dt == LRC_BF16 ? go(uint16_t{}) : go(float{});
}
