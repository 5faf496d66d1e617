// Layer norm of token rows: forward (with the input's 8-bit checkpoint) and backward.
#include "lrc_train.h"

#include <algorithm>

namespace lrc {
namespace {

constexpr int NT = 256;
constexpr int ROWS_PER_CHUNK = 64;   // tokens per partial of a column sum

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
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
  for (int j = threadIdx.x; j < d; j += NT) s += ld_elem(row + j);
  const float mu = block_sum(s, red) / float(d);
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
    const float xh = (input_at<T, CK>(x, ldx, codes, exps, nb, t, j, d) - mu) * rs;
    const float g = ld_elem(dy + t * lddy + j) * (gamma ? gamma[j] : 1.f);
    s1 += g;
    s2 = fmaf(g, xh, s2);
  }
  const float c1 = block_sum(s1, red) / float(d), c2 = block_sum(s2, red) / float(d);
  for (int j = threadIdx.x; j < d; j += NT) {
    const float xh = (input_at<T, CK>(x, ldx, codes, exps, nb, t, j, d) - mu) * rs;
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
    const float xh = (input_at<T, CK>(x, ldx, codes, exps, nb, t, j, d) - mean[t]) * rstd[t];
    const float g = ld_elem(dy + t * lddy + j);
    a = fmaf(g, xh, a);
    b += g;
  }
  partial[(int64_t(blockIdx.y) * 2 + 0) * d + j] = a;
  partial[(int64_t(blockIdx.y) * 2 + 1) * d + j] = b;
}

// chunks of tokens of a column sum: at most 1024 of them, 64 tokens at least in each
struct ColPlan {
  int64_t rows, chunks;
};
ColPlan col_plan(int64_t n) {
  ColPlan p;
  p.rows = std::max<int64_t>(ROWS_PER_CHUNK, cdiv(n, 1024));
  p.chunks = cdiv(n, p.rows);
  return p;
}

// out[c] = sum_p partial[p stride + c]: 16 columns x 16 slices of the parts per workgroup,
// the slices added in order
__global__ __launch_bounds__(NT) void reduce_partials_kernel(const float* __restrict__ partial, int64_t parts,
                                                             int64_t stride, int64_t cols, float* __restrict__ out) {
  __shared__ float acc[16][17];
  const int cx = threadIdx.x & 15, sl = threadIdx.x >> 4;
  const int64_t c = int64_t(blockIdx.x) * 16 + cx;
  float s = 0.f;
  if (c < cols)
    for (int64_t p = sl; p < parts; p += 16) s += partial[p * stride + c];
  acc[sl][cx] = s;
  __syncthreads();
  if (sl == 0 && c < cols) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v += acc[i][cx];
    out[c] = v;
  }
}

template <class T>
lrc_status norm_forward(hipStream_t st, const T* x, int64_t n, int64_t d, int64_t ldx, const float* gamma,
                        const float* beta, float eps, T* y, int64_t ldy, float* mean, float* rstd, int8_t* codes,
                        int8_t* exps, int32_t* info) {
  const int64_t nb = cdiv(d, CKB);
  ProfScope scope("ln_fwd_kernel", st, 8.0 * double(n) * double(d),
                  double(n) * double(d) * (2 * sizeof(T) + (codes ? 1 : 0)) + 8.0 * double(n + d));
  ln_fwd_rows_kernel<T><<<unsigned(n), NT, 0, st>>>(x, ldx, int(d), gamma, beta, eps, y, ldy, mean, rstd, codes, exps,
                                                    nb, info);
  LRC_LAUNCHED();
  return LRC_OK;
}

template <class T, bool CK>
lrc_status norm_backward(hipStream_t st, const T* dy, int64_t n, int64_t d, int64_t lddy, const T* x, int64_t ldx,
                         const int8_t* codes, const int8_t* exps, const float* mean, const float* rstd,
                         const float* gamma, T* dx, int64_t lddx, float* dgamma, float* dbeta, float* partial) {
  const int64_t nb = cdiv(d, CKB);
  const ColPlan p = col_plan(n);
  {
    ProfScope scope("ln_bwd_kernel", st, 14.0 * double(n) * double(d),
                    double(n) * double(d) * (2 * sizeof(T) + (CK ? 1 : sizeof(T))) + 8.0 * double(n) + 12.0 * d);
    if (dx != nullptr) {
      ln_bwd_rows_kernel<T, CK><<<unsigned(n), NT, 0, st>>>(dy, lddy, int(d), x, ldx, codes, exps, nb, mean, rstd,
                                                            gamma, dx, lddx);
      LRC_LAUNCHED();
    }
    if (dgamma == nullptr && dbeta == nullptr) return LRC_OK;
    ln_bwd_cols_kernel<T, CK><<<dim3(unsigned(cdiv(d, NT)), unsigned(p.chunks)), NT, 0, st>>>(
        dy, lddy, n, int(d), x, ldx, codes, exps, nb, mean, rstd, p.rows, partial);
    LRC_LAUNCHED();
  }
  if (dgamma != nullptr) LRC_TRY(reduce_partials(st, partial, p.chunks, 2 * d, d, dgamma));
  if (dbeta != nullptr) LRC_TRY(reduce_partials(st, partial + d, p.chunks, 2 * d, d, dbeta));
  return LRC_OK;
}

bool sizes_ok(int64_t n, int64_t d) { return n >= 0 && n < (int64_t(1) << 31) && d >= 1 && d <= (int64_t(1) << 24); }

}  // namespace

lrc_status reduce_partials(hipStream_t st, const float* partial, int64_t parts, int64_t stride, int64_t cols,
                           float* out) {
  reduce_partials_kernel<<<unsigned(cdiv(cols, 16)), NT, 0, st>>>(partial, parts, stride, cols, out);
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
  cv.take<float>(size_t(col_plan(n_tokens).chunks) * 2 * d);
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
    if (dgamma != nullptr) LRC_TRY(reduce_partials(st, nullptr, 0, 0, d, dgamma));
    if (dbeta != nullptr) LRC_TRY(reduce_partials(st, nullptr, 0, 0, d, dbeta));
    return LRC_OK;
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
