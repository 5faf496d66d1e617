// Norms around a block of a residual network, with the block's gate and residual scale: forward and backward.
//   p = post-norm(b) (or b),  s = residual + scale * gate * p,  h = norm(s)
// and, with total gradient t = ds + (gradient of h through the norm),
//   dresidual = t,  db = gradient of p = scale * gate * t through the post-norm.
//
// A token lies in the registers of 1 to 8 waves (lrc_rows.h): b and the residual are read once, s and h written
// once, the statistics of both norms are taken from registers in between (values centred before they are squared).
// The next token's loads are in flight while the present one is worked on.
// Bound by memory: forward 65536 x 4096 bf16, both norms, 445 us (2.15 GB, 4.8 TB/s), backward 32768 x 4096 308 us
// (1.61 GB, 5.2 TB/s) and 9 for the shares' sums; one token 4.4 us, a launch.  Rows of no whole 16-byte pieces reach
// 2 to 3 TB/s (334 or 5114 bf16 channels): every piece straddles two, and the last one is read element by element.
// Backward: all parameter gradients follow from four column sums over the tokens,
//   A = sum dh s^, B = sum dh, C = sum t b^, D = sum t      (^: normalised; b^ = b without a post-norm)
//   dgamma = A, dbeta = B, dpost_gamma = scale gate C, dpost_beta = scale gate D,
//   dgate = scale (post_gamma C + post_beta D),
// each lane keeping those of its channels over all tokens of the workgroup; a second kernel adds the workgroups'
// shares in a fixed order.
#include "lrc_rows.h"

#include <algorithm>

namespace lrc {
namespace {

struct NormForward {
  const void *b, *res;
  int64_t n, ldb, ldr;
  int d;
  const float *post_gamma, *post_beta, *gate, *gamma, *beta;
  float scale, eps;
  void *s, *h;
  int64_t lds, ldh;
  float *mean_b, *rstd_b, *mean_s, *rstd_s;
  int8_t* q;
  int64_t ldq;
  float* qscale;
  int32_t* info;
};

// Sums and maxima over a token's waves; consecutive calls take turns between two slots, so that the barrier
// inside the next call lies between reading a slot and writing it again.
template <int WPR, int GROUPS>
struct RowReduce {
  static constexpr int SLOTS = WPR > 1 ? GROUPS * WPR : 1, LANES = row_lanes(WPR) < 64 ? row_lanes(WPR) : 64;
  int slot = 0;
  template <int N>
  __device__ __forceinline__ void sums(float (&v)[N], float (*red)[SLOTS][2], int wave, int lane, int group) {
    static_assert(N <= 2, "two values to a slot");
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = lanes_sum<LANES>(v[k]);
    if (WPR <= 1) return;
    if (lane == 0) {
#pragma unroll
      for (int k = 0; k < N; ++k) red[slot][group * WPR + wave][k] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < WPR; ++w) s += red[slot][group * WPR + w][k];
      v[k] = s;
    }
    slot ^= 1;
  }
  __device__ __forceinline__ float sum(float x, float (*red)[SLOTS][2], int wave, int lane, int group) {
    float v[1] = {x};
    sums(v, red, wave, lane, group);
    return v[0];
  }
  __device__ __forceinline__ uint32_t largest(uint32_t v, float (*red)[SLOTS][2], int wave, int lane, int group) {
    v = lanes_max<LANES>(v);
    if (WPR <= 1) return v;
    if (lane == 0) red[slot][group * WPR + wave][0] = __uint_as_float(v);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WPR; ++w) v = max(v, __float_as_uint(red[slot][group * WPR + w][0]));
    slot ^= 1;
    return v;
  }
};

template <class T, int WPR, int V, bool LAYER, bool POST>
__global__ __launch_bounds__(row_threads(WPR)) void block_norm_kernel(NormForward a) {
  using S = RowShape<T, WPR, V>;
  using R = RowReduce<WPR, S::GROUPS>;
  constexpr int E = S::E;
  __shared__ float red[2][R::SLOTS][2];
  const int lane = threadIdx.x & 63, group = threadIdx.x / S::LANES, l = threadIdx.x % S::LANES;
  const int wave = l >> 6, d = a.d;
  const T *b = static_cast<const T*>(a.b), *res = static_cast<const T*>(a.res);
  // what the (normalised) block is multiplied with and what is added, gate and scale included
  float pa[E], pb[POST ? E : 1], ga[E], be[LAYER ? E : 1];
  row_params<S, V>(a.gate, 1.f, d, l, pa);
#pragma unroll
  for (int i = 0; i < E; ++i) pa[i] *= a.scale;
  if constexpr (POST) {
    row_params<S, V>(a.post_beta, 0.f, d, l, pb);
    row_params<S, V>(a.post_gamma, 1.f, d, l, ga);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      pb[i] *= pa[i];
      pa[i] *= ga[i];
    }
  }
  row_params<S, V>(a.gamma, 1.f, d, l, ga);
  if constexpr (LAYER) row_params<S, V>(a.beta, 0.f, d, l, be);
  const float inv_d = 1.f / float(d);
  const int64_t step = int64_t(gridDim.x) * S::GROUPS;
  int64_t t = int64_t(blockIdx.x) * S::GROUPS + group;
  RawRow<T, WPR, V> rb, rr;
  auto load = [&](int64_t u) {
    rb.load(b + u * a.ldb, d, l, u < a.n);
    rr.load(res + u * a.ldr, d, l, u < a.n && res != nullptr);
  };
  constexpr bool AHEAD = V * sizeof(T) < 16;   // the widest fp32 rows leave no registers for the next token
  if (AHEAD) load(t);
  R reduce;
  bool bad = false;
  // centres (LAYER) and returns 1 / spread; what lies behind the last channel stays zero
  auto standardise = [&](float (&v)[E], float& mu) {
    mu = 0.f;
    if (LAYER) {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < E; ++i) m = fmaf(v[i], 0.5f * inv_d, m);
      mu = mean_of(reduce.sum(m, red, wave, lane, group));
    }
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      if (LAYER) v[i] = S::col(i, l) < d ? v[i] - mu : 0.f;
      q = fmaf(v[i], v[i], q);
    }
    return 1.f / sqrtf(reduce.sum(q, red, wave, lane, group) * inv_d + a.eps);
  };
  for (int64_t t0 = int64_t(blockIdx.x) * S::GROUPS; t0 < a.n; t0 += step, t += step) {
    const bool live = t < a.n;
    float v[E], r[E];
    if (!AHEAD) load(t);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      v[i] = rb.at(i);
      r[i] = rr.at(i);
    }
    if (AHEAD) load(t + step);
    float mu;
    if constexpr (POST) {
      const float rs = standardise(v, mu);
      if (live && l == 0) {
        if (LAYER && a.mean_b != nullptr) a.mean_b[t] = mu;
        if (a.rstd_b != nullptr) a.rstd_b[t] = rs;
      }
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = r[i] + fmaf(v[i] * rs, pa[i], pb[i]);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = fmaf(v[i], pa[i], r[i]);
    }
    if (a.s != nullptr && live) {
      T* o = static_cast<T*>(a.s) + t * a.lds;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int c = (k * S::LANES + l) * 8;
        float p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = v[8 * k + e];
        if (c < d) st8(o + c, d - c, p);
      }
    }
    if (a.h == nullptr && a.q == nullptr) continue;
    const float rs = standardise(v, mu);
    if (live && l == 0) {
      if (LAYER && a.mean_s != nullptr) a.mean_s[t] = mu;
      if (a.rstd_s != nullptr) a.rstd_s[t] = rs;
    }
#pragma unroll
    for (int i = 0; i < E; ++i) {
      if constexpr (LAYER)
        v[i] = fmaf(v[i] * rs, ga[i], be[i]);
      else
        v[i] = v[i] * rs * ga[i];
    }
    if (a.h != nullptr && live) {
      T* o = static_cast<T*>(a.h) + t * a.ldh;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int c = (k * S::LANES + l) * 8;
        float p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = v[8 * k + e];
        if (c < d) st8(o + c, d - c, p);
      }
    }
    if (a.q == nullptr) continue;
    // codes of h as it is in T, the bits of the quantiser of a written h (places without a token count for nothing: with
    // eps = 0 they hold 0 / 0)
    uint32_t m = 0;
    float p[V][8];
#pragma unroll
    for (int k = 0; k < V; ++k) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        p[k][e] = live && S::col(8 * k + e, l) < d ? round_to(v[8 * k + e], static_cast<const T*>(nullptr)) : 0.f;
      m = mag8(p[k], m, bad);
    }
    const float qs = token_step(reduce.largest(m, red, wave, lane, group));
    if (!live) continue;
    if (l == 0) a.qscale[t] = qs;
    const float inv = token_inverse(qs);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c = (k * S::LANES + l) * 8;
      if (c < d) st8_token_codes(a.q + t * a.ldq + c, d - c, p[k], qs, inv, bad);
    }
  }
  if (a.info != nullptr && bad) *a.info = LRC_ENONFINITE;
}

struct NormBackward {
  const void *dh, *ds, *s, *b;
  int64_t n, lddh, ldds, lds, ldb;
  int d;
  const float *mean_b, *rstd_b, *mean_s, *rstd_s, *post_gamma, *gate, *gamma;
  float scale;
  void *dres, *db;
  int64_t lddr, lddb;
  float* partial;   // [workgroup][4][d] (LAYER) or [workgroup][2][d]: A, C(, B, D)
};

// a row of the backward pass of a norm: g = dy gamma -> r (g - mean(g) - x^ mean(g x^))
template <class T, int WPR, int V, bool LAYER, bool POST>
__global__ __launch_bounds__(row_threads(WPR)) void block_norm_bwd_kernel(NormBackward a) {
  using S = RowShape<T, WPR, V>;
  using R = RowReduce<WPR, S::GROUPS>;
  constexpr int E = S::E, NS = LAYER ? 4 : 2;
  // rows past 8192 channels: A and C are kept in LDS (a lane's own places, 16 bytes a time), B and D in registers,
  // and tokens are not loaded ahead where that spills (6100 x 11008 rms 193 us; 412 with all sums in registers)
  constexpr bool WIDE = V > 2, AHEAD = !WIDE || (V * sizeof(T) <= 6 && !LAYER);
  constexpr int NR = WIDE ? NS / 2 : NS;   // sums in registers
  __shared__ __attribute__((aligned(16))) f32x4 wide[WIDE ? 2 * 2 * V * S::LANES : 1];
  __shared__ float red[2][R::SLOTS][2];
  __shared__ float share[S::GROUPS > 1 ? (S::GROUPS - 1) * NS * E * S::LANES : 1];
  const int lane = threadIdx.x & 63, group = threadIdx.x / S::LANES, l = threadIdx.x % S::LANES;
  const int wave = l >> 6, d = a.d;
  const T *dh = static_cast<const T*>(a.dh), *ds = static_cast<const T*>(a.ds), *s = static_cast<const T*>(a.s),
          *b = static_cast<const T*>(a.b);
  float ga[E], gs[E];   // gamma; scale * gate, and * post_gamma
  row_params<S, V>(a.gate, 1.f, d, l, gs);
  if constexpr (POST) {
    row_params<S, V>(a.post_gamma, 1.f, d, l, ga);
#pragma unroll
    for (int i = 0; i < E; ++i) gs[i] *= a.scale * ga[i];
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) gs[i] *= a.scale;
  }
  row_params<S, V>(a.gamma, 1.f, d, l, ga);
  // A, C (in LDS where WIDE), B, D
  float acc[NR > 0 ? NR : 1][E];
#pragma unroll
  for (int k = 0; k < NR; ++k)
#pragma unroll
    for (int i = 0; i < E; ++i) acc[k][i] = 0.f;
  constexpr int AT_B = WIDE ? 0 : 2, AT_D = AT_B + 1;
  auto wide_at = [&](int sum, int half) -> f32x4& { return wide[(sum * 2 * V + half) * S::LANES + l]; };
  if constexpr (WIDE) {
#pragma unroll
    for (int h = 0; h < 4 * V; ++h) wide[h * S::LANES + l] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  // adds x y to A (0) or C (1)
  auto add = [&](int sum, const float (&x)[E], const float (&y)[E]) {
    if constexpr (WIDE) {
#pragma unroll
      for (int h = 0; h < 2 * V; ++h) {
        f32x4 v = wide_at(sum, h);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = fmaf(x[4 * h + e], y[4 * h + e], v[e]);
        wide_at(sum, h) = v;
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) acc[sum][i] = fmaf(x[i], y[i], acc[sum][i]);
    }
  };
  const float inv_d = 1.f / float(d);
  const int64_t step = int64_t(gridDim.x) * S::GROUPS;
  int64_t t = int64_t(blockIdx.x) * S::GROUPS + group;
  RawRow<T, WPR, V> rh, rd, rs, rb;
  float mu_s = 0.f, r_s = 0.f, mu_b = 0.f, r_b = 0.f;
  auto load = [&](int64_t u) {
    const bool live = u < a.n;
    rh.load(dh + u * a.lddh, d, l, live && dh != nullptr);
    rs.load(s + u * a.lds, d, l, live && dh != nullptr);
    rd.load(ds + u * a.ldds, d, l, live && ds != nullptr);
    rb.load(b + u * a.ldb, d, l, live && b != nullptr);
    if (LAYER) mu_s = live && dh != nullptr ? a.mean_s[u] : 0.f;
    r_s = live && dh != nullptr ? a.rstd_s[u] : 0.f;
    if (POST) {
      if (LAYER) mu_b = live ? a.mean_b[u] : 0.f;
      r_b = live ? a.rstd_b[u] : 0.f;
    }
  };
  if (AHEAD) load(t);
  R reduce;
  // v = gamma dy -> its gradient through the norm whose normalised row is xh
  auto through = [&](float (&v)[E], const float (&xh)[E], float r) {
    float c[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < E; ++i) {
      c[0] = fmaf(v[i], xh[i], c[0]);
      if (LAYER) c[1] += v[i];
    }
    if (LAYER) {
      reduce.sums(c, red, wave, lane, group);
    } else {
      c[0] = reduce.sum(c[0], red, wave, lane, group);
    }
    c[0] *= inv_d;
    c[1] *= inv_d;
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = LAYER ? r * (v[i] - c[1] - xh[i] * c[0]) : r * (v[i] - xh[i] * c[0]);
  };
  for (int64_t t0 = int64_t(blockIdx.x) * S::GROUPS; t0 < a.n; t0 += step, t += step) {
    float g[E], xh[E], total[E], bh[E];
    if (!AHEAD) load(t);
    const float rsv = r_s, rbv = r_b;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const bool in = S::col(i, l) < d;
      g[i] = rh.at(i);
      xh[i] = in ? (LAYER ? rs.at(i) - mu_s : rs.at(i)) * rsv : 0.f;
      total[i] = rd.at(i);
      bh[i] = rb.at(i);
      if (POST) bh[i] = in ? (LAYER ? bh[i] - mu_b : bh[i]) * rbv : 0.f;
    }
    if (AHEAD) load(t + step);
    const bool live = t < a.n;
    if (a.dh != nullptr) {
      add(0, g, xh);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        if constexpr (LAYER) acc[AT_B][i] += g[i];
        g[i] *= ga[i];
      }
      through(g, xh, rsv);
#pragma unroll
      for (int i = 0; i < E; ++i) total[i] += S::col(i, l) < d ? g[i] : 0.f;
    }
    add(1, total, bh);
    if constexpr (LAYER) {
#pragma unroll
      for (int i = 0; i < E; ++i) acc[AT_D][i] += total[i];
    }
    auto store = [&](void* to, int64_t ld, const float (&v)[E]) {
      if (to == nullptr || !live) return;
      T* o = static_cast<T*>(to) + t * ld;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int c = (k * S::LANES + l) * 8;
        float p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = v[8 * k + e];
        if (c < d) st8(o + c, d - c, p);
      }
    };
    store(a.dres, a.lddr, total);
    if (a.db == nullptr) continue;
#pragma unroll
    for (int i = 0; i < E; ++i) total[i] *= gs[i];
    if constexpr (POST) through(total, bh, rbv);
    store(a.db, a.lddb, total);
  }
  if (a.partial == nullptr) return;
  if (S::GROUPS > 1) {   // the workgroup's tokens of one pass, added in order
    if (group > 0) {
#pragma unroll
      for (int k = 0; k < NS; ++k)
#pragma unroll
        for (int i = 0; i < E; ++i) share[(((group - 1) * NS + k) * E + i) * S::LANES + l] = acc[k][i];
    }
    __syncthreads();
    if (group > 0) return;
#pragma unroll 1
    for (int w = 0; w < S::GROUPS - 1; ++w)
#pragma unroll
      for (int k = 0; k < NS; ++k)
#pragma unroll
        for (int i = 0; i < E; ++i) acc[k][i] += share[((w * NS + k) * E + i) * S::LANES + l];
  }
  float* o = a.partial + int64_t(blockIdx.x) * NS * d;
#pragma unroll
  for (int k = 0; k < NS; ++k)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * S::LANES + l) * 8;
      float p[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        p[e] = !WIDE ? acc[k % (NR > 0 ? NR : 1)][8 * j + e]
               : k < 2 ? wide_at(k, 2 * j + e / 4)[e % 4] : acc[NR > 0 ? (k - 2) % NR : 0][8 * j + e];
      if (c < d) st8(o + k * int64_t(d) + c, d - c, p);
    }
}

// The four sums of 32 channels from `parts` shares, eight slices of them added in order, and the gradients.
struct ParamGrads {
  float *dgamma, *dbeta, *dpost_gamma, *dpost_beta, *dgate;
  const float *post_gamma, *post_beta, *gate;
  float scale;
  bool post;
};
__global__ __launch_bounds__(256) void block_norm_params_kernel(const float* __restrict__ partial, int64_t parts,
                                                                int sums, int d, ParamGrads g) {
  __shared__ float acc[4][8][33];
  const int cx = threadIdx.x & 31, sl = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + cx;
  float v[4] = {};
  if (c < d) {
    for (int k = 0; k < sums; ++k) {
      float x = 0.f;
#pragma unroll 8
      for (int64_t p = sl; p < parts; p += 8) x += partial[(p * sums + k) * d + c];
      v[k] = x;
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) acc[k][sl][cx] = v[k];
  __syncthreads();
  if (sl != 0 || c >= d) return;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[k] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[k] += acc[k][i][cx];
  }
  const float A = v[0], C = v[1], B = v[2], D = v[3];
  const float w = g.scale * (g.gate != nullptr ? g.gate[c] : 1.f);
  if (g.dgamma != nullptr) g.dgamma[c] = A;
  if (g.dbeta != nullptr) g.dbeta[c] = B;
  if (g.dpost_gamma != nullptr) g.dpost_gamma[c] = w * C;
  if (g.dpost_beta != nullptr) g.dpost_beta[c] = w * D;
  if (g.dgate != nullptr)
    g.dgate[c] = g.scale * (g.post ? (g.post_gamma != nullptr ? g.post_gamma[c] : 1.f) * C +
                                         (g.post_beta != nullptr ? g.post_beta[c] * D : 0.f)
                                   : C);
}

// Shapes of the backward kernel: up to 2048 channels a lane holds eight, so that more waves are resident.
template <class F>
lrc_status with_bwd_shape(int64_t d, F f) {
  using std::integral_constant;
  if (d > 512 && d <= 1024) return f(integral_constant<int, 2>{}, integral_constant<int, 1>{});
  if (d > 1024 && d <= 1536) return f(integral_constant<int, 3>{}, integral_constant<int, 1>{});
  if (d > 1536 && d <= 2048) return f(integral_constant<int, 4>{}, integral_constant<int, 1>{});
  return with_any_row_shape(d, f);
}
// Workgroups of the backward kernel: at least four tokens to a group of lanes, so that the shares stay a small part
// of the traffic.
int64_t bwd_groups(int64_t n, int64_t d) {
  const int64_t at_once = d <= 128 ? 16 : d <= 256 ? 8 : d <= 512 ? 4 : d <= 1024 ? 2 : 1;
  return std::max<int64_t>(1, std::min<int64_t>(d <= 2048 ? 1024 : 512, cdiv(n, 4 * at_once)));
}

bool sizes_ok(int64_t n, int64_t d) { return n >= 0 && n < (int64_t(1) << 31) && d >= 1 && d <= ROW_MAX; }
bool kind_ok(int k) { return k == LRC_NORM_LAYER || k == LRC_NORM_RMS; }

// f(waves, pieces, LAYER, POST) as compile-time constants
template <class F>
auto with_norm(int kind, bool post, F f) {
  return [=](auto w, auto v) -> lrc_status {
    using std::false_type;
    using std::true_type;
    if (kind == LRC_NORM_LAYER) return post ? f(w, v, true_type{}, true_type{}) : f(w, v, true_type{}, false_type{});
    return post ? f(w, v, false_type{}, true_type{}) : f(w, v, false_type{}, false_type{});
  };
}

template <class T>
lrc_status forward(hipStream_t st, const NormForward& a, int kind, bool post) {
  const double cells = double(a.n) * double(a.d);
  const int streams = 1 + (a.res != nullptr) + (a.s != nullptr) + (a.h != nullptr);
  ProfScope scope("block_norm_kernel", st, 16.0 * cells, cells * double(streams * sizeof(T) + (a.q != nullptr)));
  return with_any_row_shape(a.d, with_norm(kind, post, [&](auto w, auto v, auto layer, auto after) -> lrc_status {
    constexpr int WPR = decltype(w)::value, V = decltype(v)::value;
    using S = RowShape<T, WPR, V>;
    const unsigned grid = unsigned(std::min<int64_t>(cdiv(a.n, S::GROUPS), 2048 / std::max(1, WPR / 4)));
    block_norm_kernel<T, WPR, V, decltype(layer)::value, decltype(after)::value><<<grid, S::THREADS, 0, st>>>(a);
    LRC_LAUNCHED();
    return LRC_OK;
  }));
}

template <class T>
lrc_status backward(hipStream_t st, const NormBackward& a, int kind, bool post) {
  const double cells = double(a.n) * double(a.d);
  ProfScope scope("block_norm_bwd_kernel", st, 30.0 * cells, 6.0 * cells * sizeof(T));
  return with_bwd_shape(a.d, with_norm(kind, post, [&](auto w, auto v, auto layer, auto after) -> lrc_status {
    constexpr int WPR = decltype(w)::value, V = decltype(v)::value;
    using S = RowShape<T, WPR, V>;
    block_norm_bwd_kernel<T, WPR, V, decltype(layer)::value, decltype(after)::value>
        <<<unsigned(bwd_groups(a.n, a.d)), S::THREADS, 0, st>>>(a);
    LRC_LAUNCHED();
    return LRC_OK;
  }));
}

}  // namespace
}  // namespace lrc

using namespace lrc;

extern "C" lrc_status lrc_block_norm(const void* b, lrc_dtype dt, int64_t n_tokens, int64_t d, int64_t ldb,
                                     const void* residual, int64_t ldr, lrc_norm kind, float eps, int post,
                                     const float* post_gamma, const float* post_beta, const float* gate, float scale,
                                     const float* gamma, const float* beta, void* s, int64_t lds, void* h,
                                     int64_t ldh, float* mean_b, float* rstd_b, float* mean_s, float* rstd_s,
                                     int8_t* q, int64_t ldq, float* qscale, int32_t* info, void* stream) {
  if ((dt != LRC_F32 && dt != LRC_BF16) || !kind_ok(kind)) return LRC_EDTYPE;
  if (!sizes_ok(n_tokens, d) || ldb < d || (residual != nullptr && ldr < d) || !(eps >= 0.f)) return LRC_EINVAL;
  if ((s != nullptr && lds < d) || (h != nullptr && ldh < d) || (q != nullptr && ldq < d)) return LRC_EINVAL;
  if ((q == nullptr) != (qscale == nullptr) || (!post && (post_gamma != nullptr || post_beta != nullptr)))
    return LRC_EINVAL;
  if (kind == LRC_NORM_RMS && (beta != nullptr || post_beta != nullptr)) return LRC_EINVAL;
  if (n_tokens == 0) return LRC_OK;
  if (b == nullptr || (s == nullptr && h == nullptr && q == nullptr)) return LRC_EINVAL;
  const NormForward a = {b,   residual, n_tokens, ldb, ldr, int(d), post_gamma, post_beta, gate,   gamma, beta, scale,
                         eps, s,        h,        lds, ldh, mean_b, rstd_b,     mean_s,    rstd_s, q,     ldq,  qscale,
                         info};
  hipStream_t st = static_cast<hipStream_t>(stream);
  return dt == LRC_BF16 ? forward<uint16_t>(st, a, kind, post != 0) : forward<float>(st, a, kind, post != 0);
}

extern "C" size_t lrc_block_norm_backward_workspace(int64_t n_tokens, int64_t d) {
  if (!sizes_ok(n_tokens, d)) return 0;
  Carve cv(nullptr);
  cv.take<float>(size_t(bwd_groups(n_tokens, d)) * 4 * d);
  return cv.bytes();
}

extern "C" lrc_status lrc_block_norm_backward(const void* dh, lrc_dtype dt, int64_t n_tokens, int64_t d, int64_t lddh,
                                              const void* ds, int64_t ldds, const void* s, int64_t lds, const void* b,
                                              int64_t ldb, const float* mean_b, const float* rstd_b,
                                              const float* mean_s, const float* rstd_s, lrc_norm kind, int post,
                                              const float* post_gamma, const float* post_beta, const float* gate,
                                              float scale, const float* gamma, void* dresidual, int64_t lddr,
                                              void* db, int64_t lddb, float* dgamma, float* dbeta,
                                              float* dpost_gamma, float* dpost_beta, float* dgate, void* ws,
                                              size_t ws_bytes, void* stream) {
  const bool layer = kind == LRC_NORM_LAYER;
  if ((dt != LRC_F32 && dt != LRC_BF16) || !kind_ok(kind)) return LRC_EDTYPE;
  if (!sizes_ok(n_tokens, d) || (dh != nullptr && (lddh < d || lds < d)) || (ds != nullptr && ldds < d))
    return LRC_EINVAL;
  if ((b != nullptr && ldb < d) || (dresidual != nullptr && lddr < d) || (db != nullptr && lddb < d)) return LRC_EINVAL;
  if (!post && (post_gamma != nullptr || post_beta != nullptr || dpost_gamma != nullptr || dpost_beta != nullptr))
    return LRC_EINVAL;
  if (!layer && (post_beta != nullptr || dbeta != nullptr || dpost_beta != nullptr)) return LRC_EINVAL;
  const bool params = dgamma != nullptr || dbeta != nullptr || dpost_gamma != nullptr || dpost_beta != nullptr ||
                      dgate != nullptr;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const ParamGrads g = {dgamma, dbeta, dpost_gamma, dpost_beta, dgate, post_gamma, post_beta, gate, scale, post != 0};
  const int sums = layer ? 4 : 2;
  const unsigned reduce_grid = unsigned(cdiv(d, 32));
  if (n_tokens == 0) {   // sums over nothing
    if (!params) return LRC_OK;
    block_norm_params_kernel<<<reduce_grid, 256, 0, st>>>(nullptr, 0, sums, int(d), g);
    LRC_LAUNCHED();
    return LRC_OK;
  }
  if (dh == nullptr && (ds == nullptr || dgamma != nullptr || dbeta != nullptr)) return LRC_EINVAL;
  if (dh != nullptr && (s == nullptr || rstd_s == nullptr || (layer && mean_s == nullptr))) return LRC_EINVAL;
  const bool after = post != 0 && (db != nullptr || dpost_gamma != nullptr || dpost_beta != nullptr ||
                                   dgate != nullptr);
  if (after && (rstd_b == nullptr || (layer && mean_b == nullptr))) return LRC_EINVAL;
  if (b == nullptr && (after || dgate != nullptr)) return LRC_EINVAL;
  const size_t need = lrc_block_norm_backward_workspace(n_tokens, d);
  if (ws_bytes < need || (need > 0 && ws == nullptr)) return LRC_EWORKSPACE;
  if (dresidual == nullptr && db == nullptr && !params) return LRC_OK;
  NormBackward a = {dh,     ds,     s,      b,      n_tokens,   lddh, ldds,  lds,   ldb,       int(d), mean_b, rstd_b,
                    mean_s, rstd_s, post_gamma, gate, gamma, scale, dresidual, db,     lddr,   lddb,
                    params ? static_cast<float*>(ws) : nullptr};
  // b^ is wanted for db through a post-norm, dgate and dpost_*; without those the row is not read
  if (!after && dgate == nullptr) a.b = nullptr;
  LRC_TRY(dt == LRC_BF16 ? backward<uint16_t>(st, a, kind, after) : backward<float>(st, a, kind, after));
  if (!params) return LRC_OK;
  block_norm_params_kernel<<<reduce_grid, 256, 0, st>>>(a.partial, bwd_groups(n_tokens, d), sums, int(d), g);
  LRC_LAUNCHED();
  return LRC_OK;
}
