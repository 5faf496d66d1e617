// Token rows held in registers: shapes, loads and sums shared by the norm and quantisation kernels.
//
// WPR waves share a token (WPR <= 0: 2^-WPR tokens share a wave), each lane holds 8 V of its channels.
// Lane l holds channels 8 (k LANES + l) .. + 7 of piece k, so eight lanes hold one checkpoint block; pieces are 16-byte
// accesses at any alignment, the last one of a ragged row is short.
#pragma once

#include "lrc_train.h"

#include <type_traits>

namespace lrc {

// Sum over the wave, in every lane: lane permutations inside the vector unit (neighbours, pairs,
// mirrored eights and sixteens, then rows and halves exchanged) instead of six trips through LDS.
__device__ __forceinline__ float wave_sum(float v) {
  auto dpp = [](float x, auto ctrl) {
    return __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(x), decltype(ctrl)::value, 0xf, 0xf, true));
  };
  v += dpp(v, std::integral_constant<int, 0xb1>{});
  v += dpp(v, std::integral_constant<int, 0x4e>{});
  v += dpp(v, std::integral_constant<int, 0x141>{});
  v += dpp(v, std::integral_constant<int, 0x140>{});
  const auto rows = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(rows[0]) + __uint_as_float(rows[1]);
  const auto halves = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(halves[0]) + __uint_as_float(halves[1]);
}
// The same over 16, 32 or all 64 lanes that share a token.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
  if (LANES >= 64) return wave_sum(v);
  auto dpp = [](float x, auto ctrl) {
    return __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(x), decltype(ctrl)::value, 0xf, 0xf, true));
  };
  v += dpp(v, std::integral_constant<int, 0xb1>{});
  v += dpp(v, std::integral_constant<int, 0x4e>{});
  v += dpp(v, std::integral_constant<int, 0x141>{});
  v += dpp(v, std::integral_constant<int, 0x140>{});
  if (LANES == 16) return v;
  const auto rows = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(rows[0]) + __uint_as_float(rows[1]);
}
// The mean from the sum of x_j / 2 d, which no finite token overflows; it ends at the largest number.
__device__ __forceinline__ float mean_of(float half) {
  const float m = 2.f * half;
  return finite_f(half) ? fminf(fmaxf(m, -3.402823466e38f), 3.402823466e38f) : m;
}

constexpr int ROW_MAX = 16384;        // widest row held in registers

constexpr int row_lanes(int wpr) { return wpr > 0 ? 64 * wpr : 64 >> -wpr; }
// tokens of a workgroup at a time
constexpr int row_groups(int wpr) { return wpr >= 4 ? 1 : wpr > 0 ? 4 / wpr : 4 << -wpr; }
constexpr int row_threads(int wpr) { return row_lanes(wpr) * row_groups(wpr); }

template <class T, int WPR, int V>
struct RowShape {
  static constexpr int E = 8 * V, LANES = row_lanes(WPR), GROUPS = row_groups(WPR), THREADS = row_threads(WPR);
  static __device__ __forceinline__ int col(int i, int l) {
    return ((i >> 3) * LANES + l) * 8 + (i & 7);
  }
};

// a token's elements as they lie in memory
template <class T, int WPR, int V>
struct RawRow {
  using S = RowShape<T, WPR, V>;
  static constexpr int W = 2 * int(sizeof(T));   // 32-bit words per piece
  uint32_t q[V * W];
  __device__ __forceinline__ void load(const T* row, int d, int l, bool live) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c = (k * S::LANES + l) * 8, left = live ? d - c : 0;
      if (left >= 8) {
        __builtin_memcpy(q + k * W, row + c, 4 * W);
      } else {
#pragma unroll
        for (int w = 0; w < W; ++w) q[k * W + w] = 0u;
        if (left > 0) {   // as ld_short
          T t[7];
#pragma unroll
          for (int e = 0; e < 7; ++e) t[e] = row[c + min(e, left - 1)];
#pragma unroll
          for (int e = 0; e < 7; ++e) {
            if (sizeof(T) == 4) {
              if (e < left) __builtin_memcpy(q + k * W + e % W, t + e, 4);
            } else {
              q[k * W + (e >> 1) % W] |= e < left ? uint32_t(t[e]) << (16 * (e & 1)) : 0u;
            }
          }
        }
      }
    }
  }
  __device__ __forceinline__ float at(int i) const {
    if (sizeof(T) == 4) return __uint_as_float(q[i % (V * W)]);
    return __uint_as_float((i & 1) ? (q[i >> 1] & 0xffff0000u) : (q[i >> 1] << 16));
  }
};
// a token's codes and exponents
template <int WPR, int V>
struct RawCodes {
  using S = RowShape<uint16_t, WPR, V>;
  uint32_t q[2 * V];
  int8_t e[V];
  __device__ __forceinline__ void load(const int8_t* codes, const int8_t* exps, int d, int l, bool live) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c = (k * S::LANES + l) * 8, left = live ? d - c : 0;
      e[k] = left > 0 ? exps[c >> 6] : int8_t(0);
      if (left >= 8) {
        __builtin_memcpy(q + 2 * k, codes + c, 8);
      } else {
        q[2 * k] = q[2 * k + 1] = 0u;
        if (left > 0) {   // as ld_short
          uint8_t t[7];
#pragma unroll
          for (int i = 0; i < 7; ++i) t[i] = uint8_t(codes[c + min(i, left - 1)]);
#pragma unroll
          for (int i = 0; i < 7; ++i) q[2 * k + (i >> 2)] |= i < left ? uint32_t(t[i]) << (8 * (i & 3)) : 0u;
        }
      }
    }
  }
  __device__ __forceinline__ float at(int i) const {
    return float(int8_t(q[i >> 2] >> (8 * (i & 3)))) * pow2f(e[i >> 3]);
  }
};

// Sums of the token's WPR waves, the same in all its lanes; one barrier when waves share a
// token (`red`: a slot per wave, not reused before the barrier after the next one).
template <int WPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*red)[N], int wave_in_row, int lane, int group) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = wave_sum(v[k]);
  if (WPR == 1) return;
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < N; ++k) red[group * WPR + wave_in_row][k] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) s += red[group * WPR + w][k];
    v[k] = s;
  }
}

// Largest of a magnitude over the lanes that share a token, in each of them (as lanes_sum; magnitudes as integers).
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  v = max_of_8(v);
  v = max(v, uint32_t(__builtin_amdgcn_mov_dpp(int(v), 0x140, 0xf, 0xf, true)));
  if (LANES == 16) return v;
  const auto rows = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max(uint32_t(rows[0]), uint32_t(rows[1]));
  if (LANES == 32) return v;
  const auto halves = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(uint32_t(halves[0]), uint32_t(halves[1]));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) { return lanes_max<64>(v); }
// largest over the token's waves (`red` as in row_sums)
template <int WPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* red, int wave_in_row, int lane, int group) {
  v = lanes_max<row_lanes(WPR) < 64 ? row_lanes(WPR) : 64>(v);
  if (WPR <= 1) return v;
  if (lane == 0) red[group * WPR + wave_in_row] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < WPR; ++w) v = max(v, red[group * WPR + w]);
  return v;
}

// ---- the symmetric int8 quantiser of a token --------------------------------------------
// s = fl32(max|x| / 127) over the finite entries, q = clamp(rint(fl32(x / s)), -127, 127); a token whose
// step is zero gives zeros, an infinity +-127, NaN 0.
__device__ __forceinline__ float token_step(uint32_t mag) { return __fdiv_rn(__uint_as_float(mag), 127.f); }
__device__ __forceinline__ int token_code(float x, float s) {
  const float q = fminf(fmaxf(rintf(__fdiv_rn(x, s)), -127.f), 127.f);
  return s > 0.f && x == x ? int(q) : 0;
}
// Eight codes of which `cnt` are stored; inv = 1 / s to one unit in the last place.  x inv is within 3.1e-5 of fl32(x / s)
// (|x / s| <= 127.0001), so that only a value that near to the middle of two codes needs the division: one in 10000,
// and a lane (`odd`) that met an entry that is not finite (8192 x 4096 bf16 22.5 us against 27.7 with every value
// divided, 24.1 against 28.4 on inputs that no cache holds).  x inv + 1.5 * 2^23 has the code in its low byte (ties to
// even).
__device__ __forceinline__ float token_inverse(float s) { return s >= 0x1p-100f ? __builtin_amdgcn_rcpf(s) : 0.f; }
__device__ __forceinline__ void st8_token_codes(int8_t* p, int cnt, const float (&v)[8], float s, float inv, bool odd) {
  uint32_t q[8];
  float far = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float t = v[e] * inv, r = t + 12582912.f;
    far = fmaxf(far, fabsf(t - (r - 12582912.f)));
    q[e] = __float_as_uint(r);
  }
  if (far > 0.49995f || odd || inv == 0.f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = uint32_t(token_code(v[e], s));
  }
  auto four = [](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {   // the low bytes of four words in one
    const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0c0c0400u), hi = __builtin_amdgcn_perm(d, c, 0x04000c0cu);
    return lo | hi;
  };
  const uint32_t w[2] = {four(q[0], q[1], q[2], q[3]), four(q[4], q[5], q[6], q[7])};
  if (cnt >= 8) {
    __builtin_memcpy(p, w, 8);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < cnt) p[e] = int8_t(w[e >> 2] >> (8 * (e & 3)));
}
// largest finite magnitude, as an integer; `bad` is set by an entry that is not finite
__device__ __forceinline__ uint32_t mag8(const float (&v)[8], uint32_t m, bool& bad) {
  uint32_t u = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) u = max(u, __float_as_uint(v[e]) & 0x7fffffffu);
  if (u >= 0x7f800000u) {
    bad = true;
    u = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) u = max(u, __float_as_uint(finite_mag(v[e])));
  }
  return max(m, u);
}

// a lane's channels of gamma or beta, `absent` where there is none
template <class S, int V>
__device__ __forceinline__ void row_params(const float* p, float absent, int d, int l, float (&v)[8 * V]) {
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = (k * S::LANES + l) * 8;
    float t[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = absent;
    if (p != nullptr) ld8(p + c, d - c, t);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[8 * k + e] = t[e];
  }
}

// Calls f(waves per token, 8-channel pieces per lane) as compile-time constants for rows of d
// channels; a lane holds 8 to 32 channels (16 waves of 16 would leave 128 registers a lane, and the
// backward kernel spills: 12192 x 11008 374 us).
template <class F>
lrc_status with_row_shape(int64_t d, F f) {
  using std::integral_constant;
  if (d <= 512) return f(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  if (d <= 1024) return f(integral_constant<int, 1>{}, integral_constant<int, 2>{});
  if (d <= 2048) return f(integral_constant<int, 2>{}, integral_constant<int, 2>{});
  if (d <= 4096) return f(integral_constant<int, 4>{}, integral_constant<int, 2>{});
  if (d <= 8192) return f(integral_constant<int, 8>{}, integral_constant<int, 2>{});
  if (d <= 12288) return f(integral_constant<int, 8>{}, integral_constant<int, 3>{});
  return f(integral_constant<int, 8>{}, integral_constant<int, 4>{});
}

// The same with narrow rows in 16 or 32 lanes.
template <class F>
lrc_status with_any_row_shape(int64_t d, F f) {
  using std::integral_constant;
  if (d <= 128) return f(integral_constant<int, -2>{}, integral_constant<int, 1>{});
  if (d <= 256) return f(integral_constant<int, -1>{}, integral_constant<int, 1>{});
  return with_row_shape(d, f);
}

}  // namespace lrc
