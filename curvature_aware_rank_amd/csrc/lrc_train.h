// Device helpers shared by the layer-norm, linear and 8-bit checkpoint kernels.
#pragma once

#include "lrc_internal.h"

namespace lrc {

constexpr int CKB = LRC_CKPT_BLOCK;   // channels that share one checkpoint exponent

// ---- element types: bf16 held as raw bits (uint16_t) or fp32 -------------------------
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float float_of(float v) { return v; }
__device__ __forceinline__ float float_of(uint16_t v) { return bf16_bits_to_f32(v); }
__device__ __forceinline__ float float_of(int8_t v) { return float(v); }
__device__ __forceinline__ float ld_elem(const float* p) { return *p; }
__device__ __forceinline__ float ld_elem(const uint16_t* p) { return bf16_bits_to_f32(*p); }

// two fp32 -> two bf16 in one word, round to nearest even (NaN stays NaN)
__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
  const f32x2 v = {a, b};
  const bf16x2 h = __builtin_convertvector(v, bf16x2);
  uint32_t u;
  __builtin_memcpy(&u, &h, 4);
  return u;
}
__device__ __forceinline__ void st_elem(float* p, float v) { *p = v; }
__device__ __forceinline__ void st_elem(uint16_t* p, float v) { *p = uint16_t(pack_bf16x2(v, v)); }
__device__ __forceinline__ float round_to(float v, const float*) { return v; }
__device__ __forceinline__ float round_to(float v, const uint16_t*) {
  return bf16_bits_to_f32(pack_bf16x2(v, v) & 0xffffu);
}

// A short piece: its loads repeat the last element that exists, so that none of them is under a
// condition of its own and all are in flight together.
template <class T>
__device__ __forceinline__ void ld_short(const T* p, int cnt, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = 0.f;
  if (cnt <= 0) return;
  T t[7];
#pragma unroll
  for (int e = 0; e < 7; ++e) t[e] = p[min(e, cnt - 1)];
#pragma unroll
  for (int e = 0; e < 7; ++e) v[e] = e < cnt ? float_of(t[e]) : 0.f;
}
// Eight consecutive elements, of which `cnt` are in range.  Whole pieces travel as 16-byte
// accesses at the element's own alignment (the memory path takes any address), so rows of any
// pitch and start are read alike.
__device__ __forceinline__ void ld8(const float* p, int cnt, float (&v)[8]) {
  if (cnt >= 8) {
    __builtin_memcpy(v, p, 32);
    return;
  }
  ld_short(p, cnt, v);
}
__device__ __forceinline__ void ld8(const uint16_t* p, int cnt, float (&v)[8]) {
  if (cnt >= 8) {
    uint32_t w[4];
    __builtin_memcpy(w, p, 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float(w[e] << 16);
      v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
    return;
  }
  ld_short(p, cnt, v);
}
__device__ __forceinline__ void st8(float* p, int cnt, const float (&v)[8]) {
  if (cnt >= 8) {
    __builtin_memcpy(p, v, 32);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < cnt) p[e] = v[e];
}
__device__ __forceinline__ void st8(uint16_t* p, int cnt, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
  if (cnt >= 8) {
    __builtin_memcpy(p, w, 16);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < cnt) p[e] = uint16_t(w[e >> 1] >> (16 * (e & 1)));
}

// rows of `ld` elements of `size` bytes starting at p are whole aligned 16-byte pieces
inline bool rows_vec16(const void* p, int64_t ld, int size) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * size) % 16 == 0;
}

// ---- 8-bit checkpoints ---------------------------------------------------------------
// A block of 64 channels of a token shares the exponent e, the smallest integer with
// max|x| <= 127 * 2^e, held to [-126, 121] so that 2^e is a normal number and 127 * 2^e is
// finite; the codes are q = clamp(rint(x * 2^-e), -127, 127), ties to even.  The scaling by
// a power of two is exact, so there is one rounding per value, and q * 2^e has at most seven
// significant bits: it is exact in bf16.
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

__device__ __forceinline__ int ckpt_exponent(float m) {   // m: largest finite magnitude
  const uint32_t u = __float_as_uint(m);
  // m = f 2^(E - 127), 1 <= f < 2: 64 f <= 127 exactly when the mantissa field is <= 0x7E0000
  const int e = int(u >> 23) - 133 + ((u & 0x7fffffu) > 0x7e0000u ? 1 : 0);
  return max(-126, min(121, e));
}
__device__ __forceinline__ bool finite_f(float v) { return fabsf(v) < __builtin_inff(); }
__device__ __forceinline__ float finite_mag(float v) { return finite_f(v) ? fabsf(v) : 0.f; }
// code of one value (inv = 2^-e); an infinity becomes +-127, NaN becomes 0
__device__ __forceinline__ int ckpt_code(float v, float inv) {
  const float q = fminf(fmaxf(rintf(v * inv), -127.f), 127.f);
  return v == v ? int(q) : 0;
}
// eight codes times their block's step
__device__ __forceinline__ void ld8_codes(const int8_t* p, int cnt, float step, float (&v)[8]) {
  if (cnt >= 8) {
    uint32_t w[2];
    __builtin_memcpy(w, p, 8);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = float(int8_t(w[e >> 2] >> (8 * (e & 3)))) * step;
    return;
  }
  ld_short(p, cnt, v);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] *= step;
}
// Largest of the values of the eight lanes 8 i .. 8 i + 7, in each of them (three lane
// permutations inside the vector unit: neighbours, pairs, mirrored halves).
__device__ __forceinline__ uint32_t max_of_8(uint32_t u) {
  u = max(u, uint32_t(__builtin_amdgcn_mov_dpp(int(u), 0xb1, 0xf, 0xf, true)));
  u = max(u, uint32_t(__builtin_amdgcn_mov_dpp(int(u), 0x4e, 0xf, 0xf, true)));
  return max(u, uint32_t(__builtin_amdgcn_mov_dpp(int(u), 0x141, 0xf, 0xf, true)));
}
// Codes of eight consecutive values held by each of the eight lanes that share a block
// (lanes 8 i .. 8 i + 7; every lane of the group takes part, `cnt` of its values exist).
// Magnitudes are compared as integers, where NaN and infinities come out above every finite
// one: a block without them, and below the exponent's upper end, needs no test per value, and
// v * 2^-e + 1.5 * 2^23 has the code in its low byte (one rounding, ties to even).
__device__ __forceinline__ void st8_codes(int8_t* p, int8_t* pe, int cnt, const float (&v)[8], int lane,
                                          bool& bad) {
  uint32_t u = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) u = max(u, e < cnt ? __float_as_uint(v[e]) & 0x7fffffffu : 0u);
  u = max_of_8(u);
  uint32_t q[8];
  int ex;
  if (u <= 0x7f7e0000u) {   // 127 * 2^121
    ex = ckpt_exponent(__uint_as_float(u));
    const float inv = pow2f(-ex);
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = __float_as_uint(fmaf(v[e], inv, 12582912.f));
  } else {
    uint32_t f = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < cnt) {
        f = max(f, __float_as_uint(finite_mag(v[e])));
        bad |= !finite_f(v[e]);
      }
    ex = ckpt_exponent(__uint_as_float(max_of_8(f)));
    const float inv = pow2f(-ex);
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = uint32_t(ckpt_code(v[e], inv));
  }
  if (cnt <= 0) return;
  if (cnt >= 8) {
    // the low bytes of four words in one
    auto four = [](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
      const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0c0c0400u), hi = __builtin_amdgcn_perm(d, c, 0x04000c0cu);
      return lo | hi;
    };
    const uint32_t w[2] = {four(q[0], q[1], q[2], q[3]), four(q[4], q[5], q[6], q[7])};
    __builtin_memcpy(p, w, 8);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < cnt) p[e] = int8_t(q[e]);
  }
  if ((lane & 7) == 0) *pe = int8_t(ex);
}

// ---- activations and their derivatives -----------------------------------------------
// Upper tail of the normal distribution at x >= 0 as e^(-x^2/2) t P(t), t = 1 / (1 + 0.3 x):
// P is a least-maximum fit of degree 7 to the scaled tail on [0, 14], relative error 1.5e-7
// (5e-7 evaluated in fp32), so that GELU costs one exponential and one reciprocal instead of
// an error function with its two branches.  The rounding of the exponential's argument adds up to
// 9e-8 x^2 (2.6e-6 seen up to x = 8, 7.6e-6 up to 14).  `e` receives e^(-x^2/2).
__device__ __forceinline__ float normal_tail(float x, float& e) {
  const float t = __builtin_amdgcn_rcpf(fmaf(0.3f, x, 1.f));
  e = __builtin_amdgcn_exp2f(x * x * -0.72134752044448170f);
  float p = 0.03567498177289963f;
  p = fmaf(p, t, -0.15720392763614655f);
  p = fmaf(p, t, 0.20635493099689484f);
  p = fmaf(p, t, -0.053684916347265244f);
  p = fmaf(p, t, 0.12856227159500122f);
  p = fmaf(p, t, 0.09991329908370972f);
  p = fmaf(p, t, 0.12075398862361908f);
  p = fmaf(p, t, 0.11962929368019104f);
  return p * t * e;
}
__device__ __forceinline__ float logistic(float z) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * -1.4426950408889634f));
}
__device__ __forceinline__ float relu(float z) { return z > 0.f ? z : (z == z ? 0.f : z); }
__device__ __forceinline__ float relu_slope(float z) { return z > 0.f ? 1.f : (z == z ? 0.f : z); }
__device__ __forceinline__ float gelu(float z) {
  float e;
  const float q = normal_tail(fabsf(z), e);
  return z * (z >= 0.f ? 1.f - q : q);
}
__device__ __forceinline__ float gelu_slope(float z) {
  float e;
  const float q = normal_tail(fabsf(z), e);
  return fmaf(z * e, 0.39894228040143268f, z >= 0.f ? 1.f - q : q);
}
__device__ __forceinline__ float silu_slope(float z) {
  const float s = logistic(z);
  return s * (1.f + z * (1.f - s));
}
// v = act(v), and g = g act'(z); the choice is made once for all N values
template <int N>
__device__ __forceinline__ void act_apply(int act, float (&v)[N]) {
  if (act == LRC_ACT_RELU) {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = relu(v[e]);
  } else if (act == LRC_ACT_GELU) {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = gelu(v[e]);
  } else if (act == LRC_ACT_SILU) {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] *= logistic(v[e]);
  }
}
template <int N>
__device__ __forceinline__ void slope_apply(int act, const float (&z)[N], float (&g)[N]) {
  if (act == LRC_ACT_RELU) {
#pragma unroll
    for (int e = 0; e < N; ++e) g[e] *= relu_slope(z[e]);
  } else if (act == LRC_ACT_GELU) {
#pragma unroll
    for (int e = 0; e < N; ++e) g[e] *= gelu_slope(z[e]);
  } else if (act == LRC_ACT_SILU) {
#pragma unroll
    for (int e = 0; e < N; ++e) g[e] *= silu_slope(z[e]);
  }
}

// ---- products of the linear layer: D[m][n] = sum_k A(m, k) B(n, k) ----------------------
// An operand is a row-major matrix whose rows run along k (K_ROWS) or whose rows are the k
// steps (K_COLS), or a checkpoint of the latter kind (K_CODES).
enum OperandKind { K_ROWS, K_COLS, K_CODES };

// What happens to a finished row piece of D.
struct Epilogue {
  const float* bias = nullptr;
  int act = LRC_ACT_NONE;
  const void* res = nullptr;
  int64_t ldr = 0;
  void* y = nullptr;
  int64_t ldy = 0;
  void* z = nullptr;
  int64_t ldz = 0;
  int8_t* codes = nullptr;
  int8_t* exps = nullptr;
  int64_t nb = 0;
  int32_t* info = nullptr;
  bool finite = false;   // a sum that is not finite counts as zero
  void* y2 = nullptr;    // of two products in one launch: the second one's y
};

// the bias of eight consecutive columns, of which `cnt` exist
__device__ __forceinline__ void bias8(const Epilogue& ep, int64_t col, int cnt, float (&b)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) b[e] = ep.bias != nullptr && e < cnt ? ep.bias[col + e] : 0.f;
}
// Eight consecutive columns of one row.  Lanes 8 i .. 8 i + 7 of a wave hold the 64 columns
// of one block of the row and call this together; `cnt` of the lane's columns exist.
template <class TO>
__device__ __forceinline__ void finish8(const Epilogue& ep, int64_t row, int64_t col, int cnt, const float (&b)[8],
                                        float (&v)[8], int lane, bool& bad) {
  float r[8];
  if (ep.res != nullptr) ld8(static_cast<const TO*>(ep.res) + row * ep.ldr + col, cnt, r);
  if (ep.finite) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = finite_f(v[e]) ? v[e] : 0.f;
  }
  if (ep.bias != nullptr) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += b[e];
  }
  if (ep.z != nullptr && cnt > 0) st8(static_cast<TO*>(ep.z) + row * ep.ldz + col, cnt, v);
  if (ep.codes != nullptr)
    st8_codes(ep.codes + row * ep.ldz + col, ep.exps + row * ep.nb + (col >> 6), cnt, v, lane, bad);
  if (cnt <= 0) return;
  act_apply(ep.act, v);
  if (ep.res != nullptr) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += r[e];
  }
  st8(static_cast<TO*>(ep.y) + row * ep.ldy + col, cnt, v);
}

// bf16 operands with 16-byte rows on the matrix cores (lrc_gemm.hip).
struct GemmOperand {
  const uint16_t* p;   // 16-byte aligned
  int64_t ld;          // elements, a multiple of 8
  int64_t plane;       // elements between the planes of a split fp32 operand
};
// The reduction may run over several pairs of planes, one after the other: segment s
// multiplies plane (pa >> 2 s) & 3 of A with plane (pb >> 2 s) & 3 of B.
//
// What the operands' elements are (fp32 and int8: one plane).  Those operands are addressed in 16-bit
// halves as the others are: ld and plane count halves, rows are whole pieces of 16 bytes.
enum Element { BF16, FP32, INT8 };
struct GemmSegments {
  int count = 1;
  uint32_t pa = 0, pb = 0;
  Element type = BF16;
};
constexpr int64_t GEMM_MAX_LD = int64_t(1) << 21;   // tile offsets stay below 2^31 bytes
constexpr int64_t GEMM_MAX_K = int64_t(1) << 27;    // stages of all segments count in 32 bits
// The rows of a K_ROWS operand are whole 16-byte pieces, zeros behind K where K is not a
// multiple of 8; the other extent of a K_COLS operand is a multiple of 8 or padded likewise.
// TO: type of the epilogue's matrices.  `partial`: workspace of gemm_bf16_workspace bytes.
// `skip`: NULL, or a device word that makes the product a no-op when it is not zero.
template <class TO, int KA, int KB>
lrc_status gemm_bf16(hipStream_t st, const char* name, GemmOperand A, GemmOperand B, int64_t M, int64_t N, int64_t K,
                     const GemmSegments& seg, const Epilogue& ep, float* partial, const int32_t* skip, double flops,
                     double bytes);
// the splits' tiles (partial[split][M][8 ceil(N / 8)]) added in order, then the epilogue
template <class TO>
lrc_status gemm_finish(hipStream_t st, const float* partial, int splits, int64_t M, int64_t N, const Epilogue& ep,
                       const int32_t* skip);
size_t gemm_bf16_workspace(int64_t M, int64_t N, int64_t K, int KA, int KB, bool f32);
// The gradients of a gated block: epx.y = Ax Bx (n x di, k of df, the operands' second planes after the first), and
// epw.y = A1^T B, epw.y2 = A2^T B (df x di, columns of all operands), these over two segments, plane 1 of A (what
// rounding left out) and then plane 0; a sum of the first that is not finite counts as zero.  dx or the two others are
// left out where epx.y or epw.y is NULL; their bits do not depend on it.
size_t gemm_gradients_workspace(int64_t n, int64_t di, int64_t df);
template <class TO>
lrc_status gemm_gradients(hipStream_t st, const char* name, GemmOperand Ax, GemmOperand Bx, GemmOperand A1,
                          GemmOperand A2, GemmOperand B, int64_t n, int64_t di, int64_t df, const Epilogue& epx,
                          const Epilogue& epw, float* partial, double flops, double bytes);
// estimates in microseconds of an fp32 product, on fp32 operands and on ones split in three
double gemm_f32_time(int64_t M, int64_t N, int64_t K);
double gemm_split_time(int64_t M, int64_t N, int64_t K, int KA, int KB);

// ---- shared by the gated block (lrc_linear.hip) ------------------------------------------------
// up to three bf16 operands, or checkpoints, laid out (lrc_operand.h)
struct OperandJobs;
lrc_status lay_out_bf16(hipStream_t st, const OperandJobs& jobs, int count);
// dx (+)= dz W and dW = dz^T x of an fp32 layer, as lrc_linear_backward without an activation computes
// them, in its workspace.  x or its checkpoint (xcodes, xexps).
lrc_status linear_grads_f32(hipStream_t st, int64_t n, int64_t di, int64_t dn, const float* dz, int64_t lddz,
                            const float* W, int64_t ldw, const float* x, int64_t ldx, const int8_t* xcodes,
                            const int8_t* xexps, float* dx, int64_t lddx, bool add, float* dW, int64_t lddw, void* ws);
// rows x cols elements of `size` bytes (2 or 4), leading dim ld, set to zero
lrc_status zero_rows(hipStream_t st, void* p, int64_t rows, int64_t cols, int64_t ld, int size);

// ---- column sums ---------------------------------------------------------------------
// out0[c] (c < split) and out1[c - split] (c >= split) = sum over p < parts of
// partial[p * cols + c], in a fixed order.  Either output may be NULL.
lrc_status reduce_partials(hipStream_t st, const float* partial, int64_t parts, int64_t cols, int64_t split,
                           float* out0, float* out1);

}  // namespace lrc
