// Operands that a matrix product cannot read where they lie, written to the workspace as rows it can.
#pragma once

#include "lrc_train.h"

#include <type_traits>

namespace lrc {

constexpr int LT = 256;
inline int64_t round8(int64_t v) { return (v + 7) & ~int64_t(7); }

// Magnitude up to which fp32 entries are split into three bf16 pieces.
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
__device__ __forceinline__ void lay_operand(const OperandJobs& jobs, int64_t block, int32_t* __restrict__ flag) {
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

// a bf16 operand, or a checkpoint (exps), as rows of round8(cols) bf16
inline OperandJob bf16_job(const void* p, const int8_t* exps, int64_t ld, int64_t rows, int64_t cols, uint16_t* out) {
  OperandJob j;
  j.p = p;
  j.exps = exps;
  j.out = out;
  j.ld = ld;
  j.nb = cdiv(cols, CKB);
  j.rows = rows;
  j.cols = cols;
  j.w8 = round8(cols);
  j.blocks = cdiv(cdiv(rows, JOB_ROWS) * (j.w8 / 8), LT);
  return j;
}

}  // namespace lrc
