// The tile of a matrix product: staging, fragments, pipeline, epilogue, and the choice of tiles and
// splits.  Shared by the products of the linear layer, the gated block and the 8-bit integers.
#pragma once

#include "lrc_train.h"

#include <algorithm>
#include <type_traits>

namespace lrc {
namespace gemm {

constexpr int NXCD = 8;

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4i16 lds_v4i16;
typedef __attribute__((address_space(3))) void lds_void_t;

// wait until at most N loads of this wave are in flight and its LDS reads are done, then the workgroup
template <int N>
__device__ __forceinline__ void wait_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

__device__ __forceinline__ void* uniform_ptr(const void* p) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(a));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(uint32_t(a >> 32));
  return reinterpret_cast<void*>((uint64_t(hi) << 32) | lo);
}

// One operand's stages: EDGE tile rows (channels for K_COLS), NW waves, elements of ES bytes.
// HW: 0, or the operand is one of two that share the tile's rows in turns of HW; the rows a wave
// loads then belong to one of them (`second` says which).
template <int KIND, int EDGE, int NW, int KS, int MF, int ES, int HW = 0>
struct Stager {
  static constexpr int LOADS = EDGE * KS * 2 / 1024 / NW;   // 1 KB loads per wave and stage
  static constexpr int ROWB = EDGE * ES;                    // K_COLS: bytes per k step
  static constexpr int KE = KS * 2 / ES;                    // k steps of a stage
  static constexpr int GE = 16 / ES;                        // elements of a 16-byte granule
  static_assert(EDGE >= 128 || (EDGE == 64 && MF == 16), "the granules of a k step hold their swizzle");
  static constexpr unsigned OOB = 0x80000000u;              // past every resource

  const uint16_t* base;   // first element of the tile (plane 0, k = 0)
  int64_t ld, plane;
  unsigned voff[LOADS];
  int kk[LOADS];          // K_ROWS: first k of the lane's granule within the stage
  int rows_rec;           // K_ROWS: bytes to the start of the tile's last row; K_COLS: bytes of a k step

  static constexpr int WAVE_ROWS = LOADS * 512 / KS;   // K_ROWS: tile rows a wave loads
  static_assert(HW == 0 || (KIND == K_ROWS && HW % WAVE_ROWS == 0), "a wave's rows belong to one of the two operands");
  static __device__ __forceinline__ bool second(int wave) {
    return HW > 0 && (wave * WAVE_ROWS / (HW > 0 ? HW : 1)) % 2 == 1;
  }

  __device__ void init(const GemmOperand& o, int64_t row0, int64_t rows, int wave, int lane) {
    ld = o.ld;
    plane = o.plane;
    constexpr int OWN = HW > 0 ? EDGE / 2 : EDGE;   // tile rows of this operand
    const int left = int(rows - row0 < OWN ? rows - row0 : OWN);
    if (KIND == K_ROWS) {
      base = o.p + row0 * ld;
#pragma unroll
      for (int j = 0; j < LOADS; ++j) {
        constexpr int GPR = KS / 8;          // granules per row
        const int r = (64 / GPR) * (LOADS * wave + j) + lane / GPR;
        const int g = (lane % GPR) ^ row_swizzle(r);
        kk[j] = GE * g;
        const int own = HW > 0 ? r / (HW > 0 ? 2 * HW : 1) * HW + r % (HW > 0 ? HW : 1) : r;
        voff[j] = own < left ? unsigned(own * ld * 2) + 16 * g : OOB;
      }
      rows_rec = int((left - 1) * ld * 2);
    } else {
      base = o.p + row0 * (ES / 2);
      constexpr int LPR = EDGE / GE;       // lanes (16-byte granules) per k step
#pragma unroll
      for (int j = 0; j < LOADS; ++j) {
        const int t = (64 / LPR) * (LOADS * wave + j) + lane / LPR;
        const int g = (lane % LPR) ^ step_swizzle(t);
        kk[j] = 0;
        voff[j] = GE * g < left ? unsigned(t * ld * 2) + 16 * g : OOB;
      }
      rows_rec = ES * ((left + GE - 1) & ~(GE - 1));
    }
  }

  // The loads of one stage: k steps [k, k + KE) of plane `pl`, of which `left` or all KE exist.
  struct Stage {
    __amdgpu_buffer_rsrc_t r;
    unsigned v[LOADS];
  };
  __device__ __forceinline__ Stage stage(int pl, int k, int left) const {
    const int kl = max(0, min(left, KE));
    // K_ROWS: rows are whole granules (zeros behind the last k where that is not one)
    const int rec = KIND == K_ROWS ? rows_rec + ES * ((kl + GE - 1) & ~(GE - 1)) : (kl - 1) * int(ld) * 2 + rows_rec;
    const uint16_t* p = base + pl * plane + (KIND == K_ROWS ? k * (ES / 2) : k * ld);
    Stage s;
    s.r = __builtin_amdgcn_make_buffer_rsrc(uniform_ptr(p), 0, __builtin_amdgcn_readfirstlane(kl > 0 ? rec : 0),
                                            0x00020000);
#pragma unroll
    for (int j = 0; j < LOADS; ++j) s.v[j] = KIND == K_ROWS && kk[j] >= kl ? OOB : voff[j];
    return s;
  }
  static __device__ __forceinline__ void issue(const Stage& s, uint8_t* dst, int wave) {
#pragma unroll
    for (int j = 0; j < LOADS; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(s.r, (lds_void_t*)(dst + (LOADS * wave + j) * 1024), 16, s.v[j], 0, 0,
                                               0);
  }

  // K_ROWS: rows 16 apart in a fragment read fall on every bank once
  static __device__ __forceinline__ int row_swizzle(int r) { return KS == 32 ? (r >> 2) & 3 : (r >> 1) & 7; }

  // K_COLS: the four k steps a group of 16 lanes reads fall on four quarters of the banks, the
  // groups of k steps 8 apart on halves of those
  static __device__ __forceinline__ int step_swizzle(int t) {
    if (ES == 4) return 4 * ((t >> 2) & 3);   // the four groups read k steps 4 apart, 64 bytes of each
    if (EDGE == 64) return (4 * ((t >> 1) & 1)) ^ (2 * ((t >> 3) & 1));   // a k step is half the banks
    return (4 * (t & 3)) ^ (MF == 16 ? 2 * ((t >> 3) & 1) : 0);
  }

  // A fragment is MF tile rows x KF = 512 / MF k steps, eight k of one row per lane.  Byte offset
  // of the lane's first one for tile rows row .. row + MF - 1.
  static constexpr int KF = 512 / MF;
  static __device__ int frag_off(int row, int lane) {
    if (KIND == K_ROWS) {
      const int r = row + lane % MF;
      return r * (2 * KS) + (((lane / MF) ^ row_swizzle(r)) << 4);
    }
    const int g = lane >> 4, sl = lane & 15;
    if (ES == 4) return 4 * g * ROWB + ((((row + sl) >> 2) ^ step_swizzle(4 * g)) << 4) + 4 * (sl & 3);
    const int ch = row + (MF == 32 ? 16 * (g & 1) : 0) + 4 * (sl & 3);
    const int tk = 8 * (MF == 32 ? g >> 1 : g) + (sl >> 2);
    return tk * ROWB + (((ch >> 3) ^ step_swizzle(tk)) << 4) + (ch & 7) * 2;
  }
  // fragment of the stage's k steps [KF q, KF q + KF)
  static __device__ bf16x8 frag(const uint8_t* lds, int off, int q) {
    if (KIND == K_ROWS) return *reinterpret_cast<const bf16x8*>(lds + (off ^ (2 * KF * q)));
    const uint8_t* p = lds + off + q * (KF * 2 / ES) * ROWB;
    if constexpr (ES == 4) {   // k steps 4 g .. 4 g + 3 of the lane's channel, as K_ROWS has them in a granule
      const float v[4] = {*reinterpret_cast<const float*>(p), *reinterpret_cast<const float*>(p + ROWB),
                          *reinterpret_cast<const float*>(p + 2 * ROWB),
                          *reinterpret_cast<const float*>(p + 3 * ROWB)};
      bf16x8 f;
      __builtin_memcpy(&f, v, sizeof(f));
      return f;
    }
    const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(p));
    const v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(p + 4 * ROWB));
    const short tmp[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    bf16x8 f;
    __builtin_memcpy(&f, tmp, sizeof(f));
    return f;
  }
};

// MF x MF accumulators of one matrix instruction
template <int MF>
struct Block;
template <>
struct Block<16> {
  typedef f32x4 acc_t;
  static constexpr int E = 4;
  static __device__ __forceinline__ i32x4 mma_i8(i32x4 a, i32x4 b, i32x4 c) {   // 64 k steps
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ int row(int e, int lane) { return 4 * (lane >> 4) + e; }
  static __device__ __forceinline__ acc_t mma(bf16x8 a, bf16x8 b, acc_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  // a lane's 16 bytes are four k steps; each instruction takes one of them from every lane
  static __device__ __forceinline__ acc_t mma_f32(f32x4 a, f32x4 b, acc_t c) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
    return c;
  }
};
template <>
struct Block<32> {
  typedef f32x16 acc_t;
  static constexpr int E = 16;
  static __device__ __forceinline__ int row(int e, int lane) { return 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3); }
  static __device__ __forceinline__ acc_t mma(bf16x8 a, bf16x8 b, acc_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};

struct TileGrid {
  int64_t nm, nn, tiles;
  int per_xcd, splits;
  int steps_per_split;   // stages of one split
  int steps;             // stages of one segment
  int64_t half = 0;      // of two products in one launch: tiles of each
  bool hold = false;     // the tiles go to the workspace also where k is not split
};

// What a product of 8-bit integers, or of two weights that share x, has besides.
struct Companion {
  GemmOperand B = {};             // the second weight (u = x B^T)
  void* z = nullptr;              // u, kept as the epilogue keeps z, which is g
  int8_t* codes = nullptr;
  int8_t* exps = nullptr;
  const float* row_scale = nullptr;   // of x's tokens, and of the two weights' channels
  const float* col_scale = nullptr;
  const float* col_scale2 = nullptr;
};
// the integer sums' bits as numbers: (sum * channel's scale) * token's scale
__device__ __forceinline__ void scale8(float row, const float (&col)[8], float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = float(__float_as_int(v[e])) * col[e] * row;
}
__device__ __forceinline__ void col8(const float* p, int cnt, float (&v)[8]) { ld8(p, cnt, v); }
// g and u of eight consecutive channels -> what is kept of them, and h = act(g) u.  For checkpoints
// lanes 8 i .. 8 i + 7 hold a block of 64 and call this together.
template <class TO>
__device__ __forceinline__ void finish_pair8(const Epilogue& ep, const Companion& co, int64_t row, int64_t col, int cnt,
                                             float (&g)[8], float (&u)[8], int lane, bool& bad) {
  if (ep.z != nullptr && cnt > 0) {
    st8(static_cast<TO*>(ep.z) + row * ep.ldz + col, cnt, g);
    st8(static_cast<TO*>(co.z) + row * ep.ldz + col, cnt, u);
  }
  if (ep.codes != nullptr) {
    const int64_t at = row * ep.ldz + col, blk = row * ep.nb + (col >> 6);
    st8_codes(ep.codes + at, ep.exps + blk, cnt, g, lane, bad);
    st8_codes(co.codes + at, co.exps + blk, cnt, u, lane, bad);
  }
  if (cnt <= 0) return;
  act_apply(ep.act, g);
#pragma unroll
  for (int e = 0; e < 8; ++e) g[e] *= u[e];
  st8(static_cast<TO*>(ep.y) + row * ep.ldy + col, cnt, g);
}

// Tile of linear index i: groups of eight tile rows, column after column inside a group, so
// that the 32 workgroups an XCD runs together form a block of 8 x 4 tiles.
__device__ __forceinline__ void tile_at(int64_t i, int64_t nm, int64_t nn, int64_t& tm, int64_t& tn) {
  const int64_t g = i / (8 * nn), first = 8 * g, rows = nm - first < 8 ? nm - first : 8;
  const int64_t r = i - g * 8 * nn;
  tm = first + r % rows;
  tn = r / rows;
}

// Stage buffer I, the same for all products of a kernel.  Named where it is chosen at run time: through pointers that a
// lambda holds the choice becomes branches (the smallest tiles' last stages: a linear layer's gradients at
// 1000 x 521 -> 303 34.2 us a call against 33.4).
template <int BYTES, int I>
static __shared__ __attribute__((aligned(1024))) uint8_t stage_room[BYTES];

// EL = INT8: the operands are addressed in 16-bit halves, K counts those; sums are exact int32.
// SEG: 0, one segment; 1, several; 2, two, and a sum of the first that is not finite counts as zero, of two products in
// one launch (the second one's A is co.B, its y ep.y2).
// PAIR: the tile holds BN / 2 channels of each of two weights; a wave's first FN MF / 2 columns are the
// first one's, the others the same channels of the second.
// block: the workgroup's place in the product's grid.
template <class TO, int KA, int KB, int MF, int WM, int WN, int FM, int FN, int KS, int NST, int SEG, Element EL,
          bool PAIR = false>
__device__ __forceinline__ void gemm_tile(const GemmOperand& A, const GemmOperand& B, int64_t M, int64_t N, int64_t K,
                                          const GemmSegments& seg, const TileGrid& tg, const Epilogue& ep,
                                          float* __restrict__ partial, const int32_t* __restrict__ skip,
                                          const Companion& co, int block) {
  constexpr int NW = WM * WN, BM = WM * FM * MF, BN = WN * FN * MF;
  constexpr int AB = BM * KS * 2, STB = (BM + BN) * KS * 2;
  constexpr int ES = EL == FP32 ? 4 : 2;
  using SA = Stager<KA, BM, NW, KS, MF, ES>;
  constexpr int HW = PAIR ? FN * MF / 2 : 0;
  using SB = Stager<KB, BN, NW, KS, MF, ES, HW>;
  constexpr int L = SA::LOADS + SB::LOADS;      // loads of a wave per stage
  // one LDS object per stage, so that a read of one stage does not wait for the loads of others
  constexpr int THIRD = NST > 2 ? 2 : 0, FOURTH = NST > 3 ? 3 : 0;
  uint8_t *const sb0 = stage_room<STB, 0>, *const sb1 = stage_room<STB, 1>;
  uint8_t *const sb2 = stage_room<STB, THIRD>, *const sb3 = stage_room<STB, FOURTH>;
  constexpr int ER = FM * MF < 32 ? FM * MF : 32;   // rows a wave finishes at a time
  constexpr int PART = ER * FN * MF * 4;
  constexpr int FIT = STB / PART;               // of them in a stage buffer
  static_assert(NST >= 2 && NST <= 4 && KS % 32 == 0 && FIT >= 1 && FIT * NST >= NW, "the epilogue rows fit the stage buffers");

  if (skip != nullptr && *skip != 0) return;
  const int local = block / NXCD;
  const int split = local / tg.per_xcd;
  const int64_t ti = int64_t(block % NXCD) * tg.per_xcd + local % tg.per_xcd;
  if (ti >= tg.tiles) return;
  const bool other = SEG == 2 && ti >= tg.half;   // of two products, the second
  int64_t tm, tn;
  tile_at(other ? ti - tg.half : ti, tg.nm, tg.nn, tm, tn);
  const int64_t m0 = tm * BM, n0 = tn * (PAIR ? BN / 2 : BN);

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave / WN, wc = wave % WN;
  SA sa;
  SB sb;
  sa.init(other ? co.B : A, m0, M, wave, lane);
  if constexpr (PAIR)
    sb.init(SB::second(wave) ? co.B : B, n0, N, wave, lane);
  else
    sb.init(B, n0, N, wave, lane);

  // stages of this split, counted over all segments
  const int total = tg.steps * (SEG ? seg.count : 1);
  const int first = split * tg.steps_per_split;
  const int nsteps = min(tg.steps_per_split, total - first);
  int sg = SEG ? first / tg.steps : 0;
  int k = (first - sg * tg.steps) * SA::KE;   // next stage to issue
  const int kend = int(K);
  typename SA::Stage ga;
  typename SB::Stage gb;
  // resources and offsets of the next stage, then (after the barrier that frees its buffer) its
  // loads
  auto next_stage = [&](bool live) {
    const int left = live ? kend - k : 0;
    ga = sa.stage(SEG ? int((seg.pa >> (2 * sg)) & 3) : 0, k, left);
    gb = sb.stage(SEG ? int((seg.pb >> (2 * sg)) & 3) : 0, k, left);
    k += SA::KE;
    if (SEG) {
      const bool next = k >= kend;
      sg += next ? 1 : 0;
      k = next ? 0 : k;
    }
  };
  auto issue = [&](uint8_t* dst) {
    SA::issue(ga, dst, wave);
    SB::issue(gb, dst + AB, wave);
  };

  int offa[FM], offb[FN];
#pragma unroll
  for (int i = 0; i < FM; ++i) offa[i] = SA::frag_off((wr * FM + i) * MF, lane);
#pragma unroll
  for (int j = 0; j < FN; ++j) offb[j] = SB::frag_off((wc * FN + j) * MF, lane);
  using Blk = Block<MF>;
  using Acc = std::conditional_t<EL == INT8, i32x4, typename Blk::acc_t>;
  Acc acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int e = 0; e < Blk::E; ++e) acc[i][j][e] = 0;

  bf16x8 fa0[FM], fb0[FN], fa1[FM], fb1[FN];
  auto read_frags = [&](const uint8_t* s, int q, bf16x8* fa, bf16x8* fb) {
#pragma unroll
    for (int i = 0; i < FM; ++i) fa[i] = SA::frag(s, offa[i], q);
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[j] = SB::frag(s + AB, offb[j], q);
  };
  auto mma = [&](const bf16x8* fa, const bf16x8* fb) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
        if constexpr (EL == FP32)
          acc[i][j] = Blk::mma_f32(__builtin_bit_cast(f32x4, fa[i]), __builtin_bit_cast(f32x4, fb[j]), acc[i][j]);
        else if constexpr (EL == INT8)
          acc[i][j] = Blk::mma_i8(__builtin_bit_cast(i32x4, fa[i]), __builtin_bit_cast(i32x4, fb[j]), acc[i][j]);
        else
          acc[i][j] = Blk::mma(fa[i], fb[j], acc[i][j]);
  };
  // Issue order of a step: the fragment reads (and the next stage's loads) go out between the
  // products, which hide them.
  constexpr int COLS = EL == FP32 ? 4 : 2, READS = FM * (KA == K_ROWS ? 1 : COLS) + FN * (KB == K_ROWS ? 1 : COLS),
                MM = FM * FN * (EL == FP32 ? 4 : 1);
  constexpr int GROUPS = MM < 8 ? 4 : 8, GRP = MM / GROUPS;   // products per group
  auto interleave_reads = [&]() {
#define LRC_PAIR                                                       \
  __builtin_amdgcn_sched_group_barrier(0x008, GRP, 0);                 \
  __builtin_amdgcn_sched_group_barrier(0x100, (READS + GROUPS - 1) / GROUPS, 0);
    LRC_PAIR LRC_PAIR LRC_PAIR LRC_PAIR
    if constexpr (GROUPS == 8) { LRC_PAIR LRC_PAIR LRC_PAIR LRC_PAIR }
  };
  auto interleave_loads = [&]() {
#define LRC_TRIPLE LRC_PAIR __builtin_amdgcn_sched_group_barrier(0x020, (L + GROUPS - 1) / GROUPS, 0);
    LRC_TRIPLE LRC_TRIPLE LRC_TRIPLE LRC_TRIPLE
    if constexpr (GROUPS == 8) { LRC_TRIPLE LRC_TRIPLE LRC_TRIPLE LRC_TRIPLE }
#undef LRC_TRIPLE
#undef LRC_PAIR
  };
  auto buf = [&](int st) -> uint8_t* {
    const int q = st % NST;
    return q == 0   ? stage_room<STB, 0>
           : q == 1 ? stage_room<STB, 1>
           : q == 2 ? stage_room<STB, THIRD>
                    : stage_room<STB, FOURTH>;
  };

  // Schedule, stage s in buffer s % NST, in STEPS steps of one fragment each.  Iteration s: read the
  // fragments of a step while the step before it is multiplied, up to the last of stage s; then a
  // barrier that leaves the loads of the stages behind s + 1 (L each per wave) in flight: stage
  // s + 1 is then in LDS and nobody reads stage s any more, so its buffer takes stage s + NST; read
  // the first step of stage s + 1, multiply the last of stage s.
  // Stages past the end are issued with empty resources (zeros, never multiplied), so that the
  // count of loads in flight stays the same to the end.
  // the tokens' scales wait in LDS for the epilogue, which else would wait for each (8192 x 4096 x 8192 230 us against 243)
  __shared__ float rows_scale[EL == INT8 ? BM : 1];
  if constexpr (EL == INT8) {
    for (int r = threadIdx.x; r < BM; r += 64 * NW) rows_scale[r] = co.row_scale[min(m0 + r, M - 1)];
  }
  next_stage(nsteps > 0);
  issue(sb0);
  next_stage(nsteps > 1);
  issue(sb1);
  if constexpr (NST > 2) {
    next_stage(nsteps > 2);
    issue(sb2);
  }
  if constexpr (NST > 3) {
    next_stage(nsteps > 3);
    issue(sb3);
  }
  wait_barrier<(NST - 1) * L>();
  read_frags(sb0, 0, fa0, fb0);
  // a stage of KS / KF steps (an even number); fa0, fb0 hold its first one
  constexpr int STEPS = KS / SA::KF;
  static_assert(STEPS % 2 == 0 && STEPS >= 2, "the two fragment sets take turns");
  auto stage = [&](uint8_t* cur, const uint8_t* nxt, bool live) {
    next_stage(live);
#pragma unroll
    for (int q = 0; q < STEPS; q += 2) {
      read_frags(cur, q + 1, fa1, fb1);
      mma(fa0, fb0);
      interleave_reads();
      __builtin_amdgcn_sched_barrier(0);
      if (q + 2 < STEPS) {
        read_frags(cur, q + 2, fa0, fb0);
        mma(fa1, fb1);
        interleave_reads();
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    wait_barrier<(NST - 2) * L>();
    __builtin_amdgcn_sched_barrier(0);
    issue(cur);
    read_frags(nxt, 0, fa0, fb0);
    mma(fa1, fb1);
    interleave_loads();
    __builtin_amdgcn_sched_barrier(0);
  };
  int s = 0;
  // stages of the first segment that end inside this split, or all
  const int inside = SEG == 2 ? tg.steps - first : nsteps;
  int limit = SEG == 2 && inside > 0 && inside < nsteps ? inside : nsteps;
  auto finite_sums = [&]() {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int e = 0; e < Blk::E; ++e) acc[i][j][e] = finite_f(acc[i][j][e]) ? acc[i][j][e] : 0.f;
  };
  for (;;) {
    if constexpr (SEG == 2) {   // up to a stage whose buffer is the first
      for (; s % NST != 0 && s < limit; ++s) stage(buf(s), buf(s + 1), s + NST < nsteps);
    }
    for (; s + 2 * NST - 1 < nsteps && (SEG != 2 || s + NST <= limit); s += NST) {
      if constexpr (NST == 2) {
        stage(sb0, sb1, true);
        stage(sb1, sb0, true);
      } else {
        static_assert(NST == 2 || NST == 4, "two or four stage buffers");
        stage(sb0, sb1, true);
        stage(sb1, sb2, true);
        stage(sb2, sb3, true);
        stage(sb3, sb0, true);
      }
    }
    // the last stages choose their buffers at run time; behind the last one only zeros are read
    for (; s < limit; ++s) stage(buf(s), buf(s + 1), s + NST < nsteps);
    if constexpr (SEG == 2) {
      if (s <= inside) finite_sums();
      if (limit < nsteps) {
        limit = nsteps;
        continue;
      }
    }
    break;
  }
  wait_barrier<0>();   // every load has landed and every read is done: the buffers are free

  // Epilogue: a wave's 32 (or 16) rows x TW columns at a time pass through its own part of LDS, so that a
  // lane holds eight consecutive columns of a row and the accesses to memory are whole pieces.
  float* tile = reinterpret_cast<float*>(buf(wave / FIT) + (wave % FIT) * PART);
  constexpr int TW = FN * MF;          // tile columns
  constexpr int CW = PAIR ? TW / 2 : TW;   // channels of a wave
  constexpr int LPR = CW / 8;          // lanes per row
  static_assert(TW >= 64, "a checkpoint's block belongs to one wave (of a pair: where CW is 64)");
  // rows that a wave writes together fall on different banks
  auto place = [&](int r, int c) { return r * TW + (c ^ (MF == 16 ? 16 * ((r >> 2) & 3) : (r & 4) << 3)); };
  bool bad = false;
  const int64_t col = n0 + wc * CW + 8 * (lane % LPR);   // the lane's columns
  const int cols = int(min(N - col, int64_t(8)));
  float bias[8], sc[8], sc2[8];
  if constexpr (!PAIR) bias8(ep, col, cols, bias);
  if constexpr (EL == INT8) {
    col8(co.col_scale + col, cols, sc);
    if constexpr (PAIR) col8(co.col_scale2 + col, cols, sc2);
  }
  auto emit = [&](const Acc (&upper)[FN], const Acc (&lower)[FN], int i) {
#pragma unroll
    for (int h = 0; h < ER / MF; ++h)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int e = 0; e < Blk::E; ++e)
          tile[place(MF * h + Blk::row(e, lane), j * MF + lane % MF)] =
              EL == INT8 ? __int_as_float(int(h ? lower[j][e] : upper[j][e])) : float(h ? lower[j][e] : upper[j][e]);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll 2
    for (int q = 0; q < ER * LPR / 64; ++q) {
      const int r = q * (64 / LPR) + lane / LPR, c = 8 * (lane % LPR);
      const float* src = tile + place(r, c);
      const f32x4 lo = *reinterpret_cast<const f32x4*>(src), hi = *reinterpret_cast<const f32x4*>(src + 4);
      float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      const int64_t row = m0 + wr * FM * MF + i * 32 + r;
      const int64_t left = row < M ? N - col : 0;
      const int cnt = int(left < 0 ? 0 : left > 8 ? 8 : left);
      if constexpr (PAIR) {
        const float* src2 = tile + place(r, CW + c);
        const f32x4 lo2 = *reinterpret_cast<const f32x4*>(src2), hi2 = *reinterpret_cast<const f32x4*>(src2 + 4);
        float u[8] = {lo2[0], lo2[1], lo2[2], lo2[3], hi2[0], hi2[1], hi2[2], hi2[3]};
        if (tg.splits > 1 || tg.hold) {
          const int64_t np = (N + 7) & ~int64_t(7);
          float* o = partial + (int64_t(split) * M + row) * 2 * np + col;
          if (cnt > 0) {
            st8(o, 8, v);
            st8(o + np, 8, u);
          }
        } else {
          if constexpr (EL == INT8) {
            const float s = rows_scale[wr * FM * MF + i * 32 + r];
            scale8(s, sc, v);
            scale8(s, sc2, u);
          }
          finish_pair8<TO>(ep, co, row, col, cnt, v, u, lane, bad);
        }
      } else if (tg.splits > 1) {
        const int64_t np = (N + 7) & ~int64_t(7), at = int64_t(SEG == 2 ? 2 * split + other : split) * M + row;
        if (cnt > 0) st8(partial + at * np + col, 8, v);
      } else if constexpr (SEG == 2) {
        if (cnt > 0) st8(static_cast<TO*>(other ? ep.y2 : ep.y) + row * ep.ldy + col, cnt, v);
      } else {
        if constexpr (EL == INT8) scale8(rows_scale[wr * FM * MF + i * 32 + r], sc, v);
        finish8<TO>(ep, row, col, cnt, bias, v, lane, bad);
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  };
  // (the accumulators' first index is a constant in each call, so that they stay in registers)
  static_assert(FM * MF == 64 || FM * MF == 32 || FM * MF == 16, "a wave holds 64, 32 or 16 rows");
  constexpr int HALF_ROWS = ER / MF;
  emit(acc[0], acc[HALF_ROWS - 1], 0);
  if constexpr (FM * MF == 64) emit(acc[HALF_ROWS], acc[2 * HALF_ROWS - 1], 1);
  if (ep.info != nullptr && bad) *ep.info = LRC_ENONFINITE;
}

// Tiles and splits from the sizes alone (256 compute units), so that workspace sizes are known
// without a device and equal inputs give equal bits.  LARGE tiles (256 x 256, one workgroup per
// compute unit, 1330 TFLOP/s at 4096^3) for products that fill the chip; SMALL ones (128 x 128, two
// per unit, 1060) and TINY ones (64 x 64, four stages ahead) otherwise, with k split when they are
// few.  Tiny ones need twice the loads but wait less for each: 1000 x 1024 x 1024 forward / dx / dW
// 7.9 / 9.0 / 9.2 us against 13.5 / 15.5 / 16.8 on small ones, 64 x 4096 x 11008 18 / 25 / 42 against
// 26 / 26 / 43; 4096 x 1024 x 1024 stays on large ones (17).  Small tiles for what a last, part
// full round of large ones holds gained nothing (8192 x 4096 x 11008, 5.4 rounds: 695 us against
// 690).  Times below in microseconds, taken at 100 x 64 x 64 to 8192 x 4096 x 11008.
enum Tile { LARGE, SMALL, TINY };
struct Plan {
  Tile tile;
  TileGrid tg;
};
// 64 k steps of every workgroup of a round; a round's first loads and its epilogue
constexpr double LARGE_STEP = 1.55, SMALL_STEP_FULL = 0.88, SMALL_STEP_HALF = 0.64, LARGE_ROUND = 14.0,
                 SMALL_ROUND = 8.0, TINY_STEP_FULL = 0.38, TINY_STEP_HALF = 0.25, TINY_ROUND = 4.0,
                 MEMORY = 4.5e6;

inline TileGrid tiles_of(int64_t m, int64_t n, int edge, int splits, int64_t per, int64_t steps) {
  const int64_t nm = cdiv(m, edge), nn = cdiv(n, edge);
  return {nm, nn, nm * nn, int(cdiv(nm * nn, NXCD)), splits, int(per), int(steps)};
}
inline double large_cost(int64_t tiles, double steps64) {
  return double(cdiv(tiles, 256)) * (steps64 * LARGE_STEP + LARGE_ROUND);
}
// small and tiny tiles: two workgroups on a unit, or one
inline double round_cost(int64_t groups, double steps64, double step_full, double step_half, double round) {
  const int64_t full = groups / 512, rest = groups % 512;
  double c = double(full) * (steps64 * step_full + round);
  if (rest > 0) c += steps64 * (rest > 256 ? step_full : step_half) + round;
  return c;
}
// One kind of tile.  KL: k steps per stage of a large one.
inline Plan plan_tiles(Tile tile, int64_t M, int64_t N, int64_t K, int count, int KL, double& cost) {
  Plan best;
  best.tile = tile;
  const int64_t steps_l = cdiv(K, KL), steps_s = cdiv(K, 64), total = steps_s * count;
  const double floor_us = 2.0 * double(K) * double(M + N) * std::min(count, 3) / MEMORY;
  if (tile == LARGE) {
    best.tg = tiles_of(M, N, 256, 1, steps_l * count, steps_l);
    cost = std::max(floor_us, large_cost(best.tg.tiles, double(total)));
    return best;
  }
  const bool small = tile == SMALL;
  const int edge = small ? 128 : 64;
  const double full = small ? SMALL_STEP_FULL : TINY_STEP_FULL, half = small ? SMALL_STEP_HALF : TINY_STEP_HALF,
               round = small ? SMALL_ROUND : TINY_ROUND;
  cost = 1e30;
  for (int64_t s = 1; s <= std::min<int64_t>(32, total); ++s) {
    const int64_t per = cdiv(total, s);
    if (cdiv(total, per) != s) continue;
    const TileGrid tg = tiles_of(M, N, edge, int(s), per, steps_s);
    double c = std::max(floor_us, round_cost(tg.tiles * s, double(per), full, half, round));
    if (s > 1) c += 4.0 + 8.0 * double(s) * double(M) * double(N) / MEMORY;
    if (c < cost) {
      cost = c;
      best.tg = tg;
    }
  }
  return best;
}
inline Plan plan_gemm(int64_t M, int64_t N, int64_t K, int count, int KL, double& cost) {
  Plan best = plan_tiles(LARGE, M, N, K, count, KL, cost);
  for (Tile tile : {SMALL, TINY}) {
    if (tile == TINY && count > 1) continue;   // no such tiles over several segments (the gradients plan theirs apart)
    double c;
    const Plan p = plan_tiles(tile, M, N, K, count, KL, c);
    if (c < cost) {
      cost = c;
      best = p;
    }
  }
  return best;
}
// fp32 products: tiles of 64 x 64, four waves of 16 x 64, up to five workgroups on a unit (tiles of
// 128 x 128, two on a unit, leave more units idle at these sizes: 2048 x 2048 x 1024 76 us against
// 68, 246 x 6316 x 2096 108 against 67).  32 k steps take a unit F32_STEP of matrix time, F32_ALONE
// if nothing else runs on it.
constexpr double F32_STEP = 0.5, F32_ALONE = 0.75, F32_START = 6.0;
inline Plan plan_f32(int64_t M, int64_t N, int64_t K, double& cost) {
  Plan best;
  best.tile = TINY;
  cost = 0;
  const int64_t steps = cdiv(K, 32);
  for (int64_t s = 1; s <= std::min<int64_t>(32, steps); ++s) {
    const int64_t per = cdiv(steps, s);
    if (cdiv(steps, per) != s) continue;
    const TileGrid tg = tiles_of(M, N, 64, int(s), per, steps);
    const int64_t each = cdiv(tg.tiles * s, 256);
    double c = F32_START + double(per) * (each == 1 ? F32_ALONE : double(each) * F32_STEP);
    if (s > 1) c += 6.0 + 8.0 * double(s) * double(M) * double(N) / MEMORY;
    if (s == 1 || c < cost) {
      cost = c;
      best.tg = tg;
    }
  }
  return best;
}
inline size_t plan_bytes(const Plan& p, int64_t M, int64_t N) {
  return p.tg.splits > 1 ? size_t(p.tg.splits) * M * ((N + 7) & ~int64_t(7)) * 4 : 0;
}
constexpr int large_stage(int ka, int kb) { return ka == K_ROWS && kb == K_ROWS ? 64 : 32; }

}  // namespace gemm
}  // namespace lrc
