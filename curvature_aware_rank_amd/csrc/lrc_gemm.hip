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
#include "lrc_train.h"

#include <algorithm>
#include <type_traits>

namespace lrc {
namespace gemm {

constexpr int NXCD = 8;

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
template <int KIND, int EDGE, int NW, int KS, int MF, int ES>
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

  __device__ void init(const GemmOperand& o, int64_t row0, int64_t rows, int wave, int lane) {
    ld = o.ld;
    plane = o.plane;
    const int left = int(rows - row0 < EDGE ? rows - row0 : EDGE);
    if (KIND == K_ROWS) {
      base = o.p + row0 * ld;
#pragma unroll
      for (int j = 0; j < LOADS; ++j) {
        constexpr int GPR = KS / 8;          // granules per row
        const int r = (64 / GPR) * (LOADS * wave + j) + lane / GPR;
        const int g = (lane % GPR) ^ row_swizzle(r);
        kk[j] = GE * g;
        voff[j] = r < left ? unsigned(r * ld * 2) + 16 * g : OOB;
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
};

// Tile of linear index i: groups of eight tile rows, column after column inside a group, so
// that the 32 workgroups an XCD runs together form a block of 8 x 4 tiles.
__device__ __forceinline__ void tile_at(int64_t i, int64_t nm, int64_t nn, int64_t& tm, int64_t& tn) {
  const int64_t g = i / (8 * nn), first = 8 * g, rows = nm - first < 8 ? nm - first : 8;
  const int64_t r = i - g * 8 * nn;
  tm = first + r % rows;
  tn = r / rows;
}

template <class TO, int KA, int KB, int MF, int WM, int WN, int FM, int FN, int KS, int NST, bool SEG, Element EL>
__device__ __forceinline__ void gemm_tile(const GemmOperand& A, const GemmOperand& B, int64_t M, int64_t N, int64_t K,
                                          const GemmSegments& seg, const TileGrid& tg, const Epilogue& ep,
                                          float* __restrict__ partial, const int32_t* __restrict__ skip) {
  constexpr int NW = WM * WN, BM = WM * FM * MF, BN = WN * FN * MF;
  constexpr int AB = BM * KS * 2, STB = (BM + BN) * KS * 2;
  constexpr int ES = EL == FP32 ? 4 : 2;
  using SA = Stager<KA, BM, NW, KS, MF, ES>;
  using SB = Stager<KB, BN, NW, KS, MF, ES>;
  constexpr int L = SA::LOADS + SB::LOADS;      // loads of a wave per stage
  // one LDS object per stage, so that a read of one stage does not wait for the loads of others
  __shared__ __attribute__((aligned(1024))) uint8_t sb0[STB], sb1[STB], sb2[NST > 2 ? STB : 16],
      sb3[NST > 3 ? STB : 16];
  constexpr int ER = FM * MF < 32 ? FM * MF : 32;   // rows a wave finishes at a time
  constexpr int PART = ER * FN * MF * 4;
  constexpr int FIT = STB / PART;               // of them in a stage buffer
  static_assert(NST >= 2 && NST <= 4 && KS % 32 == 0 && FIT >= 1 && FIT * NST >= NW, "the epilogue rows fit the stage buffers");

  if (skip != nullptr && *skip != 0) return;
  const int b = blockIdx.x;
  const int local = b / NXCD;
  const int split = local / tg.per_xcd;
  const int64_t ti = int64_t(b % NXCD) * tg.per_xcd + local % tg.per_xcd;
  if (ti >= tg.tiles) return;
  int64_t tm, tn;
  tile_at(ti, tg.nm, tg.nn, tm, tn);
  const int64_t m0 = tm * BM, n0 = tn * BN;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave / WN, wc = wave % WN;
  SA sa;
  SB sb;
  sa.init(A, m0, M, wave, lane);
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
  typename Blk::acc_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int e = 0; e < Blk::E; ++e) acc[i][j][e] = 0.f;

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
    return q == 0 ? sb0 : q == 1 ? sb1 : q == 2 ? sb2 : sb3;
  };

  // Schedule, stage s in buffer s % NST, in STEPS steps of one fragment each.  Iteration s: read the
  // fragments of a step while the step before it is multiplied, up to the last of stage s; then a
  // barrier that leaves the loads of the stages behind s + 1 (L each per wave) in flight: stage
  // s + 1 is then in LDS and nobody reads stage s any more, so its buffer takes stage s + NST; read
  // the first step of stage s + 1, multiply the last of stage s.
  // Stages past the end are issued with empty resources (zeros, never multiplied), so that the
  // count of loads in flight stays the same to the end.
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
  for (; s + 2 * NST - 1 < nsteps; s += NST) {
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
  for (; s < nsteps; ++s) stage(buf(s), buf(s + 1), s + NST < nsteps);
  wait_barrier<0>();   // every load has landed and every read is done: the buffers are free

  // Epilogue: a wave's 32 (or 16) rows x TW columns at a time pass through its own part of LDS, so that a
  // lane holds eight consecutive columns of a row and the accesses to memory are whole pieces.
  float* tile = reinterpret_cast<float*>(buf(wave / FIT) + (wave % FIT) * PART);
  constexpr int TW = FN * MF;          // tile columns
  constexpr int LPR = TW / 8;          // lanes per row
  static_assert(TW >= 64, "a checkpoint's block belongs to one wave");
  // rows that a wave writes together fall on different banks
  auto place = [&](int r, int c) { return r * TW + (c ^ (MF == 16 ? 16 * ((r >> 2) & 3) : (r & 4) << 3)); };
  bool bad = false;
  const int64_t col = n0 + wc * TW + 8 * (lane % LPR);   // the lane's columns
  float bias[8];
  bias8(ep, col, int(min(N - col, int64_t(8))), bias);
  auto emit = [&](const typename Blk::acc_t (&upper)[FN], const typename Blk::acc_t (&lower)[FN], int i) {
#pragma unroll
    for (int h = 0; h < ER / MF; ++h)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int e = 0; e < Blk::E; ++e)
          tile[place(MF * h + Blk::row(e, lane), j * MF + lane % MF)] = h ? lower[j][e] : upper[j][e];
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
      if (tg.splits > 1) {
        const int64_t np = (N + 7) & ~int64_t(7);
        if (cnt > 0) st8(partial + (int64_t(split) * M + row) * np + col, 8, v);
      } else {
        finish8<TO>(ep, row, col, cnt, bias, v, lane, bad);
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  };
  // (the accumulators' first index is a constant in each call, so that they stay in registers)
  static_assert(FM * MF == 64 || FM * MF == 16, "a wave holds 64 or 16 rows");
  constexpr int HALF_ROWS = ER / MF;
  emit(acc[0], acc[HALF_ROWS - 1], 0);
  if constexpr (FM * MF == 64) emit(acc[HALF_ROWS], acc[2 * HALF_ROWS - 1], 1);
  if (ep.info != nullptr && bad) *ep.info = LRC_ENONFINITE;
}

template <class TO, int KA, int KB, int MF, int WM, int WN, int FM, int FN, int KS, int NST, bool SEG, Element EL>
__global__ __launch_bounds__(64 * WM * WN, 2) void gemm_bf16_kernel(GemmOperand A, GemmOperand B, int64_t M, int64_t N,
                                                                    int64_t K, GemmSegments seg, TileGrid tg,
                                                                    Epilogue ep, float* __restrict__ partial,
                                                                    const int32_t* __restrict__ skip) {
  gemm_tile<TO, KA, KB, MF, WM, WN, FM, FN, KS, NST, SEG, EL>(A, B, M, N, K, seg, tg, ep, partial, skip);
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
  const int64_t row = g / blocks, col = g % blocks * CKB + 8 * (lane & 7);
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
  finish8<TO>(ep, row, col, cnt, bias, v, lane, bad);
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

static TileGrid tiles_of(int64_t m, int64_t n, int edge, int splits, int64_t per, int64_t steps) {
  const int64_t nm = cdiv(m, edge), nn = cdiv(n, edge);
  return {nm, nn, nm * nn, int(cdiv(nm * nn, NXCD)), splits, int(per), int(steps)};
}
static double large_cost(int64_t tiles, double steps64) {
  return double(cdiv(tiles, 256)) * (steps64 * LARGE_STEP + LARGE_ROUND);
}
// small and tiny tiles: two workgroups on a unit, or one
static double round_cost(int64_t groups, double steps64, double step_full, double step_half, double round) {
  const int64_t full = groups / 512, rest = groups % 512;
  double c = double(full) * (steps64 * step_full + round);
  if (rest > 0) c += steps64 * (rest > 256 ? step_full : step_half) + round;
  return c;
}
// KL: k steps per stage of a large tile
static Plan plan_gemm(int64_t M, int64_t N, int64_t K, int count, int KL, double& cost) {
  Plan best;
  const int64_t steps_l = cdiv(K, KL), steps_s = cdiv(K, 64);
  const double s64 = double(steps_s) * count;
  const double floor_us = 2.0 * double(K) * double(M + N) * (count > 1 ? 3 : 1) / MEMORY;
  best.tile = LARGE;
  best.tg = tiles_of(M, N, 256, 1, steps_l * count, steps_l);
  cost = std::max(floor_us, large_cost(best.tg.tiles, s64));
  const int64_t total = steps_s * count;
  for (int64_t s = 1; s <= std::min<int64_t>(32, total); ++s) {
    const int64_t per = cdiv(total, s);
    if (cdiv(total, per) != s) continue;
    const TileGrid tg = tiles_of(M, N, 128, int(s), per, steps_s);
    double c = std::max(floor_us, round_cost(tg.tiles * s, double(per), SMALL_STEP_FULL, SMALL_STEP_HALF, SMALL_ROUND));
    if (s > 1) c += 4.0 + 8.0 * double(s) * double(M) * double(N) / MEMORY;
    if (c < cost) {
      cost = c;
      best = {SMALL, tg};
    }
  }
  for (int64_t s = 1; count == 1 && s <= std::min<int64_t>(32, total); ++s) {
    const int64_t per = cdiv(total, s);
    if (cdiv(total, per) != s) continue;
    const TileGrid tg = tiles_of(M, N, 64, int(s), per, steps_s);
    double c = std::max(floor_us, round_cost(tg.tiles * s, double(per), TINY_STEP_FULL, TINY_STEP_HALF, TINY_ROUND));
    if (s > 1) c += 4.0 + 8.0 * double(s) * double(M) * double(N) / MEMORY;
    if (c < cost) {
      cost = c;
      best = {TINY, tg};
    }
  }
  return best;
}
// fp32 products: tiles of 64 x 64, four waves of 16 x 64, up to five workgroups on a unit (tiles of
// 128 x 128, two on a unit, leave more units idle at these sizes: 2048 x 2048 x 1024 76 us against
// 68, 246 x 6316 x 2096 108 against 67).  32 k steps take a unit F32_STEP of matrix time, F32_ALONE
// if nothing else runs on it.
constexpr double F32_STEP = 0.5, F32_ALONE = 0.75, F32_START = 6.0;
static Plan plan_f32(int64_t M, int64_t N, int64_t K, double& cost) {
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
static size_t plan_bytes(const Plan& p, int64_t M, int64_t N) {
  return p.tg.splits > 1 ? size_t(p.tg.splits) * M * ((N + 7) & ~int64_t(7)) * 4 : 0;
}
constexpr int large_stage(int ka, int kb) { return ka == K_ROWS && kb == K_ROWS ? 64 : 32; }

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
  auto launch = [&](auto many, auto type) {
    constexpr bool SEG = decltype(many)::value;
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
    else if constexpr (!SEG)
      gemm_bf16_kernel<TO, KA, KB, 16, 4, 1, 1, 4, 64, 4, SEG, EL><<<unsigned(grid), 256, 0, st>>>(
          A, B, M, N, K, seg, tg, ep, partial, skip);
    else
      return false;
    return true;
  };
  using std::integral_constant;
  // bf16 layers have one plane; an fp32 result may come of one (dW of a bf16 layer) or more.  What no
  // caller asks for has no kernel, and is refused.
  constexpr bool BITS = std::is_same<TO, uint16_t>::value;
  bool launched = false;
  if (seg.type == FP32) {
    if constexpr (!BITS) launched = launch(std::false_type{}, integral_constant<Element, FP32>{});
  } else if (seg.count == 1) {
    if constexpr (BITS || KA == K_COLS) launched = launch(std::false_type{}, integral_constant<Element, BF16>{});
  } else if constexpr (!BITS) {
    launched = launch(std::true_type{}, integral_constant<Element, BF16>{});
  }
  if (!launched) return LRC_EINVAL;
  LRC_LAUNCHED();
  if (tg.splits == 1) return LRC_OK;
  const int splits = tg.splits;
  return gemm_finish<TO>(st, partial, splits, M, N, ep, skip);
}

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
