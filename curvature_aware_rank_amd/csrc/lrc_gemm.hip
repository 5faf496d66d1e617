// bf16 matrix products on the matrix cores with a fused epilogue: the linear layer's forward,
// dx and dW products.
//
// An output tile of BM x BN belongs to one workgroup; its waves hold blocks of 32 x 32
// accumulators.  Both operands travel from memory straight into LDS (16 bytes per lane, no
// staging registers) in stages of 32 k steps, four stage buffers, three stages in flight
// while one is multiplied.  A buffer resource bounds each operand, so rows past the matrix and
// k past its end read as zeros without any masking of data.
//   K_ROWS: a tile row's 32 k steps are 64 bytes; the 16-byte granule g of row r sits in slot
//     g ^ ((r / 4) % 4), so the 16 rows of a fragment read cover every bank once.
//   K_COLS: a k step's BM channels lie together; fragments come from transposing LDS reads
//     (ds_read_b64_tr_b16), granule g of step t in slot g ^ 4 (t % 4).
// Few tiles leave compute units idle, so k may be split: every split writes its fp32 tile and
// a second kernel adds them in split order and runs the epilogue (bit-reproducible).
#include "lrc_train.h"

#include <algorithm>
#include <type_traits>

namespace lrc {
namespace gemm {

constexpr int KS = 32;      // k steps per stage
constexpr int NXCD = 8;

typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4i16 lds_v4i16;
typedef __attribute__((address_space(3))) void lds_void_t;

#define LRC_WAIT_BARRIER(N) asm volatile("s_waitcnt vmcnt(" #N ") lgkmcnt(0)\n\ts_barrier" ::: "memory")

__device__ __forceinline__ void* uniform_ptr(const void* p) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(a));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(uint32_t(a >> 32));
  return reinterpret_cast<void*>((uint64_t(hi) << 32) | lo);
}

// One operand's stages: EDGE tile rows (channels for K_COLS), NW waves.
template <int KIND, int EDGE, int NW>
struct Stager {
  static constexpr int LOADS = EDGE * KS * 2 / 1024 / NW;   // 1 KB loads per wave and stage
  static constexpr int ROWB = EDGE * 2;                     // K_COLS: bytes per k step
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
        const int r = 16 * (LOADS * wave + j) + (lane >> 2);
        const int g = (lane & 3) ^ ((r >> 2) & 3);
        kk[j] = 8 * g;
        voff[j] = r < left ? unsigned(r * ld * 2) + 16 * g : OOB;
      }
      rows_rec = int((left - 1) * ld * 2);
    } else {
      base = o.p + row0;
      constexpr int LPR = EDGE / 8;        // lanes (16-byte granules) per k step
#pragma unroll
      for (int j = 0; j < LOADS; ++j) {
        const int t = (64 / LPR) * (LOADS * wave + j) + lane / LPR;
        const int g = (lane % LPR) ^ (4 * (t & 3));
        kk[j] = 0;
        voff[j] = 8 * g < left ? unsigned(t * ld * 2) + 16 * g : OOB;
      }
      rows_rec = 2 * ((left + 7) & ~7);
    }
  }

  // The loads of one stage: k steps [k, k + 32) of plane `pl`, of which `left` or all 32 exist.
  struct Stage {
    __amdgpu_buffer_rsrc_t r;
    unsigned v[LOADS];
  };
  __device__ __forceinline__ Stage stage(int pl, int k, int left) const {
    const int kl = max(0, min(left, KS));
    // K_ROWS: rows are whole granules (zeros behind the last k where that is not one)
    const int rec = KIND == K_ROWS ? rows_rec + 2 * ((kl + 7) & ~7) : (kl - 1) * int(ld) * 2 + rows_rec;
    const uint16_t* p = base + pl * plane + (KIND == K_ROWS ? k : k * ld);
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

  // byte offset of the lane's fragment of tile rows row .. row + 31, k half 0
  static __device__ int frag_off(int row, int lane) {
    if (KIND == K_ROWS) {
      const int r = row + (lane & 31);
      return r * 64 + (((lane >> 5) ^ ((r >> 2) & 3)) << 4);
    }
    const int g = lane >> 4, sl = lane & 15;
    const int ch = row + 16 * (g & 1) + 4 * (sl & 3);
    const int tk = 8 * (g >> 1) + (sl >> 2);
    return tk * ROWB + (((ch >> 3) ^ (4 * (tk & 3))) << 4) + (ch & 7) * 2;
  }
  // fragment of k half `half` (16 steps)
  static __device__ bf16x8 frag(const uint8_t* lds, int off, int half) {
    if (KIND == K_ROWS) return *reinterpret_cast<const bf16x8*>(lds + (half ? off ^ 32 : off));
    const uint8_t* p = lds + off + half * 16 * ROWB;
    const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(p));
    const v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(p + 4 * ROWB));
    const short tmp[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    bf16x8 f;
    __builtin_memcpy(&f, tmp, sizeof(f));
    return f;
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

template <class TO, int KA, int KB, int WM, int WN, int FM, int FN, bool SEG>
__device__ __forceinline__ void gemm_tile(const GemmOperand& A, const GemmOperand& B, int64_t M, int64_t N, int64_t K,
                                          const GemmSegments& seg, const TileGrid& tg, const Epilogue& ep,
                                          float* __restrict__ partial, const int32_t* __restrict__ skip) {
  constexpr int NW = WM * WN, BM = WM * FM * 32, BN = WN * FN * 32;
  constexpr int AB = BM * KS * 2, STB = (BM + BN) * KS * 2;
  using SA = Stager<KA, BM, NW>;
  using SB = Stager<KB, BN, NW>;
  static_assert(SA::LOADS + SB::LOADS == 4, "the stage barrier counts four loads per wave and stage");
  // one LDS object per stage, so that a read of one stage does not wait for the loads of others
  __shared__ __attribute__((aligned(1024))) uint8_t sb0[STB], sb1[STB], sb2[STB], sb3[STB];
  static_assert(2 * 32 * FN * 32 * 4 <= STB && NW <= 8, "two waves' epilogue rows per stage buffer");

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
  int k = (first - sg * tg.steps) * KS;   // next stage to issue
  const int kend = int(K);
  typename SA::Stage ga;
  typename SB::Stage gb;
  // resources and offsets of the next stage, then (after the barrier that frees its buffer) its
  // loads
  auto next_stage = [&](bool live) {
    const int left = live ? kend - k : 0;
    ga = sa.stage(SEG ? int((seg.pa >> (2 * sg)) & 3) : 0, k, left);
    gb = sb.stage(SEG ? int((seg.pb >> (2 * sg)) & 3) : 0, k, left);
    k += KS;
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
  for (int i = 0; i < FM; ++i) offa[i] = SA::frag_off((wr * FM + i) * 32, lane);
#pragma unroll
  for (int j = 0; j < FN; ++j) offb[j] = SB::frag_off((wc * FN + j) * 32, lane);
  f32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

  bf16x8 fa0[FM], fb0[FN], fa1[FM], fb1[FN];
  auto read_half = [&](const uint8_t* s, int half, bf16x8* fa, bf16x8* fb) {
#pragma unroll
    for (int i = 0; i < FM; ++i) fa[i] = SA::frag(s, offa[i], half);
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[j] = SB::frag(s + AB, offb[j], half);
  };
  auto mma = [&](const bf16x8* fa, const bf16x8* fb) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[i], fb[j], acc[i][j], 0, 0, 0);
  };
  // Issue orders of the two halves of a step: the fragment reads (and the next stage's loads)
  // go out between the products, which hide them.
  constexpr int RD = (FM * (KA == K_ROWS ? 1 : 2) + FN * (KB == K_ROWS ? 1 : 2) + FM * FN - 1) / (FM * FN);
  auto interleave_reads = [&]() {
#define LRC_PAIR                                         \
  __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);     \
  __builtin_amdgcn_sched_group_barrier(0x100, RD, 0);
    LRC_PAIR LRC_PAIR LRC_PAIR LRC_PAIR
    if constexpr (FM * FN == 8) { LRC_PAIR LRC_PAIR LRC_PAIR LRC_PAIR }
  };
  auto interleave_loads = [&]() {
#define LRC_TRIPLE LRC_PAIR __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    LRC_TRIPLE LRC_TRIPLE LRC_TRIPLE LRC_TRIPLE
    if constexpr (FM * FN == 8) { LRC_PAIR LRC_PAIR LRC_PAIR LRC_PAIR }
#undef LRC_TRIPLE
#undef LRC_PAIR
  };
  auto buf = [&](int st) -> uint8_t* {
    const int q = st & 3;
    return q == 0 ? sb0 : q == 1 ? sb1 : q == 2 ? sb2 : sb3;
  };

  // Schedule, stage s in buffer s % 4.  Iteration s: read the second half of stage s, multiply
  // its first half, then a barrier that leaves the loads of stages s + 2 and s + 3 (four each
  // per wave) in flight: stage s + 1 is then in LDS and nobody reads stage s any more, so its
  // buffer takes stage s + 4; read the first half of stage s + 1, multiply the second half of
  // stage s.  Stages past the end are issued with empty resources (zeros, never multiplied), so
  // that the count of loads in flight stays the same to the end.
  next_stage(nsteps > 0);
  issue(sb0);
  next_stage(nsteps > 1);
  issue(sb1);
  next_stage(nsteps > 2);
  issue(sb2);
  next_stage(nsteps > 3);
  issue(sb3);
  LRC_WAIT_BARRIER(12);
  read_half(sb0, 0, fa0, fb0);
  int s = 0;
#define LRC_STEP(CUR, NXT)             \
  next_stage(true);                    \
  read_half(CUR, 1, fa1, fb1);         \
  mma(fa0, fb0);                       \
  interleave_reads();                  \
  __builtin_amdgcn_sched_barrier(0);   \
  LRC_WAIT_BARRIER(8);                 \
  __builtin_amdgcn_sched_barrier(0);   \
  issue(CUR);                          \
  read_half(NXT, 0, fa0, fb0);         \
  mma(fa1, fb1);                       \
  interleave_loads();                  \
  __builtin_amdgcn_sched_barrier(0);
  for (; s + 7 < nsteps; s += 4) {
    LRC_STEP(sb0, sb1)
    LRC_STEP(sb1, sb2)
    LRC_STEP(sb2, sb3)
    LRC_STEP(sb3, sb0)
  }
#undef LRC_STEP
  for (; s < nsteps; ++s) {
    read_half(buf(s), 1, fa1, fb1);
    mma(fa0, fb0);
    LRC_WAIT_BARRIER(8);
    next_stage(s + 4 < nsteps);
    issue(buf(s));
    read_half(buf(s + 1), 0, fa0, fb0);   // zeros behind the last stage
    mma(fa1, fb1);
  }
  LRC_WAIT_BARRIER(0);   // every load has landed and every read is done: the buffers are free

  // Epilogue: a wave's 32 rows x (32 FN) columns pass through its own part of LDS, so that a
  // lane holds eight consecutive columns of a row and the accesses to memory are whole pieces.
  // Accumulator element e of lane l is row 8 (e / 4) + 4 (l / 32) + e % 4, column l % 32.
  float* tile = reinterpret_cast<float*>(buf(wave >> 1) + (wave & 1) * (32 * FN * 32 * 4));
  constexpr int TW = FN * 32;          // tile columns
  constexpr int LPR = TW / 8;          // lanes per row
  bool bad = false;
  auto emit = [&](const f32x16 (&rows)[FN], int i) {
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int r = 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
        tile[r * TW + ((j * 32 + (lane & 31)) ^ ((r & 4) << 3))] = rows[j][e];
      }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll 1
    for (int q = 0; q < 32 * LPR / 64; ++q) {
      const int r = q * (64 / LPR) + lane / LPR, c = 8 * (lane % LPR);
      const float* src = tile + r * TW + (c ^ ((r & 4) << 3));
      const f32x4 lo = *reinterpret_cast<const f32x4*>(src), hi = *reinterpret_cast<const f32x4*>(src + 4);
      float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      const int64_t row = m0 + (wr * FM + i) * 32 + r, col = n0 + wc * TW + c;
      const int64_t left = row < M ? N - col : 0;
      const int cnt = int(left < 0 ? 0 : left > 8 ? 8 : left);
      if (tg.splits > 1) {
        const int64_t np = (N + 7) & ~int64_t(7);
        if (cnt > 0) st8(partial + (int64_t(split) * M + row) * np + col, true, 8, v);
      } else {
        finish8<TO>(ep, row, col, cnt, v, lane, bad);
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  };
  static_assert(FM == 2, "the accumulator rows are named, so that they stay in registers");
  emit(acc[0], 0);
  emit(acc[1], 1);
  if (ep.info != nullptr && bad) *ep.info = LRC_ENONFINITE;
}

template <class TO, int KA, int KB, int WM, int WN, int FM, int FN, bool SEG>
__global__ __launch_bounds__(64 * WM * WN, 1) void gemm_bf16_kernel(GemmOperand A, GemmOperand B, int64_t M, int64_t N,
                                                                    int64_t K, GemmSegments seg, TileGrid tg,
                                                                    Epilogue ep, float* __restrict__ partial,
                                                                    const int32_t* __restrict__ skip) {
  gemm_tile<TO, KA, KB, WM, WN, FM, FN, SEG>(A, B, M, N, K, seg, tg, ep, partial, skip);
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
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
      const f32x4 lo = *reinterpret_cast<const f32x4*>(p + int64_t(s) * M * np);
      const f32x4 hi = *reinterpret_cast<const f32x4*>(p + int64_t(s) * M * np + 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] += lo[e];
        v[4 + e] += hi[e];
      }
    }
  }
  bool bad = false;
  finish8<TO>(ep, row, col, cnt, v, lane, bad);
  if (ep.info != nullptr && bad) *ep.info = LRC_ENONFINITE;
}

// Tiles and splits from the sizes alone (256 compute units), so that workspace sizes are known
// without a device and equal inputs give equal bits.
struct Plan {
  bool big;
  TileGrid tg;
};
static Plan plan_gemm(int64_t M, int64_t N, int64_t K, int count) {
  Plan best{};
  double cost = 1e300;
  for (int big = 0; big < 2; ++big) {
    const int64_t edge = big ? 256 : 128;
    const int64_t nm = cdiv(M, edge), nn = cdiv(N, edge), tiles = nm * nn;
    const int64_t steps = std::max<int64_t>(1, cdiv(K, KS)), total = steps * count;
    // workgroups that run at once: one big tile or two small ones per compute unit; a stage of a
    // big tile costs 1, of a small one 0.3 (two of them share a unit), a split's partial tile
    // about 12 stages
    const double slots = big ? 256 : 512, stage = big ? 1.0 : 0.6, fixed = big ? 20.0 : 12.0;
    for (int64_t s = 1; s <= std::min<int64_t>(32, total); ++s) {
      const int64_t per = cdiv(total, s), real = cdiv(total, per);
      if (real != s) continue;
      const double rounds = std::ceil(double(cdiv(tiles, NXCD) * NXCD * s) / slots);
      const double extra = s > 1 ? double(s) * double(M) * double(N) * 8.0 / 4e6 / 1.3 * 0.5 + 8.0 : 0.0;
      const double c = rounds * (double(per) * stage + fixed) + extra;
      if (c < cost * 0.999) {
        cost = c;
        best.big = big;
        best.tg = {nm, nn, tiles, int(cdiv(tiles, NXCD)), int(s), int(per), int(steps)};
      }
    }
  }
  return best;
}

}  // namespace gemm

using namespace gemm;

size_t gemm_bf16_workspace(int64_t M, int64_t N, int64_t K) {
  size_t most = 0;
  for (int count : {1, 3, 6}) {
    const Plan p = plan_gemm(M, N, K, count);
    if (p.tg.splits > 1) most = std::max(most, size_t(p.tg.splits) * M * ((N + 7) & ~int64_t(7)) * 4);
  }
  return most;
}

template <class TO, int KA, int KB>
lrc_status gemm_bf16(hipStream_t st, const char* name, GemmOperand A, GemmOperand B, int64_t M, int64_t N, int64_t K,
                     const GemmSegments& seg, const Epilogue& ep, float* partial, const int32_t* skip, double flops,
                     double bytes) {
  const Plan p = plan_gemm(M, N, K, seg.count);
  const int64_t grid = int64_t(NXCD) * p.tg.per_xcd * p.tg.splits;
  if (grid >= (int64_t(1) << 31)) return LRC_EINVAL;
  ProfScope scope(name, st, flops, bytes);
  auto launch = [&](auto many) {
    constexpr bool SEG = decltype(many)::value;
    if (p.big)
      gemm_bf16_kernel<TO, KA, KB, 4, 2, 2, 4, SEG><<<unsigned(grid), 512, 0, st>>>(A, B, M, N, K, seg, p.tg, ep,
                                                                                   partial, skip);
    else
      gemm_bf16_kernel<TO, KA, KB, 2, 2, 2, 2, SEG><<<unsigned(grid), 256, 0, st>>>(A, B, M, N, K, seg, p.tg, ep,
                                                                                   partial, skip);
  };
  // bf16 layers have one plane; an fp32 result may come of one (dW of a bf16 layer) or more
  if (std::is_same<TO, uint16_t>::value || seg.count == 1)
    launch(std::false_type{});
  else if constexpr (!std::is_same<TO, uint16_t>::value)
    launch(std::true_type{});
  LRC_LAUNCHED();
  if (p.tg.splits == 1) return LRC_OK;
  const int64_t np = (N + 7) & ~int64_t(7), blocks = cdiv(N, CKB), threads = M * blocks * 8;
  if (cdiv(threads, 256) >= (int64_t(1) << 31)) return LRC_EINVAL;
  gemm_finish_kernel<TO><<<unsigned(cdiv(threads, 256)), 256, 0, st>>>(partial, p.tg.splits, M, N, np, blocks, ep,
                                                                          skip);
  LRC_LAUNCHED();
  return LRC_OK;
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
