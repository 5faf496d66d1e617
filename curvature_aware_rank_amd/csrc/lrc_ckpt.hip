// Activation checkpoints in 8 bits: codes and block exponents of token rows, and back.
//
// The activations that the backward pass of a calibration (or healing) step needs, kept as
// int8 codes with one power-of-two step per 64 channels of a token.
#include "lrc_train.h"

#include <algorithm>

namespace lrc {
namespace {

constexpr int CT = 256;

// One lane per eight channels, eight lanes per block: a wave covers eight blocks, taken in
// order over (token, block).  Bound by memory (32768 x 11008 bf16, 1.09 GB
// each way: pack 200 us, unpack 225; 5.4 and 4.8 TB/s).  A launch holds less than 2^32 threads, so past
// GRID_MAX workgroups (2^29 blocks, 2^35 channels in whole blocks) they take blocks in turn.
constexpr int64_t GRID_MAX = (int64_t(1) << 24) - 1;

template <class T>
__global__ __launch_bounds__(CT) void pack_kernel(const T* __restrict__ x, int64_t ldx, int64_t n, int d, int64_t nb,
                                                  int8_t* __restrict__ codes, int8_t* __restrict__ exps,
                                                  int32_t* __restrict__ info) {
  const int lane = threadIdx.x & 63;
  bool bad = false;
  for (int64_t g = (int64_t(blockIdx.x) * CT + threadIdx.x) >> 3; g < n * nb; g += int64_t(gridDim.x) * (CT / 8)) {
    const int64_t t = g / nb;
    const int c = int(g % nb) * CKB + 8 * (lane & 7);
    const int cnt = min(8, d - c);
    float v[8];
    ld8(x + t * ldx + c, cnt, v);
    st8_codes(codes + t * d + c, exps + g, cnt, v, lane, bad);
  }
  if (info != nullptr && bad) *info = LRC_ENONFINITE;
}

template <class T>
__global__ __launch_bounds__(CT) void unpack_kernel(const int8_t* __restrict__ codes, const int8_t* __restrict__ exps,
                                                    int64_t n, int d, int64_t nb, T* __restrict__ x, int64_t ldx) {
  for (int64_t g = (int64_t(blockIdx.x) * CT + threadIdx.x) >> 3; g < n * nb; g += int64_t(gridDim.x) * (CT / 8)) {
    const int64_t t = g / nb;
    const int c = int(g % nb) * CKB + 8 * (threadIdx.x & 7);
    const int cnt = min(8, d - c);
    if (cnt <= 0) continue;
    float v[8];
    ld8_codes(codes + t * d + c, cnt, pow2f(exps[g]), v);
    st8(x + t * ldx + c, cnt, v);
  }
}

bool sizes_ok(int64_t n, int64_t d, int64_t ld) {
  return n >= 0 && n < (int64_t(1) << 31) && d >= 1 && d <= (int64_t(1) << 24) && ld >= d;
}

}  // namespace
}  // namespace lrc

using namespace lrc;

extern "C" lrc_status lrc_pack_activations(const void* x, lrc_dtype dt, int64_t n_tokens, int64_t d, int64_t ldx,
                                           int8_t* codes, int8_t* exps, int32_t* info, void* stream) {
  if (dt != LRC_F32 && dt != LRC_BF16) return LRC_EDTYPE;
  if (!sizes_ok(n_tokens, d, ldx)) return LRC_EINVAL;
  if (n_tokens == 0) return LRC_OK;
  if (x == nullptr || codes == nullptr || exps == nullptr) return LRC_EINVAL;
  const int64_t nb = cdiv(d, CKB), grid = std::min(cdiv(n_tokens * nb * 8, CT), GRID_MAX);
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int size = dt == LRC_BF16 ? 2 : 4;
  ProfScope scope("pack_kernel", st, 0.0, double(n_tokens) * (double(d) * (size + 1) + double(nb)));
  if (dt == LRC_BF16)
    pack_kernel<<<unsigned(grid), CT, 0, st>>>(static_cast<const uint16_t*>(x), ldx, n_tokens, int(d), nb, codes, exps,
                                               info);
  else
    pack_kernel<<<unsigned(grid), CT, 0, st>>>(static_cast<const float*>(x), ldx, n_tokens, int(d), nb, codes, exps, info);
  LRC_LAUNCHED();
  return LRC_OK;
}

extern "C" lrc_status lrc_unpack_activations(const int8_t* codes, const int8_t* exps, int64_t n_tokens, int64_t d,
                                             void* x, lrc_dtype dt, int64_t ldx, void* stream) {
  if (dt != LRC_F32 && dt != LRC_BF16) return LRC_EDTYPE;
  if (!sizes_ok(n_tokens, d, ldx)) return LRC_EINVAL;
  if (n_tokens == 0) return LRC_OK;
  if (x == nullptr || codes == nullptr || exps == nullptr) return LRC_EINVAL;
  const int64_t nb = cdiv(d, CKB), grid = std::min(cdiv(n_tokens * nb * 8, CT), GRID_MAX);
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int size = dt == LRC_BF16 ? 2 : 4;
  ProfScope scope("unpack_kernel", st, 0.0, double(n_tokens) * (double(d) * (size + 1) + double(nb)));
  if (dt == LRC_BF16)
    unpack_kernel<<<unsigned(grid), CT, 0, st>>>(codes, exps, n_tokens, int(d), nb, static_cast<uint16_t*>(x), ldx);
  else
    unpack_kernel<<<unsigned(grid), CT, 0, st>>>(codes, exps, n_tokens, int(d), nb, static_cast<float*>(x), ldx);
  LRC_LAUNCHED();
  return LRC_OK;
}
