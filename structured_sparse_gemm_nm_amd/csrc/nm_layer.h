// Shared by the units of the operators around the product: their refusals, and
// what their kernels have in common.
#pragma once
#include "nm_device.h"
#include "nm_internal.h"

namespace nm {

// A status with its message; no exception leaves it.
inline nm_status_t layer_fail(nm_status_t st, const char* msg) noexcept {
  try {
    set_error(msg);
  } catch (...) {   // no memory for the message: the status still tells
  }
  return st;
}

inline nm_status_t layer_hip(hipError_t e) noexcept {
  return e == hipSuccess ? NM_OK : layer_fail(NM_ERR_HIP, hipGetErrorString(e));
}

inline bool layer_aligned(const void* p, unsigned to) { return ((uintptr_t)p & (to - 1)) == 0; }

// Whether a matrix of rows x len elements of es bytes, ld elements apart, keeps the rules.
inline nm_status_t layer_rows(int64_t rows, int64_t len, int64_t ld, int es) {
  const int64_t limit = (int64_t)1 << 46;
  if (ld < (len > 0 ? len : 1)) return layer_fail(NM_ERR_SHAPE, "leading dimension smaller than the row length");
  if (ld > limit || (double)rows * (double)ld > (double)limit) return layer_fail(NM_ERR_SHAPE, "matrix too large");
  if (len * es >= 16 && ld * es % 16 != 0)
    return layer_fail(NM_ERR_ALIGN, "rows of 16 bytes or more must start on 16-byte boundaries (ld * elem size % 16)");
  return NM_OK;
}

// v of another lane of the 16 that lane l shares a row of the wave with
template <int CTRL> __device__ __forceinline__ float lane_dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}

// f over the wave, the same in every lane: within 16 lanes without LDS, the four rows' results as scalars. Where a
// single row's time is a sum of latencies, exchanges through LDS (130 clocks each) are most of it.
template <typename F> __device__ __forceinline__ float wave_all(float v, F f) {
  v = f(v, lane_dpp<0xB1>(v));
  v = f(v, lane_dpp<0x4E>(v));
  v = f(v, lane_dpp<0x141>(v));
  v = f(v, lane_dpp<0x140>(v));
  const int bits = __builtin_bit_cast(int, v);
  float r[4];
#pragma unroll
  for (int i = 0; i < 4; i++) r[i] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(bits, 16 * i));
  return f(f(r[0], r[1]), f(r[2], r[3]));
}
__device__ __forceinline__ float wave_max(float v) { return wave_all(v, [](float a, float b) { return fmaxf(a, b); }); }
__device__ __forceinline__ float wave_min(float v) { return wave_all(v, [](float a, float b) { return fminf(a, b); }); }
__device__ __forceinline__ float wave_sum(float v) { return wave_all(v, [](float a, float b) { return a + b; }); }

// Sum over G neighbouring lanes (8, 16, 32 or 64), in each of them: neighbours,
// pairs, the halves of 8 and of 16 mirrored, then across rows of 16.
template <int G> __device__ __forceinline__ float lane_sum(float v) {
  v += lane_dpp<0xB1>(v);
  v += lane_dpp<0x4E>(v);
  v += lane_dpp<0x141>(v);
  if constexpr (G >= 16) v += lane_dpp<0x140>(v);
  if constexpr (G >= 32) v += __shfl_xor(v, 16);
  if constexpr (G >= 64) v += __shfl_xor(v, 32);
  return v;
}

}  // namespace nm
