// Low-rank adapters of many requests beside a shared projection:
//
//   y[j] = base[j] + s[a] xs[j] B[a] (A[a] x[j]),   a = index[j]
//
// in two kernels: the inner product t = A x in parts along k (lora_inner_kernel),
// and y from t, B and base (lora_outer_kernel). Tokens are taken 64 at a time; those
// of one adapter become the columns of the 16x16x32 matrix instructions, so an adapter's
// weights are read once for all of its tokens among the 64, whatever their order.
#include <math.h>

#include <new>

#include "nm_layer.h"

struct nm_lora_plan {
  nm_lora_problem_t p;
  int tiles;              // of 64 tokens
  int splits, loops;      // parts of k; a wave takes LORA_KW k that many times
  int slots_in, slots_out; // blocks that share out a tile's adapters
};

namespace nm {

constexpr int LORA_TILE = 64;      // tokens that are sorted into adapters together: a wave's lanes
constexpr int LORA_WAVES = 8;      // waves of the inner product's blocks
constexpr int LORA_KW = 128;       // k that a wave takes at a time
constexpr int LORA_FEATURES = 256; // outputs a block of the outer product

struct LoraArgs {
  const uint8_t* x;
  const float* x_scale;
  const uint16_t* a;
  const uint16_t* b;
  const float* scale;
  const int64_t* index;
  const uint8_t* base;
  const float* row_scale;
  const float* col_scale;
  uint16_t* y;
  float* t;               // splits x n x rank
  int64_t m, n, k, ldx, lda, ldc, ldy;
  int adapters, rank, splits, loops;
  bool in_place;          // base is y: rows without an adapter stay
};

template <int IO> struct LoraType;
template <> struct LoraType<DT_F16> { typedef half8_t v; };
template <> struct LoraType<DT_BF16> { typedef bf16x8_t v; };

template <int IO>
__device__ __forceinline__ floatx4 lora_mma(typename LoraType<IO>::v a, typename LoraType<IO>::v b, floatx4 c) {
  if constexpr (IO == DT_F16) return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  else return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// What a wave's lanes wrote to LDS its other lanes read, and write over once all have
// read: a wave's LDS operations keep their order, and the compiler keeps to it.
__device__ __forceinline__ void lora_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// The adapters of a tile's tokens, one lane a token: its adapter, -1 for none, -2 for one
// that does not exist, -3 behind the last token.
__device__ __forceinline__ int lora_named(const LoraArgs& A, int64_t tile0) {
  const int64_t at = tile0 + (threadIdx.x & 63);
  if (at >= A.n) return -3;
  const int64_t i = A.index[at];
  return i < 0 ? -1 : i < A.adapters ? (int)i : -2;
}

// The tokens of the next adapter among `left`, which loses them; named is that adapter.
__device__ __forceinline__ uint64_t lora_group(int mine, uint64_t& left, int& named) {
  named = __builtin_amdgcn_readlane(mine, __builtin_ctzll(left));
  const uint64_t group = __ballot(mine == named);
  left &= ~group;
  return group;
}

// Sixteen bytes of a row's elements from k on; those from `end` on are 0.
template <int ES>
__device__ __forceinline__ u32x4 lora_piece(const uint8_t* row, int64_t k, int64_t end) {
  constexpr int E = 16 / ES;
  if (k + E <= end) return *(const u32x4*)(row + k * ES);
  u32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < E; e++)
    if (k + e < end) {
      if constexpr (ES == 2) v[e / 2] |= (uint32_t)((const uint16_t*)row)[k + e] << (16 * (e % 2));
      else v[e / 4] |= (uint32_t)row[k + e] << (8 * (e % 4));
    }
  return v;
}

// Eight codes of 8 bits as 16-bit values, exact in both types.
template <int IO>
__device__ __forceinline__ u32x4 lora_codes(uint32_t lo, uint32_t hi) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const uint32_t v = (i < 2 ? lo : hi) >> (16 * (i % 2));
    const uint16_t a = to_bits16<IO>((float)(int8_t)v), b = to_bits16<IO>((float)(int8_t)(v >> 8));
    r[i] = (uint32_t)a | (uint32_t)b << 16;
  }
  return r;
}

// A wave's columns: the tokens of a group, in their order. Up to 16 tokens are their own
// columns, so that what does not depend on their adapters need not wait for it.
template <int NT> struct LoraColumns {
  static constexpr bool OWN = NT == 1;
  int* list;              // this wave's, in LDS
  uint64_t group;
  int count;              // columns that may be taken

  __device__ __forceinline__ void set(int* l, uint64_t g, int64_t n) {
    list = l;
    group = g;
    count = OWN ? (int)n : __popcll(g);
    if constexpr (!OWN) {
      const int lane = threadIdx.x & 63;
      lora_lds_order();
      if (g >> lane & 1)
        list[__builtin_amdgcn_mbcnt_hi((uint32_t)(g >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)g, 0))] = lane;
      lora_lds_order();
    }
  }
  // whether a column holds one of the group's tokens, and its token (any of the tile's where it does not)
  __device__ __forceinline__ bool has(int col) const { return col < count && (!OWN || (group >> col & 1)); }
  __device__ __forceinline__ int token(int col) const {
    const int c = min(col, count - 1);
    return OWN ? c : list[c];
  }
};

// t of one adapter's tokens, part blockIdx.x of k. A wave takes one tile of 16 ranks and,
// LORA_KW at a time, its share of the part; the waves of a rank tile are added in LDS in
// their order. The instruction's rows are ranks, its columns tokens.
template <int IO, bool X8, int NT>
__global__ void __launch_bounds__(64 * LORA_WAVES) lora_inner_kernel(LoraArgs A) {
  typedef typename LoraType<IO>::v v_t;
  typedef LoraColumns<NT> cols_t;
  constexpr int XS = X8 ? 2 : 4;
  __shared__ floatx4 red[LORA_WAVES][NT][64];
  __shared__ int tokens[cols_t::OWN ? 1 : LORA_WAVES][LORA_TILE];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l16 = lane & 15, q = lane >> 4;
  const int64_t tile0 = (int64_t)blockIdx.y * LORA_TILE;
  const int mine = lora_named(A, tile0);
  const int rank_tiles = (A.rank + 15) / 16, across = rank_tiles <= 1 ? 1 : rank_tiles <= 2 ? 2 : rank_tiles <= 4 ? 4 : 8;
  const int rt = wave % across, part = wave / across, parts = LORA_WAVES / across;
  const bool works = 16 * rt < A.rank;
  auto first_k = [&](int i) { return (((int64_t)blockIdx.x * A.loops + i) * parts + part) * LORA_KW; };

  u32x4 xv[NT][XS];
  auto load_x = [&](const uint8_t* const (&xr)[NT], int64_t k0, int count) {
#pragma unroll
    for (int j = 0; j < NT; j++)
      if (16 * j < count) {
#pragma unroll
        for (int s = 0; s < XS; s++) xv[j][s] = lora_piece<X8 ? 1 : 2>(xr[j], k0 + (X8 ? 64 * s + 16 * q : 32 * s + 8 * q), A.k);
      }
  };
  const uint8_t* xr[NT];
  if constexpr (cols_t::OWN) {
    xr[0] = A.x + min(l16, (int)A.n - 1) * A.ldx * (X8 ? 1 : 2);
    if (works && first_k(0) < A.k) load_x(xr, first_k(0), 16);
  }
  uint64_t left = __ballot(mine >= 0);
  for (int d = 0, next = blockIdx.z; left; d++) {
    int adapter;
    const uint64_t group = lora_group(mine, left, adapter);
    if (d != next) continue;
    next += gridDim.z;
    cols_t cols;
    cols.set(tokens[cols_t::OWN ? 0 : wave], group, A.n);
    const uint8_t* const ar = (const uint8_t*)(A.a + ((int64_t)adapter * A.rank + min(16 * rt + l16, A.rank - 1)) * A.lda);
    if constexpr (!cols_t::OWN) {
#pragma unroll
      for (int j = 0; j < NT; j++) xr[j] = A.x + (tile0 + cols.token(16 * j + l16)) * A.ldx * (X8 ? 1 : 2);
    }
    floatx4 acc[NT];
#pragma unroll
    for (int j = 0; j < NT; j++) acc[j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    if (works) {
      for (int i = 0; i < A.loops; i++) {
        const int64_t k0 = first_k(i);
        if (k0 >= A.k) break;
        u32x4 av[4];
#pragma unroll
        for (int s = 0; s < 4; s++) av[s] = lora_piece<2>(ar, k0 + (X8 ? 64 * (s / 2) + 16 * q + 8 * (s % 2) : 32 * s + 8 * q), A.k);
        if (!cols_t::OWN || i > 0 || d > (int)blockIdx.z) load_x(xr, k0, cols.count);
#pragma unroll
        for (int j = 0; j < NT; j++)
          if (16 * j < cols.count) {
#pragma unroll
            for (int s = 0; s < 4; s++) {
              u32x4 b;
              if constexpr (X8) b = lora_codes<IO>(xv[j][s / 2][2 * (s % 2)], xv[j][s / 2][2 * (s % 2) + 1]);
              else b = xv[j][s];
              acc[j] = lora_mma<IO>(__builtin_bit_cast(v_t, av[s]), __builtin_bit_cast(v_t, b), acc[j]);
            }
          }
      }
    }
#pragma unroll
    for (int j = 0; j < NT; j++) red[wave][j][lane] = acc[j];
    __syncthreads();
    for (int u = wave; u < across * NT; u += LORA_WAVES) {
      const int r = u % across, j = u / across, col = 16 * j + l16, rank = 16 * r + 4 * q;
      floatx4 v = red[r][j][lane];
      for (int w = 1; w < parts; w++) v += red[r + w * across][j][lane];
      if (cols.has(col) && rank < A.rank)
        *(floatx4*)(A.t + ((int64_t)blockIdx.x * A.n + tile0 + cols.token(col)) * A.rank + rank) = v;
    }
    __syncthreads();
  }
}

// y of one adapter's tokens (or of those without one), LORA_FEATURES outputs a block, 64 a
// wave. The instruction's rows are outputs, its columns tokens, its k the ranks twice: t
// goes in as two 16-bit parts, the second what the first left over, so that 16 to 22 bits of
// it meet B (f16: against the token's largest, brought to 1 by a power of two, which f16
// would not hold otherwise). Row 4 q + r of instruction f is output 32 (f / 2) + 8 q + 4 (f % 2)
// + r: a lane ends with two pieces of eight outputs in a row, 16 bytes each.
// SETS: chunks of eight ranks a lane takes; 0: up to 16 ranks, both parts in one instruction.
template <int IO, bool ACC, int SETS, int NT>
__global__ void __launch_bounds__(256) lora_outer_kernel(LoraArgs A) {
  typedef typename LoraType<IO>::v v_t;
  typedef LoraColumns<NT> cols_t;
  constexpr int NS = SETS == 0 ? 1 : SETS;
  constexpr int PER = (SETS == 0 ? 16 : 32 * SETS) / 4;   // threads that bring a token's t
  constexpr int RS = 4 * PER + 4;                         // floats of it in LDS: 16 tokens on distinct banks
  constexpr int BQ = ACC ? 4 : 2;                         // pieces of 16 bytes a lane's outputs take of the base
  __shared__ float ts[16 * NT][RS];
  __shared__ float most[16 * NT];
  __shared__ int tokens[cols_t::OWN ? 1 : 4][LORA_TILE];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l16 = lane & 15, q = lane >> 4;
  const int64_t tile0 = (int64_t)blockIdx.y * LORA_TILE;
  const int64_t f0 = (int64_t)blockIdx.x * LORA_FEATURES + 64 * wave;
  const bool all = f0 + 64 <= A.m;                        // the wave's outputs are whole
  const int mine = lora_named(A, tile0);
  const int chunks = A.rank / 8;

  // what y adds to, as it lies in memory: outputs 32 h + 8 q .. + 7, h = 0, 1
  u32x4 base[NT][BQ];
  floatx4 cs[ACC ? 4 : 1];
  float xs[NT], rs[NT];
  int64_t token[NT];
  auto load_base = [&](int j) {
    xs[j] = A.x_scale ? A.x_scale[token[j]] : 1.0f;
    if constexpr (ACC) rs[j] = A.row_scale[token[j]];
    if (!all) return;
    const uint8_t* p = A.base + (token[j] * A.ldc + f0 + 8 * q) * (ACC ? 4 : 2);
#pragma unroll
    for (int i = 0; i < BQ; i++) base[j][i] = *(const u32x4*)(p + (ACC ? 128 * (i / 2) + 16 * (i % 2) : 64 * i));
  };
  // one of the lane's 16 outputs of column j
  auto value = [&](int j, int h, int e) -> float {
    if (all) {
      if constexpr (ACC) {
        const uint32_t c = base[j][2 * h + e / 4][e % 4];
        return (float)(int32_t)c * rs[j] * cs[2 * h + e / 4][e % 4];
      } else {
        return from_bits16<IO>((uint16_t)(base[j][h][e / 2] >> (16 * (e % 2))));
      }
    }
    const int64_t out = f0 + 32 * h + 8 * q + e;
    if (out >= A.m) return 0.0f;
    if constexpr (ACC) return (float)((const int32_t*)A.base)[token[j] * A.ldc + out] * rs[j] * A.col_scale[out];
    else return from_bits16<IO>(((const uint16_t*)A.base)[token[j] * A.ldc + out]);
  };
  if constexpr (ACC) {
    if (all) {
#pragma unroll
      for (int i = 0; i < 4; i++) cs[i] = *(const floatx4*)(A.col_scale + f0 + 8 * q + 32 * (i / 2) + 4 * (i % 2));
    }
  }
  if constexpr (cols_t::OWN) {
    token[0] = min(l16, (int)A.n - 1);
    load_base(0);
  }

  uint64_t left = __ballot(mine >= -2);
  for (int d = 0, next = blockIdx.z; left; d++) {
    int adapter;
    const uint64_t group = lora_group(mine, left, adapter);
    if (d != next) continue;
    next += gridDim.z;
    if (adapter == -1 && A.in_place) continue;
    cols_t cols;
    cols.set(tokens[cols_t::OWN ? 0 : wave], group, A.n);
    // B's pieces: chunk 4 s + q (up to 16 ranks: q % 2) of the lane's output row
    v_t bv[NS][4];
#pragma unroll
    for (int s = 0; s < NS; s++) {
      const int chunk = SETS == 0 ? q % 2 : 4 * s + q;
#pragma unroll
      for (int f = 0; f < 4; f++) {
        const int64_t out = f0 + 32 * (f / 2) + 8 * (l16 / 4) + 4 * (f % 2) + l16 % 4;
        u32x4 v = {0, 0, 0, 0};
        if (adapter >= 0 && chunk < chunks)
          v = *(const u32x4*)(A.b + ((int64_t)adapter * A.m + min(out, A.m - 1)) * A.rank + 8 * chunk);
        bv[s][f] = __builtin_bit_cast(v_t, v);
      }
    }
    const float sa = adapter >= 0 ? A.scale[adapter] : adapter == -1 ? 0.0f : __builtin_nanf("");
    if constexpr (!cols_t::OWN) {
#pragma unroll
      for (int j = 0; j < NT; j++)
        if (16 * j < cols.count) {
          token[j] = tile0 + cols.token(16 * j + l16);
          load_base(j);
        }
    }
    if (adapter >= 0) {
      // t: the parts of k in their order
#pragma unroll 1
      for (int e = threadIdx.x; e < 16 * NT * PER; e += 256) {
        const int j = e / PER, r = e % PER * 4;
        floatx4 v = {0.0f, 0.0f, 0.0f, 0.0f};
        if (cols.has(j) && r < A.rank) {
          const float* p = A.t + (tile0 + cols.token(j)) * A.rank + r;
          for (int s = 0; s < A.splits; s += 4) {
            floatx4 w[4];
#pragma unroll
            for (int i = 0; i < 4; i++) w[i] = *(const floatx4*)(p + (int64_t)min(s + i, A.splits - 1) * A.n * A.rank);
#pragma unroll
            for (int i = 0; i < 4; i++)
              if (s + i < A.splits) v += w[i];
          }
        }
        *(floatx4*)&ts[j][r] = v;
        if constexpr (IO == DT_F16) {
          float top = 0.0f;                       // a NaN is not among them; it stays in t
#pragma unroll
          for (int i = 0; i < 4; i++) top = fmaxf(top, __builtin_fabsf(v[i]));
#pragma unroll
          for (int off = 1; off < PER; off *= 2) top = fmaxf(top, __shfl_xor(top, off));
          if (r == 0) most[j] = top;
        }
      }
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < NT; j++) {
      if (16 * j >= cols.count) break;
      float v[2][8];
#pragma unroll
      for (int h = 0; h < 2; h++)
#pragma unroll
        for (int e = 0; e < 8; e++) v[h][e] = value(j, h, e);
      if (adapter >= 0) {
        // t in two parts, and the factor that they leave
        float up = 1.0f, fac = sa * xs[j];
        if constexpr (IO == DT_F16) {
          // the largest below 1: times 2^-e with e its exponent's distance; not for 0, infinities and NaN
          const int e = (int)(__builtin_bit_cast(uint32_t, most[16 * j + l16]) >> 23) - 126;
          if (e > -126 && e < 129) {
            up = __builtin_ldexpf(1.0f, -min(e, 120));        // 2^-127 is none; 2^8 f16 still holds
            fac *= __builtin_ldexpf(1.0f, min(e, 120));
          }
        }
        floatx4 acc[4];
#pragma unroll
        for (int f = 0; f < 4; f++) acc[f] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int s = 0; s < NS; s++) {
          const float* p = &ts[16 * j + l16][8 * (SETS == 0 ? q % 2 : 4 * s + q)];
          uint16_t hi[8], lo[8];
#pragma unroll
          for (int e = 0; e < 8; e++) {
            const float w = p[e] * up;
            hi[e] = to_bits16<IO>(w);
            lo[e] = to_bits16<IO>(w - from_bits16<IO>(hi[e]));
          }
          u32x4 hv, lv;
#pragma unroll
          for (int i = 0; i < 4; i++) {
            hv[i] = (uint32_t)hi[2 * i] | (uint32_t)hi[2 * i + 1] << 16;
            lv[i] = (uint32_t)lo[2 * i] | (uint32_t)lo[2 * i + 1] << 16;
          }
          if constexpr (SETS == 0) {
#pragma unroll
            for (int i = 0; i < 4; i++) hv[i] = q < 2 ? hv[i] : lv[i];
          }
#pragma unroll
          for (int f = 0; f < 4; f++) {
            acc[f] = lora_mma<IO>(bv[s][f], __builtin_bit_cast(v_t, hv), acc[f]);
            if constexpr (SETS > 0) acc[f] = lora_mma<IO>(bv[s][f], __builtin_bit_cast(v_t, lv), acc[f]);
          }
        }
#pragma unroll
        for (int f = 0; f < 4; f++)
#pragma unroll
          for (int e = 0; e < 4; e++) v[f / 2][4 * (f % 2) + e] = __builtin_fmaf(fac, acc[f][e], v[f / 2][4 * (f % 2) + e]);
      } else if (adapter == -2) {
#pragma unroll
        for (int e = 0; e < 8; e++) v[0][e] = v[1][e] = sa;
      }
      if (!cols.has(16 * j + l16)) continue;
      uint16_t* const yr = A.y + token[j] * A.ldy;
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const int64_t out = f0 + 32 * h + 8 * q;
        uint16_t o[8];
#pragma unroll
        for (int e = 0; e < 8; e++) o[e] = to_bits16<IO>(v[h][e]);
        if (all) {
          u32x4 w;
#pragma unroll
          for (int i = 0; i < 4; i++) w[i] = (uint32_t)o[2 * i] | (uint32_t)o[2 * i + 1] << 16;
          *(u32x4*)(yr + out) = w;
        } else {
#pragma unroll
          for (int e = 0; e < 8; e++)
            if (out + e < A.m) yr[out + e] = o[e];
        }
      }
    }
    __syncthreads();                              // t is read: the next group's may come
  }
}

template <int IO, bool X8>
hipError_t lora_inner(const LoraArgs& a, const nm_lora_plan& pl, hipStream_t s) {
  const dim3 grid((unsigned)a.splits, (unsigned)pl.tiles, (unsigned)pl.slots_in);
  if (a.n <= 16) hipLaunchKernelGGL((lora_inner_kernel<IO, X8, 1>), grid, dim3(64 * LORA_WAVES), 0, s, a);
  else hipLaunchKernelGGL((lora_inner_kernel<IO, X8, 4>), grid, dim3(64 * LORA_WAVES), 0, s, a);
  return hipGetLastError();
}

template <int IO, bool ACC, int SETS>
hipError_t lora_outer(const LoraArgs& a, const nm_lora_plan& pl, hipStream_t s) {
  const dim3 grid((unsigned)((a.m + LORA_FEATURES - 1) / LORA_FEATURES), (unsigned)pl.tiles, (unsigned)pl.slots_out);
  if (a.n <= 16) hipLaunchKernelGGL((lora_outer_kernel<IO, ACC, SETS, 1>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((lora_outer_kernel<IO, ACC, SETS, 4>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

template <int IO>
hipError_t lora_go(const LoraArgs& a, const nm_lora_plan& pl, hipStream_t s) {
  const bool acc = pl.p.type_base == NM_I32;
  hipError_t e = pl.p.type_x == NM_I8 ? lora_inner<IO, true>(a, pl, s) : lora_inner<IO, false>(a, pl, s);
  if (e != hipSuccess) return e;
  const int r = a.rank;
  if (r <= 16) return acc ? lora_outer<IO, true, 0>(a, pl, s) : lora_outer<IO, false, 0>(a, pl, s);
  if (r <= 32) return acc ? lora_outer<IO, true, 1>(a, pl, s) : lora_outer<IO, false, 1>(a, pl, s);
  if (r <= 64) return acc ? lora_outer<IO, true, 2>(a, pl, s) : lora_outer<IO, false, 2>(a, pl, s);
  return acc ? lora_outer<IO, true, 4>(a, pl, s) : lora_outer<IO, false, 4>(a, pl, s);
}

static bool lora_empty(const nm_lora_problem_t& p) { return p.n == 0 || p.m == 0; }

}  // namespace nm

using namespace nm;

extern "C" {

nm_status_t nm_lora_plan_init(nm_lora_plan_t* plan, const nm_lora_problem_t* p) {
  if (!plan) return layer_fail(NM_ERR_INVALID_ARG, "plan is NULL");
  *plan = nullptr;
  if (!p) return layer_fail(NM_ERR_INVALID_ARG, "problem is NULL");
  if (p->type_y != NM_F16 && p->type_y != NM_BF16) return layer_fail(NM_ERR_INVALID_ARG, "type_y must be NM_F16 or NM_BF16");
  if (p->type_x != p->type_y && p->type_x != NM_I8) return layer_fail(NM_ERR_INVALID_ARG, "type_x must be type_y or NM_I8");
  if (p->type_base != p->type_y && p->type_base != NM_I32)
    return layer_fail(NM_ERR_INVALID_ARG, "type_base must be type_y or NM_I32");
  if (p->m < 0 || p->n < 0 || p->k < 1) return layer_fail(NM_ERR_SHAPE, "m and n must be >= 0, k >= 1");
  if (p->m > ((int64_t)1 << 24) || p->n > ((int64_t)1 << 20) || p->k > ((int64_t)1 << 20))
    return layer_fail(NM_ERR_SHAPE, "m must be <= 2^24, n and k <= 2^20");
  if (p->rank < 8 || p->rank > 128 || p->rank % 8) return layer_fail(NM_ERR_SHAPE, "rank must be a multiple of 8 from 8 to 128");
  if (p->adapters < 1 || p->adapters > (1 << 20)) return layer_fail(NM_ERR_SHAPE, "adapters must be 1 to 2^20");
  nm_status_t st = layer_rows(p->n, p->k, p->ldx, p->type_x == NM_I8 ? 1 : 2);
  if (st == NM_OK) st = layer_rows((int64_t)p->adapters * p->rank, p->k, p->lda, 2);
  if (st == NM_OK) st = layer_rows(p->n, p->m, p->ldc, p->type_base == NM_I32 ? 4 : 2);
  if (st == NM_OK) st = layer_rows(p->n, p->m, p->ldy, 2);
  if (st != NM_OK) return st;
  nm_lora_plan* pl = new (std::nothrow) nm_lora_plan();
  if (!pl) return layer_fail(NM_ERR_INVALID_ARG, "out of host memory");
  pl->p = *p;
  pl->tiles = (int)((p->n + LORA_TILE - 1) / LORA_TILE);
  const int64_t tile = p->n < LORA_TILE ? p->n : LORA_TILE, tiles = pl->tiles ? pl->tiles : 1;
  // a block for each adapter that a tile can name, while that leaves the GPU room
  auto slots = [&](int64_t most, int64_t blocks) {
    int64_t want = 2048 / blocks;
    if (want > most) want = most;
    return (int)(want < 1 ? 1 : want);
  };
  const int rank_tiles = (p->rank + 15) / 16, across = rank_tiles <= 1 ? 1 : rank_tiles <= 2 ? 2 : rank_tiles <= 4 ? 4 : 8;
  const int64_t step = (int64_t)LORA_KW * (LORA_WAVES / across), steps = (p->k + step - 1) / step;
  const int64_t named = tile < p->adapters ? tile : p->adapters;
  int64_t splits = 1024 / tiles;
  if (splits > 16) splits = 16;
  if (splits > steps) splits = steps;
  if (splits < 1) splits = 1;
  pl->loops = (int)((steps + splits - 1) / splits);
  pl->splits = (int)((steps + pl->loops - 1) / pl->loops);
  pl->slots_in = slots(named, tiles * pl->splits);
  pl->slots_out = slots(tile < p->adapters + 2 ? tile : p->adapters + 2, tiles * ((p->m + LORA_FEATURES - 1) / LORA_FEATURES + 1));
  *plan = pl;
  return layer_fail(NM_OK, "");
}

nm_status_t nm_lora_plan_destroy(nm_lora_plan_t plan) {
  delete plan;
  return NM_OK;
}

nm_status_t nm_lora_workspace_size(nm_lora_plan_t plan, size_t* bytes) {
  if (!plan || !bytes) return layer_fail(NM_ERR_INVALID_ARG, "plan / bytes is NULL");
  const nm_lora_problem_t& p = plan->p;
  *bytes = lora_empty(p) ? 0 : (size_t)plan->splits * p.n * p.rank * sizeof(float);
  return NM_OK;
}

nm_status_t nm_lora(nm_lora_plan_t plan, const void* dX, const float* d_x_scale, const void* dA, const void* dB,
                    const float* d_scale, const int64_t* d_index, const void* d_base, const float* d_row_scale,
                    const float* d_col_scale, void* dY, void* d_workspace, void* stream) {
  if (!plan) return layer_fail(NM_ERR_INVALID_ARG, "plan is NULL");
  const nm_lora_problem_t& p = plan->p;
  if (!layer_aligned(dX, 16) || !layer_aligned(dA, 16) || !layer_aligned(dB, 16) || !layer_aligned(d_base, 16) ||
      !layer_aligned(d_col_scale, 16) || !layer_aligned(dY, 16) || !layer_aligned(d_workspace, 16) ||
      !layer_aligned(d_index, 8) || !layer_aligned(d_x_scale, 4) || !layer_aligned(d_scale, 4) || !layer_aligned(d_row_scale, 4))
    return layer_fail(NM_ERR_ALIGN, "matrices, d_col_scale and d_workspace must be 16-byte aligned, the others as their elements");
  if (lora_empty(p)) return NM_OK;
  if (!dX || !dA || !dB || !d_scale || !d_index || !d_base || !dY)
    return layer_fail(NM_ERR_INVALID_ARG, "dX / dA / dB / d_scale / d_index / d_base / dY is NULL");
  if (!d_workspace) return layer_fail(NM_ERR_INVALID_ARG, "d_workspace is NULL");
  if ((d_x_scale != nullptr) != (p.type_x == NM_I8))
    return layer_fail(NM_ERR_INVALID_ARG, "d_x_scale must be given exactly where x is int8");
  const bool acc = p.type_base == NM_I32;
  if ((d_row_scale != nullptr) != acc || (d_col_scale != nullptr) != acc)
    return layer_fail(NM_ERR_INVALID_ARG, "d_row_scale and d_col_scale must be given exactly where the base is int32");
  LoraArgs a = {};
  a.x = (const uint8_t*)dX;
  a.x_scale = d_x_scale;
  a.a = (const uint16_t*)dA;
  a.b = (const uint16_t*)dB;
  a.scale = d_scale;
  a.index = d_index;
  a.base = (const uint8_t*)d_base;
  a.row_scale = d_row_scale;
  a.col_scale = d_col_scale;
  a.y = (uint16_t*)dY;
  a.t = (float*)d_workspace;
  a.m = p.m;
  a.n = p.n;
  a.k = p.k;
  a.ldx = p.ldx;
  a.lda = p.lda;
  a.ldc = p.ldc;
  a.ldy = p.ldy;
  a.adapters = p.adapters;
  a.rank = p.rank;
  a.splits = plan->splits;
  a.loops = plan->loops;
  a.in_place = !acc && d_base == dY && p.ldc == p.ldy;
  hipStream_t s = (hipStream_t)stream;
  return layer_hip(p.type_y == NM_F16 ? lora_go<DT_F16>(a, *plan, s) : lora_go<DT_BF16>(a, *plan, s));
}

}  // extern "C"
