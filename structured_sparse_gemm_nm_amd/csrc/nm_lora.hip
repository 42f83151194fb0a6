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
  bool sorted;            // the tokens are sorted by their adapters first
};

namespace nm {

constexpr int LORA_TILE = 64;      // tokens that are sorted into adapters together: a wave's lanes
constexpr int LORA_WAVES = 8;      // waves a block
constexpr int LORA_KW = 128;       // k that a wave takes at a time
constexpr int LORA_SORT_THREADS = 1024;
constexpr int LORA_SORT_BINS = 4096;
constexpr int LORA_FEATURES = 256; // outputs a block of the outer product, or twice as many
// Outputs of all groups that are more than the CUs take at a time: a wave then takes twice as many. 16 tokens to 22016
// features 10.5 us and 11.0 without; one token to 4096 or 22016 7.1 us and 7.5 with it.
constexpr int64_t LORA_MANY = 1 << 17;

typedef int intx2 __attribute__((ext_vector_type(2)));

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
  const intx2* order;     // (name, token) sorted by names, or NULL: the tokens as they come
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

// An index as the kernels take it: its adapter, -1 for none, -2 for one that does not exist.
__device__ __forceinline__ int lora_name(const LoraArgs& A, int64_t i) { return i < 0 ? -1 : i < A.adapters ? (int)i : -2; }

// A tile's tokens, one a lane, and their names (-3 behind the last token): in their own order, or in that of
// lora_sort_kernel.
__device__ __forceinline__ int lora_named(const LoraArgs& A, int64_t tile0, int& token) {
  const int64_t at = tile0 + (threadIdx.x & 63);
  token = (int)at;
  if (at >= A.n) return -3;
  if (A.order) {
    const intx2 o = A.order[at];
    token = o[1];
    return o[0];
  }
  return lora_name(A, A.index[at]);
}

// Tokens by their adapters, so that a tile holds few of them: a count of each bin of names, the
// counts' sums, and the tokens put behind them. Adapters 4096 apart share a bin, and a tile holds
// whatever it gets: the order is for speed alone. One block; the order within a bin is that in
// which the atomics are served, and no token's result depends on it: each is a column of its own.
// It takes 4 us with its launch, at 256 tokens as at 4096 (latency: the index, places, sums, the
// order), which a prompt in runs pays for nothing: 4096 tokens, 64 adapters of rank 16, k = m =
// 4096, bf16, in runs 24.5 us without it and 27.9 with it, scattered 174 and 34.8. So it runs from
// where scattered tokens gain about that: 256 tokens over 64 adapters 26.4 us without and 22.9
// with, over 8 12.0 and 16.3; 1024 over 8 28.4 and 23.2, over 4 22.3 and 23.4; 4096 over 4 33.7
// and 29.8, over 2 27.6 and 30.8; 128 over 64 15.1 and 18.5. It stays one block: k = m = 1024, 64
// adapters, without it and with it, 65536 tokens scattered 690 and 159, in runs 89 and 127; 262144
// tokens 2620 and 577, in runs 322 and 464.
__global__ void __launch_bounds__(LORA_SORT_THREADS) lora_sort_kernel(LoraArgs A, intx2* order) {
  constexpr int T = LORA_SORT_THREADS, B = LORA_SORT_BINS / T, U = 4;
  __shared__ int bins[LORA_SORT_BINS];
  __shared__ int taken;
  const int lane = threadIdx.x & 63;
  int name[U], nth[U];
  auto load = [&](int64_t b) {
    int64_t v[U];
#pragma unroll
    for (int u = 0; u < U; u++) v[u] = A.index[min(b + u * T + threadIdx.x, A.n - 1)];
#pragma unroll
    for (int u = 0; u < U; u++) name[u] = b + u * T + threadIdx.x < A.n ? lora_name(A, v[u]) + 2 : -1;
  };
  auto bin = [](int of) { return of & (LORA_SORT_BINS - 1); };
  // Each token's place in its bin. A wave whose tokens are of one name takes its places at
  // once, by lane 0 (behind the last token there are only last lanes); other lanes add 0.
  auto place = [&] {
#pragma unroll
    for (int u = 0; u < U; u++) {
      const uint64_t here = __ballot(name[u] >= 0);
      const int lead = __builtin_amdgcn_readfirstlane(name[u]);
      const bool one = here && __ballot(name[u] == lead) == here;
      const int add = one ? (lane == 0 ? __popcll(here) : 0) : name[u] >= 0;
      nth[u] = atomicAdd(&bins[add ? bin(name[u]) : lane], add);
      if (one) nth[u] = __builtin_amdgcn_readfirstlane(nth[u]) + lane;
    }
  };
  load(0);
#pragma unroll
  for (int i = 0; i < B; i++) bins[threadIdx.x + i * T] = 0;
  if (threadIdx.x == 0) taken = 0;
  __syncthreads();
  place();
  for (int64_t b = U * T; b < A.n; b += U * T) {
    load(b);
    place();
  }
  __syncthreads();
  // the bins' first places, in whatever order the threads come
#pragma unroll
  for (int i = 0; i < B; i++) {
    const int tokens = bins[threadIdx.x + i * T];
    if (tokens) bins[threadIdx.x + i * T] = atomicAdd(&taken, tokens);
  }
  __syncthreads();
  if (A.n <= U * T) {
#pragma unroll
    for (int u = 0; u < U; u++)
      if (name[u] >= 0) order[bins[bin(name[u])] + nth[u]] = intx2{name[u] - 2, (int)(u * T + threadIdx.x)};
    return;
  }
  for (int64_t b = 0; b < A.n; b += U * T) {
    load(b);
    place();
#pragma unroll
    for (int u = 0; u < U; u++)
      if (name[u] >= 0) order[nth[u]] = intx2{name[u] - 2, (int)(b + u * T + threadIdx.x)};
  }
}

// The groups of a tile (the tokens of one adapter, or of none) that fall to one of gridDim.z
// blocks: with a block for each token, the group that the token leads; with fewer, every
// gridDim.z-th group in the order of their first tokens.
struct LoraGroups {
  int mine, d;
  uint64_t left;
  bool each;

  // tokens: those to be taken
  __device__ __forceinline__ void init(int m, uint64_t tokens, int64_t in_tile) {
    mine = m;
    left = tokens;
    d = 0;
    each = (int64_t)gridDim.z >= in_tile;
    if (each) left = tokens >> blockIdx.z & 1 ? 1ull << blockIdx.z : 0;
  }
  __device__ __forceinline__ bool next(uint64_t& group, int& named) {
    while (left) {
      const int lead = __builtin_ctzll(left);
      named = __builtin_amdgcn_readlane(mine, lead);
      group = __ballot(mine == named);
      left &= ~group;
      if (each ? __builtin_ctzll(group) == lead : d++ % gridDim.z == blockIdx.z) return true;
    }
    return false;
  }
};

// Sixteen bytes at any address: those of a row's last elements start anywhere.
struct __attribute__((packed, aligned(1))) LoraAny { u32x4 v; };
__device__ __forceinline__ u32x4 lora_load(const void* p) { return ((const LoraAny*)p)->v; }

// Eight 16-bit elements without the first `drop`, which become 0.
__device__ __forceinline__ u32x4 lora_drop(u32x4 v, int drop) {
#pragma unroll
  for (int i = 0; i < 4; i++) v[i] &= (2 * i >= drop ? 0xFFFFu : 0) | (2 * i + 1 >= drop ? 0xFFFF0000u : 0);
  return v;
}

// Between the matrix instructions and the first other use of their results: where the two
// were in different blocks the compiler left out the wait states between them (LDS then got
// sums without their last instructions). The build reads the unit for it.
__device__ __forceinline__ void lora_settle(floatx4& v) { asm volatile("s_nop 15" : "+v"(v)); }

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
template <bool OWN> struct LoraColumns {
  int* list;              // this wave's, in LDS
  uint64_t group;
  int count;              // columns that may hold one

  // mine: the lane's token
  __device__ __forceinline__ void set(int* l, uint64_t g, int mine) {
    list = l;
    group = g;
    count = OWN ? 16 : __popcll(g);
    if constexpr (!OWN) {
      const int lane = threadIdx.x & 63;
      lora_lds_order();
      if (g >> lane & 1)
        list[__builtin_amdgcn_mbcnt_hi((uint32_t)(g >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)g, 0))] = mine;
      lora_lds_order();
    }
  }
  // whether a column holds one of the group's tokens, and its token (another of the group where it does not;
  // up to 16 tokens are one tile in their own order)
  __device__ __forceinline__ bool has(int col) const { return OWN ? group >> col & 1 : col < count; }
  __device__ __forceinline__ int token(int col) const {
    return OWN ? (has(col) ? col : __builtin_ctzll(group)) : list[min(col, count - 1)];
  }
};

template <int N> struct LoraCount { static constexpr int n = N; };
template <int J, int XS> struct LoraStep { u32x4 a[4], x[J][XS]; };   // what LORA_KW k of J columns need

// t of one adapter's tokens, part blockIdx.x of k. A wave takes one tile of 16 ranks and,
// LORA_KW at a time, its share of the part; the waves of a rank tile are added in LDS in
// their order. The instruction's rows are ranks, its columns tokens.
// Latency bounds it for few tokens (16 of them, k = 4096, rank 16: 4.6 us for 2 MB), loads for
// more (37 tokens of 24 adapters of rank 64, k = 11008: 10.3 us for 27 MB, 2.6 TB/s: 285 blocks on
// 256 CUs; 4096 tokens of int8 codes 8.2 us for 17 MB). More than 64 tokens of a 16-bit x spill 8
// registers, which are not needed in the loop over k.
template <int IO, bool X8, int NT, bool OWN>
__global__ void __launch_bounds__(64 * LORA_WAVES, 4) lora_inner_kernel(LoraArgs A) {
  typedef typename LoraType<IO>::v v_t;
  typedef LoraColumns<OWN> cols_t;
  constexpr int XS = X8 ? 2 : 4;
  __shared__ floatx4 red[LORA_WAVES][NT][64];
  __shared__ int tokens[OWN ? 1 : LORA_WAVES][LORA_TILE];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l16 = lane & 15, q = lane >> 4;
  const int64_t tile0 = (int64_t)blockIdx.y * LORA_TILE;
  int at_lane;
  const int mine = lora_named(A, tile0, at_lane);
  const int rank_tiles = (A.rank + 15) / 16, across = rank_tiles <= 1 ? 1 : rank_tiles <= 2 ? 2 : rank_tiles <= 4 ? 4 : 8;
  const int rt = wave % across, part = wave / across, parts = LORA_WAVES / across;

  LoraGroups groups;
  groups.init(mine, __ballot(mine >= 0), min((int64_t)LORA_TILE, A.n - tile0));
  uint64_t group;
  int adapter;
  while (groups.next(group, adapter)) {
    cols_t cols;
    cols.set(tokens[OWN ? 0 : wave], group, at_lane);
    const uint8_t* const ar = (const uint8_t*)(A.a + ((int64_t)adapter * A.rank + min(16 * rt + l16, A.rank - 1)) * A.lda);
    for (int c0 = 0; c0 < cols.count; c0 += 16 * NT) {
      floatx4 acc[NT];
#pragma unroll
      for (int j = 0; j < NT; j++) acc[j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
      // J columns of 16 tokens
      auto product = [&](auto J) {
        const uint8_t* xr[J.n];
#pragma unroll
        for (int j = 0; j < J.n; j++) xr[j] = A.x + (int64_t)cols.token(c0 + 16 * j + l16) * A.ldx * (X8 ? 1 : 2);
        constexpr int JN = decltype(J)::n;
        typedef LoraStep<JN, XS> step_t;
        auto first_k = [&](int i) { return (((int64_t)blockIdx.x * A.loops + i) * parts + part) * LORA_KW; };
        // What lies behind k is loaded from the row's last elements, and those that came before are dropped from A, and
        // from a 16-bit x too, whose infinities would make NaN of A's zeros.
        auto load = [&](step_t& S, int64_t k0, bool whole) {
          constexpr int E = X8 ? 16 : 8;          // elements of x in 16 bytes
#pragma unroll
          for (int s = 0; s < XS; s++) {
            const int64_t at = k0 + 4 * E * s + E * q, from = whole ? at : min(at, A.k - E);
#pragma unroll
            for (int h = 0; h < E / 8; h++) {
              u32x4& a = S.a[E / 8 * s + h];
              a = lora_load(ar + (from + 8 * h) * 2);
              if (!whole) a = lora_drop(a, (int)min(at - from - 8 * h, (int64_t)8));
            }
#pragma unroll
            for (int j = 0; j < JN; j++) {
              S.x[j][s] = lora_load(xr[j] + from * (X8 ? 1 : 2));
              if (!X8 && !whole) S.x[j][s] = lora_drop(S.x[j][s], (int)min(at - from, (int64_t)E));
            }
          }
          __builtin_amdgcn_sched_barrier(0);      // all are on their way
        };
        auto multiply = [&](const step_t& S) {
#pragma unroll
          for (int j = 0; j < JN; j++)
#pragma unroll
            for (int s = 0; s < 4; s++) {
              u32x4 b;
              if constexpr (X8) {
                uint32_t lo = S.x[j][s / 2][2 * (s % 2)], hi = S.x[j][s / 2][2 * (s % 2) + 1];
                asm volatile("" : "+v"(lo), "+v"(hi));          // not before they are needed: values are twice the registers
                b = lora_codes<IO>(lo, hi);
              } else {
                b = S.x[j][s];
              }
              acc[j] = lora_mma<IO>(__builtin_bit_cast(v_t, S.a[s]), __builtin_bit_cast(v_t, b), acc[j]);
            }
        };
        // The same of 16 bytes of x a lane, for many tokens: a whole step of them, dropped, costs time
        // (4096 tokens of k = m = 4096, 16-bit, no tail among them, 28.0 us beside 27.4).
        auto last_pieces = [&](int64_t k0) {
          constexpr int E = X8 ? 16 : 8;
#pragma unroll 1
          for (int s = 0; s < XS && k0 + 4 * E * s < A.k; s++) {
            const int64_t at = k0 + 4 * E * s + E * q, from = min(at, A.k - E);
            const int drop = (int)min(at - from, (int64_t)E);
            u32x4 a[E / 8], x[JN];
#pragma unroll
            for (int h = 0; h < E / 8; h++) a[h] = lora_load(ar + (from + 8 * h) * 2);
#pragma unroll
            for (int j = 0; j < JN; j++) x[j] = lora_load(xr[j] + from * (X8 ? 1 : 2));
#pragma unroll
            for (int h = 0; h < E / 8; h++) a[h] = lora_drop(a[h], drop - 8 * h);
#pragma unroll
            for (int j = 0; j < JN; j++)
#pragma unroll
              for (int h = 0; h < E / 8; h++) {
                const u32x4 b = X8 ? lora_codes<IO>(x[j][2 * h], x[j][2 * h + 1]) : lora_drop(x[j], drop);
                acc[j] = lora_mma<IO>(__builtin_bit_cast(v_t, a[h]), __builtin_bit_cast(v_t, b), acc[j]);
              }
          }
        };
        int steps = 0;                            // of the wave's, those that lie within k whole
        while (steps < A.loops && first_k(steps) + LORA_KW <= A.k) steps++;
        step_t S, N;
        if (steps > 0) {
          load(S, first_k(0), true);
#pragma unroll 1
          for (int i = 1; i < steps; i++) {
            if constexpr (JN == 1) {
              load(N, first_k(i), true);          // the next ones behind the present one's products
              multiply(S);
              S = N;
            } else {
              multiply(S);
              load(S, first_k(i), true);
            }
          }
          multiply(S);
        }
        if (steps < A.loops && first_k(steps) < A.k) {
          if constexpr (NT > 1) {
            last_pieces(first_k(steps));
          } else {
            load(S, first_k(steps), false);
            multiply(S);
          }
        }
      };
      if (16 * rt < A.rank) {
        if (NT == 1 || cols.count <= 16) product(LoraCount<1>());
        else product(LoraCount<NT>());
      }
#pragma unroll
      for (int j = 0; j < NT; j++) {
        lora_settle(acc[j]);
        red[wave][j][lane] = acc[j];
      }
      __syncthreads();
      for (int u = wave; u < across * NT; u += LORA_WAVES) {
        const int r = u % across, j = u / across, col = c0 + 16 * j + l16, rank = 16 * r + 4 * q;
        floatx4 v = red[r][j][lane];
        for (int w = 1; w < parts; w++) v += red[r + w * across][j][lane];
        if (cols.has(col) && rank < A.rank)
          *(floatx4*)(A.t + ((int64_t)blockIdx.x * A.n + cols.token(col)) * A.rank + rank) = v;
      }
      __syncthreads();
    }
  }
}

// y of one adapter's tokens (or of those without one), LORA_FEATURES outputs a block, 32 a
// wave. The instruction's rows are outputs, its columns tokens, its k the ranks twice: t
// goes in as two 16-bit parts, the second what the first left over, so that 16 to 22 bits of
// it meet B (f16: against the token's largest, brought to 1 by a power of two, which f16
// would not hold otherwise). Row 4 q + r of instruction f is output 8 q + 4 f + r: a lane
// ends with eight outputs in a row, 16 bytes.
// SETS: chunks of eight ranks a lane takes; 0: up to 16 ranks, both parts in one instruction.
// Memory bounds it for prompts: 4096 tokens to 6144 features beside accumulators, 151 MB, 33 us,
// 4.6 TB/s (with 64 outputs a wave 40 us: half the waves); for few tokens latency, 3.4 us for one
// and 6.4 for 16 tokens to 22016 features (13 MB). Six of the 64 variants spill, all beside
// accumulators, whose loads are in flight together: f16 4 registers for ranks 17 to 32 (17 to 64
// tokens, many outputs), 6 and 23 for ranks over 64 (up to 64 tokens and more), bf16 4 for ranks
// 33 to 64 (more than 64 tokens), 4 and 18 over 64. f16, rank 128: 37 tokens of k = 11008 31 us
// with the inner product, 1024 tokens of k = m = 4096 42 us.
template <int IO, bool ACC, int SETS, int NT, bool OWN, int FB>
__global__ void __launch_bounds__(64 * LORA_WAVES, 4) lora_outer_kernel(LoraArgs A) {
  typedef typename LoraType<IO>::v v_t;
  typedef LoraColumns<OWN> cols_t;
  constexpr int THREADS = 64 * LORA_WAVES;
  constexpr int NS = SETS == 0 ? 1 : SETS;
  constexpr int RANKS = SETS == 0 ? 16 : 32 * SETS;
  constexpr int PER = RANKS / 4;                          // threads that bring a token's t
  // Parts of t on their way together. In us with 4 and 8: k = 16384, m = 4096, rank 64, 8 tokens 12.1 and 11.2; rank 128,
  // 37 tokens of k = 11008 27.6 and 30.6; rank 16, 16 tokens of k = 4096 10.4 and 10.8, 4096 tokens 44.9 and 51.1.
  constexpr int WS = NT == 1 && SETS == 2 ? 8 : 4;
  constexpr int BQ = ACC ? 2 : 1;                         // pieces of 16 bytes a lane's outputs take of the base
  alignas(16) __shared__ uint16_t ts[16 * NT][2 * RANKS + 8];   // both parts of t, read in 16 bytes; 16 tokens lie on distinct banks
  __shared__ float factor[16 * NT];
  __shared__ int tokens[OWN ? 1 : LORA_WAVES][LORA_TILE];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l16 = lane & 15, q = lane >> 4;
  const int64_t tile0 = (int64_t)blockIdx.y * LORA_TILE;
  const int64_t f0 = ((int64_t)blockIdx.x * LORA_WAVES + wave) * (32 * FB);
  // A lane's eight outputs; behind the last output the last eight, of which it stores what is its own.
  auto first_out = [&](int b, int of) { return min(f0 + 32 * b + 8 * of, A.m - 8); };
  int64_t out[FB];
#pragma unroll
  for (int b = 0; b < FB; b++) out[b] = first_out(b, q);
  int at_lane;
  const int mine = lora_named(A, tile0, at_lane);
  const int chunks = A.rank / 8;

  floatx4 cs[FB][2];
  if constexpr (ACC) {
#pragma unroll
    for (int b = 0; b < FB; b++)
#pragma unroll
      for (int i = 0; i < 2; i++) cs[b][i] = __builtin_bit_cast(floatx4, lora_load(A.col_scale + out[b] + 4 * i));
  }

  LoraGroups groups;
  groups.init(mine, __ballot(mine >= -2), min((int64_t)LORA_TILE, A.n - tile0));
  uint64_t group;
  int adapter;
  while (groups.next(group, adapter)) {
    if (adapter == -1 && A.in_place) continue;
    cols_t cols;
    cols.set(tokens[OWN ? 0 : wave], group, at_lane);
    const float sa = adapter >= 0 ? A.scale[adapter] : adapter == -1 ? 0.0f : __builtin_nanf("");
    for (int c0 = 0; c0 < cols.count; c0 += 16 * NT) {
      // t first: what is behind it is not waited for until it is in LDS
      auto part = [&](int e, int s) {
        const float* p = A.t + (int64_t)cols.token(c0 + e / PER) * A.rank + min(e % PER * 4, A.rank - 4);
        return *(const floatx4*)(p + (int64_t)min(s, A.splits - 1) * A.n * A.rank);
      };
      floatx4 w[WS];
      float xs = 1.0f;
      if (adapter >= 0 && (int)threadIdx.x < 16 * NT * PER) {
#pragma unroll
        for (int i = 0; i < WS; i++) w[i] = part(threadIdx.x, i);
      }
      // B's pieces: chunk 4 s + q (up to 16 ranks: q % 2) of the lane's output row
      v_t bv[FB][NS][2];
#pragma unroll
      for (int s = 0; s < NS; s++) {
        const int chunk = SETS == 0 ? q % 2 : 4 * s + q;
#pragma unroll
        for (int f = 0; f < 2 * FB; f++) {
          const int64_t row = first_out(f / 2, l16 / 4) + 4 * (f % 2) + l16 % 4;
          u32x4 v = {0, 0, 0, 0};
          if (adapter >= 0 && chunk < chunks) v = *(const u32x4*)(A.b + ((int64_t)adapter * A.m + row) * A.rank + 8 * chunk);
          bv[f / 2][s][f % 2] = __builtin_bit_cast(v_t, v);
        }
      }
      // what y adds to, as it lies in memory
      u32x4 base[FB][NT][BQ];
      float rs[NT];
      int token[NT];
      bool in[NT];
#pragma unroll
      for (int j = 0; j < NT; j++) {
        if (j > 0 && c0 + 16 * j >= cols.count) break;    // most groups of a prompt's scattered tokens are small
        in[j] = cols.has(c0 + 16 * j + l16);
        token[j] = cols.token(c0 + 16 * j + l16);
        rs[j] = ACC ? A.row_scale[token[j]] : 1.0f;
        const uint8_t* const p = A.base + (int64_t)token[j] * A.ldc * (ACC ? 4 : 2);
#pragma unroll
        for (int b = 0; b < FB; b++)
#pragma unroll
          for (int i = 0; i < BQ; i++) base[b][j][i] = lora_load(p + out[b] * (ACC ? 4 : 2) + 16 * i);
      }
      if (adapter >= 0) {
#pragma unroll 1
        for (int e = threadIdx.x; e < min(16 * NT, (cols.count - c0 + 15) / 16 * 16) * PER; e += THREADS) {
          const int j = e / PER, r = e % PER * 4;
          if (A.x_scale) xs = A.x_scale[cols.token(c0 + j)];
          floatx4 v = {0.0f, 0.0f, 0.0f, 0.0f};
          for (int s = 0; s < A.splits; s += WS) {          // the parts of k in their order
            if (e >= THREADS || s > 0) {
#pragma unroll
              for (int i = 0; i < WS; i++) w[i] = part(e, s + i);
            }
#pragma unroll
            for (int i = 0; i < WS; i++)
              if (s + i < A.splits) v += w[i];
          }
          if (r >= A.rank || !cols.has(c0 + j)) v = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
          float up = 1.0f, fac = sa * xs, top = 0.0f;       // a NaN is not the largest; it stays in t
#pragma unroll
          for (int i = 0; i < 4; i++) top = fmaxf(top, __builtin_fabsf(v[i]));
          if constexpr (IO == DT_F16) {
            // the token's largest below 1: times 2^-x with x its exponent's distance; not for 0
#pragma unroll
            for (int off = 1; off < PER; off *= 2) top = fmaxf(top, __shfl_xor(top, off));
            const int x = (int)(__builtin_bit_cast(uint32_t, top) >> 23) - 126;
            if (x > -126) {
              up = __builtin_ldexpf(1.0f, -min(x, 120));      // 2^-127 is none; 2^8 f16 still holds
              fac *= __builtin_ldexpf(1.0f, min(x, 120));
            }
          }
          uint32_t hi[2], lo[2];
#pragma unroll
          for (int i = 0; i < 2; i++) {
            const float a = v[2 * i] * up, b = v[2 * i + 1] * up;
            const uint16_t ha = to_bits16<IO>(a), hb = to_bits16<IO>(b);
            hi[i] = (uint32_t)ha | (uint32_t)hb << 16;
            lo[i] = (uint32_t)to_bits16<IO>(a - from_bits16<IO>(ha)) | (uint32_t)to_bits16<IO>(b - from_bits16<IO>(hb)) << 16;
          }
          // Infinities have no second part (and decide what the token's others are next to them). A finite t that bf16
          // rounds to one becomes the type's largest value and the rest.
          if (!(top < (IO == DT_F16 ? INFINITY : 0x1.FEp127f))) {
            lo[0] = lo[1] = 0;
            if constexpr (IO == DT_BF16) {
#pragma unroll
              for (int i = 0; i < 4; i++) {
                const int at = 16 * (i % 2);
                if ((hi[i / 2] >> at & 0x7FFF) == 0x7F80 && __builtin_fabsf(v[i]) < INFINITY) hi[i / 2] -= 1u << at;
                if (__builtin_fabsf(v[i]) < INFINITY)
                  lo[i / 2] |= (uint32_t)to_bits16<IO>(v[i] - from_bits16<IO>((uint16_t)(hi[i / 2] >> at))) << at;
              }
            }
          }
          *(u32x2*)&ts[j][r] = u32x2{hi[0], hi[1]};
          *(u32x2*)&ts[j][RANKS + r] = u32x2{lo[0], lo[1]};
          if (r == 0) factor[j] = fac;
        }
        __syncthreads();
      }
#pragma unroll
      for (int j = 0; j < NT; j++) {
        if (c0 + 16 * j >= cols.count) break;
        const int64_t at = token[j];
        const uint16_t* const tj = ts[16 * j + l16];
        const float fac = factor[16 * j + l16];
#pragma unroll
        for (int b = 0; b < FB; b++) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; e++) {
            if constexpr (ACC) {
              const uint32_t c = base[b][j][e / 4][e % 4];
              v[e] = (float)(int32_t)c * rs[j] * cs[b][e / 4][e % 4];
            } else {
              v[e] = from_bits16<IO>((uint16_t)(base[b][j][0][e / 2] >> (16 * (e % 2))));
            }
          }
          if (adapter >= 0) {
            floatx4 acc[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
            for (int s = 0; s < NS; s++) {
              const v_t first = *(const v_t*)(tj + (SETS == 0 ? 8 * q : 8 * (4 * s + q)));  // up to 16 ranks: q / 2 is the part
#pragma unroll
              for (int f = 0; f < 2; f++) acc[f] = lora_mma<IO>(bv[b][s][f], first, acc[f]);
              if constexpr (SETS > 0) {
                const v_t second = *(const v_t*)(tj + RANKS + 8 * (4 * s + q));
#pragma unroll
                for (int f = 0; f < 2; f++) acc[f] = lora_mma<IO>(bv[b][s][f], second, acc[f]);
              }
            }
#pragma unroll
            for (int e = 0; e < 8; e++) v[e] = __builtin_fmaf(fac, acc[e / 4][e % 4], v[e]);
          } else if (adapter == -2) {
#pragma unroll
            for (int e = 0; e < 8; e++) v[e] = sa;
          }
          if (in[j]) {
            uint16_t* const yr = A.y + at * A.ldy + out[b];
            const int skip = (int)min(f0 + 32 * b + 8 * q - out[b], (int64_t)8);   // another lane's
            u32x4 p;
#pragma unroll
            for (int i = 0; i < 4; i++) p[i] = (uint32_t)to_bits16<IO>(v[2 * i]) | (uint32_t)to_bits16<IO>(v[2 * i + 1]) << 16;
            if (skip == 0) {
              ((LoraAny*)yr)->v = p;
            } else {
#pragma unroll
              for (int e = 0; e < 8; e++)
                if (e >= skip) yr[e] = (uint16_t)(p[e / 2] >> (16 * (e % 2)));
            }
          }
        }
      }
      __syncthreads();                            // t is read: the next may come
    }
  }
}

template <int IO, bool X8>
hipError_t lora_inner(const LoraArgs& a, const nm_lora_plan& pl, hipStream_t s) {
  const dim3 grid((unsigned)a.splits, (unsigned)pl.tiles, (unsigned)pl.slots_in);
  const dim3 threads(64 * LORA_WAVES);
  // Up to 16 tokens as their own columns: 16 tokens to 22016 features 10.5 us, sorted into columns 11.1, one token 7.1 and
  // 7.4. Then 16 columns at a time for a tile, 64 for more: 256 tokens in runs of two adapters 12.2 us with 64 and 19.4
  // with 16, scattered over 64 adapters 27.2 and 26.5.
  if (a.n <= 16) hipLaunchKernelGGL((lora_inner_kernel<IO, X8, 1, true>), grid, threads, 0, s, a);
  else if (a.n <= LORA_TILE) hipLaunchKernelGGL((lora_inner_kernel<IO, X8, 1, false>), grid, threads, 0, s, a);
  else hipLaunchKernelGGL((lora_inner_kernel<IO, X8, 4, false>), grid, threads, 0, s, a);
  return hipGetLastError();
}

template <int IO, bool ACC, int SETS>
hipError_t lora_outer(const LoraArgs& a, const nm_lora_plan& pl, hipStream_t s) {
  auto go = [&](auto kernel, int outputs) {
    const dim3 grid((unsigned)((a.m + outputs - 1) / outputs), (unsigned)pl.tiles, (unsigned)pl.slots_out);
    hipLaunchKernelGGL(kernel, grid, dim3(64 * LORA_WAVES), 0, s, a);
    return hipGetLastError();
  };
  if (a.n > LORA_TILE) return go(lora_outer_kernel<IO, ACC, SETS, 4, false, 1>, LORA_FEATURES);
  if constexpr (SETS < 2) {
    if (a.m * pl.slots_out > LORA_MANY) {
      if (a.n <= 16) return go(lora_outer_kernel<IO, ACC, SETS, 1, true, 2>, 2 * LORA_FEATURES);
      return go(lora_outer_kernel<IO, ACC, SETS, 1, false, 2>, 2 * LORA_FEATURES);
    }
  }
  if (a.n <= 16) return go(lora_outer_kernel<IO, ACC, SETS, 1, true, 1>, LORA_FEATURES);
  return go(lora_outer_kernel<IO, ACC, SETS, 1, false, 1>, LORA_FEATURES);
}

template <int IO>
hipError_t lora_go(const LoraArgs& a, const nm_lora_plan& pl, hipStream_t s) {
  const bool acc = pl.p.type_base == NM_I32;
  if (a.order) hipLaunchKernelGGL(lora_sort_kernel, dim3(1), dim3(LORA_SORT_THREADS), 0, s, a, (intx2*)a.order);
  hipError_t e = pl.p.type_x == NM_I8 ? lora_inner<IO, true>(a, pl, s) : lora_inner<IO, false>(a, pl, s);
  if (e != hipSuccess) return e;
  const int r = a.rank;
  if (r <= 16) return acc ? lora_outer<IO, true, 0>(a, pl, s) : lora_outer<IO, false, 0>(a, pl, s);
  if (r <= 32) return acc ? lora_outer<IO, true, 1>(a, pl, s) : lora_outer<IO, false, 1>(a, pl, s);
  if (r <= 64) return acc ? lora_outer<IO, true, 2>(a, pl, s) : lora_outer<IO, false, 2>(a, pl, s);
  return acc ? lora_outer<IO, true, 4>(a, pl, s) : lora_outer<IO, false, 4>(a, pl, s);
}

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
  if (p->m < 8 || p->n < 0 || p->k < 16) return layer_fail(NM_ERR_SHAPE, "m must be >= 8, n >= 0, k >= 16");
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
  // A block for each token of a tile while that are few, then fewer for its groups. With 64 adapters of rank 16, k = m =
  // 4096, scattered, in us: up to 4096 blocks 256 tokens 27.1 and 4096 tokens 36, up to 16384 26.4 and 67, runs of 256
  // tokens 15.4 and 20.5; then 512 over the tiles 256 tokens 23.1 and 4096 34.9, 256 24.6 and 37.3, 1024 27.2 and 35.9,
  // 2048 34.8 and 37.3.
  auto slots = [&](int64_t blocks) {
    if (blocks * tile <= 4096) return (int)tile;
    const int64_t want = 512 / blocks;
    return (int)(want < 1 ? 1 : want > tile ? tile : want);
  };
  const int rank_tiles = (p->rank + 15) / 16, across = rank_tiles <= 1 ? 1 : rank_tiles <= 2 ? 2 : rank_tiles <= 4 ? 4 : 8;
  const int64_t step = (int64_t)LORA_KW * (LORA_WAVES / across), steps = (p->k + step - 1) / step;
  // Parts of k, each of which the outer product reads t of. 32 instead of 16 for a few tokens: one token, k = 65536, rank
  // 128 28.4 us instead of 44.4, 8 tokens, k = 16384, rank 64 12.1 and 12.5; but 16 tokens of 32 adapters, k = 11008, rank
  // 64 14.2 instead of 12.3, 64 tokens of rank 32 18.5 and 16.3.
  const int64_t parts = p->n <= 8 ? 32 : 16;
  int64_t splits = 1024 / tiles;
  if (splits > parts) splits = parts;
  if (splits > steps) splits = steps;
  if (splits < 1) splits = 1;
  pl->loops = (int)((steps + splits - 1) / splits);
  pl->splits = (int)((steps + pl->loops - 1) / pl->loops);
  pl->slots_in = slots(tiles * pl->splits);
  pl->slots_out = slots(tiles * ((p->m + LORA_FEATURES - 1) / LORA_FEATURES + 1));
  pl->sorted = p->n >= 256 && p->adapters >= 4 && p->n * p->adapters >= 8192;  // figures at lora_sort_kernel
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
  *bytes = (size_t)plan->splits * p.n * p.rank * sizeof(float) + (plan->sorted ? (size_t)p.n * 8 : 0);
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
  if (p.n == 0) return NM_OK;
  if (!dX || !dA || !dB || !d_scale || !d_index || !d_base || !dY)
    return layer_fail(NM_ERR_INVALID_ARG, "dX / dA / dB / d_scale / d_index / d_base / dY is NULL");
  if (!d_workspace) return layer_fail(NM_ERR_INVALID_ARG, "d_workspace is NULL");
  if ((d_x_scale != nullptr) != (p.type_x == NM_I8))
    return layer_fail(NM_ERR_INVALID_ARG, "d_x_scale must be given exactly where x is int8");
  const bool acc = p.type_base == NM_I32;
  if ((d_row_scale != nullptr) != acc || (d_col_scale != nullptr) != acc)
    return layer_fail(NM_ERR_INVALID_ARG, "d_row_scale and d_col_scale must be given exactly where the base is int32");
  if (dY == d_base && (acc || (p.n > 1 && p.ldc != p.ldy)))
    return layer_fail(NM_ERR_INVALID_ARG, "dY may be d_base only where the base is of type_y and ldc == ldy");
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
  if (plan->sorted) a.order = (const intx2*)(a.t + (size_t)plan->splits * p.n * p.rank);
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
