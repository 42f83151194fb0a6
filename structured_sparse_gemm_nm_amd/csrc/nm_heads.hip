// Norms of queries and keys for each head with the rotation by position, in one
// pass over the joint query/key/value product, and its gradient (formulas in
// include/nmsparse.h).
//
// A head sits in G lanes, eight elements a lane, and the lanes' pairs are chosen so
// that a rotation stays within a lane: for pairs of halves a lane takes four
// elements of each half. Every head is read once and written once; memory bounds
// both directions (figures at the kernels).
#include <math.h>

#include <new>

#include "nm_layer.h"

struct nm_heads_plan {
  nm_heads_problem_t p;
};

namespace nm {

struct HeadArgs {
  const uint8_t* x;
  const float* row_scale;
  const float* col_scale;
  const uint16_t* gamma_q;
  const uint16_t* gamma_k;
  const int64_t* positions;
  const float* table;
  const uint16_t* dy;
  uint16_t* y;          // backward: dx
  float* part;          // backward: the blocks' shares of the gains' gradients, 2 x dim each
  int64_t rows, table_rows, ldx, ldy, lddy;
  int q, normed, heads, dim, rotary, zero_rows;
  float eps, rdim;      // rdim = 1 / dim
};

constexpr int HEAD_THREADS = 256;
// Blocks of the backward pass, two a CU: forward and backward of 8192 tokens of 48 heads of 128
// 102.8 us, with 1024 106.4 (before loads ran a round ahead: 512 105.2, 768 118.4, 1024 108.8, 2048 114.8).
constexpr int HEAD_MOST = 512;
constexpr int HEAD_CHAIN = 32;      // tokens whose gains' gradients are one chain of sums
// Heads that a group of lanes has on their way at a time: 4096 tokens of 48 heads of 128 from
// accumulators 31.6 us, with 2 32.2, with 8 42.9; 777 tokens of 25 heads of 80 4.6, 4.3, 5.6.
constexpr int HEAD_U = 4;

// Four 16-bit elements at an address of 8 bytes' alignment.
template <int IO> __device__ __forceinline__ void four16(float* o, u32x2 w) {
#pragma unroll
  for (int i = 0; i < 4; i++) o[i] = from_bits16<IO>((uint16_t)(w[i / 2] >> (16 * (i % 2))));
}
template <int IO> __device__ __forceinline__ u32x2 pack16(const float* v) {
  uint16_t o[4];
#pragma unroll
  for (int i = 0; i < 4; i++) o[i] = to_bits16<IO>(v[i]);
  return u32x2{(uint32_t)o[0] | (uint32_t)o[1] << 16, (uint32_t)o[2] | (uint32_t)o[3] << 16};
}

// Where a lane's eight elements lie in a head, four from lo on and four from hi
// on, and its angles. Lane j turns the pairs 4j .. 4j + 3; behind the turned part
// lanes take eight elements each.
template <bool HALVES> struct HeadLane {
  int lo, hi;
  bool in, turns;
  float c[4], s[4];

  __device__ __forceinline__ void place(const HeadArgs& A, int j) {
    in = 8 * j < A.dim;
    turns = 8 * j < A.rotary;
    lo = HALVES && turns ? 4 * j : 8 * j;
    hi = HALVES && turns ? A.rotary / 2 + 4 * j : 8 * j + 4;
    if (!in) lo = hi = 0;
  }
  // A position behind the table has no angles: NaN.
  __device__ __forceinline__ void angles(const HeadArgs& A, int j, int64_t pos) {
    if (!turns) return;
    const bool known = pos < A.table_rows;
    const float* t = A.table + (known ? pos : 0) * A.rotary + 4 * j;
    const floatx4 cv = *(const floatx4*)t, sv = *(const floatx4*)(t + A.rotary / 2);
#pragma unroll
    for (int i = 0; i < 4; i++) {
      c[i] = known ? cv[i] : __builtin_nanf("");
      s[i] = known ? sv[i] : __builtin_nanf("");
    }
  }
  // The lane's pairs (a, b) turned to (a c - b s, b c + a s), or back.
  __device__ __forceinline__ void turn(float (&v)[8], float sign) const {
    if (!turns) return;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int ia = HALVES ? i : 2 * i, ib = HALVES ? 4 + i : 2 * i + 1;
      const float a = v[ia], b = v[ib], sn = sign * s[i];
      v[ia] = a * c[i] - b * sn;
      v[ib] = b * c[i] + a * sn;
    }
  }
};

// What a lane loads for one head.
template <bool ACC> struct HeadRaw;
template <> struct HeadRaw<false> { u32x2 v[2]; };
template <> struct HeadRaw<true> { u32x4 v[2]; floatx4 s[2]; };

template <bool ACC, typename L>
__device__ __forceinline__ HeadRaw<ACC> head_load(const HeadArgs& A, const uint8_t* row, int head, const L& l) {
  HeadRaw<ACC> r;
  const int64_t at = (int64_t)head * A.dim;
  if constexpr (ACC) {
    r.v[0] = *(const u32x4*)((const uint32_t*)row + at + l.lo);
    r.v[1] = *(const u32x4*)((const uint32_t*)row + at + l.hi);
    r.s[0] = *(const floatx4*)(A.col_scale + at + l.lo);
    r.s[1] = *(const floatx4*)(A.col_scale + at + l.hi);
  } else {
    r.v[0] = *(const u32x2*)((const uint16_t*)row + at + l.lo);
    r.v[1] = *(const u32x2*)((const uint16_t*)row + at + l.hi);
  }
  return r;
}

template <int IO, bool ACC>
__device__ __forceinline__ void head_values(float (&v)[8], const HeadRaw<ACC>& r, float rs, bool in) {
#pragma unroll
  for (int h = 0; h < 2; h++) {
    if constexpr (ACC) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const uint32_t bits = r.v[h][i];
        v[4 * h + i] = (float)(int32_t)bits * rs * r.s[h][i];
      }
    } else {
      four16<IO>(v + 4 * h, r.v[h]);
    }
  }
  if (!in) {
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = 0.0f;
  }
}

// 1 / sqrt(v): the instruction's own, off by one step, but for the values that it would flush.
__device__ __forceinline__ float head_rsqrt(float v) {
  if (v < 0x1p-100f) return 1.0f / __builtin_sqrtf(v);
  return __builtin_amdgcn_rsqf(v);
}

// One block a token (and, for few tokens of many heads, a share of its heads): a group of
// G lanes loads the token's angles once and takes head after head, HEAD_U of them on
// their way together. Memory bounds it: 4096 tokens of 48 heads of 128 from accumulators,
// 153 MB, 31.7 us, 4.8 TB/s; one token 2.4 us, a launch. The exchanges of a head's sum
// stay within 16 lanes' rows, without LDS.
template <int IO, bool ACC, bool HALVES, int G>
__global__ void __launch_bounds__(HEAD_THREADS) heads_kernel(HeadArgs A) {
  const int64_t token = blockIdx.x;
  const int64_t pos = A.positions[token];
  if (pos < 0 && !A.zero_rows) return;            // no token: its row stays as it was
  const int j = threadIdx.x % G;
  const int first = blockIdx.y * (HEAD_THREADS / G) + threadIdx.x / G, step = gridDim.y * (HEAD_THREADS / G);
  HeadLane<HALVES> l;
  l.place(A, j);
  const uint8_t* const row = A.x + token * A.ldx * (ACC ? 4 : 2);
  uint16_t* const out = A.y + token * A.ldy;
  if (pos < 0) {
    for (int h = first; h < A.heads && l.in; h += step) {
      uint16_t* const to = out + (int64_t)h * A.dim;
      *(u32x2*)(to + l.lo) = *(u32x2*)(to + l.hi) = u32x2{0, 0};
    }
    return;
  }
  const float rs = ACC ? A.row_scale[token] : 1.0f;
  float gq[8], gk[8];
  l.angles(A, j, pos);
  four16<IO>(gq, *(const u32x2*)(A.gamma_q + l.lo));
  four16<IO>(gq + 4, *(const u32x2*)(A.gamma_q + l.hi));
  four16<IO>(gk, *(const u32x2*)(A.gamma_k + l.lo));
  four16<IO>(gk + 4, *(const u32x2*)(A.gamma_k + l.hi));

  for (int h0 = first; h0 < A.heads; h0 += HEAD_U * step) {
    HeadRaw<ACC> raw[HEAD_U];
#pragma unroll
    for (int u = 0; u < HEAD_U; u++)
      raw[u] = head_load<ACC>(A, row, min(h0 + u * step, A.heads - 1), l);
#pragma unroll
    for (int u = 0; u < HEAD_U; u++) {
      const int h = h0 + u * step;
      if (h >= A.heads) break;
      float v[8];
      head_values<IO, ACC>(v, raw[u], rs, l.in);
      if (h < A.normed) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; i++) sum = __builtin_fmaf(v[i], v[i], sum);
        sum = lane_sum<G>(sum);
        const float f = head_rsqrt(__builtin_fmaf(sum, A.rdim, A.eps));
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] *= f * (h < A.q ? gq[i] : gk[i]);
        l.turn(v, 1.0f);
      }
      if (l.in) {
        uint16_t* const to = out + (int64_t)h * A.dim;
        *(u32x2*)(to + l.lo) = pack16<IO>(v);
        *(u32x2*)(to + l.hi) = pack16<IO>(v + 4);
      }
    }
  }
}

// The gradient. With g the turned-back gradient of a head, u its input, f its
// factor and w = gamma g: dx = f w - u f^3 / dim * sum(w u), dgamma = sum over
// tokens and heads of g u f. Blocks walk over the tokens, their groups over the
// heads, and keep their shares of dgamma in registers; the groups' shares are added
// in LDS in their order and written out, and heads_gain_kernel adds the blocks'. Memory
// bounds it: 8192 tokens of 48 heads of 128, 302 MB, 62.6 us, 4.8 TB/s (70 us where a round's
// loads were asked for in the round itself). Rounds of 3 heads a group; what a round is short of
// is loaded for nothing. Forward and backward of 8192 tokens with rounds of 2, 3 and 4, in us:
// 48 heads of 128 113.6, 103.4 and 106.8; 40 of 128 103.9, 94.2 and 99.3; 24 of 256 110.6, 99.6
// and 103.8; 48 of 80 96.6, 86.0 and 91.0; but 64 of 128 134.8, 142.2 and 134.4, 40 of 64 63.1,
// 83.1 and 87.0.
template <int IO, bool HALVES, int G, bool GAIN>
__global__ void __launch_bounds__(HEAD_THREADS) heads_backward_kernel(HeadArgs A) {
  constexpr int U = 3;
  const int j = threadIdx.x % G, group = threadIdx.x / G, step = HEAD_THREADS / G;
  HeadLane<HALVES> l, ahead;
  l.place(A, j);
  ahead = l;
  float gq[8], gk[8], dq[8], dk[8], qs[8], ks[8];   // of HEAD_CHAIN tokens, and of all before
  four16<IO>(gq, *(const u32x2*)(A.gamma_q + l.lo));
  four16<IO>(gq + 4, *(const u32x2*)(A.gamma_q + l.hi));
  four16<IO>(gk, *(const u32x2*)(A.gamma_k + l.lo));
  four16<IO>(gk + 4, *(const u32x2*)(A.gamma_k + l.hi));
#pragma unroll
  for (int i = 0; i < 8; i++) dq[i] = dk[i] = qs[i] = ks[i] = 0.0f;
  auto flush = [&] {
#pragma unroll
    for (int i = 0; i < 8; i++) {
      qs[i] += dq[i];
      ks[i] += dk[i];
      dq[i] = dk[i] = 0.0f;
    }
  };

  struct Heads { HeadRaw<false> x[U], g[U]; };
  auto load = [&](Heads& r, int64_t token, int h0) {
    const uint8_t* const row = A.x + token * A.ldx * 2;
    const uint8_t* const drow = (const uint8_t*)(A.dy + token * A.lddy);
#pragma unroll
    for (int n = 0; n < U; n++) {
      const int h = min(h0 + n * step, A.heads - 1);
      r.x[n] = head_load<false>(A, row, h, l);
      r.g[n] = head_load<false>(A, drow, h, l);
    }
  };
  auto take = [&](const Heads& r, int64_t token, int h0, bool some) {
    uint16_t* const out = A.y + token * A.ldy;
#pragma unroll
    for (int n = 0; n < U; n++) {
      const int h = h0 + n * step;
      if (h >= A.heads) break;
      float u[8], g[8];
      head_values<IO, false>(u, r.x[n], 1.0f, l.in);
      head_values<IO, false>(g, r.g[n], 1.0f, l.in);
      if (!some) {                                // no token: no gradient
#pragma unroll
        for (int i = 0; i < 8; i++) g[i] = 0.0f;
      } else if (h < A.normed) {
        const bool query = h < A.q;
        float w[8], uu = 0.0f, wu = 0.0f;
        l.turn(g, -1.0f);
#pragma unroll
        for (int i = 0; i < 8; i++) {
          w[i] = g[i] * (query ? gq[i] : gk[i]);
          uu = __builtin_fmaf(u[i], u[i], uu);
          wu = __builtin_fmaf(w[i], u[i], wu);
        }
        uu = lane_sum<G>(uu);
        wu = lane_sum<G>(wu);
        const float f = head_rsqrt(__builtin_fmaf(uu, A.rdim, A.eps));
        const float back = wu * A.rdim * f * f;
        if constexpr (GAIN) {
          if (query) {
#pragma unroll
            for (int i = 0; i < 8; i++) dq[i] = __builtin_fmaf(g[i], u[i] * f, dq[i]);
          } else {
#pragma unroll
            for (int i = 0; i < 8; i++) dk[i] = __builtin_fmaf(g[i], u[i] * f, dk[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < 8; i++) g[i] = f * (w[i] - u[i] * back);
      }
      if (l.in) {
        uint16_t* const to = out + (int64_t)h * A.dim;
        *(u32x2*)(to + l.lo) = pack16<IO>(g);
        *(u32x2*)(to + l.hi) = pack16<IO>(g + 4);
      }
    }
  };

  // A token's heads go by in rounds of U * step; the next round's loads, and the next token's
  // angles, are on their way before a round's heads are taken. The first round is loaded
  // again where it is a token's last: a position that is not a token's is not followed.
  const int rounds = (A.heads + U * step - 1) / (U * step);
  int64_t token = blockIdx.x;
  if (token < A.rows) {
    auto position = [&](int64_t t) { return A.positions[min(t, A.rows - 1)]; };
    int64_t pos = position(token), then = position(token + gridDim.x);
    Heads now, next;
    int chain = 0;
    load(now, token, group);
    l.angles(A, j, pos < 0 ? 0 : pos);
    for (; token < A.rows; token += gridDim.x) {
      const int64_t after = position(token + 2 * (int64_t)gridDim.x);
      ahead.angles(A, j, then < 0 ? 0 : then);
#pragma unroll 1
      for (int k = 0; k < rounds; k++) {
        const bool last = k + 1 == rounds;
        load(next, last ? min(token + gridDim.x, A.rows - 1) : token, last ? group : group + (k + 1) * U * step);
        take(now, token, group + k * U * step, pos >= 0);
        now = next;
      }
      l = ahead;
      pos = then;
      then = after;
      if (GAIN && ++chain == HEAD_CHAIN) {        // a million tokens are no chain of thousands of sums
        flush();
        chain = 0;
      }
    }
  }
  if constexpr (GAIN) {
    flush();
    __shared__ float share[HEAD_THREADS * 8];
    float* const mine = A.part + (int64_t)blockIdx.x * 2 * A.dim;
#pragma unroll
    for (int which = 0; which < 2; which++) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; i++) share[threadIdx.x * 8 + i] = which ? ks[i] : qs[i];
      __syncthreads();
      // lane j of the first group adds up its elements over the groups
      if (group == 0 && l.in) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
          float sum = 0.0f;
          for (int g = 0; g < step; g++) sum += share[(g * G + j) * 8 + i];
          mine[which * A.dim + (i < 4 ? l.lo + i : l.hi + i - 4)] = sum;
        }
      }
    }
  }
}

// dgamma of 4 elements a block from the blocks' shares, in an order that the shape alone decides. Latency: 4.8 us for
// 512 shares of 256 elements.
template <int IO>
__global__ void __launch_bounds__(1024) heads_gain_kernel(const float* part, int shares, int dim, uint16_t* dq, uint16_t* dk) {
  __shared__ double sums[1024];
  const int e = blockIdx.x * 4 + threadIdx.x % 4, r = threadIdx.x / 4;      // 2 * dim is a multiple of 4
  float v[HEAD_MOST / 256];
#pragma unroll
  for (int i = 0; i < HEAD_MOST / 256; i++) v[i] = r + 256 * i < shares ? part[(int64_t)(r + 256 * i) * 2 * dim + e] : 0.0f;
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < HEAD_MOST / 256; i++) sum += (double)v[i];
  sums[threadIdx.x] = sum;
  for (int half = 128; half > 0; half /= 2) {
    __syncthreads();
    if (r < half) sums[threadIdx.x] += sums[threadIdx.x + 4 * half];
  }
  if (r > 0) return;
  sum = sums[threadIdx.x];
  if (e < dim) dq[e] = to_bits16<IO>((float)sum);
  else if (dk) dk[e - dim] = to_bits16<IO>((float)sum);
}

static int head_blocks(const nm_heads_problem_t& p) { return (int)(p.rows < HEAD_MOST ? p.rows : HEAD_MOST); }

template <int IO, bool ACC, bool HALVES>
hipError_t heads_go(const HeadArgs& a, hipStream_t s) {
  auto go = [&](auto kernel, int g) {
    // One token of 144 heads of 512: 4.0 us over nine blocks, 18.0 in one. A block takes a full round of heads:
    // 48 heads of 128 in one block 3.3 us, 3.5 in three.
    const int64_t per = HEAD_U * HEAD_THREADS / g, most = (a.heads + per - 1) / per;
    int64_t split = (256 + a.rows - 1) / a.rows;
    if (split > most) split = most;
    hipLaunchKernelGGL(kernel, dim3((unsigned)a.rows, (unsigned)split), dim3(HEAD_THREADS), 0, s, a);
    return hipGetLastError();
  };
  if (a.dim <= 64) return go(heads_kernel<IO, ACC, HALVES, 8>, 8);
  if (a.dim <= 128) return go(heads_kernel<IO, ACC, HALVES, 16>, 16);
  if (a.dim <= 256) return go(heads_kernel<IO, ACC, HALVES, 32>, 32);
  return go(heads_kernel<IO, ACC, HALVES, 64>, 64);
}

template <int IO, bool HALVES, bool GAIN>
hipError_t heads_back(const HeadArgs& a, int blocks, hipStream_t s) {
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(HEAD_THREADS), 0, s, a);
    return hipGetLastError();
  };
  if (a.dim <= 64) return go(heads_backward_kernel<IO, HALVES, 8, GAIN>);
  if (a.dim <= 128) return go(heads_backward_kernel<IO, HALVES, 16, GAIN>);
  if (a.dim <= 256) return go(heads_backward_kernel<IO, HALVES, 32, GAIN>);
  return go(heads_backward_kernel<IO, HALVES, 64, GAIN>);
}

static HeadArgs head_args(const nm_heads_problem_t& p, const void* gamma_q, const void* gamma_k, const int64_t* positions,
                          const float* table) {
  HeadArgs a = {};
  a.gamma_q = (const uint16_t*)gamma_q;
  a.gamma_k = (const uint16_t*)(p.heads_k ? gamma_k : gamma_q);   // loaded in any case
  a.positions = positions;
  a.table = table;
  a.rows = p.rows;
  a.table_rows = p.table_rows;
  a.q = p.heads_q;
  a.normed = p.heads_q + p.heads_k;
  a.heads = p.heads_q + p.heads_k + p.heads_v;
  a.dim = p.head_dim;
  a.rotary = p.rotary_dim;
  a.eps = p.eps;
  a.zero_rows = p.zero_rows;
  a.rdim = (float)(1.0 / (double)p.head_dim);
  return a;
}

// What both directions check alike.
static nm_status_t head_check(nm_heads_plan_t plan, const void* dX, const void* gamma_q, const void* gamma_k,
                              const int64_t* positions, const float* table) {
  if (!plan) return layer_fail(NM_ERR_INVALID_ARG, "plan is NULL");
  const nm_heads_problem_t& p = plan->p;
  if (!layer_aligned(dX, 16) || !layer_aligned(gamma_q, 16) || !layer_aligned(gamma_k, 16) || !layer_aligned(table, 16) ||
      !layer_aligned(positions, 8))
    return layer_fail(NM_ERR_ALIGN, "device pointers must be 16-byte aligned (the positions 8)");
  if (p.rows == 0) return NM_OK;
  if (!dX || !positions) return layer_fail(NM_ERR_INVALID_ARG, "dX / d_positions is NULL");
  if (!gamma_q || (p.heads_k && !gamma_k)) return layer_fail(NM_ERR_INVALID_ARG, "d_gamma_q / d_gamma_k is NULL");
  if (p.rotary_dim && !table) return layer_fail(NM_ERR_INVALID_ARG, "d_table is NULL");
  return NM_OK;
}

}  // namespace nm

using namespace nm;

extern "C" {

nm_status_t nm_heads_plan_init(nm_heads_plan_t* plan, const nm_heads_problem_t* p) {
  if (!plan) return layer_fail(NM_ERR_INVALID_ARG, "plan is NULL");
  *plan = nullptr;
  if (!p) return layer_fail(NM_ERR_INVALID_ARG, "problem is NULL");
  if (p->type_io != NM_F16 && p->type_io != NM_BF16)
    return layer_fail(NM_ERR_INVALID_ARG, "type_io must be NM_F16 or NM_BF16");
  if (p->type_x != p->type_io && p->type_x != NM_I32)
    return layer_fail(NM_ERR_INVALID_ARG, "type_x must be type_io or NM_I32");
  if (p->pairs != NM_PAIRS_HALVES && p->pairs != NM_PAIRS_NEIGHBOURS)
    return layer_fail(NM_ERR_INVALID_ARG, "pairs must be NM_PAIRS_HALVES or NM_PAIRS_NEIGHBOURS");
  if (!(isfinite(p->eps) && p->eps >= 0.0f)) return layer_fail(NM_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (p->zero_rows != 0 && p->zero_rows != 1) return layer_fail(NM_ERR_INVALID_ARG, "zero_rows must be 0 or 1");
  if (p->rows < 0 || p->rows >= ((int64_t)1 << 24)) return layer_fail(NM_ERR_SHAPE, "rows must be >= 0 and < 2^24");
  if (p->heads_q < 1 || p->heads_k < 0 || p->heads_v < 0 || p->heads_q > 65536 || p->heads_k > 65536 || p->heads_v > 65536)
    return layer_fail(NM_ERR_SHAPE, "heads_q must be 1 to 65536, heads_k and heads_v 0 to 65536");
  if (p->head_dim < 8 || p->head_dim > 512 || p->head_dim % 8)
    return layer_fail(NM_ERR_SHAPE, "head_dim must be a multiple of 8 from 8 to 512");
  if (p->rotary_dim < 0 || p->rotary_dim > p->head_dim || p->rotary_dim % 8)
    return layer_fail(NM_ERR_SHAPE, "rotary_dim must be a multiple of 8 from 0 to head_dim");
  if (p->table_rows < 0 || p->table_rows > ((int64_t)1 << 31) || (p->rotary_dim && p->table_rows < 1))
    return layer_fail(NM_ERR_SHAPE, "table_rows must be 1 to 2^31 (0 allowed without a rotation)");
  const int64_t cols = ((int64_t)p->heads_q + p->heads_k + p->heads_v) * p->head_dim;
  nm_status_t st = layer_rows(p->rows, cols, p->ldx, p->type_x == NM_I32 ? 4 : 2);
  if (st == NM_OK) st = layer_rows(p->rows, cols, p->ldy, 2);
  if (st == NM_OK && p->ldg != 0) st = layer_rows(p->rows, cols, p->ldg, 2);
  if (st != NM_OK) return st;
  nm_heads_plan* pl = new (std::nothrow) nm_heads_plan();
  if (!pl) return layer_fail(NM_ERR_INVALID_ARG, "out of host memory");
  pl->p = *p;
  *plan = pl;
  return layer_fail(NM_OK, "");
}

nm_status_t nm_heads_plan_destroy(nm_heads_plan_t plan) {
  delete plan;
  return NM_OK;
}

nm_status_t nm_heads_workspace_size(nm_heads_plan_t plan, size_t* bytes) {
  if (!plan || !bytes) return layer_fail(NM_ERR_INVALID_ARG, "plan / bytes is NULL");
  *bytes = plan->p.type_x == NM_I32 ? 0 : (size_t)head_blocks(plan->p) * 2 * plan->p.head_dim * sizeof(float);
  return NM_OK;
}

nm_status_t nm_head_norm_rope(nm_heads_plan_t plan, const void* dX, const float* d_row_scale, const float* d_col_scale,
                              const void* d_gamma_q, const void* d_gamma_k, const int64_t* d_positions,
                              const float* d_table, void* dY, void* stream) {
  nm_status_t st = head_check(plan, dX, d_gamma_q, d_gamma_k, d_positions, d_table);
  if (st != NM_OK) return st;
  const nm_heads_problem_t& p = plan->p;
  const bool acc = p.type_x == NM_I32;
  if (!layer_aligned(dY, 16) || !layer_aligned(d_row_scale, 4) || !layer_aligned(d_col_scale, 16))
    return layer_fail(NM_ERR_ALIGN, "device pointers must be 16-byte aligned (the row scales 4)");
  if (p.rows == 0) return NM_OK;
  if (!dY) return layer_fail(NM_ERR_INVALID_ARG, "dY is NULL");
  if ((d_row_scale != nullptr) != acc || (d_col_scale != nullptr) != acc)
    return layer_fail(NM_ERR_INVALID_ARG, "d_row_scale and d_col_scale must be given exactly where x is int32");
  if (dY == dX && (acc || (p.rows > 1 && p.ldx != p.ldy)))
    return layer_fail(NM_ERR_INVALID_ARG, "dY may equal dX only where x is of type_io and ldx == ldy");
  HeadArgs a = head_args(p, d_gamma_q, d_gamma_k, d_positions, d_table);
  a.x = (const uint8_t*)dX;
  a.row_scale = d_row_scale;
  a.col_scale = d_col_scale;
  a.y = (uint16_t*)dY;
  a.ldx = p.ldx;
  a.ldy = p.ldy;
  hipStream_t s = (hipStream_t)stream;
  const bool halves = p.pairs == NM_PAIRS_HALVES;
  hipError_t e;
  if (p.type_io == NM_F16) {
    if (acc) e = halves ? heads_go<DT_F16, true, true>(a, s) : heads_go<DT_F16, true, false>(a, s);
    else e = halves ? heads_go<DT_F16, false, true>(a, s) : heads_go<DT_F16, false, false>(a, s);
  } else {
    if (acc) e = halves ? heads_go<DT_BF16, true, true>(a, s) : heads_go<DT_BF16, true, false>(a, s);
    else e = halves ? heads_go<DT_BF16, false, true>(a, s) : heads_go<DT_BF16, false, false>(a, s);
  }
  return layer_hip(e);
}

nm_status_t nm_head_norm_rope_backward(nm_heads_plan_t plan, const void* dX, const void* d_gamma_q, const void* d_gamma_k,
                                       const int64_t* d_positions, const float* d_table, const void* d_grad_y,
                                       void* d_grad_x, void* d_grad_gamma_q, void* d_grad_gamma_k, void* d_workspace,
                                       void* stream) {
  nm_status_t st = head_check(plan, dX, d_gamma_q, d_gamma_k, d_positions, d_table);
  if (st != NM_OK) return st;
  const nm_heads_problem_t& p = plan->p;
  if (p.type_x == NM_I32) return layer_fail(NM_ERR_UNSUPPORTED, "accumulators have no gradient");
  if (!layer_aligned(d_grad_y, 16) || !layer_aligned(d_grad_x, 16) || !layer_aligned(d_grad_gamma_q, 16) ||
      !layer_aligned(d_grad_gamma_k, 16) || !layer_aligned(d_workspace, 16))
    return layer_fail(NM_ERR_ALIGN, "device pointers must be 16-byte aligned");
  const bool gain = d_grad_gamma_q != nullptr;
  if ((d_grad_gamma_k != nullptr) != (gain && p.heads_k > 0))
    return layer_fail(NM_ERR_INVALID_ARG, "d_grad_gamma_k must be given exactly with d_grad_gamma_q where there are key heads");
  if (p.rows && (!d_grad_y || !d_grad_x)) return layer_fail(NM_ERR_INVALID_ARG, "d_grad_y / d_grad_x is NULL");
  if (p.rows && gain && !d_workspace) return layer_fail(NM_ERR_INVALID_ARG, "the gains' gradients need a workspace");
  const int64_t ldg = p.ldg ? p.ldg : p.ldx;
  if (p.rows > 1 && d_grad_x == d_grad_y && ldg != p.ldy)
    return layer_fail(NM_ERR_INVALID_ARG, "d_grad_x may equal d_grad_y only where ldg == ldy");
  if (p.rows > 1 && d_grad_x == dX && ldg != p.ldx)
    return layer_fail(NM_ERR_INVALID_ARG, "d_grad_x may not equal dX where ldg != ldx");
  HeadArgs a = head_args(p, d_gamma_q, d_gamma_k, d_positions, d_table);
  a.x = (const uint8_t*)dX;
  a.dy = (const uint16_t*)d_grad_y;
  a.y = (uint16_t*)d_grad_x;
  a.part = (float*)d_workspace;
  a.ldx = p.ldx;
  a.ldy = ldg;
  a.lddy = p.ldy;
  hipStream_t s = (hipStream_t)stream;
  const bool f16 = p.type_io == NM_F16, halves = p.pairs == NM_PAIRS_HALVES;
  const int blocks = head_blocks(p);
  hipError_t e = hipSuccess;
  if (blocks) {
    if (f16 && halves) e = gain ? heads_back<DT_F16, true, true>(a, blocks, s) : heads_back<DT_F16, true, false>(a, blocks, s);
    else if (f16) e = gain ? heads_back<DT_F16, false, true>(a, blocks, s) : heads_back<DT_F16, false, false>(a, blocks, s);
    else if (halves) e = gain ? heads_back<DT_BF16, true, true>(a, blocks, s) : heads_back<DT_BF16, true, false>(a, blocks, s);
    else e = gain ? heads_back<DT_BF16, false, true>(a, blocks, s) : heads_back<DT_BF16, false, false>(a, blocks, s);
  }
  if (e == hipSuccess && gain) {
    const dim3 grid((unsigned)(2 * p.head_dim / 4));
    if (f16)
      hipLaunchKernelGGL((heads_gain_kernel<DT_F16>), grid, dim3(1024), 0, s, (const float*)a.part, blocks, p.head_dim,
                         (uint16_t*)d_grad_gamma_q, (uint16_t*)d_grad_gamma_k);
    else
      hipLaunchKernelGGL((heads_gain_kernel<DT_BF16>), grid, dim3(1024), 0, s, (const float*)a.part, blocks, p.head_dim,
                         (uint16_t*)d_grad_gamma_q, (uint16_t*)d_grad_gamma_k);
    e = hipGetLastError();
  }
  return layer_hip(e);
}

}  // extern "C"
