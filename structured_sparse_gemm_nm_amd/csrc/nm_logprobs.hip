// Log probabilities of given tokens with entropy and the most probable
// alternatives, from rows of logits, and the logits' gradient (formulas in
// include/nmsparse.h).
//
// The forward pass reads a row once: every thread keeps the largest logit it has
// seen and, against it, the sum of exponentials and their weighted sum, and every
// wave keeps a short list of candidates above a threshold that rises. Few long rows
// are cut into slices, whose results a second kernel joins.
#include <float.h>
#include <math.h>

#include <new>

#include "nm_layer.h"

struct nm_logprobs_plan {
  nm_logprobs_problem_t p;
  int slices;             // of a row
  int64_t slice;          // pieces of LP_V columns a slice
};

namespace nm {

constexpr int LP_V = 8;              // columns a thread takes at a time
constexpr int LP_THREADS = 256;
constexpr int LP_TOP = 32;           // most alternatives
constexpr int LP_CAP = 128;          // candidates a wave holds
constexpr int LP_MOST_SLICES = 64;
constexpr int64_t LP_LONGEST = 1 << 17;   // columns a slice: a thread's chain of sums stays under 64 pieces

enum LpType { LP_F16 = 0, LP_BF16 = 1, LP_F32 = 2, LP_I32 = 3 };

struct LpArgs {
  const uint8_t* x;
  const float* row_scale;
  const float* col_scale;
  const int64_t* tokens;
  float* logprob;
  float* entropy;
  float* stats;
  float* top_logprob;
  int64_t* top_index;
  floatx4* part;          // rows x slices: largest, sum, weighted sum
  uint64_t* keys;         // rows x slices x top: the slices' candidates
  int64_t rows, cols, ldx, slice;
  int slices, top;
  float scale, scale2;    // scale2 = scale * log2(e)
};

struct LpBackArgs {
  const uint8_t* x;
  const int64_t* tokens;
  const float* stats;
  const float* entropy;
  const float* g_logprob;
  const float* g_entropy;
  uint8_t* dx;
  int64_t rows, cols, ldx, ldg;
  int parts;              // blocks a row
  float scale;
};

// ---- a wave's candidates -------------------------------------------------------
// A candidate's key: the logit's bits so that they order as the values do, above the
// complement of its column; keys are unique, the lower of two equal logits' columns
// ranks first, and 0 is none.
__device__ __forceinline__ uint64_t lp_key(float x, uint32_t col) {
  uint32_t u = __builtin_bit_cast(uint32_t, x + 0.0f);            // -0 is 0
  u ^= (uint32_t)((int32_t)u >> 31) | 0x80000000u;
  return (uint64_t)u << 32 | (uint32_t)~col;
}
__device__ __forceinline__ float lp_value(uint64_t key) {
  const uint32_t u = (uint32_t)(key >> 32);
  return __builtin_bit_cast(float, u & 0x80000000u ? u ^ 0x80000000u : ~u);
}

// What a wave's lanes wrote to LDS its other lanes read, and write over once all have
// read: a wave's LDS operations keep their order, and the compiler keeps to it.
__device__ __forceinline__ void lp_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

struct LpTop {
  uint64_t* buf;          // LP_CAP keys of this wave, in LDS
  int count, top;
  uint64_t least;         // keys up to this one need not be kept
  float value;            // and logits below this one

  __device__ __forceinline__ void init(uint64_t* b, int k) {
    buf = b;
    count = 0;
    top = k;
    least = 0;
    value = -INFINITY;
  }
  // The top largest, in their order, at the list's start: a key's place is the number
  // of larger ones. Every lane of the wave takes part.
  __device__ __forceinline__ void compact() {
    const int lane = threadIdx.x & 63;
    lp_lds_order();
    const uint64_t a = lane < count ? buf[lane] : 0, b = lane + 64 < count ? buf[lane + 64] : 0;
    int ra = 0, rb = 0;
    for (int i = 0; i < count; i++) {
      const uint64_t k = buf[i];
      ra += k > a;
      rb += k > b;
    }
    lp_lds_order();
    if (a && ra < top) buf[ra] = a;
    if (b && rb < top) buf[rb] = b;
    lp_lds_order();
    if (count >= top) {
      count = top;
      least = buf[top - 1];
      value = lp_value(least);
    }
  }
  // The keys of the lanes for which it holds; every lane of the wave takes part.
  __device__ __forceinline__ void add(uint64_t key, bool holds) {
    holds = holds && key > least;
    uint64_t mask = __ballot(holds);
    if (!mask) return;
    if (count + __popcll(mask) > LP_CAP) {
      compact();
      holds = holds && key > least;
      mask = __ballot(holds);
    }
    if (holds)
      buf[count + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0))] = key;
    count += __popcll(mask);
  }
  // A first threshold from the lanes' largest logits: at least top of them reach the top-th largest.
  __device__ __forceinline__ void estimate(float most) {
    float* const f = (float*)buf;
    const int lane = threadIdx.x & 63;
    lp_lds_order();
    f[lane] = most;
    lp_lds_order();
    int above = 0;
    for (int i = 0; i < 64; i++) above += f[i] > most;
    float v = above < top ? most : INFINITY;
    for (int off = 32; off > 0; off >>= 1) v = fminf(v, __shfl_xor(v, off));
    lp_lds_order();
    value = v;
  }
};

// The waves' lists joined by the first wave, whose list then holds the result. Every
// thread of the block takes part.
__device__ __forceinline__ void lp_top_join(LpTop& t, uint64_t (*lists)[LP_CAP]) {
  const int waves = blockDim.x >> 6, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  t.compact();
  if (waves == 1) return;
  if (lane >= t.count && lane < LP_TOP) t.buf[lane] = 0;
  __syncthreads();
  if (wave == 0) {
    for (int w = 1; w < waves; w += 2) {
      const int from = w + lane / LP_TOP, at = lane % LP_TOP;
      const uint64_t key = from < waves ? lists[from][at] : 0;
      t.add(key, key != 0);
    }
    t.compact();
  }
}

// ---- the running sums ----------------------------------------------------------
// s = sum exp(scale (x - m)), w = sum exp(scale (x - m)) (x - m); m starts at the lowest
// value, so that no difference is that of two infinities.
struct LpSum {
  float m, s, w;
};

// The sums against the larger m2.
__device__ __forceinline__ void lp_shift(LpSum& t, float m2, float scale2) {
  const float d = fmaxf(t.m - m2, -FLT_MAX), f = __builtin_amdgcn_exp2f(d * scale2);
  t.s *= f;
  t.w = __builtin_fmaf(t.s, d, f * t.w);          // no product of a vast d with sums that f makes 0
  t.m = m2;
}

__device__ __forceinline__ float lp_max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));   // NaN reach the sums, not the largest
  return r;
}

// Over the block; every thread takes part and has the result.
__device__ __forceinline__ LpSum lp_join(LpSum t, float scale2) {
  __shared__ floatx4 part[LP_THREADS / 64];
  float m = t.m;
  for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
  lp_shift(t, m, scale2);
  t.s = lane_sum<64>(t.s);
  t.w = lane_sum<64>(t.w);
  const int waves = blockDim.x >> 6;
  if (waves == 1) return t;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = floatx4{t.m, t.s, t.w, 0.0f};
  __syncthreads();
  m = part[0][0];
  for (int i = 1; i < waves; i++) m = fmaxf(m, part[i][0]);
  LpSum r = {m, 0.0f, 0.0f};
  for (int i = 0; i < waves; i++) {
    LpSum o = {part[i][0], part[i][1], part[i][2]};
    lp_shift(o, m, scale2);
    r.s += o.s;
    r.w += o.w;
  }
  return r;
}

// ---- loads ----------------------------------------------------------------------
template <int XT> struct LpRaw { u32x4 v[XT == LP_F16 || XT == LP_BF16 ? 1 : 2]; floatx4 cs[XT == LP_I32 ? 2 : 1]; };
template <int XT> constexpr int LP_SIZE = XT == LP_F16 || XT == LP_BF16 ? 2 : 4;

// A whole piece of LP_V columns from column c on; where it is not whole, the row's first one, not used.
template <int XT>
__device__ __forceinline__ void lp_load(LpRaw<XT>& r, const uint8_t* row, const float* col_scale, int64_t c, bool whole,
                                        int64_t cols) {
  if (cols < LP_V) return;
  const int64_t at = whole ? c : 0;
  const u32x4* p = (const u32x4*)(row + at * LP_SIZE<XT>);
  r.v[0] = p[0];
  if constexpr (LP_SIZE<XT> == 4) r.v[1] = p[1];
  if constexpr (XT == LP_I32) {
    r.cs[0] = *(const floatx4*)(col_scale + at);
    r.cs[1] = *(const floatx4*)(col_scale + at + 4);
  }
}

template <int XT>
__device__ __forceinline__ float lp_one(const uint8_t* row, const float* col_scale, float rs, int64_t c) {
  if constexpr (XT == LP_F16) return from_bits16<DT_F16>(((const uint16_t*)row)[c]);
  else if constexpr (XT == LP_BF16) return from_bits16<DT_BF16>(((const uint16_t*)row)[c]);
  else if constexpr (XT == LP_F32) return ((const float*)row)[c];
  else return (float)((const int32_t*)row)[c] * rs * col_scale[c];
}

template <int XT>
__device__ __forceinline__ void lp_values(float (&x)[LP_V], const LpRaw<XT>& r, float rs) {
#pragma unroll
  for (int i = 0; i < LP_V; i++) {
    if constexpr (XT == LP_F16 || XT == LP_BF16) {
      x[i] = from_bits16<XT == LP_F16 ? DT_F16 : DT_BF16>((uint16_t)(r.v[0][i / 2] >> (16 * (i % 2))));
    } else {
      const uint32_t bits = r.v[i / 4][i % 4];
      if constexpr (XT == LP_F32) x[i] = __builtin_bit_cast(float, bits);
      else x[i] = (float)(int32_t)bits * rs * r.cs[i / 4][i % 4];
    }
  }
}

// ---- results --------------------------------------------------------------------
// By a row's first thread: a row without any weight (every logit -infinity) has log
// probabilities -infinity and entropy 0; a NaN or +infinity has made s NaN.
template <int XT>
__device__ __forceinline__ void lp_write(const LpArgs& A, int64_t row, const LpSum& t) {
  const bool none = t.s == 0.0f;
  const float logs = logf(t.s);
  if (A.stats) {
    A.stats[2 * row] = t.s == t.s ? t.m : NAN;
    A.stats[2 * row + 1] = none ? INFINITY : logs;
  }
  if (A.entropy) A.entropy[row] = none ? 0.0f : logs - A.scale * (t.w / t.s);
  if (A.logprob) {
    const int64_t token = A.tokens[row];
    float lp = 0.0f;
    if (token >= A.cols) {
      lp = NAN;
    } else if (token >= 0) {
      const float x = lp_one<XT>(A.x + row * A.ldx * LP_SIZE<XT>, A.col_scale, XT == LP_I32 ? A.row_scale[row] : 1.0f, token);
      lp = none ? -INFINITY : (x - t.m) * A.scale - logs;
    }
    A.logprob[row] = lp;
  }
}

// By a row's first wave, lane k the k-th alternative.
__device__ __forceinline__ void lp_write_top(const LpArgs& A, int64_t row, const LpSum& t, const LpTop& top) {
  const int lane = threadIdx.x & 63;
  if (lane >= A.top) return;
  const uint64_t key = lane < top.count ? top.buf[lane] : 0;
  const bool known = t.s == t.s && key != 0;
  const float lp = t.s == 0.0f ? -INFINITY : (lp_value(key) - t.m) * A.scale - logf(t.s);
  A.top_logprob[row * A.top + lane] = known ? lp : NAN;
  A.top_index[row * A.top + lane] = known ? (int64_t)(uint32_t)~(uint32_t)key : -1;
}

// One block a slice of a row.
template <int XT, bool ENT, bool TOP>
__global__ void __launch_bounds__(LP_THREADS) lp_kernel(LpArgs A) {
  __shared__ uint64_t lists[TOP ? LP_THREADS / 64 : 1][LP_CAP];
  const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (block >= A.rows * A.slices) return;
  const int64_t row = block / A.slices;
  const int slice = (int)(block % A.slices);
  const uint8_t* const xr = A.x + row * A.ldx * LP_SIZE<XT>;
  const float rs = XT == LP_I32 ? A.row_scale[row] : 1.0f;
  const int64_t begin = slice * A.slice, end = min(begin + A.slice, (A.cols + LP_V - 1) / LP_V);

  LpSum t = {-FLT_MAX, 0.0f, 0.0f};
  LpTop top;
  if constexpr (TOP) top.init(lists[threadIdx.x >> 6], A.top);
  auto whole = [&](int64_t p) { return p < end && (p + 1) * LP_V <= A.cols; };

  auto take = [&](const LpRaw<XT>& raw, int64_t p, bool first) {
    float x[LP_V];
    const int64_t c = p * LP_V;
    if (whole(p)) {
      lp_values<XT>(x, raw, rs);
    } else {
#pragma unroll
      for (int i = 0; i < LP_V; i++)
        x[i] = p < end && c + i < A.cols ? lp_one<XT>(xr, A.col_scale, rs, c + i) : -INFINITY;
    }
    const float most = lp_max3(lp_max3(lp_max3(x[0], x[1], x[2]), x[3], x[4]), lp_max3(x[5], x[6], x[7]), x[7]);
    if (most > t.m) lp_shift(t, most, A.scale2);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < LP_V; i++) {
      const float d = x[i] - t.m, e = __builtin_amdgcn_exp2f(d * A.scale2);
      s += e;
      if constexpr (ENT) t.w = __builtin_fmaf(e, fmaxf(d, -FLT_MAX), t.w);   // e is 0 where d is infinite
    }
    t.s += s;
    if constexpr (TOP) {
      if (first) top.estimate(most);
      if (__any(most >= top.value)) {
#pragma unroll
        for (int i = 0; i < LP_V; i++) {
          const bool holds = x[i] >= top.value && p < end && c + i < A.cols;
          if (__any(holds)) top.add(lp_key(x[i], (uint32_t)(c + i)), holds);
        }
      }
    }
  };

  LpRaw<XT> raw, next;
  int64_t p = begin + threadIdx.x;
  lp_load<XT>(raw, xr, A.col_scale, p * LP_V, whole(p), A.cols);
  for (int64_t b = begin; b < end; b += blockDim.x) {
    p = b + threadIdx.x;
    const int64_t q = p + blockDim.x;
    lp_load<XT>(next, xr, A.col_scale, q * LP_V, whole(q), A.cols);
    take(raw, p, b == begin);
    raw = next;
  }

  t = lp_join(t, A.scale2);
  if constexpr (TOP) lp_top_join(top, lists);
  if (A.slices == 1) {
    if (threadIdx.x == 0) lp_write<XT>(A, row, t);
    if constexpr (TOP) {
      if (threadIdx.x < 64) lp_write_top(A, row, t, top);
    }
  } else {
    if (threadIdx.x == 0) A.part[block] = floatx4{t.m, t.s, t.w, 0.0f};
    if constexpr (TOP) {
      if ((int)threadIdx.x < A.top) A.keys[block * A.top + threadIdx.x] = (int)threadIdx.x < top.count ? top.buf[threadIdx.x] : 0;
    }
  }
}

// The slices of a row joined, one wave a row (a block without alternatives to join is one wave).
template <int XT, bool TOP>
__global__ void __launch_bounds__(LP_THREADS) lp_join_kernel(LpArgs A) {
  __shared__ uint64_t lists[TOP ? LP_THREADS / 64 : 1][LP_CAP];
  const int64_t row = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (row >= A.rows) return;
  LpSum t = {-FLT_MAX, 0.0f, 0.0f};
  if ((int)threadIdx.x < A.slices) {
    const floatx4 v = A.part[row * A.slices + threadIdx.x];
    t = LpSum{v[0], v[1], v[2]};
  }
  LpTop top;
  if constexpr (TOP) {
    top.init(lists[threadIdx.x >> 6], A.top);
    const int total = A.slices * A.top;
    const uint64_t* const keys = A.keys + row * total;
    for (int b = 0; b < total; b += blockDim.x) {         // the slices' first candidates before their second ones
      const int i = b + threadIdx.x;
      const uint64_t key = i < total ? keys[(i % A.slices) * A.top + i / A.slices] : 0;
      top.add(key, key != 0);
    }
  }
  t = lp_join(t, A.scale2);
  if constexpr (TOP) lp_top_join(top, lists);
  if (threadIdx.x == 0) lp_write<XT>(A, row, t);
  if constexpr (TOP) {
    if (threadIdx.x < 64) lp_write_top(A, row, t, top);
  }
}

// dx_i = scale (g [i = t] - p_i (g + h (log p_i + H))), g and h the gradients of the
// row's log probability and entropy H; p_i from the forward's largest and sum. Below
// e^-200 p is 0 in fp32, and the log is held there for infinite ones.
template <int XT, bool ENT>
__global__ void __launch_bounds__(LP_THREADS) lp_backward_kernel(LpBackArgs A) {
  constexpr int U = 4;
  const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (block >= A.rows * A.parts) return;
  const int64_t row = block / A.parts, first = (block % A.parts) * (U * LP_THREADS) + threadIdx.x;
  const uint8_t* const xr = A.x + row * A.ldx * LP_SIZE<XT>;
  uint8_t* const dr = A.dx + row * A.ldg * LP_SIZE<XT>;
  LpRaw<XT> raw[U];
#pragma unroll
  for (int u = 0; u < U; u++) {
    const int64_t c = (first + u * LP_THREADS) * LP_V;
    lp_load<XT>(raw[u], xr, nullptr, c, c + LP_V <= A.cols, A.cols);
  }
  const int64_t token = A.tokens ? A.tokens[row] : -1;
  const float m = A.stats[2 * row], logs = A.stats[2 * row + 1];
  float g = A.g_logprob && token >= 0 ? A.g_logprob[row] : 0.0f;
  if (A.g_logprob && token >= A.cols) g = NAN;
  if (logs == INFINITY) g = 0.0f;                 // no weight in the row
  float h = 0.0f, H = 0.0f;
  if constexpr (ENT) { h = A.g_entropy[row]; H = A.entropy[row]; }
#pragma unroll
  for (int u = 0; u < U; u++) {
    const int64_t c = (first + u * LP_THREADS) * LP_V;
    if (c >= A.cols) break;
    const bool whole = c + LP_V <= A.cols;
    float x[LP_V];
    if (whole) {
      lp_values<XT>(x, raw[u], 1.0f);
    } else {
#pragma unroll
      for (int i = 0; i < LP_V; i++) x[i] = c + i < A.cols ? lp_one<XT>(xr, nullptr, 1.0f, c + i) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < LP_V; i++) {
      const float lp = __builtin_fmaf(x[i] - m, A.scale, -logs);
      const float p = __builtin_amdgcn_exp2f(lp * 1.44269504088896f);
      float k = g;
      if constexpr (ENT) k = __builtin_fmaf(h, fmaxf(lp, -200.0f) + H, g);
      x[i] = p * k;
    }
    const uint64_t at = (uint64_t)(token - c);
#pragma unroll
    for (int i = 0; i < LP_V; i++) x[i] = A.scale * ((at == (uint64_t)i ? g : 0.0f) - x[i]);
    if constexpr (LP_SIZE<XT> == 4) {
      if (whole) {
        ((floatx4*)(dr + c * 4))[0] = floatx4{x[0], x[1], x[2], x[3]};
        ((floatx4*)(dr + c * 4))[1] = floatx4{x[4], x[5], x[6], x[7]};
      } else {
#pragma unroll
        for (int i = 0; i < LP_V; i++)
          if (c + i < A.cols) ((float*)dr)[c + i] = x[i];
      }
    } else {
      uint16_t o[LP_V];
#pragma unroll
      for (int i = 0; i < LP_V; i++) o[i] = to_bits16<XT == LP_F16 ? DT_F16 : DT_BF16>(x[i]);
      if (whole) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; i++) w[i] = (uint32_t)o[2 * i] | (uint32_t)o[2 * i + 1] << 16;
        *(u32x4*)(dr + c * 2) = w;
      } else {
#pragma unroll
        for (int i = 0; i < LP_V; i++)
          if (c + i < A.cols) ((uint16_t*)dr)[c + i] = o[i];
      }
    }
  }
}

// A grid dimension holds under 2^32 threads.
static dim3 lp_grid(int64_t blocks) {
  const int64_t across = blocks < ((int64_t)1 << 20) ? blocks : (int64_t)1 << 20;
  return dim3((unsigned)across, (unsigned)((blocks + across - 1) / across));
}

template <int XT, bool ENT, bool TOP>
hipError_t lp_go(const LpArgs& a, hipStream_t s) {
  const int64_t waves = (a.slice + 63) / 64;
  const dim3 threads((unsigned)(64 * (waves < LP_THREADS / 64 ? waves : LP_THREADS / 64)));
  hipLaunchKernelGGL((lp_kernel<XT, ENT, TOP>), lp_grid(a.rows * a.slices), threads, 0, s, a);
  if (a.slices > 1) {
    hipLaunchKernelGGL((lp_join_kernel<XT, TOP>), lp_grid(a.rows), dim3(TOP ? LP_THREADS : 64), 0, s, a);
  }
  return hipGetLastError();
}

template <int XT>
hipError_t lp_types(const LpArgs& a, hipStream_t s) {
  if (a.top_index) return a.entropy ? lp_go<XT, true, true>(a, s) : lp_go<XT, false, true>(a, s);
  return a.entropy ? lp_go<XT, true, false>(a, s) : lp_go<XT, false, false>(a, s);
}

template <int XT>
hipError_t lp_back(const LpBackArgs& a, hipStream_t s) {
  const dim3 grid = lp_grid(a.rows * a.parts), threads(LP_THREADS);
  if (a.g_entropy) hipLaunchKernelGGL((lp_backward_kernel<XT, true>), grid, threads, 0, s, a);
  else hipLaunchKernelGGL((lp_backward_kernel<XT, false>), grid, threads, 0, s, a);
  return hipGetLastError();
}

}  // namespace nm

using namespace nm;

extern "C" {

nm_status_t nm_logprobs_plan_init(nm_logprobs_plan_t* plan, const nm_logprobs_problem_t* p) {
  if (!plan) return layer_fail(NM_ERR_INVALID_ARG, "plan is NULL");
  *plan = nullptr;
  if (!p) return layer_fail(NM_ERR_INVALID_ARG, "problem is NULL");
  if (p->type_x != NM_F16 && p->type_x != NM_BF16 && p->type_x != NM_F32 && p->type_x != NM_I32)
    return layer_fail(NM_ERR_INVALID_ARG, "type_x must be NM_F16, NM_BF16, NM_F32 or NM_I32");
  if (!(isfinite(p->scale) && p->scale > 0.0f)) return layer_fail(NM_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (p->rows < 0 || p->rows >= ((int64_t)1 << 24)) return layer_fail(NM_ERR_SHAPE, "rows must be >= 0 and < 2^24");
  if (p->cols < 1 || p->cols > ((int64_t)1 << 22)) return layer_fail(NM_ERR_SHAPE, "cols must be 1 to 2^22");
  if (p->top < 0 || p->top > LP_TOP || p->top > p->cols)
    return layer_fail(NM_ERR_SHAPE, "top must be 0 to 32, and at most cols");
  const bool wide = p->type_x == NM_F32 || p->type_x == NM_I32;
  nm_status_t st = layer_rows(p->rows, p->cols, p->ldx, wide ? 4 : 2);
  if (st == NM_OK && p->type_x != NM_I32) st = layer_rows(p->rows, p->cols, p->ldg, wide ? 4 : 2);
  if (st != NM_OK) return st;
  nm_logprobs_plan* pl = new (std::nothrow) nm_logprobs_plan();
  if (!pl) return layer_fail(NM_ERR_INVALID_ARG, "out of host memory");
  pl->p = *p;
  // Slices: four blocks a CU where the row has a whole round of pieces for each.
  const int64_t pieces = (p->cols + LP_V - 1) / LP_V, rounds = (pieces + LP_THREADS - 1) / LP_THREADS;
  int64_t n = p->rows ? (1024 + p->rows - 1) / p->rows : 1;
  if (n > rounds) n = rounds;
  if (n > LP_MOST_SLICES) n = LP_MOST_SLICES;
  const int64_t least = (p->cols + LP_LONGEST - 1) / LP_LONGEST;
  if (n < least) n = least;
  pl->slice = ((rounds + n - 1) / n) * LP_THREADS;
  if (n == 1) pl->slice = pieces;
  pl->slices = (int)((pieces + pl->slice - 1) / pl->slice);
  *plan = pl;
  return layer_fail(NM_OK, "");
}

nm_status_t nm_logprobs_plan_destroy(nm_logprobs_plan_t plan) {
  delete plan;
  return NM_OK;
}

nm_status_t nm_logprobs_workspace_size(nm_logprobs_plan_t plan, size_t* bytes) {
  if (!plan || !bytes) return layer_fail(NM_ERR_INVALID_ARG, "plan / bytes is NULL");
  const size_t parts = (size_t)plan->p.rows * plan->slices;
  *bytes = plan->slices > 1 ? parts * (16 + 8 * (size_t)plan->p.top) : 0;
  return NM_OK;
}

nm_status_t nm_logprobs(nm_logprobs_plan_t plan, const void* dX, const float* d_row_scale, const float* d_col_scale,
                        const int64_t* d_tokens, float* d_logprob, float* d_entropy, float* d_stats, float* d_top_logprob,
                        int64_t* d_top_index, void* d_workspace, void* stream) {
  if (!plan) return layer_fail(NM_ERR_INVALID_ARG, "plan is NULL");
  const nm_logprobs_problem_t& p = plan->p;
  if (!layer_aligned(dX, 16) || !layer_aligned(d_col_scale, 16) || !layer_aligned(d_workspace, 16) ||
      !layer_aligned(d_tokens, 8) || !layer_aligned(d_top_index, 8) || !layer_aligned(d_row_scale, 4) ||
      !layer_aligned(d_logprob, 4) || !layer_aligned(d_entropy, 4) || !layer_aligned(d_stats, 4) ||
      !layer_aligned(d_top_logprob, 4))
    return layer_fail(NM_ERR_ALIGN, "dX, d_col_scale and d_workspace must be 16-byte aligned, the others as their elements");
  if (p.rows == 0) return NM_OK;
  const bool acc = p.type_x == NM_I32;
  if (!dX) return layer_fail(NM_ERR_INVALID_ARG, "dX is NULL");
  if ((d_row_scale != nullptr) != acc || (d_col_scale != nullptr) != acc)
    return layer_fail(NM_ERR_INVALID_ARG, "d_row_scale and d_col_scale must be given exactly where x is int32");
  if ((d_tokens != nullptr) != (d_logprob != nullptr))
    return layer_fail(NM_ERR_INVALID_ARG, "d_tokens and d_logprob must be given together");
  if ((d_top_logprob != nullptr) != (p.top > 0) || (d_top_index != nullptr) != (p.top > 0))
    return layer_fail(NM_ERR_INVALID_ARG, "d_top_logprob and d_top_index must be given exactly where top > 0");
  if (plan->slices > 1 && !d_workspace) return layer_fail(NM_ERR_INVALID_ARG, "the plan needs a workspace");
  LpArgs a = {};
  a.x = (const uint8_t*)dX;
  a.row_scale = d_row_scale;
  a.col_scale = d_col_scale;
  a.tokens = d_tokens;
  a.logprob = d_logprob;
  a.entropy = d_entropy;
  a.stats = d_stats;
  a.top_logprob = d_top_logprob;
  a.top_index = d_top_index;
  if (plan->slices > 1) {
    a.part = (floatx4*)d_workspace;
    a.keys = (uint64_t*)((uint8_t*)d_workspace + (size_t)p.rows * plan->slices * 16);
  }
  a.rows = p.rows;
  a.cols = p.cols;
  a.ldx = p.ldx;
  a.slice = plan->slice;
  a.slices = plan->slices;
  a.top = p.top;
  a.scale = p.scale;
  a.scale2 = (float)((double)p.scale * 1.4426950408889634);
  hipStream_t s = (hipStream_t)stream;
  switch (p.type_x) {
    case NM_F16: return layer_hip(lp_types<LP_F16>(a, s));
    case NM_BF16: return layer_hip(lp_types<LP_BF16>(a, s));
    case NM_F32: return layer_hip(lp_types<LP_F32>(a, s));
    default: return layer_hip(lp_types<LP_I32>(a, s));
  }
}

nm_status_t nm_logprobs_backward(nm_logprobs_plan_t plan, const void* dX, const int64_t* d_tokens, const float* d_stats,
                                 const float* d_entropy, const float* d_grad_logprob, const float* d_grad_entropy,
                                 void* d_grad_x, void* stream) {
  if (!plan) return layer_fail(NM_ERR_INVALID_ARG, "plan is NULL");
  const nm_logprobs_problem_t& p = plan->p;
  if (p.type_x == NM_I32) return layer_fail(NM_ERR_UNSUPPORTED, "accumulators have no gradient");
  if (!layer_aligned(dX, 16) || !layer_aligned(d_grad_x, 16) || !layer_aligned(d_tokens, 8) || !layer_aligned(d_stats, 4) ||
      !layer_aligned(d_entropy, 4) || !layer_aligned(d_grad_logprob, 4) || !layer_aligned(d_grad_entropy, 4))
    return layer_fail(NM_ERR_ALIGN, "dX and d_grad_x must be 16-byte aligned, the others as their elements");
  if (p.rows == 0) return NM_OK;
  if (!dX || !d_stats || !d_grad_x) return layer_fail(NM_ERR_INVALID_ARG, "dX / d_stats / d_grad_x is NULL");
  if (!d_grad_logprob && !d_grad_entropy) return layer_fail(NM_ERR_INVALID_ARG, "no gradient is given");
  if (d_grad_logprob && !d_tokens) return layer_fail(NM_ERR_INVALID_ARG, "d_grad_logprob needs d_tokens");
  if (d_grad_entropy && !d_entropy) return layer_fail(NM_ERR_INVALID_ARG, "d_grad_entropy needs d_entropy");
  LpBackArgs a = {};
  a.x = (const uint8_t*)dX;
  a.tokens = d_tokens;
  a.stats = d_stats;
  a.entropy = d_entropy;
  a.g_logprob = d_grad_logprob;
  a.g_entropy = d_grad_entropy;
  a.dx = (uint8_t*)d_grad_x;
  a.rows = p.rows;
  a.cols = p.cols;
  a.ldx = p.ldx;
  a.ldg = p.ldg;
  a.parts = (int)((p.cols + 4 * LP_THREADS * LP_V - 1) / (4 * LP_THREADS * LP_V));
  a.scale = p.scale;
  hipStream_t s = (hipStream_t)stream;
  switch (p.type_x) {
    case NM_F16: return layer_hip(lp_back<LP_F16>(a, s));
    case NM_BF16: return layer_hip(lp_back<LP_BF16>(a, s));
    default: return layer_hip(lp_back<LP_F32>(a, s));
  }
}

}  // extern "C"
