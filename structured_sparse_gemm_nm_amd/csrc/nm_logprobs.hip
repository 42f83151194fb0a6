// Log probabilities of given tokens with entropy and the most probable
// alternatives, from rows of logits, and the logits' gradient (formulas in
// include/nmsparse.h).
//
// The forward pass reads a row once: every thread keeps the largest logit it has
// seen and, against it, the sum of exponentials and their weighted sum. Few long rows
// are cut into slices, whose results a second kernel joins. The alternatives cost the
// pass nothing: the K largest logits lie among the columns of threads (or of groups of
// threads) whose largest is not below the K-th largest of such, and these columns
// alone are read again.
#include <float.h>
#include <math.h>

#include <new>

#include "nm_layer.h"

struct nm_logprobs_plan {
  nm_logprobs_problem_t p;
  int slices;             // of a row
  int64_t slice;          // pieces of LP_V columns a slice
  int threads, group;     // of a block; see LpArgs
};

namespace nm {

constexpr int LP_V = 8;              // columns a thread takes at a time
constexpr int LP_THREADS = 256;
constexpr int LP_JOIN = 512;         // most threads where the slices' alternatives are joined
constexpr int LP_U = 2;              // pieces a thread takes at a time: 4096 x 131072 508 us, with 1 513; accumulators 60, with 4 77
constexpr int LP_TOP = 32;           // most alternatives
constexpr int LP_ROUNDS = 8;        // of 64 columns that a wave looks through together
constexpr int LP_CAP = 128;          // candidates a wave holds
constexpr int LP_CHUNKS = 2048;      // most groups of columns whose largest are kept for the alternatives
constexpr int LP_ALL = LP_CHUNKS / LP_JOIN;   // of them a thread of the join keeps, all of a row's
constexpr int LP_MOST_SLICES = 32;   // 16 rows of 131072 fp32 logits with 20 alternatives 11.8 us, 64 slices 13.1, 16 12.8
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
  float* largest;         // rows x chunks: the largest logits of the threads' groups
  int64_t rows, cols, ldx, slice;
  int slices, top;
  int group;              // neighbouring threads whose columns are one chunk: 1 or 4
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
  float scale, scale2;    // scale2 = scale * log2(e)
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
    if (lane < 8 && count + lane < LP_CAP) buf[count + lane] = 0;       // they are read eight at a time
    lp_lds_order();
    const uint64_t a = lane < count ? buf[lane] : 0, b = lane + 64 < count ? buf[lane + 64] : 0;
    int ra = 0, rb = 0;
#pragma unroll 1
    for (int i = 0; i < count; i += 8) {
      uint64_t k[8];
#pragma unroll
      for (int j = 0; j < 8; j++) k[j] = buf[i + j];
#pragma unroll
      for (int j = 0; j < 8; j++) {
        ra += k[j] > a;
        rb += k[j] > b;
      }
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
};

// The top-th largest of the lanes' values (-infinity where there are fewer), by the
// same counting; buf holds 64 floats of this wave, in LDS.
__device__ __forceinline__ float lp_nth(float most, int top, float* buf) {
  const int lane = threadIdx.x & 63;
  lp_lds_order();
  buf[lane] = most;
  lp_lds_order();
  int above = 0;
#pragma unroll 4
  for (int i = 0; i < 64; i += 4) {
    const floatx4 o = *(const floatx4*)(buf + i);
    above += (o[0] > most) + (o[1] > most) + (o[2] > most) + (o[3] > most);
  }
  const float v = wave_min(above < top ? most : INFINITY);
  lp_lds_order();
  return v;
}

// The waves' lists joined by the first wave, whose list then holds the result. Every
// thread of the block takes part. Lists that fit one are put behind each other and
// ranked once; longer ones are first cut to their own largest.
template <int W>
__device__ __forceinline__ void lp_top_join(LpTop& t, uint64_t (*lists)[LP_CAP], int* counts) {
  const int waves = blockDim.x >> 6, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  if (waves > 1) {
    if (lane == 0) counts[wave] = t.count;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < W; i++) {
      const int c = i < waves ? counts[i] : 0;
      before += i < wave ? c : 0;
      all += c;
    }
    if (all <= LP_CAP) {
      if (wave > 0) {
        for (int i = lane; i < t.count; i += 64) lists[0][before + i] = t.buf[i];
      }
      __syncthreads();
      t.count = all;
    } else {
      t.compact();
      if (lane >= t.count && lane < LP_TOP) t.buf[lane] = 0;
      __syncthreads();
      if (wave == 0) {
#pragma unroll 1
        for (int w = 1; w < waves; w += 2) {
          const int from = w + lane / LP_TOP, at = lane % LP_TOP;
          const uint64_t key = from < waves ? lists[from][at] : 0;
          t.add(key, key != 0);
        }
      }
    }
  }
  if (wave == 0) t.compact();
}

// ---- the running sums ----------------------------------------------------------
// Exponents are in base 2: of a logit x against the largest m, (x - m) scale2. That takes
// two instructions, u = x scale2 - ms with ms = m scale2 rounded one, and its rounding is the
// same for every logit: u is off by r = m scale2 - ms, which a fused multiply-add gives
// exactly, and the sums are put right when m changes. From |m scale2| = 2^20 on r is too
// large for that and the two instructions are taken.
// s = sum 2^u, w = sum 2^u u; m starts at the lowest value, so that no difference is that of
// two infinities.
struct LpSum {
  float m, s, w;
  float ms, r;            // where the sums are against ms, and else 0
};

__device__ __forceinline__ bool lp_near(float ms) { return __builtin_fabsf(ms) < 0x1p20f; }

// The sums against m2, the largest so far or m itself; against its rounded multiple where `fast` allows it.
__device__ __forceinline__ void lp_shift(LpSum& t, float m2, float scale2, bool fast) {
  const float ms2 = m2 * scale2, r2 = fast && lp_near(ms2) ? __builtin_fmaf(m2, scale2, -ms2) : 0.0f;
  const float d = fmaxf((t.m - m2) * scale2, -FLT_MAX) + (r2 - t.r), f = __builtin_amdgcn_exp2f(d);
  t.s *= f;
  t.w = __builtin_fmaf(t.s, d, f * t.w);          // no product of a vast d with sums that f makes 0
  t.m = m2;
  t.ms = ms2;
  t.r = r2;
}

__device__ __forceinline__ float lp_max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));   // NaN reach the sums, not the largest
  return r;
}

// Over the block; every thread takes part and has the result.
template <int W>
__device__ __forceinline__ LpSum lp_join(LpSum t, float scale2) {
  __shared__ floatx4 part[W];
  float m = wave_max(t.m);
  lp_shift(t, m, scale2, false);
  t.s = wave_sum(t.s);
  t.w = wave_sum(t.w);
  const int waves = blockDim.x >> 6;
  if (waves == 1) return t;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = floatx4{t.m, t.s, t.w, 0.0f};
  __syncthreads();
  floatx4 o[W];
#pragma unroll
  for (int i = 0; i < W; i++) o[i] = part[min(i, waves - 1)];
#pragma unroll
  for (int i = 0; i < W; i++) m = fmaxf(m, o[i][0]);
  LpSum r = {m, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < W; i++) {
    LpSum w = {o[i][0], o[i][1], o[i][2], 0.0f, 0.0f};
    lp_shift(w, m, scale2, false);
    r.s += i < waves ? w.s : 0.0f;
    r.w += i < waves ? w.w : 0.0f;
  }
  return r;
}

// ---- loads ----------------------------------------------------------------------
template <int XT> struct LpRaw { u32x4 v[XT == LP_F16 || XT == LP_BF16 ? 1 : 2]; floatx4 cs[XT == LP_I32 ? 2 : 1]; };
template <int XT> constexpr int LP_SIZE = XT == LP_F16 || XT == LP_BF16 ? 2 : 4;

// A whole piece of LP_V columns from column c on; where it is not whole, the row's first one, not used. STREAM: past
// the caches' reuse.
template <int XT, bool STREAM>
__device__ __forceinline__ void lp_load(LpRaw<XT>& r, const uint8_t* row, const float* col_scale, int64_t c, bool whole,
                                        int64_t cols) {
  if (cols < LP_V) return;
  const int64_t at = whole ? c : 0;
  const u32x4* p = (const u32x4*)(row + at * LP_SIZE<XT>);
#pragma unroll
  for (int i = 0; i < LP_SIZE<XT> / 2; i++) {
    if constexpr (STREAM) r.v[i] = __builtin_nontemporal_load(p + i);
    else r.v[i] = p[i];
  }
  if constexpr (XT == LP_I32) {
    r.cs[0] = *(const floatx4*)(col_scale + at);
    r.cs[1] = *(const floatx4*)(col_scale + at + 4);
  }
}

template <bool STREAM, typename V> __device__ __forceinline__ void lp_store(V* p, V v) {
  if constexpr (STREAM) __builtin_nontemporal_store(v, p);
  else *p = v;
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
// The logit of a row's token, 0 where it has none. Asked for early: two loads, one behind the other.
template <int XT>
__device__ __forceinline__ float lp_given(const LpArgs& A, int64_t row, int64_t& token) {
  token = A.logprob ? A.tokens[row] : -1;
  if (token < 0 || token >= A.cols) return 0.0f;
  return lp_one<XT>(A.x + row * A.ldx * LP_SIZE<XT>, A.col_scale, XT == LP_I32 ? A.row_scale[row] : 1.0f, token);
}

// By one thread of a row's: a row without any weight (every logit -infinity) has log
// probabilities -infinity and entropy 0; a NaN or +infinity has made s NaN.
__device__ __forceinline__ void lp_write(const LpArgs& A, int64_t row, const LpSum& t, int64_t token, float given) {
  const bool none = t.s == 0.0f;
  const float logs = logf(t.s);
  if (A.stats) {
    A.stats[2 * row] = t.s == t.s ? t.m : NAN;
    A.stats[2 * row + 1] = none ? INFINITY : logs;
  }
  if (A.entropy) A.entropy[row] = none ? 0.0f : logs - 0.693147180559945f * (t.w / t.s);
  if (A.logprob) {
    float lp = none ? -INFINITY : (given - t.m) * A.scale - logs;
    if (token < 0) lp = 0.0f;
    if (token >= A.cols) lp = NAN;
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

// What the alternatives of a row need in LDS.
template <int W> struct LpLists {
  alignas(16) uint64_t keys[W][LP_CAP];   // and lp_nth's floats, read four at a time
  int chunks[W][LP_CHUNKS / W];
  int counts[W];
  int tied;               // columns of the bound at the row's start
};

// The alternatives of a row, from the largest logits of its chunks; every thread of the
// block takes part, and the first wave has the result. A chunk is the columns of `group`
// neighbouring threads of lp_kernel's block in a slice: group * LP_V in a row, and as
// many again each `threads` pieces further on. At least top chunks reach the top-th
// largest of a wave's lanes' (each the largest of some chunks), so the top largest logits
// lie in chunks that reach it.
template <int XT, int W>
__device__ __forceinline__ void lp_alternatives(LpTop& t, const LpArgs& A, const uint8_t* xr, float rs, const float* largest,
                                                int threads, LpLists<W>& lds) {
  const int waves = blockDim.x >> 6, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int per = threads / A.group, chunks = per * A.slices;
  float most = -INFINITY;
#pragma unroll 1
  for (int i = lane; i < chunks; i += 8 * 64) {
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; u++) v[u] = largest[min(i + 64 * u, chunks - 1)];
#pragma unroll
    for (int u = 0; u < 8; u++) most = i + 64 * u < chunks ? fmaxf(most, v[u]) : most;
  }
  t.init(lds.keys[wave], A.top);
  const float bound = lp_nth(most, A.top, (float*)lds.keys[wave]);
  t.value = bound;
  // Where half the lanes' largest are the bound itself, most columns may be (logits ruled out with one value): chunks are
  // then looked through for larger ones alone, and the lowest columns of the bound are found by themselves. With this
  // rule and without: 16 rows of 131072 of -infinity, 20 alternatives, 11.0 us and 113, of random logits 12.1 and 11.9;
  // 2048 rows of 32768, 5 alternatives, of -infinity 41.0 and 158, of random logits 41.4 and 38.6.
  const bool flood = __popcll(__ballot(most == bound)) >= 32;
  // this wave's chunks
  int* const list = lds.chunks[wave];
  int count = 0;
#pragma unroll 1
  for (int b = 64 * wave + lane; b - lane < chunks; b += 4 * 64 * waves) {
    float v[4];
#pragma unroll
    for (int u = 0; u < 4; u++) v[u] = largest[min(b + 64 * waves * u, chunks - 1)];
#pragma unroll
    for (int u = 0; u < 4; u++) {
      const int at = b + 64 * waves * u;
      const bool holds = at < chunks && (flood ? v[u] > bound : v[u] >= bound);
      const uint64_t mask = __ballot(holds);
      if (holds) list[count + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0))] = at;
      count += __popcll(mask);
    }
  }
  lp_lds_order();
  // their columns, 64 at a time and LP_ROUNDS such rounds on their way; a chunk's rounds are taken for a power of two
  const int rounds = (int)((A.slice + threads - 1) / threads), lw = 31 - __builtin_clz((unsigned)A.group * LP_V);
  const int le = lw + (rounds > 1 ? 32 - __builtin_clz((unsigned)rounds - 1) : 0), total = count << le;
  const int lp = 31 - __builtin_clz((unsigned)per);        // more slices than one have 256 threads
  auto column = [&](int e, int& piece) -> int64_t {
    const int chunk = e < total ? list[e >> le] : 0, in = e & ((1 << le) - 1), at = in & ((1 << lw) - 1);
    const int first = A.slices == 1 ? 0 : chunk >> lp;
    piece = (in >> lw) * threads + (chunk - (first << lp)) * A.group + at / LP_V;       // of its slice
    return (first * A.slice + piece) * LP_V + at % LP_V;
  };
#pragma unroll 1
  for (int b = lane; b - lane < total; b += LP_ROUNDS * 64) {
    float x[LP_ROUNDS];
    uint32_t hold = 0;
#pragma unroll
    for (int u = 0; u < LP_ROUNDS; u++) {
      const int e = b + 64 * u;
      int piece;
      const int64_t c = column(e, piece);
      const bool there = e < total && piece < A.slice && c < A.cols;
      hold |= (uint32_t)there << u;
      x[u] = lp_one<XT>(xr, A.col_scale, rs, there ? c : 0);       // no branch: all on their way
    }
#pragma unroll
    for (int u = 0; u < LP_ROUNDS; u++)
      if (!(x[u] >= t.value) || (flood && x[u] == bound)) hold &= ~(1u << u);
    while (__any(hold != 0)) {                             // one a lane at a time: few reach the bound
      const int u = __builtin_ctz(hold | 1u << 31);
      float v = x[0];
#pragma unroll
      for (int i = 1; i < LP_ROUNDS; i++) v = u == i ? x[i] : v;
      int piece;
      t.add(lp_key(v, (uint32_t)column(b + 64 * u, piece)), hold != 0);
      hold &= hold - 1;
    }
  }
  if (flood) {
    int found = 0;
    // the columns of the bound among 64 * LP_V from b's on, those from `from` on
    auto look = [&](int64_t b, int64_t from) {
      float x[LP_V];
#pragma unroll
      for (int u = 0; u < LP_V; u++) x[u] = lp_one<XT>(xr, A.col_scale, rs, min(b + 64 * u, A.cols - 1));
#pragma unroll
      for (int u = 0; u < LP_V; u++) {
        const bool holds = b + 64 * u < A.cols && b + 64 * u >= from && x[u] == bound;
        if (found < A.top) t.add(lp_key(x[u], (uint32_t)(b + 64 * u)), holds);
        found += __popcll(__ballot(holds));
      }
    };
    // Mostly the row's start has enough of them, and the first wave is done at once.
    constexpr int64_t START = 2 * 64 * LP_V;
    if (wave == 0) {
#pragma unroll 1
      for (int64_t b = lane; b < START && b - lane < A.cols && found < A.top; b += 64 * LP_V) look(b, 0);
      if (lane == 0) lds.tied = found;
    }
    __syncthreads();
    found = lds.tied;
    // Else every wave takes one of the 64 pieces' places in a round, slice by slice: columns in their order, until it has
    // found as many as can be asked for. Slices whose place does not reach the bound are passed over. 20 alternatives of 4
    // rows of 2^21 f16 logits, the value from three quarters on: 62 us, with one wave over the whole row 2630; of 16 rows
    // of 131072 19 and 152; the value at the start 12.8 and 12.3; at every 997th column 39.9 and 40.8, of 2^21 77 and 58.
    const int places = threads / 64, side = waves / places, place = 64 * (wave % places);
#pragma unroll 1
    for (int slice = wave / places; slice < A.slices && found < A.top; slice += side) {
      if (!__any(largest[slice * per + (place + lane) / A.group] >= bound)) continue;
      int64_t b = (slice * A.slice + place) * LP_V + lane;
#pragma unroll 1
      for (int r = 0; r < rounds && found < A.top && b - lane < A.cols; r++, b += (int64_t)threads * LP_V) look(b, START);
    }
  }
  lp_top_join<W>(t, lds.keys, lds.counts);
}

// One block a slice of a row, LP_U pieces a thread at a time and the next ones on their way.
// Memory bounds it: 4096 x 131072 bf16, 1.07 GB, 199 us, 5.4 TB/s; 2048 x 32768 accumulators,
// 268 MB, 57 us, 4.7 TB/s. A logit costs a multiply-add, an exponential, an addition, half a
// maximum and its conversion, and with the entropy two more: a change of the largest, which
// scales the sums, comes once for LP_U pieces at most and rarely after the first.
template <int XT, bool ENT, bool TOP, bool STREAM>
__global__ void __launch_bounds__(LP_THREADS) lp_kernel(LpArgs A) {
  const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (block >= A.rows * A.slices) return;
  const int64_t row = A.slices == 1 ? block : block / A.slices;
  const int slice = (int)(block - row * A.slices);
  const uint8_t* const xr = A.x + row * A.ldx * LP_SIZE<XT>;
  const float rs = XT == LP_I32 ? A.row_scale[row] : 1.0f;
  const int begin = (int)(slice * A.slice), end = (int)min(begin + A.slice, (A.cols + LP_V - 1) / LP_V);
  const int full = min(end, (int)(A.cols / LP_V));        // pieces that are whole
  int64_t token = -1;
  const float given = A.slices == 1 ? lp_given<XT>(A, row, token) : 0.0f;

  LpSum t = {-FLT_MAX, 0.0f, 0.0f, -FLT_MAX, 0.0f};
  float mine = -INFINITY;                         // the thread's largest: t.m, or below it where that is none's
  auto take = [&](const LpRaw<XT> (&raw)[LP_U], int b) {
    float x[LP_U][LP_V], most = -INFINITY;
#pragma unroll
    for (int u = 0; u < LP_U; u++) {
      const int at = b + u * (int)blockDim.x + (int)threadIdx.x;
      if (u > 0 && b + u * (int)blockDim.x >= end) break;
      if (at < full) {
        lp_values<XT>(x[u], raw[u], rs);
      } else {
#pragma unroll
        for (int i = 0; i < LP_V; i++)
          x[u][i] = at < end && at * LP_V + i < A.cols ? lp_one<XT>(xr, A.col_scale, rs, at * LP_V + i) : -INFINITY;
      }
#pragma unroll
      for (int i = 0; i < LP_V; i += 2) most = lp_max3(most, x[u][i], x[u][i + 1]);
    }
    if constexpr (TOP) mine = fmaxf(mine, most);
    if (most > t.m) lp_shift(t, most, A.scale2, true);
    const bool near = lp_near(t.ms);
#pragma unroll
    for (int u = 0; u < LP_U; u++) {
      if (u > 0 && b + u * (int)blockDim.x >= end) break;
      float s = 0.0f;
      auto sums = [&](auto exponent) {
#pragma unroll
        for (int i = 0; i < LP_V; i++) {
          const float d = exponent(x[u][i]), e = __builtin_amdgcn_exp2f(d);
          s += e;
          if constexpr (ENT) t.w = __builtin_fmaf(e, fmaxf(d, -200.0f), t.w);   // e is 0 below that, infinite d among them
        }
      };
      if (near) sums([&](float v) { return __builtin_fmaf(v, A.scale2, -t.ms); });
      else sums([&](float v) { return (v - t.m) * A.scale2; });
      t.s += s;
    }
  };
  auto load = [&](LpRaw<XT> (&raw)[LP_U], int b) {
#pragma unroll
    for (int u = 0; u < LP_U; u++) {
      const int at = b + u * (int)blockDim.x + (int)threadIdx.x;
      lp_load<XT, STREAM>(raw[u], xr, A.col_scale, (int64_t)at * LP_V, at < full, A.cols);
    }
  };

  LpRaw<XT> raw[LP_U], next[LP_U];
  const int step = LP_U * (int)blockDim.x;
  load(raw, begin);
#pragma unroll 1
  for (int b = begin; b < end; b += 2 * step) {
    if (b + step < end) load(next, b + step);
    take(raw, b);
    if (b + step >= end) break;
    if (b + 2 * step < end) load(raw, b + 2 * step);
    take(next, b + step);
  }

  if (A.slices == 1) {
    if constexpr (TOP) {
      __shared__ LpLists<LP_THREADS / 64> lds;
      __shared__ float largest[LP_THREADS];
      largest[threadIdx.x] = mine;
      t = lp_join<LP_THREADS / 64>(t, A.scale2);
      __syncthreads();
      LpTop top;
      lp_alternatives<XT>(top, A, xr, rs, largest, blockDim.x, lds);
      if (threadIdx.x < 64) lp_write_top(A, row, t, top);
    } else {
      t = lp_join<LP_THREADS / 64>(t, A.scale2);
    }
    if (threadIdx.x == blockDim.x - 1) lp_write(A, row, t, token, given);    // the first wave has the alternatives
  } else {
    if constexpr (TOP) {
      if (A.group == 4) {
        mine = fmaxf(mine, lane_dpp<0xB1>(mine));
        mine = fmaxf(mine, lane_dpp<0x4E>(mine));
      }
      if (threadIdx.x % A.group == 0) A.largest[(block * LP_THREADS + threadIdx.x) / A.group] = mine;
    }
    t = lp_join<LP_THREADS / 64>(t, A.scale2);
    if (threadIdx.x == 0) A.part[block] = floatx4{t.m, t.s, t.w, 0.0f};
  }
}

// The slices of a row joined; one wave a row where there are no alternatives. Latency bounds it:
// 6.0 us for 32003 logits and 5 alternatives, about 8 for 16 rows of 131072 and 20 (the largest of
// the chunks, their columns, the lists: one behind the other).
template <int XT, bool TOP>
__global__ void __launch_bounds__(LP_JOIN) lp_join_kernel(LpArgs A) {
  const int64_t row = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (row >= A.rows) return;
  int64_t token;
  const float given = lp_given<XT>(A, row, token);
  LpSum t = {-FLT_MAX, 0.0f, 0.0f, -FLT_MAX, 0.0f};
  if ((int)threadIdx.x < A.slices) {
    const floatx4 v = A.part[row * A.slices + threadIdx.x];
    t = LpSum{v[0], v[1], v[2], -FLT_MAX, 0.0f};
  }
  if constexpr (TOP) {
    __shared__ LpLists<LP_JOIN / 64> lds;
    __shared__ float largest[LP_CHUNKS];
    const int chunks = A.slices * (LP_THREADS / A.group);
    const float* const from = A.largest + row * chunks;
    float v[LP_ALL];
#pragma unroll
    for (int i = 0; i < LP_ALL; i++) v[i] = from[min((int)threadIdx.x + i * (int)blockDim.x, chunks - 1)];
#pragma unroll
    for (int i = 0; i < LP_ALL; i++) largest[threadIdx.x + i * blockDim.x] = v[i];
    t = lp_join<LP_JOIN / 64>(t, A.scale2);
    __syncthreads();
    LpTop top;
    lp_alternatives<XT>(top, A, A.x + row * A.ldx * LP_SIZE<XT>, XT == LP_I32 ? A.row_scale[row] : 1.0f, largest, LP_THREADS, lds);
    if (threadIdx.x < 64) lp_write_top(A, row, t, top);
  } else {
    t = lp_join<LP_JOIN / 64>(t, A.scale2);
  }
  if (threadIdx.x == blockDim.x - 1) lp_write(A, row, t, token, given);      // the first wave has the alternatives
}

// dx_i = scale (g [i = t] - p_i (g + h (log p_i + H))), g and h the gradients of the
// row's log probability and entropy H; p_i from the forward's largest and sum. Below
// 2^-300 p is 0 in fp32, and the log is held there for infinite ones. Memory bounds it:
// 4096 x 131072 bf16, 2.1 GB, 343 us, 6.3 TB/s.
template <int XT, bool ENT, bool STREAM>
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
    lp_load<XT, STREAM>(raw[u], xr, nullptr, c, c + LP_V <= A.cols, A.cols);
  }
  const int64_t token = A.tokens ? A.tokens[row] : -1;
  const float m = A.stats[2 * row], logs = A.stats[2 * row + 1];
  float g = A.g_logprob && token >= 0 ? A.g_logprob[row] : 0.0f;
  if (token >= A.cols && g != 0.0f) g = NAN;
  if (logs == INFINITY) g = 0.0f;                 // no weight in the row
  float h = 0.0f, H = 0.0f;
  if constexpr (ENT) { h = A.g_entropy[row]; H = A.entropy[row]; }
  const bool none = g == 0.0f && h == 0.0f;       // zeros, also where the logits are NaN
  const float own = A.scale * g, g2 = none ? 0.0f : -A.scale * __builtin_fmaf(h, H, g), h2 = -A.scale * h * 0.693147180559945f;
  const float logs2 = logs * 1.44269504088896f;
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
    // with the token's own term where it is: - scale (g + h (log p + H)) p, its logs in base 2
#pragma unroll
    for (int i = 0; i < LP_V; i++) {
      const float lp = none ? -INFINITY : __builtin_fmaf(x[i] - m, A.scale2, -logs2), p = __builtin_amdgcn_exp2f(lp);
      x[i] = p * (ENT ? __builtin_fmaf(h2, fmaxf(lp, -300.0f), g2) : g2);
    }
    const uint64_t at = (uint64_t)(token - c);
    if (at < LP_V) {
#pragma unroll
      for (int i = 0; i < LP_V; i++) x[i] += at == (uint64_t)i ? own : 0.0f;
    }
    if constexpr (LP_SIZE<XT> == 4) {
      if (whole) {
        lp_store<STREAM>((floatx4*)(dr + c * 4), floatx4{x[0], x[1], x[2], x[3]});
        lp_store<STREAM>((floatx4*)(dr + c * 4) + 1, floatx4{x[4], x[5], x[6], x[7]});
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
        lp_store<STREAM>((u32x4*)(dr + c * 2), w);
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

// Logits that the caches do not hold until they are read again (256 MB on this card) are read past them, and so is
// their gradient written: 4096 x 131072 bf16 (1 GB) forward and backward 566 us without, 522 with loads and 509 with
// stores past them; 2048 x 32768 accumulators (268 MB) 60 us without and 66 with. bf16 rows of 131072, forward and
// backward, without and with: 512 MB 308 and 278, 640 MB 392 and 364; below the edge, which the accumulators set, 450 MB
// 273 and 246, 384 MB 228 and 206, 275 MB 167 and 151.
static bool lp_streams(int64_t rows, int64_t cols, int size) { return rows * cols * size >= (int64_t)1 << 29; }

// Half the threads where that keeps the chunks' list: 32003 f16 logits with 5 alternatives 9.7 us, 10.3 with all; but 16
// rows of 131072 12.4 with half where there are 2048 chunks, 11.8 with all, and 1024 threads are slower for both (12.8, 15.5).
static unsigned lp_join_threads(const LpArgs& a) {
  return a.slices * (LP_THREADS / a.group) <= LP_ALL * LP_JOIN / 2 ? LP_JOIN / 2 : LP_JOIN;
}

template <int XT, bool ENT, bool TOP>
hipError_t lp_go(const LpArgs& a, int threads, hipStream_t s) {
  const dim3 grid = lp_grid(a.rows * a.slices);
  if (lp_streams(a.rows, a.cols, LP_SIZE<XT>)) hipLaunchKernelGGL((lp_kernel<XT, ENT, TOP, true>), grid, dim3((unsigned)threads), 0, s, a);
  else hipLaunchKernelGGL((lp_kernel<XT, ENT, TOP, false>), grid, dim3((unsigned)threads), 0, s, a);
  if (a.slices > 1) hipLaunchKernelGGL((lp_join_kernel<XT, TOP>), lp_grid(a.rows), dim3(TOP ? lp_join_threads(a) : 64), 0, s, a);
  return hipGetLastError();
}

template <int XT>
hipError_t lp_types(const LpArgs& a, int threads, hipStream_t s) {
  if (a.top_index) return a.entropy ? lp_go<XT, true, true>(a, threads, s) : lp_go<XT, false, true>(a, threads, s);
  return a.entropy ? lp_go<XT, true, false>(a, threads, s) : lp_go<XT, false, false>(a, threads, s);
}

template <int XT>
hipError_t lp_back(const LpBackArgs& a, hipStream_t s) {
  const dim3 grid = lp_grid(a.rows * a.parts), threads(LP_THREADS);
  if (lp_streams(a.rows, a.cols, LP_SIZE<XT>)) {
    if (a.g_entropy) hipLaunchKernelGGL((lp_backward_kernel<XT, true, true>), grid, threads, 0, s, a);
    else hipLaunchKernelGGL((lp_backward_kernel<XT, false, true>), grid, threads, 0, s, a);
  } else {
    if (a.g_entropy) hipLaunchKernelGGL((lp_backward_kernel<XT, true, false>), grid, threads, 0, s, a);
    else hipLaunchKernelGGL((lp_backward_kernel<XT, false, false>), grid, threads, 0, s, a);
  }
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
  if (!(p->scale > 0.0f && p->scale <= 0x1p127f)) return layer_fail(NM_ERR_INVALID_ARG, "scale must be > 0 and at most 2^127");
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
  // Slices: four blocks a CU where the row has a whole round of pieces for each. 256 rows of 131072 fp32 logits 33.6 us;
  // with two blocks a CU 36.1, with one 46.3, with eight 33.2; 64 rows 17.7, 17.0, 19.2, 17.0.
  const int64_t pieces = (p->cols + LP_V - 1) / LP_V, rounds = (pieces + LP_THREADS - 1) / LP_THREADS;
  int64_t n = p->rows ? (1024 + p->rows - 1) / p->rows : 1;
  if (n > rounds) n = rounds;
  if (n > LP_MOST_SLICES) n = LP_MOST_SLICES;
  const int64_t least = (p->cols + LP_LONGEST - 1) / LP_LONGEST;
  if (n < least) n = least;
  pl->slice = n == 1 ? pieces : ((rounds + n - 1) / n) * LP_THREADS;
  pl->slices = (int)((pieces + pl->slice - 1) / pl->slice);
  pl->threads = pl->slices > 1 || pieces >= LP_THREADS ? LP_THREADS : (int)((pieces + 63) / 64 * 64);
  const int64_t all = (int64_t)pl->slices * pl->threads;
  pl->group = all <= LP_CHUNKS ? 1 : 4;                    // LP_MOST_SLICES blocks of LP_THREADS are 4 LP_CHUNKS
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
  *bytes = plan->slices > 1 ? parts * (16 + (plan->p.top ? 4 * (size_t)(LP_THREADS / plan->group) : 0)) : 0;
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
    a.largest = (float*)((uint8_t*)d_workspace + (size_t)p.rows * plan->slices * 16);
  }
  a.rows = p.rows;
  a.cols = p.cols;
  a.ldx = p.ldx;
  a.slice = plan->slice;
  a.slices = plan->slices;
  a.group = plan->group;
  a.top = p.top;
  a.scale = p.scale;
  a.scale2 = (float)((double)p.scale * 1.4426950408889634);
  hipStream_t s = (hipStream_t)stream;
  switch (p.type_x) {
    case NM_F16: return layer_hip(lp_types<LP_F16>(a, plan->threads, s));
    case NM_BF16: return layer_hip(lp_types<LP_BF16>(a, plan->threads, s));
    case NM_F32: return layer_hip(lp_types<LP_F32>(a, plan->threads, s));
    default: return layer_hip(lp_types<LP_I32>(a, plan->threads, s));
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
  if (d_grad_x == dX && p.rows > 1 && p.ldg != p.ldx)
    return layer_fail(NM_ERR_INVALID_ARG, "d_grad_x may equal dX only where ldg == ldx");
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
  a.scale2 = (float)((double)p.scale * 1.4426950408889634);
  hipStream_t s = (hipStream_t)stream;
  switch (p.type_x) {
    case NM_F16: return layer_hip(lp_back<LP_F16>(a, s));
    case NM_BF16: return layer_hip(lp_back<LP_BF16>(a, s));
    default: return layer_hip(lp_back<LP_F32>(a, s));
  }
}

}  // extern "C"
