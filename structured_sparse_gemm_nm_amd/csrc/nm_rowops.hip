// Row operators: the RMS norm with the residual's addition and the gated SiLU
// product, from 16-bit rows or an int8 product's int32 accumulators, to 16 bits
// or to 8 bits with one scale a row (formulas in include/nmsparse.h).
//
// Both are one pass over memory: a row is read once into registers, its
// statistics (the sum of squares, the largest magnitude) are reduced over the
// row's threads, and the row is written. Rows too long for that are read twice,
// the second time from the caches. Memory bounds them (figures at row_op_kernel).
#include <math.h>

#include <new>

#include "nm_device.h"
#include "nm_internal.h"

struct nm_rows_plan {
  nm_rows_problem_t p;
};

namespace nm {

struct RowArgs {
  const uint8_t* x;
  const float* row_scale;
  const float* col_scale;
  const uint16_t* residual;
  const uint16_t* gamma;
  uint16_t* h;
  uint8_t* y;
  float* y_scale;
  int64_t rows, cols, ldx, ldr, ldh, ldy;
  float eps, rcols;     // rcols = 1 / cols
};

constexpr int ROW_V = 8;          // columns a thread takes at a time
constexpr int ROW_MOST = 1024;    // threads a row

// 16 bytes at an address that may be off the 16-byte grid (the up half of a
// row starts at any column)
struct __attribute__((packed, aligned(2))) U16x8 { u32x4 v; };
// 8 bytes anywhere: 8-bit rows of fewer than 16 columns start at any byte
struct __attribute__((packed, aligned(1))) U8x8 { u32x2 v; };

// ROW_V columns of a row as they lie in memory. The loads of a row are all on
// their way before the first is used, so they are free of branches: a thread past
// the last whole piece loads the row's last ROW_V columns and shifts its own down.
template <int W> struct RowRaw { u32x4 v[W / 4]; };   // W dwords

template <int W>
__device__ __forceinline__ RowRaw<W> row_raw(const void* at) {
  RowRaw<W> r;
#pragma unroll
  for (int i = 0; i < W / 4; i++) r.v[i] = ((const U16x8*)at)[i].v;
  return r;
}

template <int IO>
__device__ __forceinline__ void unpack16(float (&o)[ROW_V], const RowRaw<4>& r) {
#pragma unroll
  for (int i = 0; i < ROW_V; i++) o[i] = from_bits16<IO>((uint16_t)(r.v[0][i / 2] >> (16 * (i % 2))));
}
template <typename T>
__device__ __forceinline__ void unpack32(T (&o)[ROW_V], const RowRaw<8>& r) {
#pragma unroll
  for (int i = 0; i < ROW_V; i++) {
    const uint32_t bits = r.v[i / 4][i % 4];   // by itself: a bit cast of the element in place reads the first
    o[i] = __builtin_bit_cast(T, bits);
  }
}

// The columns from k on, zeros behind them: 16-bit and 32-bit columns.
__device__ __forceinline__ void row_shift(RowRaw<4>& r, int k) {
  u32x4& v = r.v[0];
  if (k & 4) v = u32x4{v[2], v[3], 0, 0};
  if (k & 2) v = u32x4{v[1], v[2], v[3], 0};
  if (k & 1) v = u32x4{v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16, v[3] >> 16};
}
__device__ __forceinline__ void row_shift(RowRaw<8>& r, int k) {
  u32x4 &a = r.v[0], &b = r.v[1];
  if (k & 4) { a = b; b = u32x4{0, 0, 0, 0}; }
  if (k & 2) { a = u32x4{a[2], a[3], b[0], b[1]}; b = u32x4{b[2], b[3], 0, 0}; }
  if (k & 1) { a = u32x4{a[1], a[2], a[3], b[0]}; b = u32x4{b[1], b[2], b[3], 0}; }
}

// The same columns of a row of fewer than ROW_V; those past the end are 0.
template <int IO>
__device__ __forceinline__ void part16(float (&o)[ROW_V], const uint16_t* row, int64_t c, int64_t cols) {
#pragma unroll
  for (int i = 0; i < ROW_V; i++) o[i] = c + i < cols ? from_bits16<IO>(row[c + i]) : 0.0f;
}
template <typename T>
__device__ __forceinline__ void part32(T (&o)[ROW_V], const T* row, int64_t c, int64_t cols) {
#pragma unroll
  for (int i = 0; i < ROW_V; i++) o[i] = c + i < cols ? row[c + i] : (T)0;
}

// silu(g) * u. For g < 0, with p = exp(-|g| / 2), as (g p / (1 + p p)) (p u): the
// first factor stays under 1 and above fp32's smallest values where exp(-|g|) is
// past them, so a large u meets all of its bits. p is the square of exp(-|g| / 4):
// the exponential instruction flushes subnormal results.
__device__ __forceinline__ float gated(float g, float u) {
  const float root = __builtin_amdgcn_exp2f(-__builtin_fabsf(g) * 0.36067376022224f), p = root * root;
  const float r = __builtin_amdgcn_rcpf(__builtin_fmaf(p, p, 1.0f)), s = g < 0.0f ? p : 1.0f;
  return g * (s * r) * (s * u);
}

template <int IO, bool TAIL>
__device__ __forceinline__ void store16(uint16_t* row, int64_t c, int64_t cols, const float (&v)[ROW_V]) {
  uint16_t o[ROW_V];
#pragma unroll
  for (int i = 0; i < ROW_V; i++) o[i] = to_bits16<IO>(v[i]);
  if (!TAIL || c + ROW_V <= cols) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; i++) w[i] = (uint32_t)o[2 * i] | (uint32_t)o[2 * i + 1] << 16;
    *(u32x4*)(row + c) = w;
  } else {
#pragma unroll
    for (int i = 0; i < ROW_V; i++)
      if (c + i < cols) row[c + i] = o[i];
  }
}

// round(v * r) in 8 bits, r = 127 / (largest magnitude), infinite for a row of
// zeros: NaN converts to 0, the rest is clamped.
template <bool TAIL>
__device__ __forceinline__ void store8(uint8_t* row, int64_t c, int64_t cols, const float (&v)[ROW_V], float r) {
  uint32_t o[ROW_V];
#pragma unroll
  for (int i = 0; i < ROW_V; i++) {
    const float t = __builtin_rintf(v[i] * r);
    o[i] = t != t ? 0u : (uint32_t)(int)__builtin_amdgcn_fmed3f(t, -127.0f, 127.0f) & 0xFFu;
  }
  if (!TAIL || c + ROW_V <= cols) {
    ((U8x8*)(row + c))->v = u32x2{o[0] | o[1] << 8 | o[2] << 16 | o[3] << 24, o[4] | o[5] << 8 | o[6] << 16 | o[7] << 24};
  } else {
#pragma unroll
    for (int i = 0; i < ROW_V; i++)
      if (c + i < cols) row[c + i] = (uint8_t)o[i];
  }
}

// v of another lane of the 16 that lane l shares a row of the wave with
template <int CTRL> __device__ __forceinline__ uint32_t row_dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}
// Sum and largest over 16 lanes, in each of them: neighbours, pairs, then the
// halves of 8 and of 16 mirrored.
__device__ __forceinline__ void reduce16(float& sum, uint32_t& top) {
  auto step = [&](uint32_t s, uint32_t t) {
    sum += __builtin_bit_cast(float, s);
    top = max(top, t);
  };
  const auto bits = [&] { return __builtin_bit_cast(uint32_t, sum); };
  step(row_dpp<0xB1>(bits()), row_dpp<0xB1>(top));
  step(row_dpp<0x4E>(bits()), row_dpp<0x4E>(top));
  step(row_dpp<0x141>(bits()), row_dpp<0x141>(top));
  step(row_dpp<0x140>(bits()), row_dpp<0x140>(top));
}

// Sum and largest magnitude over the block. Magnitudes are compared as the bits
// of |v|, which order as the values do and put a NaN above infinity, so that it
// reaches the scale. Within 16 lanes without LDS, and one read of it for the waves'
// shares: for a single row the time is the sum of such latencies.
__device__ __forceinline__ void row_reduce(float& sum, uint32_t& top) {
  __shared__ u32x2 part[ROW_MOST / 64];
  reduce16(sum, top);
  const int bits = (int)__builtin_bit_cast(uint32_t, sum);
  float s[4];
  uint32_t t = 0;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    s[i] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(bits, 16 * i));
    t = max(t, (uint32_t)__builtin_amdgcn_readlane((int)top, 16 * i));
  }
  sum = (s[0] + s[1]) + (s[2] + s[3]);
  top = t;
  const int n = blockDim.x >> 6, l16 = threadIdx.x & 15;
  if (n == 1) return;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = u32x2{__builtin_bit_cast(uint32_t, sum), top};
  __syncthreads();
  const u32x2 w = l16 < n ? part[l16] : u32x2{0, 0};
  const uint32_t ws = w[0];
  sum = __builtin_bit_cast(float, ws);
  top = w[1];
  reduce16(sum, top);
}

// What a thread loads for ROW_V columns: x (for the activation the gate), the
// second operand (the residual; the up half), and what the rows have in common
// (gamma and, for accumulators, the column scales).
template <int OP, bool ACC> struct RowPiece {
  RowRaw<ACC ? 8 : 4> x;
  RowRaw<OP == NM_ROWS_SWIGLU && ACC ? 8 : 4> second;
  RowRaw<4> gamma;
  RowRaw<8> cs[OP == NM_ROWS_SWIGLU ? 2 : 1];
};

// One block a row. C > 0: the row sits in C pieces of ROW_V columns a thread;
// C = 0: any length, read twice. TAIL: the columns are no whole pieces (one row of
// 4095, 16 bits: 3.8 us, and 4.5 with the last columns loaded one by one; with the
// shifts in every kernel the norm of 4096x16384 takes 96 us, without 83). A row
// gets as many threads as it has pieces, up to 1024, and then two or four pieces each:
// with 256 threads and up to eight pieces, each waiting for its own loads, the norm
// of 8192x4096 took 47 us, the activation 6.6 for 16x11008 and 94 for 4096x11008
// accumulators. Memory bounds it: norm of 8192x4096 in 8 bits 41 us (235 MB, 5.7 TB/s),
// of 4096x4096 accumulators 31.5 (168 MB, 5.3 TB/s), activation of 4096x11008
// accumulators 82 (406 MB, 4.9 TB/s); few rows by latency: 16x11008 4.7 us, one row
// of 4096 2.3.
template <int OP, int IO, bool ACC, bool Y8, int C, bool TAIL>
__global__ void __launch_bounds__(ROW_MOST) row_op_kernel(RowArgs A) {
  constexpr bool NORM = OP == NM_ROWS_RMSNORM;
  typedef RowPiece<OP, ACC> piece_t;
  const int64_t row = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (row >= A.rows) return;
  const float rs = ACC ? A.row_scale[row] : 1.0f;
  const uint8_t* const x = A.x + row * A.ldx * (ACC ? 4 : 2);
  const uint16_t* const res = A.residual ? A.residual + row * A.ldr : nullptr;
  constexpr int XS = ACC ? 4 : 2;

  auto load_scales = [&](piece_t& P, int64_t at) {
    if constexpr (ACC) {
      P.cs[0] = row_raw<8>(A.col_scale + at);
      if constexpr (!NORM) P.cs[1] = row_raw<8>(A.col_scale + A.cols + at);
    }
  };
  // Column scales lie in the caches. With two pieces a thread they come last, or their
  // registers would leave a CU one block (4096x11008 accumulators: 96 us, so 84).
  constexpr bool LATE = ACC && C > 1;
  auto load = [&](piece_t& P, int64_t c) {
    const int64_t at = TAIL ? min(c, A.cols - ROW_V) : c < A.cols ? c : 0;
    P.x = row_raw<ACC ? 8 : 4>(x + at * XS);
    if constexpr (NORM) {
      if (res) P.second = row_raw<4>(res + at);
      P.gamma = row_raw<4>(A.gamma + at);
    } else {
      P.second = row_raw<ACC ? 8 : 4>(x + (A.cols + at) * XS);
    }
    if constexpr (!LATE) load_scales(P, at);
  };
  auto value = [&](float (&o)[ROW_V], const RowRaw<ACC ? 8 : 4>& raw, const RowRaw<8>& scales) {
    if constexpr (ACC) {
      int32_t a[ROW_V];
      float cs[ROW_V];
      unpack32(a, raw);
      unpack32(cs, scales);
#pragma unroll
      for (int i = 0; i < ROW_V; i++) o[i] = (float)a[i] * rs * cs[i];
    } else {
      unpack16<IO>(o, raw);
    }
  };
  auto value_part = [&](float (&o)[ROW_V], int64_t first, int64_t c) {
    if constexpr (ACC) {
      int32_t a[ROW_V];
      float cs[ROW_V];
      part32(a, (const int32_t*)x + first, c, A.cols);
      part32(cs, A.col_scale + first, c, A.cols);
#pragma unroll
      for (int i = 0; i < ROW_V; i++) o[i] = (float)a[i] * rs * cs[i];
    } else {
      part16<IO>(o, (const uint16_t*)x + first, c, A.cols);
    }
  };

  // v before the row's factor, of columns that exist; the norm's u goes to h and into the sum
  auto make = [&](float (&v)[ROW_V], piece_t& P, int64_t c, float& sum, uint32_t& top, bool write_h) {
    float s[ROW_V], g[ROW_V];
    if (!TAIL || A.cols >= ROW_V) {
      if constexpr (LATE) load_scales(P, TAIL ? min(c, A.cols - ROW_V) : c);
      if (TAIL && c + ROW_V > A.cols) {
        const int k = (int)(c + ROW_V - A.cols);
        row_shift(P.x, k);
        if (!NORM || res) row_shift(P.second, k);
        if constexpr (NORM) row_shift(P.gamma, k);
        if constexpr (ACC) {
          row_shift(P.cs[0], k);
          if constexpr (!NORM) row_shift(P.cs[1], k);
        }
      }
      value(v, P.x, P.cs[0]);
      if constexpr (NORM) {
        if (res) unpack16<IO>(s, P.second);
        unpack16<IO>(g, P.gamma);
      } else {
        value(s, P.second, P.cs[1]);
      }
    } else {
      value_part(v, 0, c);
      if constexpr (NORM) {
        if (res) part16<IO>(s, res, c, A.cols);
        part16<IO>(g, A.gamma, c, A.cols);
      } else {
        value_part(s, A.cols, c);
      }
    }
    if constexpr (NORM) {
      if (res) {
#pragma unroll
        for (int i = 0; i < ROW_V; i++) v[i] += s[i];
      }
      if (write_h && A.h) store16<IO, TAIL>(A.h + row * A.ldh, c, A.cols, v);
#pragma unroll
      for (int i = 0; i < ROW_V; i++) {
        sum = __builtin_fmaf(v[i], v[i], sum);
        v[i] *= g[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < ROW_V; i++) v[i] = gated(v[i], s[i]);
    }
    if constexpr (Y8) {
#pragma unroll
      for (int i = 0; i < ROW_V; i++) top = max(top, __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu);
    }
  };

  const int64_t first = (int64_t)threadIdx.x * ROW_V, stride = (int64_t)blockDim.x * ROW_V;
  float sum = 0.0f;
  uint32_t top = 0;
  float v[C > 0 ? C : 1][ROW_V];
  if constexpr (C > 0) {
    piece_t P[C];
    if (!TAIL || A.cols >= ROW_V) {
#pragma unroll
      for (int p = 0; p < C; p++) load(P[p], first + p * stride);
      asm volatile("" ::: "memory");   // and here, not where they are used
    }
#pragma unroll
    for (int p = 0; p < C; p++)
      if (first + p * stride < A.cols) make(v[p], P[p], first + p * stride, sum, top, true);
  } else {
    // Up to 2^17 pieces a thread: a chain of 2^20 equal squares in fp32 is off by up to 0.8 %,
    // so pieces join in 64 bits (2 x 2^24 columns: 2868 us, 2854 with one fp32 chain)
    double total = 0.0;
    for (int64_t c = first; c < A.cols; c += stride) {
      piece_t P;
      float part = 0.0f;
      load(P, c);
      make(v[0], P, c, part, top, false);
      if constexpr (NORM) total += (double)part;
    }
    sum = (float)total;
  }
  float f = 1.0f, r = 0.0f;
  bool small = false;
  if constexpr (NORM || Y8) row_reduce(sum, top);
  if constexpr (NORM) f = 1.0f / __builtin_sqrtf(__builtin_fmaf(sum, A.rcols, A.eps));
  if constexpr (Y8) {
    float a = __builtin_bit_cast(float, top);
    if (threadIdx.x == 0) A.y_scale[row] = a * f / 127.0f;
    small = a < 0x1p-64f;              // 127 / a may be past fp32: both by 2^64
    if (small) a *= 0x1p64f;
    r = 127.0f / a;
  }
  auto write = [&](float (&w)[ROW_V], int64_t c) {
    if constexpr (Y8) {
      if (small) {
#pragma unroll
        for (int i = 0; i < ROW_V; i++) w[i] *= 0x1p64f;
      }
      store8<TAIL>(A.y + row * A.ldy, c, A.cols, w, r);
    } else {
#pragma unroll
      for (int i = 0; i < ROW_V; i++) w[i] *= f;
      store16<IO, TAIL>((uint16_t*)A.y + row * A.ldy, c, A.cols, w);
    }
  };
  if constexpr (C > 0) {
#pragma unroll
    for (int p = 0; p < C; p++)
      if (first + p * stride < A.cols) write(v[p], first + p * stride);
  } else {
    for (int64_t c = first; c < A.cols; c += stride) {
      float unused = 0.0f;
      uint32_t none = 0;
      piece_t P;
      load(P, c);
      make(v[0], P, c, unused, none, true);
      write(v[0], c);
    }
  }
}

template <int OP, int IO, bool ACC, bool Y8, int C>
hipError_t row_go(const RowArgs& a, int threads, hipStream_t s) {
  // a grid dimension holds under 2^32 threads
  const int64_t across = a.rows < ((int64_t)1 << 20) ? a.rows : (int64_t)1 << 20;
  const dim3 grid((unsigned)across, (unsigned)((a.rows + across - 1) / across));
  if (a.cols % ROW_V) hipLaunchKernelGGL((row_op_kernel<OP, IO, ACC, Y8, C, true>), grid, dim3(threads), 0, s, a);
  else hipLaunchKernelGGL((row_op_kernel<OP, IO, ACC, Y8, C, false>), grid, dim3(threads), 0, s, a);
  return hipGetLastError();
}

template <int OP, int IO, bool ACC, bool Y8>
hipError_t row_len(const RowArgs& a, hipStream_t s) {
  const int64_t pieces = (a.cols + ROW_V - 1) / ROW_V;
  auto threads = [&](int c) { return (int)((pieces + 64 * c - 1) / (64 * c)) * 64; };
  if (pieces <= ROW_MOST) return row_go<OP, IO, ACC, Y8, 1>(a, threads(1), s);
  if (pieces <= 2 * ROW_MOST) return row_go<OP, IO, ACC, Y8, 2>(a, threads(2), s);
  if constexpr (!ACC) {
    if (pieces <= 4 * ROW_MOST) return row_go<OP, IO, ACC, Y8, 4>(a, threads(4), s);
  }
  return row_go<OP, IO, ACC, Y8, 0>(a, ROW_MOST, s);
}

template <int OP, int IO>
hipError_t row_types(const nm_rows_problem_t& p, const RowArgs& a, hipStream_t s) {
  const bool y8 = p.type_y == NM_I8;
  if (p.type_x == NM_I32) return y8 ? row_len<OP, IO, true, true>(a, s) : row_len<OP, IO, true, false>(a, s);
  return y8 ? row_len<OP, IO, false, true>(a, s) : row_len<OP, IO, false, false>(a, s);
}

static nm_status_t row_fail(nm_status_t st, const char* msg) {
  try {
    set_error(msg);
  } catch (...) {   // no memory for the message: the status still tells
  }
  return st;
}

static bool row_aligned(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// What nm_rmsnorm and nm_swiglu check alike; NM_OK with go = false: nothing to do.
static nm_status_t row_check(nm_rows_plan_t plan, int op, const void* dX, const float* d_row_scale,
                             const float* d_col_scale, const void* dY, const float* d_y_scale, bool& go) {
  go = false;
  if (!plan) return row_fail(NM_ERR_INVALID_ARG, "plan is NULL");
  const nm_rows_problem_t& p = plan->p;
  if (p.op != op) return row_fail(NM_ERR_INVALID_ARG, "the plan is for the other row operator");
  const bool empty = p.rows == 0 || p.cols == 0, acc = p.type_x == NM_I32, y8 = p.type_y == NM_I8;
  if (!row_aligned(dX) || !row_aligned(d_row_scale) || !row_aligned(d_col_scale) || !row_aligned(dY) ||
      !row_aligned(d_y_scale))
    return row_fail(NM_ERR_ALIGN, "device pointers must be 16-byte aligned");
  if (empty) return NM_OK;
  if (!dX || !dY) return row_fail(NM_ERR_INVALID_ARG, "dX / dY is NULL");
  if ((d_row_scale != nullptr) != acc || (d_col_scale != nullptr) != acc)
    return row_fail(NM_ERR_INVALID_ARG, "d_row_scale and d_col_scale must be given exactly where x is int32");
  if ((d_y_scale != nullptr) != y8)
    return row_fail(NM_ERR_INVALID_ARG, "d_y_scale must be given exactly where y is int8");
  go = true;
  return NM_OK;
}

static RowArgs row_args(const nm_rows_problem_t& p, const void* dX, const float* d_row_scale,
                        const float* d_col_scale, void* dY, float* d_y_scale) {
  RowArgs a = {};
  a.x = (const uint8_t*)dX;
  a.row_scale = d_row_scale;
  a.col_scale = d_col_scale;
  a.y = (uint8_t*)dY;
  a.y_scale = d_y_scale;
  a.rows = p.rows;
  a.cols = p.cols;
  a.ldx = p.ldx;
  a.ldr = p.ldr;
  a.ldh = p.ldh;
  a.ldy = p.ldy;
  a.eps = p.eps;
  a.rcols = (float)(1.0 / (double)p.cols);
  return a;
}

static nm_status_t row_hip(hipError_t e) {
  return e == hipSuccess ? NM_OK : row_fail(NM_ERR_HIP, hipGetErrorString(e));
}

}  // namespace nm

using namespace nm;

extern "C" {

nm_status_t nm_rows_plan_init(nm_rows_plan_t* plan, const nm_rows_problem_t* p) {
  if (!plan) return row_fail(NM_ERR_INVALID_ARG, "plan is NULL");
  *plan = nullptr;
  if (!p) return row_fail(NM_ERR_INVALID_ARG, "problem is NULL");
  if (p->op != NM_ROWS_RMSNORM && p->op != NM_ROWS_SWIGLU)
    return row_fail(NM_ERR_INVALID_ARG, "op must be NM_ROWS_RMSNORM or NM_ROWS_SWIGLU");
  if (p->type_io != NM_F16 && p->type_io != NM_BF16)
    return row_fail(NM_ERR_INVALID_ARG, "type_io must be NM_F16 or NM_BF16");
  if (p->type_x != p->type_io && p->type_x != NM_I32)
    return row_fail(NM_ERR_INVALID_ARG, "type_x must be type_io or NM_I32");
  if (p->type_y != p->type_io && p->type_y != NM_I8)
    return row_fail(NM_ERR_INVALID_ARG, "type_y must be type_io or NM_I8");
  const bool norm = p->op == NM_ROWS_RMSNORM;
  if (norm && !(isfinite(p->eps) && p->eps >= 0.0f))
    return row_fail(NM_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (p->rows < 0 || p->cols < 0) return row_fail(NM_ERR_SHAPE, "rows and cols must be >= 0");
  if (p->rows >= ((int64_t)1 << 24) || p->cols > ((int64_t)1 << 30))
    return row_fail(NM_ERR_SHAPE, "rows must be < 2^24 and cols <= 2^30");
  const int64_t limit = (int64_t)1 << 46, width = norm ? p->cols : 2 * p->cols;
  struct { int64_t ld, len; int es; } lines[4] = {{p->ldx, width, p->type_x == NM_I32 ? 4 : 2},
                                                  {p->ldy, p->cols, p->type_y == NM_I8 ? 1 : 2},
                                                  {p->ldr, p->cols, 2},
                                                  {p->ldh, p->cols, 2}};
  for (int i = 0; i < (norm ? 4 : 2); i++) {
    if (lines[i].ld < (lines[i].len > 0 ? lines[i].len : 1))
      return row_fail(NM_ERR_SHAPE, "leading dimension smaller than the row length");
    if (lines[i].ld > limit || (double)p->rows * (double)lines[i].ld > (double)limit)
      return row_fail(NM_ERR_SHAPE, "matrix too large");
    if (lines[i].len * lines[i].es >= 16 && lines[i].ld * lines[i].es % 16 != 0)
      return row_fail(NM_ERR_ALIGN, "rows of 16 bytes or more must start on 16-byte boundaries (ld * elem size % 16)");
  }
  nm_rows_plan* pl = new (std::nothrow) nm_rows_plan();
  if (!pl) return row_fail(NM_ERR_INVALID_ARG, "out of host memory");
  pl->p = *p;
  *plan = pl;
  return row_fail(NM_OK, "");
}

nm_status_t nm_rows_plan_destroy(nm_rows_plan_t plan) {
  delete plan;
  return NM_OK;
}

nm_status_t nm_rmsnorm(nm_rows_plan_t plan, const void* dX, const float* d_row_scale, const float* d_col_scale,
                       const void* d_residual, const void* d_gamma, void* d_h, void* dY, float* d_y_scale,
                       void* stream) {
  bool go;
  const nm_status_t st = row_check(plan, NM_ROWS_RMSNORM, dX, d_row_scale, d_col_scale, dY, d_y_scale, go);
  if (st != NM_OK) return st;
  if (!row_aligned(d_residual) || !row_aligned(d_gamma) || !row_aligned(d_h))
    return row_fail(NM_ERR_ALIGN, "device pointers must be 16-byte aligned");
  if (!go) return NM_OK;
  if (!d_gamma) return row_fail(NM_ERR_INVALID_ARG, "d_gamma is NULL");
  RowArgs a = row_args(plan->p, dX, d_row_scale, d_col_scale, dY, d_y_scale);
  a.residual = (const uint16_t*)d_residual;
  a.gamma = (const uint16_t*)d_gamma;
  a.h = (uint16_t*)d_h;
  hipStream_t s = (hipStream_t)stream;
  return row_hip(plan->p.type_io == NM_F16 ? row_types<NM_ROWS_RMSNORM, DT_F16>(plan->p, a, s)
                                           : row_types<NM_ROWS_RMSNORM, DT_BF16>(plan->p, a, s));
}

nm_status_t nm_swiglu(nm_rows_plan_t plan, const void* dX, const float* d_row_scale, const float* d_col_scale,
                      void* dY, float* d_y_scale, void* stream) {
  bool go;
  const nm_status_t st = row_check(plan, NM_ROWS_SWIGLU, dX, d_row_scale, d_col_scale, dY, d_y_scale, go);
  if (st != NM_OK || !go) return st;
  const RowArgs a = row_args(plan->p, dX, d_row_scale, d_col_scale, dY, d_y_scale);
  hipStream_t s = (hipStream_t)stream;
  return row_hip(plan->p.type_io == NM_F16 ? row_types<NM_ROWS_SWIGLU, DT_F16>(plan->p, a, s)
                                           : row_types<NM_ROWS_SWIGLU, DT_BF16>(plan->p, a, s));
}

}  // extern "C"
