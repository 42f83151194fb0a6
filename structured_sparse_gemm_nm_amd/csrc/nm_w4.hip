// 4-bit weight product: plan validation, argument checks, the packing kernels
// and dispatch. The product's kernels are in nm_w4_kernels.h.
#include <new>

#include "nm_device.h"
#include "nm_w4.h"

namespace nm {

static nm_status_t w4_fail(nm_status_t st, const char* msg) {
  try {
    set_error(msg);
  } catch (...) {   // no memory for the message: the status still tells
  }
  return st;
}

static nm_status_t w4_hip(hipError_t e) {
  return e == hipSuccess ? NM_OK : w4_fail(NM_ERR_HIP, hipGetErrorString(e));
}

static bool w4_aligned(const void* p) { return ((uintptr_t)p & 15u) == 0; }

static const int64_t kW4MaxK = (int64_t)1 << 20;   // keeps offsets inside a row of x and of a row tile's codes in 32 bits
static const int64_t kW4MaxM = (int64_t)1 << 24;   // the grid: m / 16 blocks of up to 512 threads, under 2^32 threads
static const int64_t kW4MaxN = (int64_t)1 << 20;   // 48 columns a grid row, under 2^16 grid rows

// One block a tile of 16 rows x 128 kept values, one thread a dword of eight
// codes: thread 4 l + d writes dword d of lane l, so the writes are contiguous.
// Values past the end of a row get the code of zero (the zero point). 32768x32768:
// 0.5 ms (537 MB each way); with the codes taken one by one 1.9.
struct W4PackArgs {
  const uint8_t* codes;
  const uint8_t* zeros;
  const uint8_t* meta;
  uint8_t* out_codes;
  uint8_t* out_meta;
  int64_t m, kept, code_ld, meta_ld, tiles, row_tiles, groups;
  int x_type;            // nm_dtype_t of the activations the codes will meet
};

struct __attribute__((packed, aligned(1))) U32 { uint32_t v; };   // rows of codes start anywhere

// nibbles 0, 2, 4, 6 of w, next to each other; and back, from the lower 16 bits
__device__ __forceinline__ uint32_t nibbles_even(uint32_t w) {
  w &= 0x0F0F0F0Fu;
  w = (w | w >> 4) & 0x00FF00FFu;
  return (w | w >> 8) & 0xFFFFu;
}
__device__ __forceinline__ uint32_t nibbles_apart(uint32_t w) {
  w = (w | w << 8) & 0x00FF00FFu;
  return (w | w << 4) & 0x0F0F0F0Fu;
}

__global__ void __launch_bounds__(256) w4_pack_kernel(W4PackArgs A) {
  const int lane = threadIdx.x >> 2, d = threadIdx.x & 3, l16 = lane & 15, q = lane >> 4;
  for (int64_t b = blockIdx.x; b < A.tiles * A.row_tiles; b += gridDim.x) {
    const int64_t rt = b / A.tiles, t = b % A.tiles;
    const int64_t row = rt * 16 + l16;
    const int64_t p0 = t * 128 + (A.x_type == NM_I8 ? (d >> 1) * 64 + q * 16 + (d & 1) * 8 : d * 32 + q * 8);
    uint32_t w = 0x88888888u;   // eight codes in order
    if (row < A.m) {
      const uint8_t* src = A.codes + row * A.code_ld + p0 / 2;
      if (p0 + 8 <= A.kept) {
        w = ((const U32*)src)->v;
      } else {
        const uint32_t zero = A.zeros ? A.zeros[row * A.groups + A.groups - 1] & 15u : 8u;
        w = 0;
        for (int i = 0; i < 8; i++)
          w |= (p0 + i < A.kept ? (uint32_t)(src[i / 2] >> (4 * (i & 1))) & 15u : zero) << (4 * i);
      }
    }
    // the orders that the kernels unpack (nm_w4_kernels.h)
    if (A.x_type == NM_F16) {
      w = nibbles_even(w) | nibbles_even(w >> 4) << 16;
    } else {
      w = nibbles_apart(w & 0xFFFFu) | nibbles_apart(w >> 16) << 4;
      if (!A.zeros) w ^= 0x88888888u;
    }
    ((uint32_t*)(A.out_codes + b * 1024))[threadIdx.x] = w;
    if (A.meta && threadIdx.x < 128) {
      const int ml = threadIdx.x >> 1, h = threadIdx.x & 1, mq = ml >> 4;
      const int64_t mrow = rt * 16 + (ml & 15);
      uint32_t v = 0;
      if (mrow < A.m) {
        for (int i = 0; i < 4; i++) {   // byte i of the dword: four kept values' offsets
          const int64_t p = t * 128 + (A.x_type == NM_I8 ? h * 64 + mq * 16 + i * 4
                                                         : (2 * h + (i >> 1)) * 32 + mq * 8 + (i & 1) * 4);
          if (p < A.kept) v |= (uint32_t)A.meta[mrow * A.meta_ld + p / 4] << (8 * i);
        }
      }
      ((uint32_t*)(A.out_meta + b * 512))[threadIdx.x] = v;
    }
  }
}

// scales [m][groups] -> [row tile][group][16 rows], zeros likewise; rows past m get 0.
__global__ void __launch_bounds__(256) w4_pack_scales_kernel(const uint16_t* scales, const uint8_t* zeros,
                                                             uint16_t* out_scales, uint8_t* out_zeros, int64_t m,
                                                             int64_t groups, int64_t total) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i % 16, g = i / 16 % groups, row = i / 16 / groups * 16 + r;
    out_scales[i] = row < m ? scales[row * groups + g] : (uint16_t)0;
    if (zeros) out_zeros[i] = row < m ? (uint8_t)(zeros[row * groups + g] & 15u) : (uint8_t)0;
  }
}

}  // namespace nm

using namespace nm;

extern "C" {

nm_status_t nm_w4_plan_init(nm_w4_plan_t* plan, const nm_w4_problem_t* p) {
  if (!plan) return w4_fail(NM_ERR_INVALID_ARG, "plan is NULL");
  *plan = nullptr;
  if (!p) return w4_fail(NM_ERR_INVALID_ARG, "problem is NULL");
  if (p->m < 0 || p->n < 0 || p->k < 0) return w4_fail(NM_ERR_SHAPE, "m, n, k must be >= 0");
  if (p->m > kW4MaxM || p->n > kW4MaxN || p->k > kW4MaxK)
    return w4_fail(NM_ERR_SHAPE, "4-bit product: m <= 2^24, n <= 2^20 and k <= 2^20");
  if (p->type_y != NM_F16 && p->type_y != NM_BF16)
    return w4_fail(NM_ERR_INVALID_ARG, "type_y (scales and y) must be NM_F16 or NM_BF16");
  if (p->type_x != p->type_y && p->type_x != NM_I8)
    return w4_fail(NM_ERR_INVALID_ARG, "type_x must be type_y or NM_I8");
  if ((p->sparse != 0 && p->sparse != 1) || (p->zeros != 0 && p->zeros != 1))
    return w4_fail(NM_ERR_INVALID_ARG, "sparse and zeros must be 0 or 1");
  if (p->sparse && p->k % 4 != 0) return w4_fail(NM_ERR_SHAPE, "2:4 weights: k must be a multiple of 4");
  const int64_t step = (p->type_x == NM_I8 ? 64 : 32) * (p->sparse ? 2 : 1);
  if (p->group < 0 || p->group % step != 0)
    return w4_fail(NM_ERR_SHAPE, "group must be 0 (one scale a row) or a multiple of the matrix instruction's k: "
                                 "32 (16-bit x) or 64 (8-bit x), twice that for 2:4 weights");
  if (p->ldx < (p->k > 0 ? p->k : 1) || p->ldy < (p->m > 0 ? p->m : 1))
    return w4_fail(NM_ERR_SHAPE, "ldx must be >= k and ldy >= m");
  const int64_t ex = p->type_x == NM_I8 ? 1 : 2, limit = (int64_t)1 << 46;
  if (p->ldx > limit || p->ldy > limit || (double)p->n * (double)p->ldx > (double)limit ||
      (double)p->n * (double)p->ldy > (double)limit)
    return w4_fail(NM_ERR_SHAPE, "matrix too large");
  if ((p->k * ex >= 16 && p->ldx * ex % 16 != 0) || (p->m * 2 >= 16 && p->ldy * 2 % 16 != 0))
    return w4_fail(NM_ERR_ALIGN, "rows of 16 bytes or more must start on 16-byte boundaries (ld * elem size % 16)");

  nm_w4_plan* pl = new (std::nothrow) nm_w4_plan();
  if (!pl) return w4_fail(NM_ERR_INVALID_ARG, "out of host memory");
  pl->p = *p;
  const int64_t kept = p->sparse ? p->k / 2 : p->k, tile_k = p->sparse ? 256 : 128;
  pl->row_tiles = (p->m + 15) / 16;
  pl->tiles = (p->k + tile_k - 1) / tile_k;
  pl->groups = p->group == 0 || p->group >= p->k ? 1 : (p->k + p->group - 1) / p->group;
  const int steps = (int)(tile_k / step);   // 4 (16-bit x) or 2 (8-bit x)
  pl->flushes = 1;
  pl->group_magic = 0;                      // one group a row: every application is group 0
  if (pl->groups > 1) {
    while (p->group % (tile_k / pl->flushes) != 0 && pl->flushes < steps) pl->flushes *= 2;
    // u < 2^15 applications, at most 2^15 a group: the rounded-up reciprocal divides exactly
    const uint64_t per = (uint64_t)(p->group / (tile_k / pl->flushes));
    pl->group_magic = (uint32_t)((((uint64_t)1 << 31) + per - 1) / per);
  }
  pl->code_ld = (kept + 1) / 2;
  pl->meta_ld = ((kept + 3) / 4 + 15) / 16 * 16;
  const size_t codes = (size_t)(pl->row_tiles * pl->tiles) * 1024;
  pl->meta_off = codes;
  pl->scale_off = pl->meta_off + (p->sparse ? codes / 2 : 0);
  pl->zero_off = pl->scale_off + (size_t)(pl->row_tiles * pl->groups) * 32;
  pl->packed_bytes = pl->zero_off + (p->zeros ? (size_t)(pl->row_tiles * pl->groups) * 16 : 0);
  *plan = pl;
  return w4_fail(NM_OK, "");
}

nm_status_t nm_w4_plan_destroy(nm_w4_plan_t plan) {
  delete plan;
  return NM_OK;
}

nm_status_t nm_w4_sizes(nm_w4_plan_t plan, size_t* packed_bytes, int64_t* groups, int64_t* code_ld, int64_t* meta_ld) {
  if (!plan) return w4_fail(NM_ERR_INVALID_ARG, "plan is NULL");
  if (packed_bytes) *packed_bytes = plan->packed_bytes;
  if (groups) *groups = plan->groups;
  if (code_ld) *code_ld = plan->code_ld;
  if (meta_ld) *meta_ld = plan->p.sparse ? plan->meta_ld : 0;
  return NM_OK;
}

nm_status_t nm_w4_pack(nm_w4_plan_t plan, const void* d_codes, const void* d_scales, const void* d_zeros,
                       const void* d_meta, void* d_packed, void* stream) {
  if (!plan) return w4_fail(NM_ERR_INVALID_ARG, "plan is NULL");
  const nm_w4_problem_t& p = plan->p;
  const bool empty = p.m == 0 || p.k == 0;
  if ((d_zeros != nullptr) != (p.zeros != 0) && !empty)
    return w4_fail(NM_ERR_INVALID_ARG, "d_zeros must be given exactly where the plan has zero points");
  if ((d_meta != nullptr) != (p.sparse != 0) && !empty)
    return w4_fail(NM_ERR_INVALID_ARG, "d_meta must be given exactly where the plan's weights are 2:4");
  if (!empty && (!d_codes || !d_scales || !d_packed))
    return w4_fail(NM_ERR_INVALID_ARG, "d_codes / d_scales / d_packed is NULL");
  if (!w4_aligned(d_codes) || !w4_aligned(d_scales) || !w4_aligned(d_zeros) || !w4_aligned(d_meta) ||
      !w4_aligned(d_packed))
    return w4_fail(NM_ERR_ALIGN, "device pointers must be 16-byte aligned");
  if (empty) return NM_OK;
  hipStream_t s = (hipStream_t)stream;
  uint8_t* out = (uint8_t*)d_packed;
  W4PackArgs a;
  a.codes = (const uint8_t*)d_codes;
  a.zeros = (const uint8_t*)d_zeros;
  a.meta = (const uint8_t*)d_meta;
  a.out_codes = out;
  a.out_meta = out + plan->meta_off;
  a.m = p.m;
  a.kept = p.sparse ? p.k / 2 : p.k;
  a.code_ld = plan->code_ld;
  a.meta_ld = plan->meta_ld;
  a.tiles = plan->tiles;
  a.row_tiles = plan->row_tiles;
  a.groups = plan->groups;
  a.x_type = p.type_x;
  const int64_t blocks = plan->tiles * plan->row_tiles, most = (int64_t)1 << 20;
  hipLaunchKernelGGL(w4_pack_kernel, dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return w4_hip(e);
  const int64_t total = plan->row_tiles * plan->groups * 16, sb = (total + 255) / 256;
  hipLaunchKernelGGL(w4_pack_scales_kernel, dim3((unsigned)(sb < most ? sb : most)), dim3(256), 0, s,
                     (const uint16_t*)d_scales, (const uint8_t*)d_zeros, (uint16_t*)(out + plan->scale_off),
                     out + plan->zero_off, p.m, plan->groups, total);
  return w4_hip(hipGetLastError());
}

nm_status_t nm_w4_matvec(nm_w4_plan_t plan, const void* d_packed, const void* dX, const float* d_x_scale, void* dY,
                         void* stream) {
  if (!plan) return w4_fail(NM_ERR_INVALID_ARG, "plan is NULL");
  const nm_w4_problem_t& p = plan->p;
  const bool empty = p.m == 0 || p.n == 0, scaled = p.type_x == NM_I8;
  if ((d_x_scale != nullptr) != scaled && !empty)
    return w4_fail(NM_ERR_INVALID_ARG, "d_x_scale must be given exactly where x is int8");
  if (!empty && (!dY || (p.k > 0 && (!d_packed || !dX))))
    return w4_fail(NM_ERR_INVALID_ARG, "d_packed / dX / dY is NULL");
  if (!w4_aligned(d_packed) || !w4_aligned(dX) || !w4_aligned(d_x_scale) || !w4_aligned(dY))
    return w4_fail(NM_ERR_ALIGN, "device pointers must be 16-byte aligned");
  if (empty) return NM_OK;
  const uint8_t* in = (const uint8_t*)d_packed;
  W4Args a;
  a.codes = in;
  a.meta = in + plan->meta_off;
  a.scales = (const uint16_t*)(in + plan->scale_off);
  a.zeros = in + plan->zero_off;
  a.x = (const uint8_t*)dX;
  a.x_scale = d_x_scale;
  a.y = (uint16_t*)dY;
  a.ldx = p.ldx;
  a.ldy = p.ldy;
  a.m = (int32_t)p.m;
  a.n = (int32_t)p.n;
  a.k = (int32_t)p.k;
  a.row_tiles = (int32_t)plan->row_tiles;
  a.tiles = (int32_t)plan->tiles;
  a.groups = (int32_t)plan->groups;
  a.group_magic = plan->group_magic;
  const W4Shape sh = {p.sparse != 0, p.zeros != 0, plan->flushes};
  hipStream_t s = (hipStream_t)stream;
  if (p.type_x == NM_F16) return w4_hip(launch_w4_f16(a, sh, s));
  if (p.type_x == NM_BF16) return w4_hip(launch_w4_bf16(a, sh, s));
  if (p.type_y == NM_F16) return w4_hip(launch_w4_i8_f16(a, sh, s));
  return w4_hip(launch_w4_i8_bf16(a, sh, s));
}

}  // extern "C"
