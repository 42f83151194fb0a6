// Product of a few tokens with 4-bit weights: templates included by the
// per-type instantiation files nm_w4_{f16,bf16,i8}.hip.
//
//   y[j][i] = xs_j * sum_g s[i][g] * sum_{k in g} (q[i][k] - z[i][g]) * x[j][k]
//
// W is m x k in codes q of 4 bits, dense or 2:4; s is one scale a group along
// k, z the group's zero point (8 without zero points); x holds n tokens.
//
// The weights are read once and are nearly all of the traffic, so the kernel
// is a stream over them: nm_w4_pack lays the codes out so that one 16-byte
// load a lane (1 KB a wave, contiguous) brings the 16 rows x 128 kept values
// that the lanes feed to the 16x16 matrix instructions, 4 steps of 32 kept
// values for 16-bit x and 2 of 64 for 8-bit x. q - z is an integer of
// magnitude at most 15, exact in f16, bf16 and int8; the products of one group
// are summed by the matrix unit in fp32 (int32 for 8-bit x) and the group's
// scale is applied to that sum in fp32, so a code costs only its unpacking.
//
// A block takes 16 rows of W; its waves share out the tiles of k and add their
// sums through LDS in wave order (the order of a sum depends on the shape
// alone). The matrix instruction's 16 columns hold the tokens; columns past n
// repeat the last token's address (the same cache line) and are not stored.
// Up to NT * 16 tokens share one pass over the weights.
//
// Lane layouts (l % 16 = row or column, q = l / 16; accumulator D[4q + r][l % 16]):
//  dense 16-bit 16x16x32: k = 8q ..; dense int8 16x16x64: k = 16q ..
//  2:4 16-bit 16x16x64: kept values 8q .., x at k = 8q .. and 32 + 8q ..
//  2:4 int8 16x16x128:  kept values 16q .., x at k = 16q .. and 64 + 16q ..
#pragma once
#include "nm_device.h"
#include "nm_w4.h"

namespace nm {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half16_t __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x16_t __attribute__((ext_vector_type(16)));

template <int XT> struct W4Type;
template <> struct W4Type<DT_F16> { typedef half8_t a; typedef half16_t b2; typedef floatx4 acc; };
template <> struct W4Type<DT_BF16> { typedef bf16x8_t a; typedef bf16x16_t b2; typedef floatx4 acc; };
template <> struct W4Type<DT_I8> { typedef intx4 a; typedef intx8 b2; typedef intx4 acc; };

// Zero point of one lane's row, in the form its unpacking subtracts.
// Unpacking of one dword of eight codes, exact in every type:
//  f16: 0x6400 | q = 1024 + q and 0x6400 | q << 4 = 1024 + 16 q as f16, so two
//       codes take one and-or and one packed subtraction (packed
//       multiply-subtraction by 1/16). Codes 0, 1 sit in nibbles 0 and 4, codes
//       2, 3 in 1 and 5, and so on.
//  bf16: there is no packed bf16 arithmetic; nibble at bit p under the exponent
//       of 2^(23-p) is the fp32 2^(23-p) + q, minus 2^(23-p) + z is q - z, whose
//       upper half is its bf16. Codes in nibble order.
//  int8: even nibbles are codes 0..3, odd nibbles 4..7. Without zero points the
//       pack step stores q - 8 as a two's complement nibble, which in the upper
//       half of a byte is 16 (q - 8). With zero points 128 + q - z never borrows
//       from its neighbour byte, and flipping the top bit leaves q - z.
template <int XT, bool ZEROS> struct W4Zero;

template <bool ZEROS> struct W4Zero<DT_F16, ZEROS> {
  half2_t z1, z16;
  __device__ __forceinline__ void set(uint32_t z) {
    z1 = __builtin_bit_cast(half2_t, 0x64006400u + z * 0x00010001u);    // 1024 + z
    z16 = __builtin_bit_cast(half2_t, 0x54005400u + z * 0x00100010u);   // 64 + z
  }
  __device__ __forceinline__ half8_t unpack(const uint32_t* w) const {
    const half2_t r16 = {(_Float16)0.0625f, (_Float16)0.0625f};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const uint32_t v = w[0] >> (8 * i);
      const half2_t a = __builtin_bit_cast(half2_t, (v & 0x000F000Fu) | 0x64006400u);
      const half2_t b = __builtin_bit_cast(half2_t, (v & 0x00F000F0u) | 0x64006400u);
      o[2 * i] = __builtin_bit_cast(uint32_t, a - z1);
      o[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(b, r16, -z16));
    }
    const u32x4 r = {o[0], o[1], o[2], o[3]};
    return __builtin_bit_cast(half8_t, r);
  }
};

template <bool ZEROS> struct W4Zero<DT_BF16, ZEROS> {
  static constexpr uint32_t magic(int p) { return (uint32_t)(127 + 23 - p) << 23; }
  uint32_t z;
  __device__ __forceinline__ void set(uint32_t zz) { z = zz; }
  __device__ __forceinline__ float one(uint32_t w, int p) const {
    return __builtin_bit_cast(float, (w & (15u << p)) | magic(p)) - __builtin_bit_cast(float, (z << p) | magic(p));
  }
  __device__ __forceinline__ bf16x8_t unpack(const uint32_t* w) const {
    const uint32_t h = w[0] >> 12;
    const float f[8] = {one(w[0], 0), one(w[0], 4), one(w[0], 8), one(w[0], 12),
                        one(w[0], 16), one(h, 8), one(h, 12), one(h, 16)};
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; i++)
      r[i] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, f[2 * i + 1]), __builtin_bit_cast(uint32_t, f[2 * i]),
                                   0x07060302u);
    return __builtin_bit_cast(bf16x8_t, r);
  }
};

template <bool ZEROS> struct W4Zero<DT_I8, ZEROS> {
  uint32_t z4;
  __device__ __forceinline__ void set(uint32_t z) { z4 = z * 0x01010101u; }
  __device__ __forceinline__ intx4 unpack(const uint32_t* w) const {
    intx4 r;
#pragma unroll
    for (int i = 0; i < 2; i++) {
      if constexpr (ZEROS) {
        r[2 * i] = (int)((((w[i] & 0x0F0F0F0Fu) | 0x80808080u) - z4) ^ 0x80808080u);
        r[2 * i + 1] = (int)(((((w[i] >> 4) & 0x0F0F0F0Fu) | 0x80808080u) - z4) ^ 0x80808080u);
      } else {
        r[2 * i] = (int)((w[i] << 4) & 0xF0F0F0F0u);
        r[2 * i + 1] = (int)(w[i] & 0xF0F0F0F0u);
      }
    }
    return r;
  }
};

template <int XT, bool SPARSE>
__device__ __forceinline__ typename W4Type<XT>::acc w4_mma(typename W4Type<XT>::a a, const u32x4 (&b)[SPARSE ? 2 : 1],
                                                          typename W4Type<XT>::acc c, int idx) {
  typedef typename W4Type<XT>::a a_t;
  typedef typename W4Type<XT>::b2 b2_t;
  if constexpr (SPARSE) {
    typedef uint32_t u32x8 __attribute__((ext_vector_type(8)));
    const u32x8 w = {b[0][0], b[0][1], b[0][2], b[0][3], b[1][0], b[1][1], b[1][2], b[1][3]};
    const b2_t bb = __builtin_bit_cast(b2_t, w);
    if constexpr (XT == DT_F16) return __builtin_amdgcn_smfmac_f32_16x16x64_f16(a, bb, c, idx, 0, 0);
    else if constexpr (XT == DT_BF16) return __builtin_amdgcn_smfmac_f32_16x16x64_bf16(a, bb, c, idx, 0, 0);
    else return __builtin_amdgcn_smfmac_i32_16x16x128_i8(a, bb, c, idx, 0, 0);
  } else {
    const a_t bb = __builtin_bit_cast(a_t, b[0]);
    if constexpr (XT == DT_F16) return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, bb, c, 0, 0, 0);
    else if constexpr (XT == DT_BF16) return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, bb, c, 0, 0, 0);
    else return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, bb, c, 0, 0, 0);
  }
}

// What one tile needs from memory besides x.
template <bool SPARSE, int F> struct W4Tile {
  u32x4 c;
  u32x2 mt;
  u32x2 sc[F];
  uint32_t z[F];
};

template <int XT, bool SPARSE, bool ZEROS, int F, int NT>
__global__ void __launch_bounds__(1024) w4_kernel(W4Args A) {
  constexpr int ESZ = XT == DT_I8 ? 1 : 2;
  constexpr int S = XT == DT_I8 ? 2 : 4;         // matrix instructions along a tile
  constexpr int SF = S / F;                      // of them, between two scales
  constexpr int TK = SPARSE ? 256 : 128;         // k per tile
  constexpr int KS = TK / S;
  constexpr int E = 16 / ESZ;                    // elements of x in 16 bytes
  constexpr int BC = SPARSE ? 2 : 1;             // 16-byte pieces of x per instruction
  typedef typename W4Type<XT>::acc acc_t;
  extern __shared__ floatx4 red[];

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int l16 = lane & 15, q = lane >> 4;
  const bool ybf = XT == DT_BF16 || (XT == DT_I8 && A.y_bf16);
  const int64_t rt = blockIdx.x;
  const int col0 = blockIdx.y * (16 * NT);

  const uint8_t* codes = A.codes + rt * A.tiles * 1024 + lane * 16;
  const uint8_t* meta = A.meta + rt * A.tiles * 512 + lane * 8;
  const uint8_t* scales = (const uint8_t*)A.scales + rt * A.groups * 32 + q * 8;
  const uint8_t* zeros = A.zeros + rt * A.groups * 16 + l16;
  const uint8_t* xp[NT];
#pragma unroll
  for (int j = 0; j < NT; j++) xp[j] = A.x + (int64_t)min(col0 + 16 * j + l16, A.n - 1) * A.ldx * ESZ;

  auto load = [&](W4Tile<SPARSE, F>& T, int t) {
    T.c = *(const u32x4*)(codes + (size_t)t * 1024);
    if constexpr (SPARSE) T.mt = *(const u32x2*)(meta + (size_t)t * 512);
#pragma unroll
    for (int f = 0; f < F; f++) {
      const uint32_t u = (uint32_t)(t * F + f);
      // the last tile may reach past the last group (its x is zero there)
      const uint32_t g = min(A.group_magic ? __umulhi(u, A.group_magic) : u, (uint32_t)A.groups - 1u);
      T.sc[f] = *(const u32x2*)(scales + (size_t)g * 32);
      if constexpr (ZEROS) T.z[f] = zeros[(size_t)g * 16];
      else T.z[f] = 8;
    }
  };
  // one 16-byte piece of a token's row; past k the values are zero
  auto piece = [&](const uint8_t* row, int k0, bool whole) -> u32x4 {
    if (whole || k0 + E <= A.k) return *(const u32x4*)(row + (size_t)k0 * ESZ);
    u32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < E; e++)
      if (k0 + e < A.k) {
        if constexpr (ESZ == 2) v[e / 2] |= (uint32_t)((const uint16_t*)row)[k0 + e] << (16 * (e % 2));
        else v[e / 4] |= (uint32_t)row[k0 + e] << (8 * (e % 4));
      }
    return v;
  };

  floatx4 y[NT];
#pragma unroll
  for (int j = 0; j < NT; j++) y[j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

  auto compute = [&](const W4Tile<SPARSE, F>& T, int t, bool whole) {
    const int k0 = t * TK + E * q;
#pragma unroll
    for (int f = 0; f < F; f++) {
      W4Zero<XT, ZEROS> zp;
      zp.set(T.z[f]);
      acc_t acc[NT];
#pragma unroll
      for (int j = 0; j < NT; j++) acc[j] = acc_t{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < SF; i++) {
        const int s = f * SF + i;
        uint32_t w[2];
        if constexpr (ESZ == 2) w[0] = T.c[s];
        else { w[0] = T.c[2 * s]; w[1] = T.c[2 * s + 1]; }
        const typename W4Type<XT>::a a = zp.unpack(w);
        int idx = 0;
        if constexpr (SPARSE) idx = ESZ == 2 ? (int)(T.mt[s / 2] >> (16 * (s % 2))) : (int)T.mt[s];
#pragma unroll
        for (int j = 0; j < NT; j++) {
          u32x4 b[BC];
#pragma unroll
          for (int c = 0; c < BC; c++) b[c] = piece(xp[j], k0 + s * KS + c * (KS / 2), whole);
          acc[j] = w4_mma<XT, SPARSE>(a, b, acc[j], idx);
        }
      }
#pragma unroll
      for (int r = 0; r < 4; r++) {
        const uint16_t raw = (uint16_t)(T.sc[f][r / 2] >> (16 * (r % 2)));
        float sc = ybf ? from_bits16<DT_BF16>(raw) : from_bits16<DT_F16>(raw);
        if constexpr (XT == DT_I8 && !ZEROS) sc *= 0.0625f;   // the codes are held times 16
#pragma unroll
        for (int j = 0; j < NT; j++) y[j][r] = __builtin_fmaf(sc, (float)acc[j][r], y[j][r]);
      }
    }
  };

  int t = wave;
  if (t < A.tiles) {
    W4Tile<SPARSE, F> cur;
    load(cur, t);
    const int full = A.k / TK;      // tiles that lie within k whole
    for (; t < A.tiles; t += waves) {
      W4Tile<SPARSE, F> next = cur;
      if (t + waves < A.tiles) load(next, t + waves);
      if (t < full) compute(cur, t, true);
      else compute(cur, t, false);
      cur = next;
    }
  }

#pragma unroll
  for (int j = 0; j < NT; j++) red[(wave * NT + j) * 64 + lane] = y[j];
  __syncthreads();
  for (int j = wave; j < NT; j += waves) {
    floatx4 v = red[j * 64 + lane];
    for (int w = 1; w < waves; w++) v += red[(w * NT + j) * 64 + lane];
    const int col = col0 + 16 * j + l16;
    const int row = (int)rt * 16 + 4 * q;
    if (col >= A.n || row >= A.m) continue;
    if constexpr (XT == DT_I8) v *= A.x_scale[col];
    uint16_t o[4];
#pragma unroll
    for (int r = 0; r < 4; r++) o[r] = ybf ? to_bits16<DT_BF16>(v[r]) : to_bits16<DT_F16>(v[r]);
    uint16_t* yp = A.y + (int64_t)col * A.ldy + row;
    if (row + 4 <= A.m && A.ldy % 4 == 0) {
      *(u32x2*)yp = u32x2{(uint32_t)o[0] | (uint32_t)o[1] << 16, (uint32_t)o[2] | (uint32_t)o[3] << 16};
    } else {
#pragma unroll
      for (int r = 0; r < 4; r++)
        if (row + r < A.m) yp[r] = o[r];
    }
  }
}

// Waves per block: as many as it takes to have work on every SIMD, at most 16,
// at least one tile of k each.
inline int w4_waves(const W4Args& a, int64_t blocks) {
  int w = 4;
  while (w < 16 && blocks * w < 8192 && w < a.tiles) w *= 2;
  return w;
}

template <int XT, bool SPARSE, bool ZEROS, int F, int NT>
hipError_t w4_go(const W4Args& a, const W4Shape& sh, hipStream_t s) {
  const int64_t cols = (a.n + 16 * NT - 1) / (16 * NT);
  const int w = w4_waves(a, sh.row_tiles * cols);
  hipLaunchKernelGGL((w4_kernel<XT, SPARSE, ZEROS, F, NT>), dim3((unsigned)sh.row_tiles, (unsigned)cols), dim3(64 * w),
                     (size_t)w * NT * 1024, s, a);
  return hipGetLastError();
}

template <int XT, bool SPARSE, bool ZEROS, int F>
hipError_t w4_cols(const W4Args& a, const W4Shape& sh, hipStream_t s) {
  if (a.n <= 16) return w4_go<XT, SPARSE, ZEROS, F, 1>(a, sh, s);
  if (a.n <= 32) return w4_go<XT, SPARSE, ZEROS, F, 2>(a, sh, s);
  return w4_go<XT, SPARSE, ZEROS, F, 3>(a, sh, s);
}

template <int XT, bool SPARSE, bool ZEROS>
hipError_t w4_flush(const W4Args& a, const W4Shape& sh, hipStream_t s) {
  if (sh.flushes == 1) return w4_cols<XT, SPARSE, ZEROS, 1>(a, sh, s);
  if (sh.flushes == 2) return w4_cols<XT, SPARSE, ZEROS, 2>(a, sh, s);
  if constexpr (XT != DT_I8) return w4_cols<XT, SPARSE, ZEROS, 4>(a, sh, s);
  return hipErrorInvalidValue;
}

template <int XT>
hipError_t w4_dispatch(const W4Args& a, const W4Shape& sh, hipStream_t s) {
  if (sh.sparse) return sh.zeros ? w4_flush<XT, true, true>(a, sh, s) : w4_flush<XT, true, false>(a, sh, s);
  return sh.zeros ? w4_flush<XT, false, true>(a, sh, s) : w4_flush<XT, false, false>(a, sh, s);
}

}  // namespace nm
