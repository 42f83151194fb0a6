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
// Two kernels. w4_kernel: a block takes R tiles of 16 rows; its waves share out
// the tiles of k, two of them in registers at a time, with their piece of x, and
// add their sums through LDS in wave order (the order of a sum depends on the
// shape alone). w4_walk_kernel (2:4 weights, 16-bit x, many rows): x lies in LDS,
// and blocks walk over the row tiles. The matrix instruction's 16 columns hold
// the tokens; columns past n repeat the last token's address (the same cache
// line) and are not stored. Up to NT * 16 tokens share one pass over the weights.
//
// Lane layouts (l % 16 = row or column, q = l / 16; accumulator D[4q + r][l % 16]):
//  dense 16-bit 16x16x32: k = 8q ..; dense int8 16x16x64: k = 16q ..
//  2:4 16-bit 16x16x64: kept values 8q .., x at k = 8q .. and 32 + 8q ..
//  2:4 int8 16x16x128:  kept values 16q .., x at k = 16q .. and 64 + 16q ..
#pragma once
#include <type_traits>

#include "nm_device.h"
#include "nm_w4.h"

namespace nm {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half16_t __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x16_t __attribute__((ext_vector_type(16)));

template <int XT> struct W4Type;
template <> struct W4Type<DT_F16> {
  typedef half8_t a; typedef floatx4 acc;
  template <bool SPARSE> using b = std::conditional_t<SPARSE, half16_t, half8_t>;
};
template <> struct W4Type<DT_BF16> {
  typedef bf16x8_t a; typedef floatx4 acc;
  template <bool SPARSE> using b = std::conditional_t<SPARSE, bf16x16_t, bf16x8_t>;
};
template <> struct W4Type<DT_I8> {
  typedef intx4 a; typedef intx4 acc;
  template <bool SPARSE> using b = std::conditional_t<SPARSE, intx8, intx4>;
};

// Zero point of one lane's row, in the form its unpacking subtracts.
// Unpacking of one dword of eight codes, exact in every type:
//  f16: 0x6400 | q = 1024 + q and 0x6400 | q << 4 = 1024 + 16 q as f16, so two
//       codes take one and-or and one packed subtraction (packed
//       multiply-subtraction by 1/16). Codes 0, 1 sit in nibbles 0 and 4, codes
//       2, 3 in 1 and 5, and so on.
//  int8: even nibbles are codes 0..3, odd nibbles 4..7. Without zero points the
//       pack step stores q - 8 as a two's complement nibble, which in the upper
//       half of a byte is 16 (q - 8). With zero points 128 + q - z never borrows
//       from its neighbour byte, and flipping the top bit leaves q - z.
//  bf16: there is no packed bf16 arithmetic; the bytes of int8 are converted to
//       fp32, whose upper half is the value's bf16.
template <int XT, bool ZEROS> struct W4Zero;

template <bool ZEROS> struct W4Zero<DT_F16, ZEROS> {
  half2_t z1, z16;
  uint32_t m1, m16, k;   // in registers: an and-or takes no literals
  __device__ __forceinline__ void set(uint32_t z) {
    m1 = 0x000F000Fu; m16 = 0x00F000F0u; k = 0x64006400u;
    asm("" : "+s"(m1), "+s"(m16), "+v"(k));
    z1 = __builtin_bit_cast(half2_t, 0x64006400u + z * 0x00010001u);    // 1024 + z
    z16 = __builtin_bit_cast(half2_t, 0x54005400u + z * 0x00100010u);   // 64 + z
  }
  __device__ __forceinline__ half8_t unpack(const uint32_t* w) const {
    const half2_t r16 = {(_Float16)0.0625f, (_Float16)0.0625f};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const uint32_t v = w[0] >> (8 * i);
      const half2_t a = __builtin_bit_cast(half2_t, (v & m1) | k);
      const half2_t b = __builtin_bit_cast(half2_t, (v & m16) | k);
      o[2 * i] = __builtin_bit_cast(uint32_t, a - z1);
      o[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(b, r16, -z16));
    }
    const u32x4 r = {o[0], o[1], o[2], o[3]};
    return __builtin_bit_cast(half8_t, r);
  }
};

template <bool ZEROS> struct W4Bytes {
  uint32_t z4;
  __device__ __forceinline__ void set(uint32_t z) { z4 = z * 0x01010101u; }
  // the eight codes of a dword minus the zero point: 0..3 in the bytes of e, 4..7 in those of o
  __device__ __forceinline__ void unpack(uint32_t w, uint32_t& e, uint32_t& o) const {
    if constexpr (ZEROS) {
      e = (((w & 0x0F0F0F0Fu) | 0x80808080u) - z4) ^ 0x80808080u;
      o = ((((w >> 4) & 0x0F0F0F0Fu) | 0x80808080u) - z4) ^ 0x80808080u;
    } else {
      e = (w << 4) & 0xF0F0F0F0u;
      o = w & 0xF0F0F0F0u;
    }
  }
};

template <bool ZEROS> struct W4Zero<DT_BF16, ZEROS> {
  W4Bytes<ZEROS> b;
  __device__ __forceinline__ void set(uint32_t z) { b.set(z); }
  __device__ __forceinline__ bf16x8_t unpack(const uint32_t* w) const {
    uint32_t h[2];
    b.unpack(w[0], h[0], h[1]);
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const uint32_t v = h[i / 2] >> (16 * (i % 2));
      r[i] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, (float)(int8_t)(v >> 8)),
                                   __builtin_bit_cast(uint32_t, (float)(int8_t)v), 0x07060302u);
    }
    return __builtin_bit_cast(bf16x8_t, r);
  }
};

template <bool ZEROS> struct W4Zero<DT_I8, ZEROS> {
  W4Bytes<ZEROS> b;
  __device__ __forceinline__ void set(uint32_t z) { b.set(z); }
  __device__ __forceinline__ intx4 unpack(const uint32_t* w) const {
    uint32_t h[4];
    b.unpack(w[0], h[0], h[1]);
    b.unpack(w[1], h[2], h[3]);
    return intx4{(int)h[0], (int)h[1], (int)h[2], (int)h[3]};
  }
};

template <int XT, bool SPARSE>
__device__ __forceinline__ typename W4Type<XT>::acc w4_mma(typename W4Type<XT>::a a, typename W4Type<XT>::template b<SPARSE> b,
                                                          typename W4Type<XT>::acc c, int idx) {
  if constexpr (SPARSE) {
    if constexpr (XT == DT_F16) return __builtin_amdgcn_smfmac_f32_16x16x64_f16(a, b, c, idx, 0, 0);
    else if constexpr (XT == DT_BF16) return __builtin_amdgcn_smfmac_f32_16x16x64_bf16(a, b, c, idx, 0, 0);
    else return __builtin_amdgcn_smfmac_i32_16x16x128_i8(a, b, c, idx, 0, 0);
  } else {
    if constexpr (XT == DT_F16) return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    else if constexpr (XT == DT_BF16) return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    else return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
  }
}

typedef const __attribute__((address_space(1))) uint8_t* gptr;
typedef const __attribute__((address_space(1))) u32x4* gptr16;
typedef const __attribute__((address_space(1))) u32x2* gptr8;

// Four rows of one column of y from `row` on.
template <int XT, bool YB, bool ZEROS>
__device__ __forceinline__ void w4_store(const W4Args& A, floatx4 v, int col, int64_t row) {
  if (col >= A.n || row >= A.m) return;
  if constexpr (XT == DT_I8) v *= A.x_scale[col];
  if constexpr (XT != DT_F16 && !ZEROS) v *= 0.0625f;    // these codes are held times 16
  uint16_t o[4];
#pragma unroll
  for (int e = 0; e < 4; e++) o[e] = to_bits16<YB ? DT_BF16 : DT_F16>(v[e]);
  uint16_t* yp = A.y + (int64_t)col * A.ldy + row;
  if (row + 4 <= A.m && A.ldy % 4 == 0) {
    *(u32x2*)yp = u32x2{(uint32_t)o[0] | (uint32_t)o[1] << 16, (uint32_t)o[2] | (uint32_t)o[3] << 16};
  } else {
#pragma unroll
    for (int e = 0; e < 4; e++)
      if (row + e < A.m) yp[e] = o[e];
  }
}

// What one tile of k of R row tiles needs from memory; x with it for up to 16 tokens.
template <int XT, bool SPARSE, int F, int NT, int R, bool XL> struct W4Tile {
  u32x4 c[R];
  u32x2 mt[R];
  u32x2 sc[R][F];
  uint32_t z[R][F];
  std::conditional_t<XL, u32x4[(XT == DT_I8 ? 2 : 4) * (SPARSE ? 2 : 1)],
                     typename W4Type<XT>::template b<SPARSE>[NT == 1 ? (XT == DT_I8 ? 2 : 4) : 1]> x;
};

// Bytes of LDS in which a wave turns a tile of x, 16 tokens 16 bytes apart in their banks.
constexpr int w4_turn(int tile_bytes) { return 16 * (tile_bytes + 16); }

// What bounds it: the loads of x. They come from the L1 cache, 1 KB (2:4: 2 KB) a
// matrix instruction against 256 to 512 bytes of codes, so each piece of x serves R row
// tiles; and R is chosen so that the blocks are whole rounds of the 256 CUs. The matrix
// instruction's order has neighbouring lanes load from different tokens, a cache line
// each; with XL they load a token's row along, and the wave turns the tile in LDS.
// 16384x4096, one f16 token, 8.5 us with R = 4 (34 MB, 4.1 TB/s; 11.1 with R = 1),
// 16 tokens 9.3 (18.7); 32768x32768, four 8-bit tokens, 87 us (559 MB, 6.4 TB/s;
// 115 with R = 1). Codes are loaded past the caches' reuse (nontemporal): x stays there.
template <int XT, bool YB, bool SPARSE, bool ZEROS, int F, int NT, int R, bool XL>
__global__ void __launch_bounds__(512) w4_kernel(W4Args A) {
  static_assert(!XL || NT == 1, "x is turned for up to 16 tokens");
  constexpr int ESZ = XT == DT_I8 ? 1 : 2;
  constexpr int S = XT == DT_I8 ? 2 : 4;         // matrix instructions along a tile
  constexpr int SF = S / F;                      // of them, between two scales
  constexpr int TK = SPARSE ? 256 : 128;         // k per tile
  constexpr int KS = TK / S;
  constexpr int E = 16 / ESZ;                    // elements of x in 16 bytes
  typedef typename W4Type<XT>::acc acc_t;
  typedef typename W4Type<XT>::template b<SPARSE> b_t;
  constexpr int TB = TK * ESZ;                   // bytes of a token's row in a tile
  constexpr int LPR = TB / 16;                   // lanes that load them
  typedef W4Tile<XT, SPARSE, F, NT, R, XL> tile_t;
  extern __shared__ floatx4 red[];

  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);   // scalar, and with it a tile's addresses
  const int l16 = lane & 15, q = lane >> 4;
  const int col0 = blockIdx.y * (16 * NT);

  int64_t rt[R];                                 // past the last row tile: that one again, not stored
#pragma unroll
  for (int r = 0; r < R; r++) rt[r] = min((int)blockIdx.x * R + r, A.row_tiles - 1);
  const uint8_t* xp[NT];
#pragma unroll
  for (int j = 0; j < NT; j++)
    xp[j] = A.x + (int64_t)min(col0 + 16 * j + l16, A.n - 1) * A.ldx * ESZ;

  // the at-th 16 bytes of a token's row from k0 on; past k the values are zero
  auto piece = [&](const uint8_t* row, int k0, int at, bool whole) -> u32x4 {
    const uint8_t* p = row + (size_t)k0 * ESZ + at * 16;
    const int left = A.k - k0 - E * at;
    if (whole || left >= E) return *(const u32x4*)p;
    u32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < E; e++)
      if (e < left) {
        if constexpr (ESZ == 2) v[e / 2] |= (uint32_t)((const uint16_t*)p)[e] << (16 * (e % 2));
        else v[e / 4] |= (uint32_t)p[e] << (8 * (e % 4));
      }
    return v;
  };

  // what one matrix instruction takes of it: one piece, or two half an instruction's k apart
  auto pieces = [&](const uint8_t* row, int k0, bool whole) -> b_t {
    if constexpr (SPARSE)
      return __builtin_bit_cast(b_t, __builtin_shufflevector(piece(row, k0, q, whole), piece(row, k0 + KS / 2, q, whole), 0, 1, 2,
                                                             3, 4, 5, 6, 7));
    else return __builtin_bit_cast(b_t, piece(row, k0, q, whole));
  };

  auto load = [&](tile_t& T, int t, bool whole) {
#pragma unroll
    for (int r = 0; r < R; r++) {
      // opaque, so that the scalar address and the lane's offset stay apart
      gptr pc = (gptr)A.codes + (rt[r] * A.tiles + t) * 1024;
      asm("" : "+s"(pc));
      T.c[r] = __builtin_nontemporal_load((gptr16)(pc + (uint32_t)lane * 16));
      if constexpr (SPARSE) {
        gptr pm = (gptr)A.meta + (rt[r] * A.tiles + t) * 512;
        asm("" : "+s"(pm));
        T.mt[r] = __builtin_nontemporal_load((gptr8)(pm + (uint32_t)lane * 8));
      }
#pragma unroll
      for (int f = 0; f < F; f++) {
        const uint32_t u = (uint32_t)(t * F + f);
        // the last tile may reach past the last group (its x is zero there)
        const uint32_t g = min(__umulhi(2 * u, A.group_magic), (uint32_t)A.groups - 1u);
        gptr ps = (gptr)A.scales + (rt[r] * A.groups + g) * 32;
        asm("" : "+s"(ps));
        T.sc[r][f] = *(gptr8)(ps + (uint32_t)q * 8);
        if constexpr (ZEROS) {
          gptr pz = (gptr)A.zeros + (rt[r] * A.groups + g) * 16;
          asm("" : "+s"(pz));
          T.z[r][f] = pz[(uint32_t)l16];
        } else T.z[r][f] = 8;
      }
    }
    if constexpr (XL) {
#pragma unroll
      for (int i = 0; i < 16 * TB / 1024; i++)
        T.x[i] = piece(A.x + (int64_t)min(i * (64 / LPR) + lane / LPR, A.n - 1) * A.ldx * ESZ, t * TK, lane % LPR, whole);
    } else if constexpr (NT == 1) {
#pragma unroll
      for (int i = 0; i < S; i++) T.x[i] = pieces(xp[0], t * TK + i * KS, whole);
    }
    __builtin_amdgcn_sched_barrier(0);           // all of them are on their way before the products that follow
  };

  floatx4 y[R][NT];
#pragma unroll
  for (int r = 0; r < R; r++)
#pragma unroll
    for (int j = 0; j < NT; j++) y[r][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

  uint8_t* const turn = (uint8_t*)(red + waves * NT * R * 64) + wave * w4_turn(TB);
  auto compute = [&](const tile_t& T, int t, bool whole) {
    if constexpr (XL) {
#pragma unroll
      for (int i = 0; i < 16 * TB / 1024; i++)
        *(u32x4*)(turn + (i * (64 / LPR) + lane / LPR) * (TB + 16) + lane % LPR * 16) = T.x[i];
    }
#pragma unroll
    for (int f = 0; f < F; f++) {
      if (!whole && t * TK + f * SF * KS >= A.k) break;
      W4Zero<XT, ZEROS> zp[R];
      acc_t acc[R][NT];
#pragma unroll
      for (int r = 0; r < R; r++) {
        zp[r].set(T.z[r][f]);
#pragma unroll
        for (int j = 0; j < NT; j++) acc[r][j] = acc_t{0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < SF; i++) {
        const int s = f * SF + i;
        b_t b[NT];
#pragma unroll
        for (int j = 0; j < NT; j++) {
          if constexpr (XL) {
            const uint8_t* p = turn + l16 * (TB + 16) + s * KS * ESZ + q * 16;
            if constexpr (SPARSE)
              b[j] = __builtin_bit_cast(b_t, __builtin_shufflevector(*(const u32x4*)p, *(const u32x4*)(p + KS / 2 * ESZ), 0, 1,
                                                                     2, 3, 4, 5, 6, 7));
            else b[j] = __builtin_bit_cast(b_t, *(const u32x4*)p);
          } else if constexpr (NT == 1) b[j] = T.x[s];
          else b[j] = pieces(xp[j], t * TK + s * KS, whole);
        }
#pragma unroll
        for (int r = 0; r < R; r++) {
          uint32_t w[2];
          if constexpr (ESZ == 2) w[0] = T.c[r][s];
          else { w[0] = T.c[r][2 * s]; w[1] = T.c[r][2 * s + 1]; }
          const typename W4Type<XT>::a a = zp[r].unpack(w);
          int idx = 0;
          if constexpr (SPARSE) idx = ESZ == 2 ? (int)(T.mt[r][s / 2] >> (16 * (s % 2))) : (int)T.mt[r][s];
#pragma unroll
          for (int j = 0; j < NT; j++) acc[r][j] = w4_mma<XT, SPARSE>(a, b[j], acc[r][j], idx);
        }
      }
#pragma unroll
      for (int r = 0; r < R; r++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const float sc = from_bits16<YB ? DT_BF16 : DT_F16>((uint16_t)(T.sc[r][f][e / 2] >> (16 * (e % 2))));
#pragma unroll
          for (int j = 0; j < NT; j++) y[r][j][e] = __builtin_fmaf(sc, (float)acc[r][j][e], y[r][j][e]);
        }
    }
  };

  // Two tiles in turn, the next one's loads behind the present one's products.
  // Every path into a product has the same loads behind it, or the wait for
  // them would be a wait for all.
  const int full = A.k / TK;      // tiles that lie within k whole
  if (wave < full) {
    int t = wave;
    tile_t T0, T1;
    load(T0, t, true);
    for (;;) {
      t += waves;
      if (t >= full) { compute(T0, t - waves, true); break; }
      load(T1, t, true);
      compute(T0, t - waves, true);
      t += waves;
      if (t >= full) { compute(T1, t - waves, true); break; }
      load(T0, t, true);
      compute(T1, t - waves, true);
    }
  }
  if (full < A.tiles && full % waves == wave) {
    tile_t T;
    load(T, full, false);
    compute(T, full, false);
  }

#pragma unroll
  for (int r = 0; r < R; r++)
#pragma unroll
    for (int j = 0; j < NT; j++) red[((wave * R + r) * NT + j) * 64 + lane] = y[r][j];
  __syncthreads();
  for (int u = wave; u < R * NT; u += waves) {
    floatx4 v = red[u * 64 + lane];
    for (int w = 1; w < waves; w++) v += red[(w * R * NT + u) * 64 + lane];
    w4_store<XT, YB, ZEROS>(A, v, col0 + 16 * (u % NT) + l16, ((int64_t)blockIdx.x * R + u / NT) * 16 + 4 * q);
  }
}

// ---------------------------------------------------------------- x in LDS

constexpr int W4_ENTRIES = 16;                     // scale applications a wave fetches at a time
constexpr int W4_SCALE_LDS = W4_ENTRIES * (32 + 16);

struct W4Walk {
  int ks_log2;   // waves that share the k of a row tile
  int x_ld;      // bytes between tokens in LDS
};

constexpr int W4_WALK_WAVES = 8;
constexpr int W4_WALK_BLOCKS = 512;                // two a CU

// Up to 16 tokens in LDS, zero past k, so that no tile of W is a special case. Each block
// takes 8 >> ks_log2 row tiles at a time, and 1 << ks_log2 waves share the k of each.
// What bounds it: the instructions that unpack the codes, together with the start
// (x has to be in LDS before the first product). 22016x4096 2:4, bf16, one token:
// 8.9 us, 35 MB at 3.9 TB/s (w4_kernel 11.2; with loads alone, 7.0).
template <int XT, bool YB, bool SPARSE, bool ZEROS, int F>
__global__ void __launch_bounds__(64 * W4_WALK_WAVES) w4_walk_kernel(W4Args A, W4Walk P) {
  constexpr int ESZ = XT == DT_I8 ? 1 : 2;
  constexpr int S = XT == DT_I8 ? 2 : 4;         // matrix instructions along a tile
  constexpr int SF = S / F;                      // of them, between two scales
  constexpr int TK = SPARSE ? 256 : 128;         // k per tile
  constexpr int KS = TK / S;
  constexpr int CI = W4_ENTRIES / F;             // tiles whose scales come at a time
  typedef typename W4Type<XT>::acc acc_t;
  typedef typename W4Type<XT>::template b<SPARSE> b_t;
  struct Item { u32x4 c; u32x2 mt; };
  extern __shared__ floatx4 lds[];

  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, q = lane >> 4;
  floatx4* const red = lds;
  uint8_t* const own = (uint8_t*)(lds + waves * 64) + wave * W4_SCALE_LDS;   // this wave's scales and zero points
  uint8_t* const xs = (uint8_t*)(lds + waves * 64) + waves * W4_SCALE_LDS;

  const int ks = 1 << P.ks_log2, slice = wave & (ks - 1), per = waves >> P.ks_log2;
  const int step = gridDim.x * per;              // row tiles in a pass
  int base = blockIdx.x * per, rt = base + (wave >> P.ks_log2);

  // Row tiles past the last: that one again, its result not stored.
  auto load = [&](Item& T, int row_tile, int t) {
    const int64_t at = (int64_t)min(row_tile, A.row_tiles - 1) * A.tiles + t;
    gptr pc = (gptr)A.codes + at * 1024;
    asm("" : "+s"(pc));
    T.c = __builtin_nontemporal_load((gptr16)(pc + (uint32_t)lane * 16));
    if constexpr (SPARSE) {
      gptr pm = (gptr)A.meta + at * 512;
      asm("" : "+s"(pm));
      T.mt = __builtin_nontemporal_load((gptr8)(pm + (uint32_t)lane * 8));
    }
  };
  // lane 4 e + i: a quarter of the scales of this wave's application e from its tile t on;
  // returns whether that application begins before k (what lies past it meets no scale)
  auto load_scales = [&](u32x2& sc, uint32_t& zp, int row_tile, int t) -> bool {
    const int64_t r = min(row_tile, A.row_tiles - 1);
    const uint32_t e = lane >> 2, u = (t + (e / F << P.ks_log2)) * F + e % F;
    const int64_t g = r * A.groups + min(__umulhi(2 * u, A.group_magic), (uint32_t)A.groups - 1u);
    sc = *(const u32x2*)((const uint8_t*)A.scales + g * 32 + (lane & 3) * 8);
    if constexpr (ZEROS) zp = *(const uint32_t*)(A.zeros + g * 16 + (lane & 3) * 4);
    return u * (TK / F) < (uint32_t)A.k;
  };

  // x to LDS, 1 KB a wave at a time, eight of them on their way
  const int row_bytes = A.tiles * TK * ESZ, kb = A.k * ESZ, row_kb = (row_bytes + 1023) & ~1023;
  int xrow = 0, xc = wave * 1024, xat[8];
  u32x4 xv[8];
  auto x_load = [&]() {
#pragma unroll
    for (int u = 0; u < 8; u++) {
      while (xc >= row_kb && xrow < A.n) { xc -= row_kb; xrow++; }
      const int b = xc + lane * 16;
      xat[u] = xrow < A.n && b < row_bytes ? xrow * P.x_ld + b : -1;
      xv[u] = u32x4{0, 0, 0, 0};
      if (xat[u] >= 0) {
        const uint8_t* p = A.x + (int64_t)xrow * A.ldx * ESZ + b;
        if (b + 16 <= kb) xv[u] = *(const u32x4*)p;
        else
          for (int e = 0; e < kb - b; e++) xv[u][e / 4] |= (uint32_t)p[e] << (8 * (e % 4));
      }
      xc += waves * 1024;
    }
  };
  auto x_store = [&]() {
#pragma unroll
    for (int u = 0; u < 8; u++)
      if (xat[u] >= 0) *(u32x4*)(xs + xat[u]) = xv[u];
  };

  const uint8_t* const xl = xs + min(l16, A.n - 1) * P.x_ld + q * 16;
  // tile t; i: its place among those whose scales are in LDS
  auto compute = [&](const Item& T, int t, int i, floatx4& y) {
    const uint8_t* const xt = xl + t * (TK * ESZ);
    const uint8_t* const st = own + i * (F * 32) + q * 8;
    const uint8_t* const zt = own + W4_ENTRIES * 32 + i * (F * 16) + l16;
#pragma unroll
    for (int f = 0; f < F; f++) {
      const u32x2 sc = *(const u32x2*)(st + f * 32);
      W4Zero<XT, ZEROS> zp;
      zp.set(ZEROS ? zt[f * 16] : 8u);
      acc_t acc = acc_t{0, 0, 0, 0};
#pragma unroll
      for (int h = 0; h < SF; h++) {
        const int s = f * SF + h;
        uint32_t w[2];
        if constexpr (ESZ == 2) w[0] = T.c[s];
        else { w[0] = T.c[2 * s]; w[1] = T.c[2 * s + 1]; }
        const typename W4Type<XT>::a a = zp.unpack(w);
        int idx = 0;
        if constexpr (SPARSE) idx = ESZ == 2 ? (int)(T.mt[s / 2] >> (16 * (s % 2))) : (int)T.mt[s];
        const u32x4 b0 = *(const u32x4*)(xt + s * KS * ESZ);
        b_t b;
        if constexpr (SPARSE) {
          const u32x4 b1 = *(const u32x4*)(xt + (s * KS + KS / 2) * ESZ);
          b = __builtin_bit_cast(b_t, __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7));
        } else b = __builtin_bit_cast(b_t, b0);
        acc = w4_mma<XT, SPARSE>(a, b, acc, idx);
      }
#pragma unroll
      for (int e = 0; e < 4; e++)
        y[e] = __builtin_fmaf(from_bits16<YB ? DT_BF16 : DT_F16>((uint16_t)(sc[e / 2] >> (16 * (e % 2)))), (float)acc[e], y[e]);
    }
  };

  auto sync = [&]() {   // of LDS alone: loads from memory stay on their way
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  // the waves' sums of a pass, added in the order of the slices
  auto finish = [&](const floatx4& y) {
    red[wave * 64 + lane] = y;
    sync();
    if (slice == 0) {
      floatx4 v = y;
#pragma unroll 4
      for (int w = 1; w < ks; w++) v += red[(wave + w) * 64 + lane];
      w4_store<XT, YB, ZEROS>(A, v, l16, (int64_t)rt * 16 + 4 * q);
    }
    sync();
  };

  x_load();
  Item T0, T1;
  u32x2 sv;
  uint32_t zv = 0;
  int lt = slice, lrt = rt, ct = slice, st = slice, srt = rt, ci = CI;
  auto fetch = [&](Item& to) {
    load(to, lrt, lt);
    lt += ks;
    if (lt >= A.tiles) { lt = slice; lrt += step; }
    __builtin_amdgcn_sched_barrier(0);           // on its way before the products that follow
  };
  bool within = load_scales(sv, zv, srt, st);
  fetch(T0);
  for (;;) {
    x_store();
    if (xrow >= A.n) break;
    x_load();
  }
  sync();

  floatx4 y = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  // One tile, the next one's loads before it. The scales that follow are asked
  // for before those, or the wait for this tile would be one for the next as well.
  auto turn = [&](Item& cur, Item& next) {
    if (ci == CI) {
      *(u32x2*)(own + lane * 8) = within ? sv : u32x2{0, 0};
      if constexpr (ZEROS) *(uint32_t*)(own + W4_ENTRIES * 32 + lane * 4) = zv;
      st += CI << P.ks_log2;
      if (st >= A.tiles) { st = slice; srt += step; }
      within = load_scales(sv, zv, srt, st);
      ci = 0;
    }
    fetch(next);
    compute(cur, ct, ci, y);
    ci++;
    ct += ks;
    if (ct >= A.tiles) {
      if (base < A.row_tiles) finish(y);
      y = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
      base += step;
      rt += step;
      ct = slice;
      ci = CI;
    }
  };
  do {
    turn(T0, T1);
    turn(T1, T0);
  } while (base < A.row_tiles);
}

template <int XT, bool YB, bool SPARSE, bool ZEROS, int F, int NT, int R, bool XL>
hipError_t w4_go(const W4Args& a, int waves, hipStream_t s) {
  constexpr int TB = (SPARSE ? 256 : 128) * (XT == DT_I8 ? 1 : 2);
  hipLaunchKernelGGL((w4_kernel<XT, YB, SPARSE, ZEROS, F, NT, R, XL>),
                     dim3((unsigned)((a.row_tiles + R - 1) / R), (unsigned)((a.n + 16 * NT - 1) / (16 * NT))),
                     dim3(64 * waves), (size_t)waves * (NT * R * 1024 + (XL ? w4_turn(TB) : 0)), s, a);
  return hipGetLastError();
}

// Row tiles a block: the fewest row tiles for the busiest of 256 CUs, and among
// equals the most a block, which shares the loads of x (12288x4096, one f16 token: 9.2,
// 8.6, 7.3 and 7.9 us with 1, 2, 3 and 4).
inline int w4_rows(const W4Args& a, int nt, int most) {
  const int64_t cols = (a.n + 16 * nt - 1) / (16 * nt);
  int best = 1;
  int64_t least = 0;
  for (int r = 1; r <= most; r++) {
    const int64_t load = ((a.row_tiles + r - 1) / r * cols + 255) / 256 * r;
    if (r == 1 || load <= least) { best = r; least = load; }
  }
  return best;
}

// Waves a block: 8 where a CU has one block, 4 where it has several (12288x4096: 7.3 and
// 7.5 us; 32003x4096: 17.0 and 15.6), at most one a tile of k.
inline int w4_waves(const W4Args& a, int nt, int r) {
  const int64_t blocks = (int64_t)((a.row_tiles + r - 1) / r) * ((a.n + 16 * nt - 1) / (16 * nt));
  int w = blocks <= 256 ? 8 : 4;
  while (w > 1 && w > a.tiles) w /= 2;
  return w;
}

// More than four tokens have x turned, where fewer than four row tiles share its loads
// (2:4 4096x11008, sixteen 8-bit tokens: 7.2 us, 8.8 without; four tokens 6.9 and 6.9;
// 16384x4096, sixteen f16 tokens: 9.0 and 8.9).
template <int XT, bool YB, bool SPARSE, bool ZEROS, int F, int NT, int R>
hipError_t w4_try(const W4Args& a, int r, hipStream_t s) {
  if constexpr (R > 1) {
    if (r < R) return w4_try<XT, YB, SPARSE, ZEROS, F, NT, R - 1>(a, r, s);
  }
  if constexpr (NT == 1 && R <= 3) {
    if (a.n > 4) return w4_go<XT, YB, SPARSE, ZEROS, F, NT, R, true>(a, w4_waves(a, NT, R), s);
  }
  return w4_go<XT, YB, SPARSE, ZEROS, F, NT, R, false>(a, w4_waves(a, NT, R), s);
}

// The walk: where w4_kernel would hold 32 registers of x a tile, twice, and a CU gets
// more than four row tiles (22016x4096 2:4: 8.9 against 11.2 us; 12288x4096: 7.7
// against 7.0), as long as two blocks' x fit a CU's LDS.
template <int XT, bool YB, bool ZEROS, int F>
bool w4_walk(const W4Args& a, hipStream_t s, hipError_t& err) {
  const int x_ld = (a.tiles * 512 + 255) / 256 * 256 + 16;   // 16 bytes on: the tokens of a read lie in different banks
  const size_t lds = (size_t)W4_WALK_WAVES * (1024 + W4_SCALE_LDS) + (size_t)a.n * x_ld;
  if (a.n > 16 || a.row_tiles <= 1024 || a.tiles == 0 || lds > 80 * 1024) return false;   // k = 0: nothing to load
  // waves a row tile: the fewest tiles, and a joining of sums that costs about one, for the busiest CU
  W4Walk w = {0, x_ld};
  int64_t least = -1;
  for (int k = 0; (1 << k) <= W4_WALK_WAVES && (1 << k) <= a.tiles; k++) {
    const int64_t per = W4_WALK_WAVES >> k, pass = W4_WALK_BLOCKS * per, half = W4_WALK_BLOCKS / 2 * per;
    const int64_t passes = (a.row_tiles + pass - 1) / pass + (a.row_tiles > half ? (a.row_tiles - half + pass - 1) / pass : 0);
    const int64_t load = passes * (((a.tiles + (1 << k) - 1) >> k) + 1);
    if (least < 0 || load < least) { least = load; w.ks_log2 = k; }
  }
  hipLaunchKernelGGL((w4_walk_kernel<XT, YB, true, ZEROS, F>), dim3(W4_WALK_BLOCKS), dim3(64 * W4_WALK_WAVES), lds, s, a, w);
  err = hipGetLastError();
  return true;
}

template <int XT, bool YB, bool SPARSE, bool ZEROS, int F>
hipError_t w4_cols(const W4Args& a, hipStream_t s) {
  if constexpr (SPARSE && XT != DT_I8) {
    hipError_t e;
    if (w4_walk<XT, YB, ZEROS, F>(a, s, e)) return e;
  }
  if (a.n <= 16) return w4_try<XT, YB, SPARSE, ZEROS, F, 1, 4>(a, w4_rows(a, 1, 4), s);
  if (a.n <= 32) return w4_try<XT, YB, SPARSE, ZEROS, F, 2, 2>(a, w4_rows(a, 2, 2), s);
  return w4_try<XT, YB, SPARSE, ZEROS, F, 3, 2>(a, w4_rows(a, 3, 2), s);
}

template <int XT, bool YB, bool SPARSE, bool ZEROS>
hipError_t w4_flush(const W4Args& a, const W4Shape& sh, hipStream_t s) {
  if (sh.flushes == 1) return w4_cols<XT, YB, SPARSE, ZEROS, 1>(a, s);
  if (sh.flushes == 2) return w4_cols<XT, YB, SPARSE, ZEROS, 2>(a, s);
  if constexpr (XT != DT_I8) return w4_cols<XT, YB, SPARSE, ZEROS, 4>(a, s);
  return hipErrorInvalidValue;
}

template <int XT, bool YB>
hipError_t w4_dispatch(const W4Args& a, const W4Shape& sh, hipStream_t s) {
  if (sh.sparse) return sh.zeros ? w4_flush<XT, YB, true, true>(a, sh, s) : w4_flush<XT, YB, true, false>(a, sh, s);
  return sh.zeros ? w4_flush<XT, YB, false, true>(a, sh, s) : w4_flush<XT, YB, false, false>(a, sh, s);
}

}  // namespace nm
