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
// A block takes R tiles of 16 rows; its waves share out the tiles of k, two of them in
// registers at a time, with their piece of x, and add their sums through LDS in wave
// order (the order of a sum depends on the shape alone). The matrix instruction's 16
// columns hold the tokens; columns past n repeat the last token's address (the same
// cache line) and are not stored. Up to NT * 16 tokens share one pass over the weights.
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
//       fp32, whose upper half is the value's bf16. Without zero points the
//       conversion of a 4-bit two's complement nibble gives (q - 8) / 16, and the
//       16 is multiplied into the result: a sum that fp32 holds cannot overflow on
//       the way, and products of bf16 values by multiples of 1/16 down to fp32's
//       smallest are exact.
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

template <> struct W4Zero<DT_BF16, true> {
  W4Bytes<true> b;
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

template <> struct W4Zero<DT_BF16, false> {
  __device__ __forceinline__ void set(uint32_t) {}
  __device__ __forceinline__ bf16x8_t unpack(const uint32_t* w) const {
    uint32_t h[2] = {w[0], w[0] >> 4};
    asm("" : "+v"(h[1]));   // shifted once, its bytes picked by the conversions
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const uint32_t v = h[i / 2] >> (16 * (i % 2));
      r[i] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_off_f32_i4((int)(v >> 8 & 0xFF))),
                                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_off_f32_i4((int)(v & 0xFF))), 0x07060302u);
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

// 8-bit codes without zero points are held times 16. Where y is bf16 the scale takes
// the 1/16, so that no sum overflows early; f16 scales times the largest sum stay under
// 2^52, and y takes it, which leaves the scale to a mixed multiply-add (2:4 4096x11008,
// sixteen tokens: 662 vector instructions a SIMD, 838 with the scale's product).
template <int XT, bool ZEROS> constexpr bool W4_SIXTEEN = XT == DT_I8 && !ZEROS;

// Four rows of one column of y from `row` on.
template <int XT, bool YB, bool ZEROS>
__device__ __forceinline__ void w4_store(const W4Args& A, floatx4 v, int col, int64_t row) {
  if (col >= A.n || row >= A.m) return;
  if constexpr (W4_SIXTEEN<XT, ZEROS> && !YB) v *= 0.0625f;
  if constexpr (XT == DT_I8) v *= A.x_scale[col];
  if constexpr (XT == DT_BF16 && !ZEROS) v *= 16.0f;     // these codes are held as sixteenths
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

// What one tile of k of R row tiles needs from memory besides scales; x with it for up to 16 tokens.
template <int XT, bool SPARSE, int NT, int R, bool XL> struct W4Tile {
  u32x4 c[R];
  u32x2 mt[R];
  std::conditional_t<XL, u32x4[(XT == DT_I8 ? 2 : 4) * (SPARSE ? 2 : 1)],
                     typename W4Type<XT>::template b<SPARSE>[NT == 1 ? (XT == DT_I8 ? 2 : 4) : 1]> x;
};

// A wave fetches the scales and zero points of 16 applications of a row tile at a time, into its own LDS.
constexpr int W4_ENTRIES = 16;
constexpr int W4_SCALE_LDS = W4_ENTRIES * (32 + 16);

// Bytes of LDS in which a wave turns a tile of x, 16 tokens 16 bytes apart in their banks.
constexpr int w4_turn(int tile_bytes) { return 16 * (tile_bytes + 16); }

// Lanes of a wave read what its other lanes wrote to LDS, and write over it once all
// have read. A wave's LDS operations are carried out in their order, so this emits no
// instruction; it keeps the compiler from moving them past each other.
__device__ __forceinline__ void w4_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// What bounds it: loads other than the codes'. x comes from the L1 cache, 1 KB (2:4:
// 2 KB) a matrix instruction against 256 to 512 bytes of codes, so each piece of x serves
// R row tiles; and R is chosen so that the blocks are whole rounds of the 256 CUs. The
// matrix instruction's order has neighbouring lanes load from different tokens, a
// cache line each; with XL they load a token's row along, and the wave turns the tile in
// LDS. Scales come for 16 applications at a time: fetched with each tile, 8 bytes a lane,
// they cost 32003x4096 (five tokens, two scales a tile) 15.6 us instead of 13.4 (70 MB,
// 5.2 TB/s). 16384x4096, one f16 token, 8.2 us with R = 4 (34 MB, 4.2 TB/s; 10.3 with
// R = 1), 16 tokens 8.9 (17.8); 32768x32768, four 8-bit tokens, 88 us (562 MB, 6.4 TB/s;
// 97 with R = 1); 2:4 22016x4096, one bf16 token, 9.2 us (35 MB, 3.8 TB/s).
// Codes are loaded past the caches' reuse (nontemporal): x stays there.
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
  typedef W4Tile<XT, SPARSE, NT, R, XL> tile_t;
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

  // Lane 4 e + i: a quarter of the scales of this wave's application e from its tile t
  // on; those that begin past k are 0, whatever the scale.
  uint8_t* const own = (uint8_t*)(red + waves * NT * R * 64) + wave * (R * W4_SCALE_LDS);
  u32x2 sv[R];
  uint32_t zv[R];
  bool within = false;
  auto load_scales = [&](int t) {
    const uint32_t e = lane >> 2, u = (uint32_t)(t + (int)(e / F) * waves) * F + e % F;
    const uint32_t g = min(__umulhi(2 * u, A.group_magic), (uint32_t)A.groups - 1u);
    within = u * (TK / F) < (uint32_t)A.k;
#pragma unroll
    for (int r = 0; r < R; r++) {
      const int64_t at = rt[r] * A.groups + g;
      sv[r] = *(const u32x2*)((const uint8_t*)A.scales + at * 32 + (lane & 3) * 8);
      if constexpr (ZEROS) zv[r] = *(const uint32_t*)(A.zeros + at * 16 + (lane & 3) * 4);
    }
  };
  constexpr int CI = W4_ENTRIES / F;             // tiles whose scales come at a time
  int ci = CI, st = wave;
  // Before the first tile of each CI: what was fetched goes to LDS, the next is asked for.
  auto scales_ready = [&]() {
    if (ci < CI) return;
    ci = 0;
    w4_lds_order();
#pragma unroll
    for (int r = 0; r < R; r++) {
      *(u32x2*)(own + r * W4_SCALE_LDS + lane * 8) = within ? sv[r] : u32x2{0, 0};
      if constexpr (ZEROS) *(uint32_t*)(own + r * W4_SCALE_LDS + W4_ENTRIES * 32 + lane * 4) = zv[r];
    }
    w4_lds_order();
    st += CI * waves;
    if (st < A.tiles) load_scales(st);
  };

  uint8_t* const turn = (uint8_t*)(red + waves * NT * R * 64) + waves * (R * W4_SCALE_LDS) + wave * w4_turn(TB);
  auto compute = [&](const tile_t& T, int t, bool whole) {
    if constexpr (XL) {
      w4_lds_order();
#pragma unroll
      for (int i = 0; i < 16 * TB / 1024; i++)
        *(u32x4*)(turn + (i * (64 / LPR) + lane / LPR) * (TB + 16) + lane % LPR * 16) = T.x[i];
      w4_lds_order();
    }
#pragma unroll
    for (int f = 0; f < F; f++) {
      W4Zero<XT, ZEROS> zp[R];
      acc_t acc[R][NT];
      u32x2 sc[R];
#pragma unroll
      for (int r = 0; r < R; r++) {
        sc[r] = *(const u32x2*)(own + r * W4_SCALE_LDS + (ci * F + f) * 32 + q * 8);
        zp[r].set(ZEROS ? own[r * W4_SCALE_LDS + W4_ENTRIES * 32 + (ci * F + f) * 16 + l16] : 8u);
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
          float s1 = from_bits16<YB ? DT_BF16 : DT_F16>((uint16_t)(sc[r][e / 2] >> (16 * (e % 2))));
          if constexpr (W4_SIXTEEN<XT, ZEROS> && YB) s1 *= 0.0625f;   // f16's scales leave room for 16 times the sums
#pragma unroll
          for (int j = 0; j < NT; j++) y[r][j][e] = __builtin_fmaf(s1, (float)acc[r][j][e], y[r][j][e]);
        }
      // The sums are taken here, in the block of the matrix instructions. Left to itself the compiler moves this
      // behind the next tile's early return, and leaves out wait states on the way there; the build reads the
      // units for it.
#pragma unroll
      for (int r = 0; r < R; r++)
#pragma unroll
        for (int j = 0; j < NT; j++) asm volatile("" : "+v"(y[r][j]));
    }
    ci++;
  };

  // Two tiles in turn, the next one's loads behind the present one's products.
  // Every path into a product has the same loads behind it, or the wait for
  // them would be a wait for all.
  const int full = A.k / TK;      // tiles that lie within k whole
  if (wave < A.tiles) load_scales(wave);
  if (wave < full) {
    int t = wave;
    tile_t T0, T1;
    load(T0, t, true);
    for (;;) {
      scales_ready();
      t += waves;
      if (t >= full) { compute(T0, t - waves, true); break; }
      load(T1, t, true);
      compute(T0, t - waves, true);
      scales_ready();
      t += waves;
      if (t >= full) { compute(T1, t - waves, true); break; }
      load(T0, t, true);
      compute(T1, t - waves, true);
    }
  }
  if (full < A.tiles && full % waves == wave) {
    tile_t T;
    load(T, full, false);
    scales_ready();
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

template <int XT, bool YB, bool SPARSE, bool ZEROS, int F, int NT, int R, bool XL>
hipError_t w4_go(const W4Args& a, int waves, hipStream_t s) {
  constexpr int TB = (SPARSE ? 256 : 128) * (XT == DT_I8 ? 1 : 2);
  hipLaunchKernelGGL((w4_kernel<XT, YB, SPARSE, ZEROS, F, NT, R, XL>),
                     dim3((unsigned)((a.row_tiles + R - 1) / R), (unsigned)((a.n + 16 * NT - 1) / (16 * NT))),
                     dim3(64 * waves), (size_t)waves * (R * (NT * 1024 + W4_SCALE_LDS) + (XL ? w4_turn(TB) : 0)), s, a);
  return hipGetLastError();
}

// Row tiles a block: the fewest row tiles for the busiest of 256 CUs, and among
// equals the most a block, which shares the loads of x (12288x4096, one f16 token: 8.3,
// 7.8, 6.7 and 7.2 us with 1, 2, 3 and 4).
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

// Waves a block: 8 where a CU has one block, 4 where it has several (12288x4096: 6.7 and
// 7.3 us; 32003x4096: 15.1 and 13.7), at most one a tile of k.
inline int w4_waves(const W4Args& a, int nt, int r) {
  const int64_t blocks = (int64_t)((a.row_tiles + r - 1) / r) * ((a.n + 16 * nt - 1) / (16 * nt));
  int w = blocks <= 256 ? 8 : 4;
  while (w > 1 && w > a.tiles) w /= 2;
  return w;
}

// More than four tokens have x turned, where fewer than four row tiles share its loads
// (2:4 4096x11008, sixteen 8-bit tokens: 7.2 us, 8.6 without; four tokens 6.7 and 6.5;
// 16384x4096, sixteen f16 tokens: 9.2 and 8.9).
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

template <int XT, bool YB, bool SPARSE, bool ZEROS, int F>
hipError_t w4_cols(const W4Args& a, hipStream_t s) {
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
