// Internal declarations of the 4-bit weight product (nm_w4_*).
#pragma once
#include "nm_internal.h"

struct nm_w4_plan {
  nm_w4_problem_t p;
  int64_t row_tiles;    // tiles of 16 rows of W
  int64_t tiles;        // tiles of 128 kept values along k
  int64_t groups;       // scales per row
  int flushes;          // scale applications per tile of k
  uint32_t group_magic; // see W4Args
  int64_t code_ld;      // bytes per row of the codes as handed to nm_w4_pack
  int64_t meta_ld;      // bytes per row of the 2:4 metadata
  size_t meta_off, scale_off, zero_off, packed_bytes;
};

namespace nm {

// One launch of the product. The packed buffer holds, for row tile r, k tile t
// and lane l of a wave:
//   codes  [r][t][l][16 bytes]   the 32 codes lane l feeds to the matrix unit
//   meta   [r][t][l][8 bytes]    their 2:4 offsets (sparse only)
//   scales [r][g][16 rows]       16-bit
//   zeros  [r][g][16 rows]       bytes (zero points only)
struct W4Args {
  const uint8_t* codes;
  const uint8_t* meta;
  const uint16_t* scales;
  const uint8_t* zeros;
  const uint8_t* x;
  const float* x_scale;
  uint16_t* y;
  int64_t ldx, ldy;
  int32_t m, n, k;
  int32_t row_tiles, tiles, groups;
  uint32_t group_magic;  // group of scale application u: umulhi(2 u, group_magic)
};

struct W4Shape {
  bool sparse, zeros;
  int flushes;
};

hipError_t launch_w4_f16(const W4Args& a, const W4Shape& sh, hipStream_t s);
hipError_t launch_w4_bf16(const W4Args& a, const W4Shape& sh, hipStream_t s);
hipError_t launch_w4_i8_f16(const W4Args& a, const W4Shape& sh, hipStream_t s);
hipError_t launch_w4_i8_bf16(const W4Args& a, const W4Shape& sh, hipStream_t s);

}  // namespace nm
