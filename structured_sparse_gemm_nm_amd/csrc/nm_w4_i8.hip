// 4-bit weight product, i8 activations and f16 output (see nm_w4_kernels.h; bf16 output: nm_w4_i8_bf16.hip).
#include "nm_w4_kernels.h"

namespace nm {

hipError_t launch_w4_i8_f16(const W4Args& a, const W4Shape& sh, hipStream_t s) { return w4_dispatch<DT_I8, false>(a, sh, s); }

}  // namespace nm
