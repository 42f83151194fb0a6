// 4-bit weight product, i8 activations and bf16 output (see nm_w4_kernels.h).
#include "nm_w4_kernels.h"

namespace nm {

hipError_t launch_w4_i8_bf16(const W4Args& a, const W4Shape& sh, hipStream_t s) { return w4_dispatch<DT_I8, true>(a, sh, s); }

}  // namespace nm
