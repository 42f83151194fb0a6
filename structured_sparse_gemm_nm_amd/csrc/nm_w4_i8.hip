// 4-bit weight product, i8 activations (see nm_w4_kernels.h).
#include "nm_w4_kernels.h"

namespace nm {

hipError_t launch_w4_i8(const W4Args& a, const W4Shape& sh, hipStream_t s) { return w4_dispatch<DT_I8>(a, sh, s); }

}  // namespace nm
