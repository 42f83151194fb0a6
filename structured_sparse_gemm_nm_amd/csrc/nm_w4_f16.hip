// 4-bit weight product, f16 activations (see nm_w4_kernels.h).
#include "nm_w4_kernels.h"

namespace nm {

hipError_t launch_w4_f16(const W4Args& a, const W4Shape& sh, hipStream_t s) { return w4_dispatch<DT_F16, false>(a, sh, s); }

}  // namespace nm
