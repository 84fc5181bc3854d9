// The norm kernels (norm_kernel.hpp) for bf16 throughout; one set of element
// types per translation unit, the kernels of one being many.
#include "norm_kernel.hpp"

namespace w8a8 {

hipError_t launch_norm_rows_bf16(const NormRowsArgs &a, hipStream_t stream) { return launch<kBF16, kBF16>(a, stream); }

}  // namespace w8a8
