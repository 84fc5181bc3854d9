// The norm kernels (norm_kernel.hpp) for an fp32 stream with fp16 activations; one set of element
// types per translation unit, the kernels of one being many.
#include "norm_kernel.hpp"

namespace w8a8 {

hipError_t launch_norm_rows_f32_f16(const NormRowsArgs &a, hipStream_t stream) { return launch<kF32, kF16>(a, stream); }

}  // namespace w8a8
