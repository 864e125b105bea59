// linear_tc_bf16.cu -- the tensor-core kernels of moe_linear for bf16 operands (a unit per type, compiled in parallel).
#include "linear_tc.cuh"

namespace moe {

cudaError_t launch_linear_tc_bf16(const LinearArgs& l, cudaStream_t st) { return launch_tc_type<false>(l, st); }

}  // namespace moe
