// moe_add_norm for x of MOE_T_BF16.
#include "add_norm.cuh"

namespace moe {

template cudaError_t add_norm_of<MOE_T_BF16>(const AddNormArgs &a, Grid grid, int sms, cudaStream_t s);

}  // namespace moe
