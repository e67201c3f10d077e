// The layer-norm kernels for bf16 elements.
#include "norm_kernels.cuh"

namespace attn {
namespace norm {

template int run_fwd<__nv_bfloat16>(const FwdArgs& a, cudaStream_t stream);
template int run_bwd<__nv_bfloat16>(const BwdArgs& a, cudaStream_t stream);

}  // namespace norm
}  // namespace attn
