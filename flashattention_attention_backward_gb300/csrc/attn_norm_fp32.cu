// The layer-norm kernels for fp32 elements.
#include "norm_kernels.cuh"

namespace attn {
namespace norm {

template int run_fwd<float>(const FwdArgs& a, cudaStream_t stream);
template int run_bwd<float>(const BwdArgs& a, cudaStream_t stream);

}  // namespace norm
}  // namespace attn
