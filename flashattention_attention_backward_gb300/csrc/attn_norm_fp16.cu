// The layer-norm kernels for fp16 elements.
#include "norm_kernels.cuh"

namespace attn {
namespace norm {

template int run_fwd<__half>(const FwdArgs& a, cudaStream_t stream);
template int run_bwd<__half>(const BwdArgs& a, cudaStream_t stream);

}  // namespace norm
}  // namespace attn
