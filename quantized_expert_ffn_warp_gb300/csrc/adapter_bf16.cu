// The adapters' products for bf16 activations.
#include "adapter_mma.cuh"

namespace qe {

cudaError_t adapter_bf16(const AdapterCall &c, cudaStream_t st)
{
    return run_adapter<__nv_bfloat16>(c, st);
}
cudaError_t adapter_grad_bf16(const AdapterGradCall &c, cudaStream_t st)
{
    return run_adapter_grad<__nv_bfloat16>(c, st);
}

}  // namespace qe
