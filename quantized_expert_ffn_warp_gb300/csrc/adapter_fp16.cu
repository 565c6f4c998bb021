// The adapters' products for fp16 activations.
#include "adapter_mma.cuh"

namespace qe {

cudaError_t adapter_fp16(const AdapterCall &c, cudaStream_t st)
{
    return run_adapter<__half>(c, st);
}
cudaError_t adapter_grad_fp16(const AdapterGradCall &c, cudaStream_t st)
{
    return run_adapter_grad<__half>(c, st);
}

}  // namespace qe
