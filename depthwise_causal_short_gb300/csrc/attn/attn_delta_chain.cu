// attn_delta_chain.cu -- launches of the chain over the chunks: the forward, and the gradient's states.
#include "attn_delta_chain.cuh"

namespace cattn {

static __device__ unsigned g_fault_chain;
static int read_fault(unsigned* out) {
  const unsigned zero = 0;
  if (report_cuda("fault word", cudaMemcpyFromSymbol(out, g_fault_chain, sizeof(*out))) != cudaSuccess ||
      (*out && report_cuda("fault word", cudaMemcpyToSymbol(g_fault_chain, &zero, sizeof(zero))) !=
                   cudaSuccess))
    return CCONV_ERR_CUDA;
  return CCONV_OK;
}
static FaultReader reader(read_fault);

template <bool BWD>
__global__ void __launch_bounds__(chain::kThreads, 1) cattn_delta_chain_kernel(const __grid_constant__ chain::Args p) {
  chain::run<BWD>(p, static_cast<int>(blockIdx.x), &g_fault_chain);
}

template <bool BWD>
static int launch_chain(const DeltaCall& c, cudaStream_t stream) {
  chain::Args a{};
  const int rc = chain::args_of(c, a);
  if (rc != CCONV_OK) return rc;
  auto kern = cattn_delta_chain_kernel<BWD>;
  if (cconv::set_max_dynamic_smem(reinterpret_cast<const void*>(kern), chain::kBytes) != CCONV_OK)
    return CCONV_ERR_CUDA;
  return launch_pdl(kern, dim3(chain::ctas(c)), dim3(chain::kThreads), chain::kBytes, stream, a) == cudaSuccess
             ? CCONV_OK
             : CCONV_ERR_CUDA;
}

int launch_delta_fwd(const DeltaCall& c, cudaStream_t stream) { return launch_chain<false>(c, stream); }
int launch_delta_states(const DeltaCall& c, cudaStream_t stream) { return launch_chain<true>(c, stream); }

}  // namespace cattn
