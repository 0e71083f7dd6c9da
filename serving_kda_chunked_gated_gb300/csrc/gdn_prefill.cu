// bf16 prefill of the scalar-gated delta rule: the per-token recurrence.
#include "kda_common.cuh"

namespace kda {
namespace gdn {

cudaError_t launch_recurrent(const kda_gdn_prefill_args& a, cudaStream_t s);

size_t chunked_workspace_size(const kda_gdn_prefill_args&) { return 256; }   // the error word

cudaError_t launch_chunked(const kda_gdn_prefill_args& a, cudaStream_t s) {
    const cudaError_t e = cudaMemsetAsync(a.workspace, 0, 4, s);
    return e != cudaSuccess ? e : launch_recurrent(a, s);
}

}  // namespace gdn
}  // namespace kda
