// Attention of drafted tokens in trees: the attention kernel's TREE instances
// (prefill_kernel.cuh).
#include "prefill_kernel.cuh"

namespace msa {

cudaError_t launch_tree(const PrefillArgs& a, cudaStream_t s) { return launch_attention<true>(a, s); }

}  // namespace msa
