// tree_attn_bf16.cu - gdn_tree_attention's kernel for a bf16 cache (tree_attn.cuh).
#include "tree_attn.cuh"

namespace gdn {
namespace tree_attn {

cudaError_t launch_bf16(const Args& a, const CUtensorMap& tmk, const CUtensorMap& tmv, int grid, cudaStream_t stream) {
  return launch_format<false>(a, tmk, tmv, grid, stream);
}

}  // namespace tree_attn
}  // namespace gdn
