// tree_attn_e4m3.cu - gdn_tree_attention's kernel for an E4M3 cache (tree_attn.cuh).
#include "tree_attn.cuh"

namespace gdn {
namespace tree_attn {

cudaError_t launch_e4m3(const Args& a, const CUtensorMap& tmk, const CUtensorMap& tmv, int grid, cudaStream_t stream) {
  return launch_format<true>(a, tmk, tmv, grid, stream);
}

}  // namespace tree_attn
}  // namespace gdn
