// Attention of trees of drafted tokens on the tensor cores: the instances of qdq_kv_attn_tc_kernel.cuh whose rows
// see what was cached before the tree, their ancestors and themselves (see qdq_kv_tree.cu).
#include "qdq_kv_attn_tc_kernel.cuh"

namespace qdq {

cudaError_t launch_attn_tree_tc(const AttnArgs &a, int head_dim, int parts, int groups, cudaStream_t s) {
  return run_attn_tc<true>(a, head_dim, parts, groups, s);
}

QDQ_CHECK_READER(read_checks_tree_tc)

int read_attn_tree_tc_timeouts() { return read_timeouts(); }

}  // namespace qdq
