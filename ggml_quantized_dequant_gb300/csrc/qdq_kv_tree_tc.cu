// Attention of trees of drafted tokens on the tensor cores: the instances of qdq_kv_attn_tc_kernel.cuh whose rows
// see what was cached before the tree, their ancestors and themselves (see qdq_kv_tree.cu).
//
// A tree has at most 64 nodes, so that a cache head's rows are mostly one tile of 128: up to heads of 128 the two groups
// of softmax warps take alternate tiles of 64 tokens of the same rows (one group alone: 243 us for the long one below, its
// chain of products, softmax and conversions waits for itself), one set of warps converts keys and one values, codes come
// for pairs of tiles in copies of whole runs of blocks, and the groups' halves are joined in shared memory at the end.
// Parts of a split line are joined by a kernel of its own, 16 dims to a CTA.
// Measured: 26 nodes behind 131045 tokens, 32 / 8 heads of 128, bf16 129 us (2.1 TB/s of codes); 16 trees of 7 to 64 nodes behind
// 300 to 8191 tokens, 24 / 8 heads 125 us.
// Bound: the chain between the warps.  Without conversions the long one takes 101 us, without softmax 127, with neither 95, with
// codes that are in the L2 122; issue slots are 53 % busy, memory 30 %.
#include "qdq_kv_attn_tc_kernel.cuh"

namespace qdq {

cudaError_t launch_attn_tree_tc(const AttnArgs &a, int head_dim, int parts, int groups, cudaStream_t s) {
  return run_attn_tc<true>(a, head_dim, parts, groups, s);
}

QDQ_CHECK_READER(read_checks_tree_tc)

int read_attn_tree_tc_timeouts() { return read_timeouts(); }

}  // namespace qdq
