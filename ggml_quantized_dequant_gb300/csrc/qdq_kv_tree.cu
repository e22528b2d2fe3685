// Attention of a sequence's tree of drafted tokens over the paged 8-bit cache.
//
//   node i of n, the i-th of the sequence's last n tokens, at position kv_len - n + depth(i), sees
//   the tokens j < kv_len - n, its ancestors and itself; scores, cap, bias, window and sums as in qdq_kv_attn.cu.
//
// The kernels are those of qdq_kv_attn_kernel.cuh and qdq_kv_attn_tc_kernel.cuh with the visibility of a tree: a row's drafted
// tokens are 64 bits, which a CTA finds by walking the parents of its sequence's nodes in shared memory (one thread per
// node, at most 64 steps), and blocks of 16 tokens below the tree need no mask.
//
// Here the instances for few rows per cache head, which read the codes once for every 16 rows.  Measured: 13 nodes behind 764
// tokens, 24 / 8 heads of 128, f32 10.0 us; 9 trees of up to 31 nodes behind 200 to 6001 tokens, 16 / 2 heads of 64, f16, cap, bias
// and a window of 1500 32.6 us.  Bound: the chain of launch, length, page, codes and the join of the parts.
#include "qdq_kv_attn_kernel.cuh"

namespace qdq {

cudaError_t launch_attn_tree(const AttnArgs &a, int head_dim, int parts, int warps, int ctas, cudaStream_t s) {
  return run_attn<true>(a, head_dim, parts, warps, ctas, s);
}

QDQ_CHECK_READER(read_checks_tree)

}  // namespace qdq
