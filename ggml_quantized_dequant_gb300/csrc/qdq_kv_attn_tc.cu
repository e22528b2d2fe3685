// Attention of many query rows over the paged 8-bit cache on the 5th-generation tensor cores
// (prompt chunks; the formulas are those of qdq_kv_attn.cu).
//
// A unit is one or two groups of 128 rows (query token, head of the group) of one key/value head;
// its work is the tiles of 64 tokens that its rows see.  All units' tiles and their parts' costs in one
// line are cut into equal shares, one per CTA (causal tiles and ragged sequences differ in length), so a
// CTA takes the end of a unit, whole units and the start of another, part by part.  A unit cut by
// shares is joined from its parts' accumulators by the CTA that finishes last, in order.  For each tile:
//   S = Q K^T (128 x 64, f32 in TMEM), P = 2^(S - reference) in f16 written over S in TMEM,
//   O += P V (128 x D, f32 in TMEM).
// Codes are exact in f16, so K and V tiles are converted in registers, without their scales, into
// the 128-byte-swizzled layout the tensor core reads (V transposed on the way, four by four bytes); a
// block's key scale multiplies its 16 columns of S, its value scale the probabilities.
//   one part (16-bit activations): the queries are exact in f16 but for elements 2^-25 below the
//     row's largest, the probabilities are rounded to f16 (2^-11 relative, as the output is);
//   two parts (f32): queries and probabilities in two f16 parts each, twice the products.
//
// Warp roles (G groups of rows):
//   4 G softmax warps: one row per thread (a TMEM lane), so its maximum and sum need no exchange;
//              O is rescaled only when a reference has grown by 2^kLazy;
//   8 warps that convert the codes, as two sets of 4 taking alternate tiles, so that the loads and
//              the fence of one tile run beside the conversion of the other;
//   G warps that issue the products of a group (the first also allocates TMEM): S of tile i + 1 before P V
//              of tile i, so that the tensor core works while the softmax of a tile runs;
//   1 warp that brings the codes (bulk copies).
// Bound: the chain of a tile (codes converted, S, softmax, P V: 1.2 us a tile, no unit more than half busy)
// and what a part costs besides (queries 5 us, output 4 us, a join 8 us).  Measured: 2 prompts of 512 queries
// over 3500 to 4600 tokens, 24 / 8 heads of 128, bf16: 85 us, 0.56 PFLOP/s; the decode kernel took 278 us.
// One CTA per SM.  Two groups (head dims up to 128) share each tile's conversion.  Every wait is
// bounded; one that runs out makes the CTA's rows NaN and counts in qdq_pipeline_timeouts.
#include "qdq_kv_attn_tc_kernel.cuh"

namespace qdq {

cudaError_t launch_attn_tc(const AttnArgs &a, int head_dim, int parts, int groups, cudaStream_t s) {
  return run_attn_tc<false>(a, head_dim, parts, groups, s);
}

QDQ_CHECK_READER(read_checks_attn_tc)

int read_attn_tc_timeouts() {  // of both
  const int tree = read_attn_tree_tc_timeouts(), own = read_timeouts();
  return tree < 0 || own < 0 ? -1 : own + tree;
}

}  // namespace qdq
