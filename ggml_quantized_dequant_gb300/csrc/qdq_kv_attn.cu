// Attention of query tokens over the paged 8-bit cache.
//
//   s[j] = scale * q . (kc[j] * ks[j / 16])        (kc, vc: int8 codes; ks, vs: a block's scales)
//   s[j] = cap * tanh(s[j] / cap)                   when cap > 0
//   s[j] -= slope * (pos - j)                       when slopes are given
//   o    = sum_j e^(s[j] - m) vc[j] vs[j / 16] / sum_j e^(s[j] - m)  over the visible j
//
// Rows are (query token, head of the group) pairs that share a key/value head.  A warp walks
// blocks of 16 tokens: their codes come through a ring of asynchronous copies in its own part of
// shared memory (16-byte chunks exchanged by row so that the fragment loads below meet no bank
// conflict) and become the operands of 16-row matrix instructions with 16-bit operands (a code
// is exact in f16).  A query row is scaled by a power of two to below 2^14 first.
//   two parts (f32 activations; a tile is 8 rows): instruction rows 0-7 hold the high f16 part
//     of the queries, rows 8-15 the rest in f16, so the products are exact and a score has f32
//     precision; the probabilities are split the same way.
//   one part (16-bit activations with more than 8 rows per head; a tile is 16 rows): the queries
//     are exact in f16 but for elements 2^-25 below the row's largest, the
//     probabilities are rounded to f16 (2^-11 relative, as the output is).
// The running maximum, the sum and the accumulators are f32.  The warps of a CTA (4, or 16 or 8
// where there are few tiles) take blocks of their split of the tokens in turn and are joined through
// shared memory; splits of one tile are joined by the CTA that finishes last, in split order.
// Bound: memory for many or long sequences (a code is read once for all rows of its head); for a short one the
// chain of a launch, length, page, codes, joins.  Measured (8 heads of 128 in the cache): one sequence of
// 777 tokens, 24 heads f32 9.0 us; 48 of 1 to 8191 78.5 us (5.2 TB/s, 76 % of a plain copy's rate); one of 131071
// tokens, 32 heads bf16 50.6 us (5.3 TB/s, 78 %).
#include <algorithm>

#include "qdq_kv_attn_kernel.cuh"

namespace qdq {

std::atomic<int> g_opt_attn_kernel{0};

namespace {

// Query rows per key/value head from which on the tensor-core kernel runs.  This file's kernel is kept all the same
// where its tiles do not outnumber the SMs (each is then an SM's, split over idle ones) and a CTA's context is at
// most kTcMinTokens, and where all rows' tokens times dims are at most kTcMinWork.  Us here and there, 24 / 8 heads
// of 128: 8 sequences of up to 6000 tokens, 8 queries bf16 39 52, 16 71 52, 64 146 67; 48 of up to 3000, 16
// queries bf16 123 157, 22 176 158; one of 4000, 64 queries bf16 28 42, 128 84 45, 43 queries f32 25 46; 30 queries
// f32 over 16000 90 57; a prompt of 100 queries over 1000 f32 31 42, 4 of 64 over 1000 bf16 50 37; 8 / 8 heads,
// 300 queries over 600 f32 21 43; heads of 64, 512 queries over themselves f32 20 34, bf16 29 30.
constexpr int kTcMinRows = 64, kTcMinTokens = 6000;
constexpr int64_t kTcMinWork = 340'000'000;
// The same for trees, whose tensor-core kernel is another one (qdq_kv_tree_tc.cu).  Us there and here, 24 / 8 heads of 128
// bf16: one sequence of 131071 tokens, 18 rows 132 112, 39 rows 131 165, 96 rows 131 323; 16 of 300 to 6000, 18 rows 74
// 80, 39 rows 75 104, 96 rows 77 171; 48 of 300 to 3000, 18 rows 119 105, 39 rows 122 142; 9 of 200 to 6001 f16, heads of 64,
// 248 rows, cap, bias and a window of 1500 35 32.
constexpr int kTreeMinRows = 32;
constexpr int64_t kTreeMinWork = 600'000'000;

struct Plan {
  bool tc;  // the tensor-core kernel of qdq_kv_attn_tc.cu
  int parts, groups, warps, tiles, splits, split_blocks, entries, ctas;
  int64_t units;
  size_t bytes;  // of the workspace, for any window
};

// tree: a sequence's queries are one.  For a window, span: how much further apart a tile's tokens may lie than its
// rows (a tree's nodes come in any order).
Plan plan(const DeviceInfo &di, int n_seqs, int max_q, int max_kv_len, int n_heads, int n_kv, int head_dim, int window,
          int type, bool tree = false) {
  Plan p{};
  const int span = tree ? max_q : 0;
  const int64_t rows = int64_t(max_q) * (n_heads / n_kv);
  p.parts = type != QDQ_TYPE_F32 && rows > 8 ? 1 : 2;
  const int64_t small = int64_t(n_seqs) * n_kv * ((rows * p.parts + 15) / 16);  // tiles of the other kernel
  const bool few = small <= di.sm_count && max_kv_len / (di.sm_count / small) <= kTcMinTokens;
  // Blocks without a window.  A window's are never more, or its plan could want a larger workspace.
  const int64_t all_blocks = (int64_t(max_kv_len) + kKvBlock - 1) / kKvBlock;
  const int64_t far = tree && window > 0 ? std::min<int64_t>(max_kv_len, int64_t(window) + max_q) : max_kv_len;
  const int64_t tokens_seen = std::max<int64_t>(1, far - max_q / 2);
  const bool light = int64_t(n_seqs) * n_kv * rows * head_dim <= (tree ? kTreeMinWork : kTcMinWork) / tokens_seen;
  const int forced = g_opt_attn_kernel.load(std::memory_order_relaxed);
  p.tc = (forced == 2 || (forced == 0 && rows > (tree ? kTreeMinRows : kTcMinRows) && !few && !light)) && (type == QDQ_TYPE_F32 || p.parts == 1) &&
         attn_tc_supported(head_dim, p.parts);
  if (p.tc) {
    p.groups = rows > kTcRows && head_dim <= 128 && !tree ? 2 : 1;
    const int R = kTcRows * p.groups;
    p.tiles = int((rows + R - 1) / R);
    p.units = int64_t(n_seqs) * n_kv * p.tiles;
    int64_t tokens = max_kv_len;
    if (window > 0 && tokens > int64_t(window) + R + span) tokens = int64_t(window) + R + span;
    const int64_t blocks = std::min(all_blocks, (tokens + kKvBlock - 1) / kKvBlock + (window > 0));
    // whole waves of CTAs (one per SM), each with at most kTcSplitBlocks of the blocks there can be
    const int64_t most = p.units * ((blocks + 4) / 4 + kTcPartCost);  // tiles of 64 tokens and parts' costs
    const int64_t wave = int64_t(di.sm_count) * ((tree && head_dim <= 128 ? kTcTreeBlocks : kTcSplitBlocks) / 4);
    const int64_t ctas = di.sm_count * ((most + wave - 1) / wave);
    p.splits = int(ctas < 0x7fffffff ? ctas : 0);
    p.bytes = workspace_for(size_t(p.units), 2 * size_t(ctas) * attn_tc_part_bytes(head_dim, p.groups));
    return p;
  }
  const int R = 16 / p.parts;
  p.tiles = int((rows + R - 1) / R);
  p.units = small;
  // blocks a tile can see: its rows span at most R queries
  int64_t tokens = max_kv_len;
  if (window > 0 && tokens > int64_t(window) + R + span) tokens = int64_t(window) + R + span;
  const int64_t blocks = std::min(all_blocks, (tokens + kKvBlock - 1) / kKvBlock + (window > 0));
  const int resident = head_dim <= 128 ? 16 : 8;  // warps per SM
  // Few tiles: CTAs that fill an SM, so that a tile is cut into few splits; many: small CTAs,
  // whose starts and ends overlap with their neighbours' work.
  p.warps = p.units <= di.sm_count || blocks > int64_t(max_splits(4)) * max_split_blocks(4) ? resident : 4;
  const int64_t per_wave = int64_t(di.sm_count) * (resident / p.warps);
  // small CTAs: four waves of them, so that sequences of different lengths even out (48 sequences
  // of up to 8K tokens, 24 / 8 heads of 128: 78 us; two waves 87 us, eight 89 us)
  int64_t splits = p.warps == 4 ? 4 * per_wave / p.units : per_wave / p.units;
  if (splits < 1) splits = 1;
  if (splits > max_splits(p.warps)) splits = max_splits(p.warps);
  int64_t per = (blocks + splits - 1) / splits;
  if (per < kMinBlocks * p.warps) per = kMinBlocks * p.warps;
  if (per > max_split_blocks(p.warps)) per = max_split_blocks(p.warps);
  p.split_blocks = int(per);
  p.splits = int((blocks + per - 1) / per);
  if (p.splits < 1) p.splits = 1;
  p.ctas = p.units * p.splits <= 0x7fffffff ? int(p.units * p.splits) : 0;
  // sequences of their own lengths: splits whose length the device chooses (above), as many as CTAs are aimed at
  const int64_t aim = p.warps == 4 ? 4 * per_wave : per_wave, entries = int64_t(n_seqs) * p.tiles;
  if (entries <= kMaxEntries && p.warps > 4 && n_seqs > 1 && per >= kEvenBlocks) {
    const int64_t least = entries * ((blocks + max_split_blocks(p.warps) - 1) / max_split_blocks(p.warps));
    const int64_t per_head = std::max(std::max(aim / n_kv, entries), least);
    p.entries = int(entries);
    p.ctas = per_head * n_kv <= 0x7fffffff ? int(per_head * n_kv) : 0;
  }
  // Parts there can be, with any window: another one can want either size of CTA.  More CTAs than units cut a unit;
  // as many do where the device chooses the splits, since a sequence without queries leaves its CTAs to the others.
  const bool chosen = n_seqs > 1 && entries <= kMaxEntries && p.units <= di.sm_count;
  int64_t slots = chosen ? p.units : 0;
  for (int warps : {4, resident})
    if (warps == resident || p.units > di.sm_count) {
      const int64_t to = (warps == 4 ? 4 : 1) * int64_t(di.sm_count) * (resident / warps);
      const int64_t forced = p.units * ((all_blocks + max_split_blocks(warps) - 1) / max_split_blocks(warps));
      for (int64_t n : {to, forced})
        if (n > p.units && n > slots) slots = n;
    }
  p.bytes = workspace_for(size_t(p.units), size_t(slots) * R * (head_dim + 2) * 4);
  return p;
}

}  // namespace

size_t kv_attention_workspace_bytes(int n_seqs, int max_q, int max_kv_len, int n_heads, int n_kv, int head_dim, bool tree) {
  DeviceInfo di;
  if (device_info(&di) != cudaSuccess) return 0;
  size_t most = 0;  // enough for every element type
  for (int type : {QDQ_TYPE_F32, QDQ_TYPE_BF16}) {
    const size_t b = plan(di, n_seqs, max_q, max_kv_len, n_heads, n_kv, head_dim, 0, type, tree).bytes;
    if (b > most) most = b;
  }
  return most;
}

int launch_kv_attention(const KvPool &c, int head_dim, const int *kv_len, const int *cu_q, const int *parent, int n_seqs,
                        int max_q, int max_kv_len, int n_heads, const void *q, int64_t q_stride, void *out, int64_t out_stride,
                        float *lse, const float *slopes, float scale, float softcap, int window, int type,
                        void *workspace, size_t workspace_bytes, cudaStream_t s) {
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return fail_cuda(e);
  // a window that hides nothing is none, and a position less a smaller one stays within 32 bits
  if (window >= max_kv_len) window = 0;
  const bool tree = parent != nullptr;
  const Plan p = plan(di, n_seqs, max_q, max_kv_len, n_heads, c.n_kv, head_dim, window, type, tree);
  if (p.splits < 1 || p.units > 0x7fffffff / (tree ? 16 : 1) || (!p.tc && p.ctas < 1)) return QDQ_ERR_UNSUPPORTED;
  AttnArgs a{};
  a.c = c;
  a.kv_len = kv_len;
  a.cu_q = cu_q;
  a.parent = parent;
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.slopes = slopes;
  a.tickets = static_cast<uint32_t *>(workspace);
  a.partial = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + workspace_tickets(workspace_bytes));
  a.room = int64_t((workspace_bytes - workspace_tickets(workspace_bytes)) / 4);
  a.units = p.units;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.n_seqs = n_seqs;
  a.max_q = max_q;
  a.max_rows = max_q * (n_heads / c.n_kv);
  a.max_kv_len = max_kv_len;
  a.n_heads = n_heads;
  a.group = n_heads / c.n_kv;
  a.group_mul = ((uint64_t(1) << 40) + uint64_t(a.group) - 1) / uint64_t(a.group);
  a.tiles = p.tiles;
  a.splits = p.splits;
  a.split_blocks = p.split_blocks;
  a.inv_splits = 1.f / float(p.splits);
  a.entries = p.entries;
  a.window = window;
  a.type = type;
  a.scale = scale;
  a.softcap = softcap;
  a.inv_cap = softcap > 0.f ? 1.f / softcap : 0.f;
  if (p.tc) {
    e = tree ? launch_attn_tree_tc(a, head_dim, p.parts, p.groups, s) : launch_attn_tc(a, head_dim, p.parts, p.groups, s);
    return e == cudaSuccess ? QDQ_OK : fail_cuda(e);
  }
  e = tree ? launch_attn_tree(a, head_dim, p.parts, p.warps, p.ctas, s) : run_attn<false>(a, head_dim, p.parts, p.warps, p.ctas, s);
  return e == cudaSuccess ? QDQ_OK : fail_cuda(e);
}

QDQ_CHECK_READER(read_checks_attn)

}  // namespace qdq
