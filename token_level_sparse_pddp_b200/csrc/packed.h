// Shared between the planner of the packed attention calls (packed_plan.cu)
// and their kernels.
#pragma once

#include "kernels.h"

namespace tlsp {

// Query tokens q0 .. q0 + nt - 1 (all query heads of one key/value head)
// against prefix keys pre0 .. pre0 + pre_n - 1, which every token sees, and
// the key rows kv0 .. kv0 + kv_n - 1 of K, of which token q0 + i sees the first
// min(kv_n, diag + i + 1) (none if that is negative).
// slot < 0: the result is final; else it is the partial result of token
// q0 + i in row slot + i of the workspace's partial rows.
struct PackedItem {
  int32_t q0, nt;
  int32_t kv0, kv_n;
  int32_t pre0, pre_n;
  int32_t diag, slot;
};
static_assert(sizeof(PackedItem) == 32, "item table layout");

// Token items of bf16 plans: tokens q0 .. q0 + nt - 1 (up to kTokenRows rows) against
// the keys of nseg segments. slot as above.
struct TokenItem {
  int32_t q0, nt;
  int32_t seg0, nseg;
  int32_t slot, pad[3];
};
// Keys k0 .. k0 + n - 1 of the prefix, which all of the item's tokens see, or of K:
// then tokens tok0 + i, i < ntok, see the first min(n, diag + i + 1) of them, the others
// none.
struct TokenSegment {
  int32_t k0, n;
  int32_t tok0, ntok;
  int32_t diag, prefix, pad[2];
};
static_assert(sizeof(TokenItem) == 32 && sizeof(TokenSegment) == 32, "item table layout");

// Tokens q0 .. q0 + nt - 1: partial rows a_slot + p * a_stride + i for p <
// a_parts, then the same with b.
struct MergeItem {
  int32_t q0, nt;
  int32_t a_slot, a_parts, a_stride;
  int32_t b_slot, b_parts, b_stride;
};
static_assert(sizeof(MergeItem) == 32, "item table layout");

constexpr int kTokenRows = 16;    // rows (tokens x heads of a group) of a token item
constexpr int kMergeTokens = 1;   // tokens of a merge item
constexpr int kMergeWarps = 4;    // of a block of the merge kernel
constexpr int kMergeAhead = 8;    // parts in flight for a warp

// With more parts than a warp has in flight, a block's warps share a row's.
inline bool merge_joint(int parts) { return parts > kMergeAhead; }
// Blocks (the grid's y) that the rows of a merge item take.
inline int64_t merge_blocks(int heads, int parts) {
  return ceil_div((int64_t)kMergeTokens * heads, merge_joint(parts) ? 1 : kMergeWarps);
}
constexpr int kMaxGridY = 65535;

constexpr int kMaxSegments = 32;  // of a token item: its tokens' sequences and the prefix
constexpr int kMaxCluster = 8;    // CTAs that share a token item (portable cluster size)
constexpr int kTcRows = 128;       // rows of one of the two query tiles of a bf16 tile item

// Rows of a tile item, fp32: 32 (twice as many items as with 64, for balance; half of
// the 64 rows' K and V reuse, which the CUDA cores do not need), or one token's.
inline int simt_tile_rows(int group) { return group <= 32 ? 32 : 64; }

// Most tokens of a tile item: whole groups of `group` rows (per query tile).
inline int tile_tokens(bool bf16, int group) {
  return bf16 ? 2 * (kTcRows / group) : simt_tile_rows(group) / group;
}

struct PackedArgs {
  const PackedItem* tiles;
  const PackedItem* tokens;    // fp32
  const TokenItem* token_items;  // bf16: the same entries
  const TokenSegment* segments;
  const MergeItem* merges;
  int n_tiles, n_tokens, n_segments, n_merges;
  int merge_parts;  // most parts of a merge item
  int cluster;  // CTAs of a token item (bf16)
  int heads, kv_heads, group, d;
  int64_t q_rows, kv_rows, prefix_len, part_rows;
  tlsp_rows Q, K, V, Kp, Vp, O;
  float* lse;       // [q_rows, heads] or null
  float scale;
  float* part_lse;  // [part_rows, heads] natural log
  float* part_o;    // [part_rows, heads, d], normalised
  int* status;
};

// An item read from device memory lies within the call's tensors and has at most
// `tokens` tokens (else the caller's table is not the plan's: it is skipped).
__device__ __forceinline__ bool item_ok(const PackedArgs& a, const PackedItem& t, int tokens) {
  const bool pieces = t.nt >= 1 && t.nt <= tokens && t.q0 >= 0 && t.kv0 >= 0 &&
                      t.kv_n >= 0 && t.pre0 >= 0 && t.pre_n >= 0;
  return pieces && (int64_t)t.q0 + t.nt <= a.q_rows &&
         (t.kv_n == 0 || (int64_t)t.kv0 + t.kv_n <= a.kv_rows) &&
         (int64_t)t.pre0 + t.pre_n <= a.prefix_len && t.diag >= -0x40000000 &&
         t.diag <= t.kv_n && (t.slot < 0 || (int64_t)t.slot + t.nt <= a.part_rows);
}

// packed_tile.cu: tile items on the tensor cores (bf16)
int packed_tile(const PackedArgs& a, cudaStream_t st);
// packed_token.cu: token items (bf16)
// `after`: behind the tile items of the call, beside which it runs
int packed_token(const PackedArgs& a, bool after, cudaStream_t st);
// packed_simt.cu: both kinds of items (fp32)
int packed_simt(const PackedArgs& a, cudaStream_t st);
// packed_merge.cu: merge items
int packed_merge(const PackedArgs& a, bool bf16, cudaStream_t st);

}  // namespace tlsp
