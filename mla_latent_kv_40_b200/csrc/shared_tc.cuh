// Decode over shared prefixes on tensor cores: plan and attention (host interface).
#pragma once

#include "kernels.cuh"

namespace mla {

// At most 256 query rows and the keys that they attend to: a sequence's rows over its own keys, or a block of a group's
// rows over the shared keys.  Own units come first, unit b for sequence b, then the shared ones.
struct SharedUnit {
  int cost0;      // place of its first tile (128 keys) in the work list
  int tiles, pages;         // 128-key tiles; 64-key pages (the last tile may hold one page only)
  int seq;        // block table row that names the pages
  int row0, rows; // first query row, counted over [B, n_q, H], and their number
  int page0;      // first page, counted over the sequence's keys
  int keys;       // keys from page0 on that exist
  int part0, part_stride;   // partial row of cluster c's piece: part0 + c * part_stride
  int vis0;       // keys from page0 on that the first query token sees; one more for each later one
  int pad;
};
static_assert(sizeof(SharedUnit) == 48, "read as three 16-byte words");

// What the plan kernel leaves for the kernels behind it.
struct SharedPlan {
  int *head;                // [4]: total cost, clusters that get a share, units, 0
  int *cluster_unit;        // [clusters]: the unit at which each cluster's share begins
  SharedUnit *units;        // [units]
  int2 *unit_parts;         // [units]: first partial row of the unit, number of partials
  int2 *seq_group;          // [B]: first shared unit of the sequence's group (-1: none), the group's first query row
  int *own_begin;           // [B] scratch: first key of the sequence's own unit
  int *group_pages;         // [num_groups] scratch
};

constexpr int kSharedMaxClusters = 64;
// Clusters of four CTAs that fit on the current device at once (0 without a device).
int shared_clusters_for_device();
// Shared units that B sequences of R query rows in num_groups groups can have.
inline int shared_max_units(int B, int R, int num_groups) {
  return (int)(((int64_t)B * R) / 256) + (num_groups < B ? num_groups : B);
}
int launch_shared_plan(const SharedPlan &pl, int B, int n_q, int H, int max_seqlen, int block_size, int num_groups,
                       const int32_t *group_offsets, const int32_t *prefix_lens, const int32_t *seqlens,
                       int *dev_status, cudaStream_t st);
// Attention of every unit over its keys: partials o_part [row][512] (bf16, normalised by their own sums) and
// lse_part [row], rows as the units say.
int launch_shared_attention(const mla_dims &d, const SharedPlan &pl, const void *q_abs, const CacheView &cache,
                            __nv_bfloat16 *o_part, float *lse_part, int *dev_status, cudaStream_t st);

}  // namespace mla
