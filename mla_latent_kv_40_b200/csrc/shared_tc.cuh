// Decode over a shared prefix on tensor cores: plan and attention over the shared keys (host interface).
#pragma once

#include "kernels.cuh"

namespace mla {

// One block of at most 256 query rows of a group and the shared keys that it attends to.
struct SharedUnit {
  int tile0;      // 128-key tiles of all units before this one
  int tiles;      // its own
  int pages;      // 64-key pages (the last tile may hold one page only)
  int seq;        // block table row that names the pages: the group's first sequence
  int row0;       // first query row, counted over [B, n_q, H]
  int rows;       // query rows, 1 .. 256
  int pad[2];
};
static_assert(sizeof(SharedUnit) == 32, "read as two 16-byte words");

// What the plan kernel leaves for the kernels behind it.
struct SharedPlan {
  int *head;                // [4]: tiles in all, clusters that get some, units, 0
  int *cluster_unit;        // [clusters]: the unit of each cluster's first tile
  SharedUnit *units;        // [units]
  int2 *unit_segs;          // [units]: first partial of the unit and their number
  int *own_begin;           // [B]: first key that the sequence attends to by itself (a multiple of 64)
  int2 *seq_unit;           // [B]: first unit of the sequence's group (-1: none), the group's first query row
  int *group_pages;         // [num_groups] scratch
};

constexpr int kSharedMaxClusters = 64;
// Clusters of four CTAs that fit on the current device at once (0 without a device).
int shared_clusters_for_device();
// Units that B sequences of R query rows in num_groups groups can have.
inline int shared_max_units(int B, int R, int num_groups) {
  return (int)(((int64_t)B * R) / 256) + (num_groups < B ? num_groups : B);
}
int launch_shared_plan(const SharedPlan &pl, int B, int n_q, int H, int max_seqlen, int block_size, int num_groups,
                       const int32_t *group_offsets, const int32_t *prefix_lens, const int32_t *seqlens,
                       int *dev_status, cudaStream_t st);
// Attention of every unit over its shared keys: partials o_part [segment][256][512] (bf16, normalised by their own
// sums) and lse_part [segment][256].
int launch_shared_attention(const mla_dims &d, const SharedPlan &pl, const void *q_abs, const CacheView &cache,
                            __nv_bfloat16 *o_part, float *lse_part, int *dev_status,
                            cudaStream_t st);

}  // namespace mla
