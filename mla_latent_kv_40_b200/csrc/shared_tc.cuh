// Decode over shared prefixes on tensor cores: plan and attention (host interface).
#pragma once

#include "kernels.cuh"

namespace mla {

// At most 256 consecutive query rows of one group, the rows of up to 32 sequences (its members), and the pages of 64
// keys that they attend to: the group's shared pages, seen by every row, then each member's own pages, seen by that
// member's rows.
struct SharedUnit {
  int cost0;      // place of its first tile (two pages) in the work list
  int tiles, pages, shared;   // tiles; pages in all and shared ones among them
  int row0, rows; // first query row, counted over [B, n_q, H], and their number
  int seq0, members;          // first sequence with rows here, number of such sequences
  int table_seq;  // block table row that names the shared pages: the group's first sequence
  int pad[3];
};
static_assert(sizeof(SharedUnit) == 48, "read as three 16-byte words");
// One cluster's share of the work list: [begin, end), the first unit there, the number of units, and that unit.
struct SharedShare {
  int begin, end, unit, units;
  SharedUnit first;
};
static_assert(sizeof(SharedShare) == 64, "read as four 16-byte words");
constexpr int kSharedPage = 64;      // keys of a page
constexpr int kSharedPartRows = 256; // rows of a partial
constexpr int kSharedMembers = 32;
// Query rows of a full unit of sequences with R rows each.
__host__ __device__ constexpr int shared_unit_rows(int R) { return R >= 8 ? 256 : kSharedMembers * R; }

// What the plan kernel leaves for the kernels behind it.
struct SharedPlan {
  SharedShare *shares;      // [clusters]
  SharedUnit *units;        // [units]
  int2 *unit_parts;         // [units]: first partial (of 256 rows) of the unit, number of partials
  int2 *seq_group;          // [B]: first unit of the sequence's group, the group's first query row
  int *own_pages;           // [B + 1]: own pages of the sequences before this one
  int *scratch;             // shared_plan_words() of the plan kernel's own
};
// Words that the plan works on (in shared memory while they fit there).
inline size_t shared_plan_words(int B, int units, int num_groups) {
  return 3 * (size_t)B + 1 + 4 * (size_t)units + 1 + 3 * (size_t)num_groups + 2;
}

constexpr int kSharedMaxClusters = 64;
// Clusters of four CTAs that fit on the current device at once (0 without a device).
int shared_clusters_for_device();
// Units that B sequences of R query rows in num_groups groups can have.
inline int shared_max_units(int B, int R, int num_groups) {
  return (int)(((int64_t)B * R) / shared_unit_rows(R)) + (num_groups < B ? num_groups : B);
}
struct SharedPlanArgs {
  SharedPlan out;
  int B, n_q, R, max_seqlen, block_size, num_groups, max_units, clusters;
  const int32_t *offsets, *prefix_lens, *seqlens;
  int *dev_status;
};
int launch_shared_plan(const SharedPlanArgs &a, cudaStream_t st);
// The plan and the query absorption in one launch (absorb_tc_supported shapes).
int launch_absorb_plan(const AbsorbArgs &ab, const SharedPlanArgs &plan, int *dev_status, cudaStream_t st);
// Attention of every unit over its pages: partials o_part [256 (u + c) + row][512] (normalised by their own sums) and
// lse_part of cluster c's share of unit u.
int launch_shared_attention(const mla_dims &d, int n_q, int max_seqlen, const SharedPlan &pl, const void *q_abs,
                            const CacheView &cache, const int32_t *seqlens, float *o_part, float *lse_part,
                            int *dev_status, cudaStream_t st);
// Merge of the partials, and the W_UV product when w_uv != NULL (else out is o_lat).
int launch_shared_combine(const mla_dims &d, int B, int n_q, const SharedPlan &pl, const float *o_part,
                          const float *lse_part, const void *w_uv, void *out, float *lse, int *dev_status,
                          cudaStream_t st);

}  // namespace mla
