// The plan of a decode over shared prefixes: one block (a kernel of its own, or one block of the absorption's launch).
//
// A group's shared keys are the whole blocks among its first min(prefix_lens[g], shortest visible run) keys, where the
// first query token of sequence b sees seqlens[b] - n_q + 1 keys.  Its rows are cut into units; a unit's tiles (two
// pages each) are the shared pages and its members' own ones.
//
// The tiles of all units, in order, are dealt out to the clusters in shares of about equal cost: a tile costs 1, and
// every unit after the first kUnitCost more (its queries go to tensor memory and the finished unit's O is written out
// while the MMAs wait; about 10 us against 1.4 us per tile).  Tile i of unit u has place cost0[u] + i in a list of length
// W, cost0[u] = tiles before u + kUnitCost (non-empty units before u), and cluster c's share is
// [floor(c W / C), floor((c + 1) W / C)).  Where there are no more units than clusters and the longest is no longer than such
// a share, every unit has a cluster to itself: no unit is cut (64 sequences of 128 heads, 32 units: 106.8 us a call instead
// of 109.0, or 99.6 instead of 106.2 with the buffers placed otherwise; most of it in the merge).  Filling the clusters
// greedily to the least load that 33 of them manage (32 loads tried at once) took 9 us: not worth it.
#pragma once

#include "shared_tc.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

constexpr int kUnitCost = 8;

// Exclusive scan of one value per thread over the block, its total added to `carry`.
__device__ __forceinline__ int64_t plan_scan(int64_t v, int64_t *part, int64_t &carry) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int64_t inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t w = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += w;
  }
  __syncthreads();
  if (lane == 31) part[warp] = inc;
  __syncthreads();
  int64_t w = lane < warps ? part[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  const int64_t before = __shfl_sync(0xffffffffu, w, warp ? warp - 1 : 0);
  const int64_t all = __shfl_sync(0xffffffffu, w, 31);
  const int64_t exc = carry + (warp ? before : 0) + inc - v;
  carry += all;
  return exc;
}

// Last i in [0, n) with a[i] <= v, for a ascending and a[0] <= v.
__device__ __forceinline__ int last_at(const int *a, int n, int v) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= v) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int cluster_of(int64_t at, int W, int C) { return (int)(((at + 1) * C + W - 1) / W - 1); }

// `words`: shared_plan_words() words of shared memory, or NULL to use a.out.scratch.
//
// The lengths and groups may be what the kernel ahead still writes, and only grid_dep_wait() makes that visible.  The plan is
// formed ahead of the wait all the same, from copies, and again behind it if a copy differs from what is there then: a
// plan behind the wait alone took 5 us of a call of 28.  Any words that are read ahead give a plan within bounds.
__device__ __forceinline__ void shared_plan_body(const SharedPlanArgs &a, int *words) {
  __shared__ int64_t part[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
  const int B = a.B, R = a.R, unit_rows = shared_unit_rows(R);
  const SharedPlan &pl = a.out;
  bool waited = !words;
  if (!words) {
    sm100::grid_dep_wait();   // an earlier call may still use the scratch words
    words = pl.scratch;
  }
  int *const own = words;                        // [B + 1] own pages before each sequence
  int *const seq_shared = own + B + 1;           // [B] shared pages
  int *const cost0 = seq_shared + B;             // [max_units + 1]
  int *const tiles_of = cost0 + a.max_units + 1;
  int *const shared_of = tiles_of + a.max_units;
  int *const span_of = shared_of + a.max_units;  // first sequence * 64 + members
  int *const group_units = span_of + a.max_units;   // [num_groups + 1] first unit
  int *const lens = group_units + a.num_groups + 1;   // [B], [num_groups + 1], [num_groups] copies of the inputs
  int *const offs = lens + B;
  int *const prefs = offs + a.num_groups + 1;
  // Every input word and its copy, past L1, which may hold what was there ahead of the wait (one load's latency up to as many
  // words as threads).
  auto inputs = [&](auto &&f) {
    for (int i = tid; i < B + 2 * a.num_groups + 1; i += threads) {
      const int g = i - B, p = g - a.num_groups - 1;
      f(lens[i], __ldcg(g < 0 ? a.seqlens + i : p < 0 ? a.offsets + g : a.prefix_lens + p));
    }
  };
  int G, bad, wrong, U, longest, W, C;
  int64_t list;
  auto first_of = [&](int g) { return bad ? g * B : offs[g]; };
  for (;;) {
    inputs([](int &copy, int word) { copy = word; });
    __syncthreads();
    G = a.num_groups;
    bad = 0;
    for (int g = tid; g < G; g += threads) {
      const int lo = offs[g], hi = offs[g + 1];
      bad |= lo < 0 || lo > hi || hi > B || (g == 0 && lo != 0) || (g == G - 1 && hi != B) || prefs[g] < 0;
    }
    bad = __syncthreads_or(bad);
    if (bad) G = 1;    // then one group that shares nothing
    // Units before each group.
    int64_t units = 0;
    for (int g0 = 0; g0 < G; g0 += threads) {
      const int g = g0 + tid;
      const int64_t rows = g < G ? (int64_t)(first_of(g + 1) - first_of(g)) * R : 0;
      const int64_t exc = plan_scan((rows + unit_rows - 1) / unit_rows, part, units);
      if (g < G) group_units[g] = (int)exc;
    }
    if (tid == 0) group_units[G] = (int)units;
    __syncthreads();
    U = (int)units;
    // Shared pages of every group.
    wrong = 0;
    for (int g = warp; g < G; g += threads / 32) {
      const int lo = first_of(g), hi = first_of(g + 1), u0 = group_units[g], n = group_units[g + 1] - u0;
      int common = bad ? 0 : prefs[g];
      for (int b = lo + lane; b < hi; b += 32) {
        const int S = lens[b];
        wrong |= S < a.n_q || S > a.max_seqlen;
        common = min(common, max(min(max(S, 0), a.max_seqlen) - a.n_q + 1, 0));
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) common = min(common, __shfl_xor_sync(0xffffffffu, common, o));
      const int shared = common / a.block_size * (a.block_size / kSharedPage);
      for (int b = lo + lane; b < hi; b += 32) seq_shared[b] = shared;
      for (int i = lane; i < n; i += 32) {
        const int row0 = lo * R + i * unit_rows, rows = min(unit_rows, hi * R - row0);
        const int seq0 = row0 / R, last = (row0 + rows - 1) / R;
        shared_of[u0 + i] = shared;
        span_of[u0 + i] = seq0 * 64 + last - seq0 + 1;
      }
    }
    __syncthreads();
    // Own pages before each sequence.
    int64_t pages_all = 0;
    for (int b0 = 0; b0 < B; b0 += threads) {
      const int b = b0 + tid;
      int n = 0;
      if (b < B) n = (max(min(max(lens[b], 0), a.max_seqlen) - kSharedPage * seq_shared[b], 0) + kSharedPage - 1) / kSharedPage;
      const int64_t exc = plan_scan(n, part, pages_all);
      if (b < B) own[b] = (int)exc;
    }
    if (tid == 0) own[B] = (int)pages_all;
    __syncthreads();
    // Tiles of every unit and its place; non-empty units are counted in the low word.
    list = 0;
    longest = 0;
    for (int u0 = 0; u0 < U; u0 += threads) {
      const int u = u0 + tid;
      int tiles = 0;
      if (u < U) {
        const int seq0 = span_of[u] >> 6;
        tiles = (shared_of[u] + own[seq0 + (span_of[u] & 63)] - own[seq0] + 1) / 2;
      }
      const int64_t exc = plan_scan((int64_t)(tiles > 0) | ((int64_t)tiles << 32), part, list);
      if (u < U) {
        cost0[u] = (int)(exc >> 32) + kUnitCost * (int)(exc & 0xffffffff);
        tiles_of[u] = tiles;
      }
      longest = max(longest, tiles);
    }
    W = (int)(list >> 32) + kUnitCost * max((int)(list & 0xffffffff) - 1, 0);
    C = min(W, a.clusters);
#pragma unroll
    for (int o = 16; o; o >>= 1) longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
    __syncthreads();
    if (lane == 0) part[warp] = longest;
    __syncthreads();
    longest = lane < threads / 32 ? (int)part[lane] : 0;
#pragma unroll
    for (int o = 16; o; o >>= 1) longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
    if (waited) break;
    sm100::grid_dep_wait();   // (earlier calls may also still read the plan that is overwritten from here on)
    waited = true;
    int news = 0;
    inputs([&](int &copy, int word) { news |= copy != word; });
    if (!__syncthreads_or(news)) break;
  }
  const bool whole = (int)(list & 0xffffffff) <= a.clusters && (int64_t)longest * C <= W;
  __syncthreads();
  if ((bad && tid == 0) || wrong) report(a.dev_status, MLA_ERR_BAD_INDEX);
  auto put = [&](int4 *dst, int u) {
    const int g = last_at(group_units, G, u);   // of groups without units, which begin where the next one does, the last
    const int lo = first_of(g), seq0 = span_of[u] >> 6, members = span_of[u] & 63;
    const int row0 = lo * R + (u - group_units[g]) * unit_rows;
    dst[0] = make_int4(cost0[u], tiles_of[u], shared_of[u] + own[seq0 + members] - own[seq0], shared_of[u]);
    dst[1] = make_int4(row0, min(unit_rows, first_of(g + 1) * R - row0), seq0, members);
    dst[2] = make_int4(lo, 0, 0, 0);
  };
  if (whole) {
    int64_t n = 0;
    for (int u0 = 0; u0 < U; u0 += threads) {
      const int u = u0 + tid;
      const int tiles = u < U ? tiles_of[u] : 0;
      const int c = (int)plan_scan(tiles > 0, part, n);
      if (u >= U) continue;
      put(reinterpret_cast<int4 *>(pl.units + u), u);
      pl.unit_parts[u] = tiles > 0 ? make_int2(u + c, 1) : make_int2(0, 0);
      if (tiles > 0) {
        int4 *sh = reinterpret_cast<int4 *>(pl.shares + c);
        sh[0] = make_int4(cost0[u], cost0[u] + tiles, u, U);
        put(sh + 1, u);
      }
    }
    for (int c = (int)n + tid; c < a.clusters; c += threads) *reinterpret_cast<int4 *>(pl.shares + c) = make_int4(0, 0, 0, 0);
  } else {
    for (int c = tid; c < a.clusters; c += threads) {
      int4 *sh = reinterpret_cast<int4 *>(pl.shares + c);
      if (c >= C) {
        sh[0] = make_int4(0, 0, 0, 0);
        continue;
      }
      const int at = (int)((int64_t)c * W / C);
      int u = last_at(cost0, U, at);
      while (u + 1 < U && at - cost0[u] >= tiles_of[u]) ++u;   // in the gap behind u (or u is empty): the next with tiles
      sh[0] = make_int4(at, (int)((int64_t)(c + 1) * W / C), u, U);
      put(sh + 1, u);
    }
    for (int u = tid; u < U; u += threads) {
      put(reinterpret_cast<int4 *>(pl.units + u), u);
      int2 parts = make_int2(0, 0);
      if (tiles_of[u] > 0) {
        const int c0 = cluster_of(cost0[u], W, C), c1 = cluster_of((int64_t)cost0[u] + tiles_of[u] - 1, W, C);
        parts = make_int2(u + c0, c1 - c0 + 1);
      }
      pl.unit_parts[u] = parts;
    }
  }
  for (int b = tid; b <= B; b += threads) pl.own_pages[b] = own[b];
  for (int g = warp; g < G; g += threads / 32) {
    const int lo = first_of(g), hi = first_of(g + 1);
    for (int b = lo + lane; b < hi; b += 32) pl.seq_group[b] = make_int2(group_units[g], lo * R);
  }
}

}  // namespace
}  // namespace mla
