// Bookkeeping of the paged latent cache on the GPU: the block tables, lengths and slot maps of a step
// from the requests' lengths (mla_plan_step), and the return of finished requests' blocks
// (mla_release_blocks).
//
// Mathematics.  With block size s, request b holding c_b tokens and receiving n_b:
//   need_b = ceil((c_b + n_b) / s) - ceil(c_b / s),   N_b = need_0 + .. + need_b,
//   b is served iff need_b = 0 or N_b <= F (F free blocks),
//   its i-th new block is free_list[F - 1 - (N_b - need_b + i)],
//   token t of the step belongs to the request whose range of the prefix sums of n holds t.
// All of it is two prefix sums over the requests and one search per four tokens (or ids).
//
// Shape.  Every CTA loads the lengths and forms the prefix sums in its own shared memory (redundantly: they are a few
// KB), then the table entries and tokens are dealt out over all threads.  Outputs that may alias inputs (lengths, free
// count) are written only when every CTA has read them, so that the state of a serving loop can be updated in place,
// also in a replayed graph.  Two forms of that:
//   * little work: one cluster of kCtas CTAs in one launch, with a cluster barrier before those outputs;
//   * much work: kBodyCtas CTAs that leave those outputs alone, and a second launch of one CTA that forms the sums again
//     (while the first kernel runs) and writes them once that has finished.
// No atomics: the result does not depend on timing.  The call is bound by latency (the dependent loads of the scan and
// of the search), not by its bytes.  Measured (device, several boxes): plan of 64 requests with one token each 10.6 to 13.6 us,
// of 256 with 16 to 1024 tokens 11.9 to 13.5, of 4096 with 4 to 32 tokens 19.3 to 20.4 (two launches); release of 64 requests
// 6.2 us, of 4096 11.5.
#include "kernels.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kCtas = 8;          // the largest portable cluster
constexpr int kBodyCtas = 128;
// Up to so many words that a call may have to write, one cluster takes it (device time, one cluster against two launches:
// plan of 256 requests with 33k tokens 10.6 and 11.6 us, 63k 13.8 and 10.8, 131k 20.7 and 10.9; release of 33k blocks 5.9
// and 8.8, 64k 7.4 and 8.6, 131k 11.0 and 9.0; the second launch takes 3 us of the host's time).
constexpr int64_t kWholeWords = 65536;
// What one launch is to do.
enum Mode { kWhole, kBody, kFinish };
constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = 4;           // consecutive tokens (or block ids) per thread and search

// Inclusive block-wide prefix sum of one value per thread.  `part` holds kWarps values; the caller
// synchronises before it is used again.
__device__ __forceinline__ long long block_scan(long long v, long long *part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) part[warp] = v;
  __syncthreads();
  long long w = part[lane];      // kWarps == 32: every warp scans the warps' totals
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += u;
  }
  const long long before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  __syncthreads();
  return v + (warp > 0 ? before : 0);
}
static_assert(kWarps == 32, "block_scan reads one total per lane");

// Exclusive prefix sums of in[0..n) into out[0..n], thread i owning items i * per .. (i + 1) * per - 1;
// values are clamped to `most` on the way out.  Returns the total to every thread.
template <typename F>
__device__ __forceinline__ long long scan_items(int n, int per, long long most, int32_t *out, long long *part, F item) {
  const int lo = min(n, (int)threadIdx.x * per), hi = min(n, lo + per);
  long long sum = 0;
  for (int i = lo; i < hi; ++i) sum += item(i);
  const long long inc = block_scan(sum, part);
  long long at = inc - sum;
  for (int i = lo; i < hi; ++i) {
    const long long v = item(i);
    out[i] = (int32_t)min(at, most);
    at += v;
  }
  if (threadIdx.x == kThreads - 1) {
    out[n] = (int32_t)min(inc, most);
    part[0] = inc;
  }
  __syncthreads();
  const long long total = part[0];
  __syncthreads();
  return total;
}

// Last i with a[i] <= v, for a[0] <= v and a ascending over [0, n).
__device__ __forceinline__ int last_le(const int32_t *a, int n, int32_t v) {
  int lo = 0, hi = n;             // a[lo] <= v < a[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= v) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Group of every request (-1: none).  Offsets that do not rise from 0 to B leave every request without one.
__device__ __forceinline__ void fill_groups(int B, int G, const int32_t *offsets, int32_t *gid, int *dev_status) {
  int bad = 0;
  for (int g = threadIdx.x; g < G; g += kThreads) {
    const int lo = offsets[g], hi = offsets[g + 1];
    bad |= lo < 0 || lo > hi || hi > B || (g == 0 && lo != 0) || (g == G - 1 && hi != B);
  }
  bad = __syncthreads_or(bad);
  if (bad && threadIdx.x == 0) report(dev_status, MLA_ERR_BAD_INDEX);
  if (bad || G == 0) {
    for (int b = threadIdx.x; b < B; b += kThreads) gid[b] = -1;
  } else {
    for (int g = threadIdx.x >> 5; g < G; g += kWarps)
      for (int b = offsets[g] + (threadIdx.x & 31); b < offsets[g + 1]; b += 32) gid[b] = g;
  }
  __syncthreads();
}

__device__ __forceinline__ int blocks_of(int tokens, int bs) { return tokens / bs + (tokens % bs != 0); }

template <Mode kMode>
__global__ void __launch_bounds__(kThreads) step_plan_kernel(const StepPlanArgs a) {
  extern __shared__ int32_t sm[];
  __shared__ long long part[kWarps];
  __shared__ int s_taken;
  const int B = a.B, bs = a.block_size, tid = threadIdx.x;
  int32_t *cu = sm;                    // [B + 1] first token of each request
  int32_t *cum = cu + B + 1;           // [B + 1] first new block of each request
  int32_t *held = cum + B + 1;         // [B] cached tokens; ~cached where the request is refused
  int32_t *gid = held + B;             // [B] group; then, where the request joins its prefix, still the group, else -1
  const int rank = blockIdx.x, threads = gridDim.x * kThreads;
  const int gtid = rank * kThreads + tid;
  // The finishing launch may form its sums while this one runs.  The other modes let nothing start early: kernels behind
  // them read lengths and positions before they wait for their predecessor.
  if (kMode == kBody) grid_dep_launch();
  int *const status = kMode == kFinish ? nullptr : a.dev_status;   // each error is reported by one launch
  const int per = (B + kThreads - 1) / kThreads;

  fill_groups(B, a.num_groups, a.group_offsets, gid, rank == 0 ? status : nullptr);
  int free = *a.free_count;
  if (free < 0 || free > a.free_capacity) {
    if (gtid == 0) report(status, MLA_ERR_BAD_INDEX);
    free = free < 0 ? 0 : a.free_capacity;
  }
  // Lengths and refusals that do not depend on the other requests.
  const int64_t room = min((int64_t)a.max_blocks_per_seq * bs, (int64_t)0x7fffffff);
  for (int b = tid; b < B; b += kThreads) {
    const int c = a.cached_lens[b], g = gid[b];
    int n = a.new_lens[b];
    const int P = g >= 0 ? a.prefix_lens[g] : 0;
    bool bad = n < 0 || n > a.max_tokens;
    if (bad) n = 0;
    const bool idle = c == 0 && n == 0 && !bad;   // a slot without a request, as a release leaves it: nothing to refuse
    bad |= c < 0 || (int64_t)c + n > room || P < 0 || P % bs != 0 || P / bs > a.max_prefix_blocks || (c < P && !idle);
    cu[b] = n;
    held[b] = bad ? ~max(c, 0) : c;
    if (bad || P <= 0 || c != P) gid[b] = -1;
    if (bad && rank == 0) report(status, MLA_ERR_BAD_INDEX);
  }
  __syncthreads();
  // First tokens.  cum holds the token counts meanwhile.
  for (int b = tid; b < B; b += kThreads) cum[b] = cu[b];
  __syncthreads();
  const long long tokens = scan_items(B, per, a.max_tokens, cu, part, [&](int b) { return (long long)cum[b]; });
  // A request whose tokens do not all fit the token arrays is refused.
  if (tokens > a.max_tokens) {
    for (int b = tid; b < B; b += kThreads)
      if (held[b] >= 0 && cum[b] > 0 && (long long)cu[b] + cum[b] > a.max_tokens) {
        held[b] = ~held[b];
        gid[b] = -1;
        if (rank == 0) report(status, MLA_ERR_BAD_INDEX);
      }
    __syncthreads();
  }
  for (int b = tid; b < B; b += kThreads) {
    const int n = cum[b];
    cum[b] = held[b] >= 0 ? blocks_of(held[b] + n, bs) - blocks_of(held[b], bs) : 0;
  }
  __syncthreads();
  // First new blocks, in place: every item is read by the thread that overwrites it, after its own reads.
  {
    const int lo = min(B, tid * per), hi = min(B, lo + per);
    long long sum = 0;
    for (int b = lo; b < hi; ++b) sum += cum[b];
    const long long inc = block_scan(sum, part);
    long long at = inc - sum;
    int taken = 0;
    for (int b = lo; b < hi; ++b) {
      const int need = cum[b];
      cum[b] = (int32_t)min(at, (long long)free);
      at += need;
      if (need > 0) {
        if (at <= free) {
          taken = (int)at;
        } else {                   // the free list ends here: this request and every later one that needs a block
          held[b] = ~held[b];
          gid[b] = -1;
          if (rank == 0) report(status, MLA_ERR_NO_BLOCKS);
        }
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) taken = max(taken, __shfl_xor_sync(0xffffffffu, taken, o));
    if ((tid & 31) == 0) part[tid >> 5] = taken;
    __syncthreads();
    if (tid < 32) {
      int t = (int)part[tid];
#pragma unroll
      for (int o = 16; o; o >>= 1) t = max(t, __shfl_xor_sync(0xffffffffu, t, o));
      if (tid == 0) s_taken = t;
    }
    __syncthreads();
  }
  const int taken = s_taken;
  if (kMode == kWhole) {   // this CTA has read the lengths and the free count
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  }

  if (kMode != kFinish) {
    // New table entries.
    for (uint32_t k0 = gtid * kPer; k0 < (uint32_t)taken; k0 += threads * kPer) {   // (unsigned: the last step may pass 2^31)
      int b = last_le(cum, B, (int)k0);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (k0 + i >= (uint32_t)taken) break;
        const int k = (int)(k0 + i);
        while (b + 1 < B && cum[b + 1] <= k) ++b;
        int id = a.free_list[free - 1 - k];
        if (id < 0 || id >= a.num_blocks) {
          report(status, MLA_ERR_BAD_INDEX);
          id = -1;
        }
        a.block_table[(int64_t)b * a.max_blocks_per_seq + blocks_of(held[b], bs) + (k - cum[b])] = id;
      }
    }
    // The shared blocks of requests that join their group's prefix.
    for (int b = gtid >> 5; b < B; b += threads / 32) {
      const int g = gid[b];
      if (g < 0) continue;
      const int np = held[b] / bs;
      const int32_t *src = a.prefix_table + (int64_t)g * a.max_prefix_blocks;
      int32_t *dst = a.block_table + (int64_t)b * a.max_blocks_per_seq;
      for (int i = tid & 31; i < np; i += 32) dst[i] = src[i];
    }
    // Tokens: request, position and pool row.
    const int T = cu[B];
    for (uint32_t t0 = gtid * kPer; t0 < (uint32_t)T; t0 += threads * kPer) {
      int b = last_le(cu, B, (int)t0);
      int32_t sq[kPer], ps[kPer];
      int64_t sl[kPer];
      int at_b = -1, at_l = -1;
      int32_t blk = -1;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        sq[i] = ps[i] = -1;
        sl[i] = -1;
        if (t0 + i < (uint32_t)T) {
          const int t = (int)(t0 + i);
          while (b + 1 < B && cu[b + 1] <= t) ++b;
          const int c = held[b];
          if (c >= 0) {
            const int p = c + (t - cu[b]), l = p / bs, have = blocks_of(c, bs);
            if (b != at_b || l != at_l) {
              blk = l < have ? a.block_table[(int64_t)b * a.max_blocks_per_seq + l]
                             : a.free_list[free - 1 - (cum[b] + l - have)];
              if (blk < 0 || blk >= a.num_blocks) {
                report(status, MLA_ERR_BAD_INDEX);
                blk = -1;
              }
              at_b = b;
              at_l = l;
            }
            if (blk >= 0) {
              sq[i] = b;
              ps[i] = p;
              sl[i] = (int64_t)blk * bs + p % bs;
            }
          }
        }
      }
      if (a.vec && t0 + kPer <= (uint32_t)T) {
        *reinterpret_cast<int4 *>(a.seq_idx + t0) = make_int4(sq[0], sq[1], sq[2], sq[3]);
        *reinterpret_cast<int4 *>(a.pos + t0) = make_int4(ps[0], ps[1], ps[2], ps[3]);
        if (a.slots) {
          *reinterpret_cast<longlong2 *>(a.slots + t0) = make_longlong2(sl[0], sl[1]);
          *reinterpret_cast<longlong2 *>(a.slots + t0 + 2) = make_longlong2(sl[2], sl[3]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (t0 + i < (uint32_t)T) {
            a.seq_idx[t0 + i] = sq[i];
            a.pos[t0 + i] = ps[i];
            if (a.slots) a.slots[t0 + i] = sl[i];
          }
      }
    }
    for (int b = gtid; b <= B; b += threads) a.cu_seqlens[b] = cu[b];
  }
  if (kMode == kBody) return;
  // In-place outputs.  new = cu[b + 1] - cu[b] for a served request (refused ones keep what they held).
  if (kMode == kWhole) {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  } else {
    grid_dep_wait();
  }
  for (int b = gtid; b < B; b += threads) {
    const int c = held[b];
    a.seqlens[b] = c >= 0 ? c + (cu[b + 1] - cu[b]) : ~c;
  }
  if (gtid == 0) *a.free_count_out = free - taken;
}

template <Mode kMode>
__global__ void __launch_bounds__(kThreads) release_kernel(const ReleaseArgs a) {
  extern __shared__ int32_t sm[];
  __shared__ long long part[kWarps];
  __shared__ int s_put;
  const int B = a.B, bs = a.block_size, tid = threadIdx.x;
  int32_t *cum = sm;                   // [B + 1] first returned block of each request
  int32_t *first = cum + B + 1;        // [B] first own table entry
  int32_t *left = first + B;           // [B] length after the call
  int32_t *gid = left + B;             // [B] group
  const int rank = blockIdx.x, threads = gridDim.x * kThreads;
  const int gtid = rank * kThreads + tid;
  // The finishing launch may form its sums while this one runs.  The other modes let nothing start early: kernels behind
  // them read lengths and positions before they wait for their predecessor.
  if (kMode == kBody) grid_dep_launch();
  int *const status = kMode == kFinish ? nullptr : a.dev_status;   // each error is reported by one launch
  const int per = (B + kThreads - 1) / kThreads;

  fill_groups(B, a.num_groups, a.group_offsets, gid, rank == 0 ? status : nullptr);
  int free = *a.free_count;
  if (free < 0 || free > a.free_capacity) {
    if (gtid == 0) report(status, MLA_ERR_BAD_INDEX);
    free = free < 0 ? 0 : a.free_capacity;
  }
  for (int b = tid; b < B; b += kThreads) {
    const int n = a.seqlens[b], g = gid[b];
    const int P = g >= 0 ? a.prefix_lens[g] : 0;
    int own = 0;
    left[b] = n;
    first[b] = 0;
    if (a.done[b]) {
      if (n < 0 || P < 0 || P % bs != 0 || blocks_of(n, bs) > a.max_blocks_per_seq) {
        if (rank == 0) report(status, MLA_ERR_BAD_INDEX);
      } else {
        own = max(0, blocks_of(n, bs) - P / bs);
        first[b] = P / bs;
        left[b] = 0;
      }
    }
    cum[b] = own;
  }
  __syncthreads();
  const long long most = a.free_capacity - free;
  {
    const int lo = min(B, tid * per), hi = min(B, lo + per);
    long long sum = 0;
    for (int b = lo; b < hi; ++b) sum += cum[b];
    const long long inc = block_scan(sum, part);
    long long at = inc - sum;
    int put = 0;
    for (int b = lo; b < hi; ++b) {
      const int own = cum[b];
      cum[b] = (int32_t)min(at, most);
      at += own;
      if (own > 0) {
        if (at <= most) {
          put = (int)at;
        } else {                   // the list is full: this request and every later one keeps its blocks
          left[b] = a.seqlens[b];
          if (rank == 0) report(status, MLA_ERR_BAD_INDEX);
        }
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) put = max(put, __shfl_xor_sync(0xffffffffu, put, o));
    if ((tid & 31) == 0) part[tid >> 5] = put;
    __syncthreads();
    if (tid < 32) {
      int t = (int)part[tid];
#pragma unroll
      for (int o = 16; o; o >>= 1) t = max(t, __shfl_xor_sync(0xffffffffu, t, o));
      if (tid == 0) s_put = t;
    }
    __syncthreads();
  }
  const int put = s_put;
  if (kMode == kWhole) {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  }
  if (kMode != kFinish) {
    for (uint32_t k0 = gtid * kPer; k0 < (uint32_t)put; k0 += threads * kPer) {
      int b = last_le(cum, B, (int)k0);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (k0 + i >= (uint32_t)put) break;
        const int k = (int)(k0 + i);
        while (b + 1 < B && cum[b + 1] <= k) ++b;
        const int id = a.block_table[(int64_t)b * a.max_blocks_per_seq + first[b] + (k - cum[b])];
        if (id < 0 || id >= a.num_blocks) report(status, MLA_ERR_BAD_INDEX);
        a.free_list[free + k] = id;
      }
    }
  }
  if (kMode == kBody) return;
  if (kMode == kWhole) {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  } else {
    grid_dep_wait();
  }
  for (int b = gtid; b < B; b += threads) a.seqlens_out[b] = left[b];
  if (gtid == 0) *a.free_count_out = free + put;
}

using Cache = std::atomic<int>[kSmemCacheDevs];

// One launch of a bookkeeping kernel: a cluster (kWhole), many CTAs (kBody), or one that may begin while the launch
// before it is still running (kFinish).
template <typename Args>
int launch(Mode mode, void (*kernel)(Args), const Args &a, size_t smem, Cache &cache, cudaStream_t st) {
  if (smem_limit(kernel, smem, cache) != cudaSuccess) return MLA_ERR_CUDA;
  if (mode == kFinish) return launch_pdl(kernel, dim3(1), dim3(kThreads), smem, st, a) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(mode == kWhole ? kCtas : kBodyCtas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = mode == kWhole ? kCtas : 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace

int launch_step_plan(const StepPlanArgs &a, cudaStream_t st) {
  static Cache cache[3];
  const size_t smem = (size_t)(4 * a.B + 2) * sizeof(int32_t);
  // The most that the call can have to write: its tokens, and whole table rows of joining requests.
  const int64_t most = (int64_t)a.max_tokens + (int64_t)a.B * min(a.max_prefix_blocks, a.max_blocks_per_seq);
  if (most <= kWholeWords) return launch(kWhole, step_plan_kernel<kWhole>, a, smem, cache[0], st);
  const int rc = launch(kBody, step_plan_kernel<kBody>, a, smem, cache[1], st);
  return rc ? rc : launch(kFinish, step_plan_kernel<kFinish>, a, smem, cache[2], st);
}

int launch_release(const ReleaseArgs &a, cudaStream_t st) {
  static Cache cache[3];
  const size_t smem = (size_t)(4 * a.B + 1) * sizeof(int32_t);
  const int64_t most = min((int64_t)a.B * a.max_blocks_per_seq, (int64_t)a.free_capacity);
  if (most <= kWholeWords) return launch(kWhole, release_kernel<kWhole>, a, smem, cache[0], st);
  const int rc = launch(kBody, release_kernel<kBody>, a, smem, cache[1], st);
  return rc ? rc : launch(kFinish, release_kernel<kFinish>, a, smem, cache[2], st);
}

}  // namespace mla
