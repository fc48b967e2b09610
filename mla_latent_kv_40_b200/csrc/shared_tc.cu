// Decode over shared prefixes: the attention of a group's query rows over the keys that its sequences share, and of
// every sequence's rows over its own keys, in one launch on tcgen05 (sm_100a).
//
// In the absorbed form every head of every sequence attends to the same cached rows [c_i | kpe_i], so over a shared
// prefix the rows of all sequences of a group are rows of one product,
//   S = Q [rows x 576] . K^T [576 x keys],   O += P [rows x keys] . C [keys x 512],
// with no mask (the shared keys end before every query).  2176 FLOPs per (row, key) against 1152 bytes per key and
// 256 rows: bound by the tensor cores.
//
// Shape.  A unit is at most 256 consecutive rows of a group, and a list of pages of 64 keys: the group's shared pages,
// then the own pages of every sequence with rows in the unit, which the other rows do not see (a mask by owner and
// length; S of such a page is computed for all rows, as an MMA with fewer rows would take the same time).  Own pages in
// units of their own were slower by what a unit costs at its start and end: 106 against 85 us of attention for 64
// sequences of 128 heads behind 4096 shared tokens and up to 512 own ones.  A cluster of four CTAs works on one unit at
// a time, as two pairs that issue M = 256 MMAs (cta_group::2: each CTA holds 128 of the rows and half of the B operand, so each SM pulls half the bytes that
// a 128-row tile of its own would need; at 128 rows the L2 -> SM path, not the tensor pipe, sets the pace):
//   * ranks 0, 1 (score pair): Q_lat of the CTA's 128 rows in tensor memory (A operand), Q_rope in shared memory; a
//     tile is 128 keys, and CTA r streams its page r (64 keys, contiguous in the tiled pool) as two half-page stages;
//     rank 0 issues S [256 x 128] into one of two tensor-memory buffers; eight warps per CTA run the online softmax
//     of its 128 rows and send each page of P (bf16) to the value CTA of the same rows by one shared-to-shared copy;
//   * ranks 2, 3 (value pair): O of the CTA's 128 rows in all 512 tensor-memory columns; CTA r streams the latent
//     dims 256 (r - 2) .. of every page (32 KB, contiguous); rank 2 issues O += P . C as two N = 256 MMAs per 16 keys.
// Per 128 keys the score pair has 36 MMAs of 64 cycles, the value pair 16 of 128: 2304 and 2048 cycles.
//
// Measured: 128 sequences of 128 heads behind 32768 shared tokens (16384 rows, 1.19e12 FLOPs): 766-780 us, 1530-1550
// TFLOP/s of the burst matrix product's 1675; 2470 cycles a tile of the 2304, on 132 of 148 SMs (33 clusters fit).
//
// The issuing warps run whole, and each MMA is issued by the elected lane: with warp-uniform descriptors the issue
// keeps up with the pipe from one warp.  Reference maximum, row sums and rounding of P as in the per-sequence kernel
// (decode_tc.cu): lazy maximum in log2 units, sums of P in fp32 before its rounding to bf16, the type of the latents that
// it is multiplied with; but O / l of a piece stays in fp32 (in bf16 it cost the merged result a rounding, 0.0034 instead
// of 0.0030 of its norm).  The (unit, tile) list is cut into equal runs, one per cluster; a unit cut between clusters
// leaves one partial per piece, merged by the combine.
// Every wait is bounded; on expiry the kernel reports MLA_ERR_TIMEOUT, drains its copies, frees its tensor memory
// and returns.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <math_constants.h>

#include <atomic>
#include <cstring>
#include <mutex>
#include <type_traits>

#include "shared_plan.cuh"
#include "shared_tc.cuh"
#include "sm100.cuh"
#include "tmap.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kPage = kSharedPage;                 // keys of a page
constexpr int kDc = 512, kDr = 64, kW = kDc + kDr;
constexpr int kRows = 128;                         // query rows per CTA
constexpr int kUnitRows = kSharedPartRows;         // two CTAs' rows
constexpr int kThreads = 384;
constexpr int kSoftWarps = 8;
constexpr uint32_t kChunkBytes = kPage * 128;      // [64 keys x 64 dims] bf16, 128-byte swizzled
constexpr int kKStages = 4;                        // half pages: chunks 0-3, then 4-8
__host__ __device__ constexpr int half_chunks(int half) { return half ? 5 : 4; }
// Even stages take first halves, odd ones second halves.
__host__ __device__ constexpr uint32_t k_stage_off(int s) { return (s >> 1) * 9 * kChunkBytes + (s & 1) * 4 * kChunkBytes; }
static_assert(kKStages % 2 == 0, "a stage always holds the same half");
constexpr int kVStages = 4;                        // a page's 256 latent dims of this CTA
constexpr uint32_t kVStageBytes = 4 * kChunkBytes;
constexpr uint32_t kPBytes = kRows * kPage * 2;
constexpr int kPSlots = 5;
// A page of P travels with its rows' rescale factors: per writer warp 32 factors, a word of flags, padding.
constexpr uint32_t kPaWords = 36;
constexpr uint32_t kMoved = 1, kOdd = 2;           // flags: some factor is not 1; some score is not finite
constexpr uint32_t kPTxBytes = kPBytes + 4 * kPaWords * 4;
constexpr uint32_t kPSlotBytes = ((kPTxBytes + 1023) / 1024) * 1024;
constexpr uint32_t kQpeOff = 0;
constexpr uint32_t kKOff = kRows * 128;
constexpr uint32_t kStgOff = kKOff + k_stage_off(kKStages);
constexpr int kStgTiles = 3;                       // staged pages of P, shared by the two softmax groups in turn
constexpr uint32_t kPOff = kVStages * kVStageBytes;
constexpr uint32_t kScoreEnd = kStgOff + kStgTiles * kPSlotBytes, kValueEnd = kPOff + kPSlots * kPSlotBytes;
constexpr uint32_t kRegion = ((kScoreEnd > kValueEnd ? kScoreEnd : kValueEnd) + 1023) & ~1023u;
constexpr float kRescaleLog2 = 8.f;
constexpr uint64_t kWaitNs = 2000000000ull;        // 2 s per wait

constexpr uint32_t kQCol = 0, kSCol = 256;         // score CTA's tensor memory; the value CTA's is all O
constexpr uint16_t kScorePair = 0x3, kValuePair = 0xc;

// Barrier slots, alike in all four CTAs.
enum Bar {
  B_KFULL = 0,                          // score: own stage has landed; at rank 0 rank 1's as well
  B_KEMPTY = B_KFULL + kKStages,        // score: the MMAs have read the stage (both CTAs, one commit)
  B_SFULL = B_KEMPTY + kKStages,        // score: S of a tile is complete (both CTAs)
  B_SEMPTY = B_SFULL + 2,               // rank 0: both CTAs' softmax warps have read S
  B_QREADY = B_SEMPTY + 2,              // rank 0: both CTAs' queries are in place
  B_PEMPTY = B_QREADY + 1,              // score: the value CTA's P slot may be written
  B_STATSEMPTY = B_PEMPTY + kPSlots,    // score: the value CTA has read the row statistics
  B_STGFULL = B_STATSEMPTY + 1,         // score: a page of P is staged
  B_STGEMPTY = B_STGFULL + kStgTiles,   // score: its copy has read the staging tile
  B_CFULL = B_STGEMPTY + kStgTiles,         // value: own latents have landed; at rank 2 also: rank 3 is ready for the page
  B_CEMPTY = B_CFULL + kVStages,        // value: the MMAs have read the stage (both CTAs)
  B_PFULL = B_CEMPTY + kVStages,        // value: a page of P has landed
  B_PVDONE = B_PFULL + kPSlots,         // value: the page's MMAs are complete (both CTAs)
  B_REQ = B_PVDONE + kPSlots,           // value: request to the epilogue warps
  B_REQDONE = B_REQ + 1,
  B_STATSFULL = B_REQDONE + 1,          // value: row statistics of a finished unit
  B_OFREE = B_STATSFULL + 1,            // value: both CTAs' O has been read (both CTAs)
  B_RUNSEEN = B_OFREE + 1,              // value: the slots' thread has seen the MMAs of the run's last pages
  B_COUNT = B_RUNSEEN + 1
};

struct Req {
  int kind;      // 0: before a page's MMAs, rescale O and/or tidy the latents; 1: the epilogue
  int rescale, slot, keys, stage, scan;
  int np, pages;   // 1: pages so far, and those of the run
};

struct Small {                          // behind the tiles
  float stat_l[kRows], stat_m[kRows];
  float m_sh[2][kRows];                 // score: reference maximum after a tile, per group
  float xl[kRows];
  int odd_seen[2];                      // score: own pages of the run with scores that are not finite, per group
  uint64_t bars[B_COUNT];
  Req req;
  uint32_t tmem_base;
  int abort;
};
constexpr size_t kSmemBytes = 1024 + kRegion + sizeof(Small);
static_assert(kSmemBytes <= 232448, "shared memory budget");

struct Params {
  const SharedShare *shares;
  const SharedUnit *units;
  const __nv_bfloat16 *q;
  const int32_t *block_table, *seqlens;
  const int *own_pages;
  int max_blocks_per_seq, num_blocks, block_size, H, n_q, max_seqlen;
  float scale_log2;
  float *o_part, *lse_part;
  int *dev_status;
  const unsigned char *tiled;           // tiled pool, or NULL: row pool through the tensor maps
  const unsigned char *rows;            // the row pool's latents
  int64_t row_bytes;
};

// ------------------------------------------------------------ cta_group::2 forms
__device__ __forceinline__ void tmem_alloc2(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tmem_relinquish2() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// The whole warp calls these; one elected lane (always the same one) issues.
__device__ __forceinline__ void mma2_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma2_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// Arrival on the barrier at this offset in every CTA of `mask` once the elected lane's MMAs so far are complete.
__device__ __forceinline__ void commit2(uint32_t bar, uint16_t mask) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
      "h"(mask)
      : "memory");
}

// ------------------------------------------------------------ waits
__device__ __noinline__ bool timed_out(Small &sm, int *dev_status) {
  *(volatile int *)&sm.abort = 1;
  report(dev_status, MLA_ERR_TIMEOUT);
  return false;
}
// One thread's bounded wait; false once any wait of the CTA has given up.  `remote`: what is waited for was written
// by another CTA's threads (not by copies or MMAs).
__device__ __forceinline__ bool wait1(Small &sm, uint32_t bar, uint32_t parity, int *dev_status, bool remote = false) {
  if (remote ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
  if (*(volatile int *)&sm.abort) return false;
  if (mbar_wait(bar, parity, kWaitNs, remote)) return true;
  return timed_out(sm, dev_status);
}
// The same for a whole warp, with one verdict.
__device__ __forceinline__ bool waitw(Small &sm, uint32_t bar, uint32_t parity, int *dev_status, bool remote = false) {
  const bool ok = remote ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity);
  if (__all_sync(0xffffffffu, ok)) return true;
  return __all_sync(0xffffffffu, wait1(sm, bar, parity, dev_status, remote));
}

// ------------------------------------------------------------ work list
// The runs of tiles of one cluster: unit by unit, the tiles whose place lies in its share.
struct Runs {
  int u, units, begin, end, cid;
  bool fresh;       // `un` came with the share
  SharedUnit un;
  int t0, t1;       // tiles of the unit in this run
  __device__ __forceinline__ void take(const int4 &a, const int4 &b, const int4 &c) {
    un.cost0 = a.x; un.tiles = a.y; un.pages = a.z; un.shared = a.w;
    un.row0 = b.x; un.rows = b.y; un.seq0 = b.z; un.members = b.w;
    un.table_seq = c.x;
  }
  __device__ __forceinline__ Runs(const Params &p, int cid_) : cid(cid_), fresh(true) {
    const int4 *src = reinterpret_cast<const int4 *>(p.shares + cid);
    const int4 h = src[0];
    take(src[1], src[2], src[3]);
    begin = h.x; end = h.y; u = h.z; units = h.w;
  }
  __device__ __forceinline__ bool next(const Params &p) {
    for (; u < units; ++u, fresh = false) {
      if (!fresh) {
        const int4 *src = reinterpret_cast<const int4 *>(p.units + u);
        take(src[0], src[1], src[2]);
      }
      if (un.cost0 >= end) break;
      t0 = max(begin - un.cost0, 0);
      t1 = min(end - un.cost0, un.tiles);
      if (t0 < t1) {
        ++u;
        fresh = false;
        return true;
      }
    }
    u = units;
    return false;
  }
  // u and cid only rise along the list, so that every (unit, cluster) has a partial of its own.
  __device__ __forceinline__ int64_t part_row() const { return (int64_t)(u - 1 + cid) * kUnitRows; }
  __device__ __forceinline__ int pages_end() const { return min(2 * t1, un.pages); }
};

__device__ __forceinline__ int64_t page_row(const Params &p, int seq, int page) {
  const int key = page * kPage;
  const int lb = key / p.block_size;
  if (lb >= p.max_blocks_per_seq) return -1;
  const int blk = p.block_table[(int64_t)seq * p.max_blocks_per_seq + lb];
  if (blk < 0 || blk >= p.num_blocks) return -1;
  return (int64_t)blk * p.block_size + key % p.block_size;
}

// The members of a unit, one per lane, and whose page is whose.  Warp-collective.
struct Members {
  int first, keys;    // this lane's member: its first page among the unit's own pages, its own keys
  int shared;
  __device__ __forceinline__ void load(const Params &p, const SharedUnit &un) {
    const int lane = threadIdx.x & 31, b = un.seq0 + min(lane, un.members - 1);
    shared = un.shared;
    first = p.own_pages[b] - p.own_pages[un.seq0];
    keys = min(max(p.seqlens[b], 0), p.max_seqlen) - kPage * shared;
    if (lane >= un.members) first = 0x7fffffff;
  }
  // Owner of page v of the unit, the same for the whole warp (-1: shared), and which of its own pages it is.
  __device__ __forceinline__ int owner(int v, int &page) const {
    const int x = v - shared;
    const int m = __popc(__ballot_sync(0xffffffffu, first <= x)) - 1;   // members without pages share their successor's place
    page = x - __shfl_sync(0xffffffffu, first, max(m, 0));
    return m;
  }
  // Pool row of page v, one page per lane.
  __device__ __forceinline__ int64_t row(const Params &p, const SharedUnit &un, int v) const {
    const int x = v - shared;
    int m = 0, f = 0;
    for (int i = 0; i < un.members; ++i) {
      const int fi = __shfl_sync(0xffffffffu, first, i);
      if (fi <= x) {
        m = i;
        f = fi;
      }
    }
    return x < 0 ? page_row(p, un.table_seq, v) : page_row(p, un.seq0 + m, shared + x - f);
  }
};

// Pool rows of a run's pages, looked up a warp-load at a time, one load ahead.
struct PageRows {
  Members mem;
  int base = 0;
  int64_t r0 = -1, r1 = -1;
  __device__ __forceinline__ int64_t look(const Params &p, const SharedUnit &un, int v) const {
    const int64_t r = mem.row(p, un, min(v, un.pages - 1));
    return v < un.pages ? r : -1;
  }
  __device__ __forceinline__ void start(const Params &p, const SharedUnit &un, int page) {
    mem.load(p, un);
    base = page;
    r0 = look(p, un, base + (threadIdx.x & 31));
    r1 = look(p, un, base + 32 + (threadIdx.x & 31));
  }
  // Pages must be asked for in ascending order from the start page on.
  __device__ __forceinline__ int64_t get(const Params &p, const SharedUnit &un, int page) {
    while (page >= base + 32) {
      base += 32;
      r0 = r1;
      r1 = look(p, un, base + 32 + (threadIdx.x & 31));
    }
    return __shfl_sync(0xffffffffu, r0, page - base);
  }
};

// The latents of a page before its MMAs, thread t of 256: rows from `keys` on become zero and, with `scan`, so does every
// value that is not finite.  The rows that see such a key have NaN from their scores, or from a sum that is made NaN at the
// end of the run.
__device__ __noinline__ void tidy_page(unsigned char *vt, int keys, int scan, int t) {
  // 4 chunks of 64 rows of 8 pieces of 16 bytes; piece t + 256 i lies in row (t >> 3) + 32 (i & 1) of chunk i >> 1.
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    uint4 *at = reinterpret_cast<uint4 *>(vt) + t + 256 * i;
    if ((t >> 3) + 32 * (i & 1) >= keys) {
      *at = make_uint4(0, 0, 0, 0);
    } else if (scan) {
      const uint4 y = *at;
      uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] &= ((w[e] & 0x7f80u) == 0x7f80u ? 0u : 0xffffu) | ((w[e] & 0x7f800000u) == 0x7f800000u ? 0u : 0xffff0000u);
      *at = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// Whether this lane's row sees a key of member `mine` whose latents are not all finite among the own pages of a run: `vis` own
// keys of that member are seen.  Warp-collective, and slow: for runs that have scores which are not finite.
__device__ __noinline__ bool sees_lost_key(const Params &p, const SharedUnit un, const Members mem, int page0, int page1, int mine,
                                           int vis) {
  const int lane = threadIdx.x & 31;
  bool sees = false;
#pragma unroll 1
  for (int v = max(page0, un.shared); v < page1; ++v) {
    int own;
    const int m = mem.owner(v, own);
    if (!__any_sync(0xffffffffu, m == mine)) continue;
    const int left = __shfl_sync(0xffffffffu, mem.keys, m) - kPage * own;
    const int64_t row = max(mem.row(p, un, v), (int64_t)0);
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      const int key = lane + 32 * half;
      bool bad = false;
#pragma unroll 1
      for (int c = 0; c < kDc / 64 && key < left; ++c) {
        const unsigned char *src = p.tiled ? p.tiled + (row / kPage) * (9 * kChunkBytes) + c * kChunkBytes + key * 128
                                           : p.rows + (row + key) * p.row_bytes + c * 128;
        for (int g = 0; g < 8; ++g) {
          const uint4 y = *reinterpret_cast<const uint4 *>(src + 16 * g);
          const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) bad |= (w[e] & 0x7f80u) == 0x7f80u || (w[e] & 0x7f800000u) == 0x7f800000u;
        }
      }
      const uint32_t lost = __ballot_sync(0xffffffffu, bad);
      const int first = lost ? __ffs(lost) - 1 + 32 * half : kPage;
      sees |= m == mine && kPage * own + first < vis && first < kPage;
    }
  }
  return sees;
}

__global__ void __cluster_dims__(4, 1, 1) __launch_bounds__(kThreads, 1)
shared_attn_kernel(const __grid_constant__ CUtensorMap map_c, const __grid_constant__ CUtensorMap map_pe,
                   const __grid_constant__ Params p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char *tiles = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Small &sm = *reinterpret_cast<Small *>(tiles + kRegion);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank(), side = rank & 1;   // side: which 128 rows
  const bool score = rank < 2, lead = side == 0;
  const int cid = (int)cluster_id_x();
  auto bar = [&](int i) { return smem_u32(&sm.bars[i]); };

  grid_dep_launch();
  if (threadIdx.x == 0) {
    for (int i = 0; i < B_COUNT; ++i) {
      uint32_t n = 1;
      if (i == B_QREADY || i == B_OFREE) n = 2 * kSoftWarps;
      if (i >= B_SEMPTY && i < B_SEMPTY + 2) n = kSoftWarps;   // four warps of each CTA
      if (lead && ((i >= B_KFULL && i < B_KFULL + kKStages) || (i >= B_CFULL && i < B_CFULL + kVStages))) n = 2;
      if (i == B_STATSEMPTY || i == B_REQDONE) n = kSoftWarps;
      if (i >= B_STGFULL && i < B_STGFULL + kStgTiles) n = 4;
      if (i == B_STATSFULL) n = kRows;
      mbar_init(bar(i), n);
    }
    if (!score)
      for (int i = 0; i < kPSlots; ++i) mbar_expect_tx(bar(B_PFULL + i), kPTxBytes);
    sm.abort = 0;
    fence_mbar_init();
  }
  if (warp == 3) {
    tmem_alloc2(smem_u32(&sm.tmem_base), 512);
    tmem_relinquish2();
  }
  if (threadIdx.x == 32 && !p.tiled) {
    tma_prefetch_desc(&map_c);
    tma_prefetch_desc(&map_pe);
  }
  tc_fence_before();
  cluster_sync();   // barriers ready in all CTAs before any remote arrival
  tc_fence_after();
  const uint32_t tbase = sm.tmem_base;
  grid_dep_wait();  // the plan and the queries come from earlier kernels, whose reads of the partials are over too

  Runs it(p, cid);
  if (warp < 4) {
    if (score) {
      if (warp == 0) {
        // ---- keys: page `side` of every tile as two stages; a tile without that page passes its stages on empty.
        uint32_t n = 0;
        PageRows pr;
        int ok = 1;
        while (ok && it.next(p)) {
          pr.start(p, it.un, 2 * it.t0);
          for (int t = it.t0; ok && t < it.t1; ++t) {
            const int page = 2 * t + (int)side;
            const bool have = page < it.un.pages;
            int64_t row = pr.get(p, it.un, have ? page : 2 * t);
            if (row < 0) {
              if (lane == 0) report(p.dev_status, MLA_ERR_BAD_INDEX);
              row = 0;
            }
            if (lane == 0)
              for (int half = 0; half < 2; ++half, ++n) {
                const int s = n % kKStages;
                if (n >= kKStages && !wait1(sm, bar(B_KEMPTY + s), (n / kKStages - 1) & 1, p.dev_status)) {
                  ok = 0;
                  break;
                }
                if (!have) {
                  mbar_arrive(bar(B_KFULL + s));
                  continue;
                }
                const uint32_t dst = smem_u32(tiles + kKOff + k_stage_off(s));
                const int c0 = 4 * half, nc = half_chunks(half);
                mbar_expect_tx(bar(B_KFULL + s), nc * kChunkBytes);
                if (p.tiled)
                  bulk_load(dst, p.tiled + (row / kPage) * (9 * kChunkBytes) + c0 * kChunkBytes, nc * kChunkBytes,
                            bar(B_KFULL + s));
                else
                  for (int c = 0; c < nc; ++c) {
                    if (c0 + c < 8) tma_load_2d(dst + c * kChunkBytes, &map_c, 64 * (c0 + c), (int32_t)row, bar(B_KFULL + s));
                    else tma_load_2d(dst + c * kChunkBytes, &map_pe, 0, (int32_t)row, bar(B_KFULL + s));
                  }
              }
            ok = __shfl_sync(0xffffffffu, ok, 0);
          }
        }
        // Drain: what was loaded last into each stage has landed before the CTA may exit.
        if (lane == 0)
          for (uint32_t i = n > kKStages ? n - kKStages : 0; i < n; ++i)
            mbar_wait(bar(B_KFULL + i % kKStages), (i / kKStages) & 1, kWaitNs);
      } else if (warp == 1 && lead) {
        // ---- S [256 x 128] = Q . K^T, the tile's two pages being the two CTAs' halves of B.
        const uint32_t idesc = idesc_bf16_f32(kUnitRows, 2 * kPage, false, false);
        const uint64_t qpe = smem_desc_sw128(smem_u32(tiles + kQpeOff), 16, 1024);
        uint32_t n = 0, ns = 0, uc = 0;
        bool ok = true;
        while (ok && it.next(p)) {
          ok = waitw(sm, bar(B_QREADY), uc & 1, p.dev_status, true);
          ++uc;
          for (int t = it.t0; ok && t < it.t1; ++t, ++ns) {
            const uint32_t sbuf = ns & 1, dcol = tbase + kSCol + 128 * sbuf;
            if (ns >= 2 && !(ok = waitw(sm, bar(B_SEMPTY + sbuf), (ns / 2 - 1) & 1, p.dev_status))) break;
#pragma unroll
            for (int half = 0; half < 2; ++half, ++n) {
              const int s = n % kKStages;
              const uint32_t par = (n / kKStages) & 1;
              ok = ok && waitw(sm, bar(B_KFULL + s), par, p.dev_status);
              if (!ok) break;
              tc_fence_after();
              const uint64_t kd = smem_desc_sw128(smem_u32(tiles + kKOff + k_stage_off(s)), 16, 1024);
#pragma unroll
              for (int c = 0; c < half_chunks(half); ++c) {
                const int j = 4 * half + c;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                  const uint64_t bd = kd + ((c * kChunkBytes + kk * 32) >> 4);
                  if (j < 8) mma2_ts(dcol, tbase + kQCol + 32 * j + 8 * kk, bd, idesc, (j | kk) ? 1u : 0u);
                  else mma2_ss(dcol, qpe + ((kk * 32) >> 4), bd, idesc, 1u);
                }
              }
              commit2(bar(B_KEMPTY + s), kScorePair);
            }
            if (ok) commit2(bar(B_SFULL + sbuf), kScorePair);
          }
        }
      } else if (warp == 1 && lane == 0) {
        // ---- rank 1: tells rank 0 about its stages.
        const uint32_t kpeer = mapa(bar(B_KFULL), 0);
        uint32_t n = 0;
        bool ok = true;
        while (ok && it.next(p))
          for (int i = 2 * it.t0; ok && i < 2 * it.t1; ++i, ++n) {
            const int s = n % kKStages;
            ok = wait1(sm, bar(B_KFULL + s), (n / kKStages) & 1, p.dev_status);
            if (ok) mbar_arrive_cluster_light(kpeer + 8 * s);
          }
      } else if (warp == 2 && lane == 0) {
        // ---- sender: every staged page, in order, to the value CTA of these rows, once the MMAs that read the slot before
        // are complete.  A staging tile is given back when the page after it is under way.  That the tiles come back in
        // order is what lets both softmax groups wait for them by parity: whoever stages page q has seen page q - 6
        // given back (with its own page before q, at most three earlier, it waited for a page at or behind q - 6).
        const uint32_t mate = 2 + side;
        const uint32_t pslot_remote = mapa(smem_u32(tiles + kPOff), mate), pfull_remote = mapa(bar(B_PFULL), mate);
        uint32_t pn = 0;
        bool ok = true;
        while (ok && it.next(p))
          for (int g = 2 * it.t0; g < it.pages_end(); ++g, ++pn) {
            const uint32_t pb = pn % kPSlots, sg = pn % kStgTiles;
            ok = wait1(sm, bar(B_STGFULL + sg), (pn / kStgTiles) & 1, p.dev_status) &&
                 (pn < kPSlots || wait1(sm, bar(B_PEMPTY + pb), (pn / kPSlots - 1) & 1, p.dev_status, true));
            if (!ok) break;
            bulk_copy_to_peer(pslot_remote + pb * kPSlotBytes, smem_u32(tiles + kStgOff + sg * kPSlotBytes), kPTxBytes,
                              pfull_remote + 8 * pb);
            bulk_commit();
            bulk_wait_read_but_last();
            if (pn > 0) mbar_arrive(bar(B_STGEMPTY + (pn - 1) % kStgTiles));
          }
        bulk_wait_all();   // the copies have landed before the CTA may exit
      }
    } else {
      if (warp == 0) {
        // ---- latents: dims 256 side .. of every page, one stage each.
        uint32_t n = 0;
        PageRows pr;
        int ok = 1;
        while (ok && it.next(p)) {
          pr.start(p, it.un, 2 * it.t0);
          for (int g = 2 * it.t0; ok && g < it.pages_end(); ++g, ++n) {
            int64_t row = pr.get(p, it.un, g);
            if (row < 0) row = 0;   // reported by the score pair
            const int s = n % kVStages;
            if (lane == 0) {
              if (n >= kVStages && !wait1(sm, bar(B_CEMPTY + s), (n / kVStages - 1) & 1, p.dev_status)) ok = 0;
              if (ok) {
                const uint32_t dst = smem_u32(tiles + s * kVStageBytes);
                mbar_expect_tx(bar(B_CFULL + s), kVStageBytes);
                if (p.tiled)
                  bulk_load(dst, p.tiled + (row / kPage) * (9 * kChunkBytes) + side * kVStageBytes, kVStageBytes,
                            bar(B_CFULL + s));
                else
                  for (int c = 0; c < 4; ++c)
                    tma_load_2d(dst + c * kChunkBytes, &map_c, 256 * (int)side + 64 * c, (int32_t)row, bar(B_CFULL + s));
              }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
          }
        }
        if (lane == 0)
          for (uint32_t i = n > kVStages ? n - kVStages : 0; i < n; ++i)
            mbar_wait(bar(B_CFULL + i % kVStages), (i / kVStages) & 1, kWaitNs);
      } else if (warp == 1) {
        // ---- O += P . C.  Both CTAs walk the pages alike: P has landed, O rescaled where the page asks for it, C has
        // landed; rank 3 then reports to rank 2, which issues for both.
        const uint32_t idesc = idesc_bf16_f32(kUnitRows, 256, false, true);
        const uint32_t ready = mapa(bar(B_CFULL), 2);
        uint32_t np = 0, uc = 0, nfix = 0;
        int run_pages = 0;
        bool ok = true;
        while (ok && it.next(p)) {
          Members mem;
          mem.load(p, it.un);
          if (uc > 0) {
            // Warp 2 must have seen the phases of the run's last slots before these go round again, or it would wait for the
            // other parity: no phase of this barrier completes before the one ahead of it has been waited for here.
            if (!(ok = waitw(sm, bar(B_OFREE), (uc - 1) & 1, p.dev_status) && waitw(sm, bar(B_RUNSEEN), (uc - 1) & 1, p.dev_status))) break;
            // The epilogue is through with the P slots of the finished run's last two pages, which it borrowed.
            if (lane < 2 && run_pages >= 2) {
              const int pb = (np - 2 + lane) % kPSlots;
              mbar_expect_tx(bar(B_PFULL + pb), kPTxBytes);
              mbar_arrive_cluster(mapa(bar(B_PEMPTY + pb), side));   // (it stored there)
            }
            __syncwarp();
          }
          for (int g = 2 * it.t0; g < it.pages_end(); ++g, ++np) {
            const int pb = np % kPSlots, sv = np % kVStages;
            const uint32_t ppar = (np / kPSlots) & 1;
            if (!(ok = waitw(sm, bar(B_PFULL + pb), ppar, p.dev_status))) break;
            const uint32_t slot = smem_u32(tiles + kPOff + pb * kPSlotBytes);
            const bool first = g == 2 * it.t0;
            // Rows past the last key may hold anything (NaN), and one member's keys may for the others, whose P is 0 there:
            // 0 * x is 0 for finite x only.
            int own;
            const int m = mem.owner(g, own);
            const int left = m < 0 ? kPage : __shfl_sync(0xffffffffu, mem.keys, m) - kPage * own;
            uint32_t flags = 0;
            const float *pa = reinterpret_cast<const float *>(tiles + kPOff + pb * kPSlotBytes + kPBytes);
#pragma unroll
            for (int w = 0; w < 4; ++w) flags |= reinterpret_cast<const uint32_t *>(pa + w * kPaWords)[32];
            const bool moved = flags & kMoved, odd = flags & kOdd;
            // At rank 2 the phase holds rank 3's arrival, which passes on what its epilogue warps stored in an own page.
            if (!(ok = waitw(sm, bar(B_CFULL + sv), (np / kVStages) & 1, p.dev_status, lead && m >= 0))) break;
            if (flags || left < kPage) {
              // O is read back for a rescale: the previous page's MMAs must be complete.
              if (moved && !(ok = waitw(sm, bar(B_PVDONE + (np - 1) % kPSlots), ((np - 1) / kPSlots) & 1, p.dev_status)))
                break;
              if (lane == 0) {
                sm.req = Req{0, moved, pb, left, sv, odd, 0, 0};
                mbar_arrive(bar(B_REQ));
              }
              if (!(ok = waitw(sm, bar(B_REQDONE), nfix & 1, p.dev_status))) break;
              tc_fence_after();
              ++nfix;
            }
            if (!lead) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) {
                if (odd || left < kPage) mbar_arrive_cluster(ready + 8 * sv);   // the page was tidied: by stores that rank 2's MMAs read
                else mbar_arrive_cluster_light(ready + 8 * sv);
              }
              continue;
            }
            tc_fence_after();
            const uint64_t ad = smem_desc_sw128(slot, 16, 1024);
            const uint64_t bd = smem_desc_sw128(smem_u32(tiles + sv * kVStageBytes), kChunkBytes, 1024);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                mma2_ss(tbase + 256 * h, ad + ((ks * 32) >> 4), bd + ((h * 2 * kChunkBytes + ks * 2048) >> 4), idesc,
                        (first && ks == 0) ? 0u : 1u);
            commit2(bar(B_CEMPTY + sv), kValuePair);
            commit2(bar(B_PVDONE + pb), kValuePair);
          }
          if (!ok) break;
          run_pages = it.pages_end() - 2 * it.t0;
          if (lane == 0) {
            sm.req = Req{1, 0, 0, 0, 0, 0, (int)np, run_pages};
            mbar_arrive(bar(B_REQ));
          }
          __syncwarp();
          ++uc;
        }
      } else if (warp == 2 && lane == 0) {
        // ---- a P slot may be written again once the MMAs that read it are complete (the last two of a run go to the
        // epilogue first: see warp 1).
        const uint32_t pempty = mapa(bar(B_PEMPTY), side);
        uint32_t np = 0;
        bool ok = true;
        while (ok && it.next(p)) {
          const int n = it.pages_end() - 2 * it.t0;
          for (int i = 0; i < n; ++i, ++np) {
            const int pb = np % kPSlots;
            if (!(ok = wait1(sm, bar(B_PVDONE + pb), (np / kPSlots) & 1, p.dev_status))) break;
            if (n >= 2 && i >= n - 2) continue;
            mbar_expect_tx(bar(B_PFULL + pb), kPTxBytes);
            mbar_arrive_cluster_light(pempty + 8 * pb);
          }
          if (ok) mbar_arrive(bar(B_RUNSEEN));
        }
      }
    }
  } else if (score) {
    // ---- softmax: two groups of four warps take the tiles in turn, group h those of S buffer h; warp (quadrant q4)
    // owns rows 32 q4 .. of both pages.  While one group waits for tensor memory, barriers or its copy, the other has
    // the SM's exponentials.  The reference maximum passes from tile to tile, so from group to group, through
    // m_sh and a pair of named barriers.  No early exit: after a timeout every wait returns at once.
    const int q4 = warp & 3, h = (warp - 4) >> 2;
    const int r = q4 * 32 + lane;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    uint32_t ns = 0, np = 0, uc = 0;
    // The staging tile of page pn, once the copy of page pn - kStgTiles has read it.  (The copies of earlier pages do not
    // wait for this one, whichever group stages them.)
    auto staging = [&](uint32_t pn) {
      if (pn >= kStgTiles)
        waitw(sm, bar(B_STGEMPTY + pn % kStgTiles), (pn / kStgTiles - 1) & 1, p.dev_status);
      return tiles + kStgOff + (pn % kStgTiles) * kPSlotBytes;
    };
    while (it.next(p)) {
      // Queries of the unit: latent dims 256 h .. of the warp's rows into tensor memory, coalesced through the warp's
      // part of a P staging tile (one that the unit's first two pages will use); half 0 also stages the RoPE dims.  Both
      // groups have read the last S of the previous unit, so its MMAs are complete.
      {
        unsigned char *stg_w = staging(np + h) + q4 * 4096;
        const int j = lane & 7;
        // This lane's rows are r0, r0 + 4, .. of the unit, contiguous in memory.
        const int r0 = kRows * (int)side + q4 * 32 + (lane >> 3);
        const int left = it.un.rows - r0;
        const uint4 *src = reinterpret_cast<const uint4 *>(p.q + (int64_t)(it.un.row0 + r0) * kW) + j;
        constexpr int kStep = 4 * kW / 8;   // 16-byte words between a lane's rows
        // Two of the four 64-dim columns in flight; a column's registers take the one after next as soon as it is staged,
        // and the RoPE dims (half 0 only) after those.
        uint4 x[2][8];
        auto load_column = [&](uint4 (&dst)[8], int word) {
#pragma unroll
          for (int k = 0; k < 8; ++k) dst[k] = 4 * k < left ? __ldg(src + k * kStep + word) : make_uint4(0, 0, 0, 0);
        };
#pragma unroll
        for (int cb = 0; cb < 2; ++cb) load_column(x[cb], h * 32 + cb * 8);
#pragma unroll
        for (int cb = 0; cb < 4; ++cb) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int lr = 4 * k + (lane >> 3);
            *reinterpret_cast<uint4 *>(stg_w + (lr >> 3) * 1024 + (lr & 7) * 128 + ((j ^ (lr & 7)) << 4)) = x[cb & 1][k];
          }
          if (cb < 2) load_column(x[cb], h * 32 + (cb + 2) * 8);
          if (cb == 2 && h == 0) load_column(x[0], 64);
          __syncwarp();
          uint32_t w[32];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 y = *reinterpret_cast<const uint4 *>(stg_w + (lane >> 3) * 1024 + (lane & 7) * 128 + ((i ^ (lane & 7)) << 4));
            w[4 * i] = y.x; w[4 * i + 1] = y.y; w[4 * i + 2] = y.z; w[4 * i + 3] = y.w;
          }
          tmem_st32(tbase + lane_off + kQCol + 128 * h + 32 * cb, w);
          __syncwarp();
        }
        if (h == 0) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int rq = q4 * 32 + 4 * k + (lane >> 3);
            *reinterpret_cast<uint4 *>(tiles + kQpeOff + (rq >> 3) * 1024 + (rq & 7) * 128 + ((j ^ (rq & 7)) << 4)) = x[0][k];
          }
          fence_proxy_async_smem();   // the MMAs read it
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        // A release for the cluster: rank 0's MMAs read the RoPE rows that these warps stored in either CTA.
        if (lane == 0) mbar_arrive_cluster(mapa(bar(B_QREADY), 0));
      }
      // This row's member and how many of that member's own keys it sees; rows past the unit's end see none.
      Members mem;
      mem.load(p, it.un);
      const int gr = it.un.row0 + kRows * (int)side + r, R = p.n_q * p.H;
      const int my_m = kRows * (int)side + r < it.un.rows ? gr / R - it.un.seq0 : -2;
      const int vis = __shfl_sync(0xffffffffu, mem.keys, max(my_m, 0)) - p.n_q + 1 + (gr % R) / p.H;
      if (q4 == 0 && lane == 0) sm.odd_seen[h] = 0;
      float m_mine = -CUDART_INF_F, l = 0.f;   // l: this group's row sum, relative to m_mine
      const uint32_t ns_end = ns + (uint32_t)(it.t1 - it.t0);
      // One tile.  Mixed: some page of it is one member's.  A copy of its own, as the checks alone that such pages need took 4 %
      // of a batch that is nearly all shared pages.
      auto tile = [&](auto mixed_tag, int t, int npg, uint32_t pn) __attribute__((always_inline)) {
        constexpr bool mixed = decltype(mixed_tag)::value;
        waitw(sm, bar(B_SFULL + h), (ns >> 1) & 1, p.dev_status);
        tc_fence_after();
        const uint32_t scol = tbase + lane_off + kSCol + 128 * h;
        uint32_t v[2][32];            // 64 scores of this row: one page
        float mx = -CUDART_INF_F;
        auto load_page = [&](int pg) {
          tmem_ld32(scol + 64 * pg, v[0]);
          tmem_ld32(scol + 64 * pg + 32, v[1]);
        };
        auto page_max = [&]() {
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            mx = max3f(mx, __uint_as_float(v[0][k]), __uint_as_float(v[0][k + 1]));
            mx = max3f(mx, __uint_as_float(v[1][k]), __uint_as_float(v[1][k + 1]));
          }
        };
        // Visible keys of both pages: 64 or more of a shared page, none of another member's page.  left: keys of the owner there.
        int n0 = kPage, n1 = kPage, left0 = -1, left1 = -1;
        auto seen = [&](int pg, int &left) {
          int own;
          const int m = mem.owner(2 * t + pg, own);
          left = m < 0 ? -1 : __shfl_sync(0xffffffffu, mem.keys, m) - kPage * own;
          return m < 0 ? kPage : (m == my_m ? vis - kPage * own : 0);
        };
        if (mixed) {
          n0 = seen(0, left0);
          if (npg == 2) n1 = seen(1, left1);
        }
        auto mask_page = [&](int n) {   // only pages that some row of the warp does not see whole
          if (!mixed || __all_sync(0xffffffffu, n >= kPage)) return;
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            v[0][k] = k < n ? v[0][k] : __float_as_uint(-CUDART_INF_F);
            v[1][k] = k + 32 < n ? v[1][k] : __float_as_uint(-CUDART_INF_F);
          }
        };
        // A latent that is not finite leaves no row's score of its key finite (0 * x is NaN), so one warp's rows tell which of
        // the pages have such.  It matters where a page is one member's among several: the others' P is 0 there, and the value
        // pair must not multiply that by NaN.  (1 to 2 us of a batch of many own pages; looking at the latents themselves
        // took 4 to 6 of 110, in shared-memory reads that the MMAs missed.)  What lies behind a member's last key is zero there
        // anyhow.
        uint32_t odd = 0;             // kOdd for the first page, kOdd << 8 for the second
        if (mixed && q4 == 0 && it.un.members > 1) {
#pragma unroll 1
          for (int pg = 0; pg < npg; ++pg) {
            const int left = pg ? left1 : left0;
            if (left < 0) continue;   // a shared page
            load_page(pg);
            tmem_wait_ld();
            float z = 0.f;
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              z = fmaf(k < left ? __uint_as_float(v[0][k]) : 0.f, 0.f, z);
              z = fmaf(k + 32 < left ? __uint_as_float(v[1][k]) : 0.f, 0.f, z);
            }
            if (__any_sync(0xffffffffu, (__float_as_uint(z) & 0x7fffffffu) != 0u)) {
              odd |= kOdd << (8 * pg);
              if (lane == 0) sm.odd_seen[h] = 1;
            }
          }
        }
        // The second page only for its maximum (it is read again below), the first one to stay.
        if (npg == 2) {
          load_page(1);
          tmem_wait_ld();
          mask_page(n1);
          page_max();
        }
        load_page(0);
        tmem_wait_ld();
        mask_page(n0);
        page_max();
        mx *= p.scale_log2;
        // The reference after the previous tile, and this tile's for the next one.
        float m_prev = -CUDART_INF_F;
        if (t != it.t0) {
          asm volatile("bar.sync %0, 256;" ::"r"(5 - h) : "memory");
          m_prev = sm.m_sh[h ^ 1][r];
        }
        const bool need = mx > m_prev + kRescaleLog2;
        const float m_ref = need ? mx : m_prev;
        const float alpha = need ? exp2f(m_prev - mx) : 1.f;
        const float m_use = m_ref == -CUDART_INF_F ? 0.f : m_ref;   // no key seen yet: every P is exp2(-inf) = 0
        sm.m_sh[h][r] = m_ref;
        asm volatile("bar.arrive %0, 256;" ::"r"(4 + h) : "memory");
        if (m_mine != m_ref) {
          l *= exp2f(m_mine - m_ref);   // m_mine = -inf: l is 0 (and m_ref, which never falls, is finite)
          m_mine = m_ref;
        }
        const uint32_t moved = __any_sync(0xffffffffu, need && t != it.t0) ? kMoved : 0u;
        float psum0 = 0.f, psum1 = 0.f;
        uint32_t pk[32];              // this row's 64 P values of a page
        auto page_p = [&]() {
#pragma unroll
          for (int c2 = 0; c2 < 2; ++c2)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float p0 = exp2f(__uint_as_float(v[c2][2 * e]) * p.scale_log2 - m_use);
              const float p1 = exp2f(__uint_as_float(v[c2][2 * e + 1]) * p.scale_log2 - m_use);
              pk[16 * c2 + e] = pack_bf16x2(p0, p1);
              psum0 += p0;
              psum1 += p1;
            }
        };
        // The first page of a tile carries its rows' rescale factors.
        auto stage = [&](uint32_t page, float factor, uint32_t flags) {
          unsigned char *stg = staging(page);
          unsigned char *prow = stg + 4096 * q4 + (lane >> 3) * 1024 + (lane & 7) * 128;
#pragma unroll
          for (int c = 0; c < 8; ++c)
            *reinterpret_cast<uint4 *>(prow + ((c ^ (lane & 7)) << 4)) = make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
          float *pa = reinterpret_cast<float *>(stg + kPBytes) + q4 * kPaWords;
          pa[lane] = factor;
          if (lane < 4) reinterpret_cast<uint32_t *>(pa + 32)[lane] = lane == 0 ? flags : 0u;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_STGFULL + page % kStgTiles));
        };
        page_p();
        load_page(1);                 // (unused columns where there is no second page)
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_light(mapa(bar(B_SEMPTY + h), 0));   // the last read of this S is done
        stage(pn, alpha, moved | (odd & kOdd));
        if (npg == 2) {
          mask_page(n1);
          page_p();
          stage(pn + 1, 1.f, odd >> 8);
        }
        l += psum0 + psum1;
      };
      for (int t = it.t0; t < it.t1; ++t, ++ns) {
        const int npg = min(2, it.un.pages - 2 * t);
        const uint32_t pn = np;             // the tile's first page
        np += npg;
        if ((int)(ns & 1) != h) continue;   // the other group's
        if (2 * t + npg > it.un.shared) tile(std::true_type{}, t, npg, pn);
        else tile(std::false_type{}, t, npg, pn);
      }
      // Row statistics of the run: the group that did not have the last tile passes its sum on, relative to the final
      // reference; the other one sends the total.
      const bool last = (int)((ns_end - 1) & 1) == h;
      if (!last) {
        asm volatile("bar.sync %0, 256;" ::"r"(5 - h) : "memory");
        const float m_end = sm.m_sh[h ^ 1][r];
        sm.xl[r] = l > 0.f ? l * exp2f(m_mine - m_end) : 0.f;   // l > 0: m_mine is finite
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (last) {
        l += sm.xl[r];
        // An infinite latent may leave a score of -inf, so a weight of 0, and is taken out of the page for the other members'
        // sake; but 0 * inf is NaN.
        if ((sm.odd_seen[0] | sm.odd_seen[1]) && sees_lost_key(p, it.un, mem, 2 * it.t0, it.pages_end(), my_m, vis)) l = CUDART_NAN_F;
        if (uc > 0) waitw(sm, bar(B_STATSEMPTY), (uc - 1) & 1, p.dev_status);
        const uint32_t mate = 2 + side;   // the value CTA of these rows
        st_cluster_f32(mapa(smem_u32(&sm.stat_l[r]), mate), l);
        st_cluster_f32(mapa(smem_u32(&sm.stat_m[r]), mate), m_mine);
        mbar_arrive_cluster(mapa(bar(B_STATSFULL), mate));
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");   // xl and m_sh may be used again
      ++uc;
    }
  } else {
    // ---- epilogue warps: group g owns O columns 256 g ..; warp w owns rows 32 (w & 3) ...
    const int g = (warp - 4) >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ocol = 256 * g;
    const uint32_t statsempty_remote = mapa(bar(B_STATSEMPTY), side);
    const uint32_t ofree2 = mapa(bar(B_OFREE), 2), ofree3 = mapa(bar(B_OFREE), 3);
    uint32_t nreq = 0, uc = 0;
    bool ok = true;
    while (ok && it.next(p)) {
      for (;;) {
        if (!(ok = waitw(sm, bar(B_REQ), nreq & 1, p.dev_status))) break;
        ++nreq;
        const Req q = sm.req;
        if (q.kind == 0) {
          if (q.rescale) {
            tc_fence_after();
            const float a = reinterpret_cast<const float *>(tiles + kPOff + q.slot * kPSlotBytes + kPBytes)[(r >> 5) * kPaWords + (r & 31)];
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t v[32];
              tmem_ld32(tbase + lane_off + ocol + 32 * c, v);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * a);
              tmem_st32(tbase + lane_off + ocol + 32 * c, v);
            }
            tmem_wait_st();
            tc_fence_before();
          }
          if (q.keys < kPage || q.scan) {
            tidy_page(tiles + q.stage * kVStageBytes, q.keys, q.scan, threadIdx.x - 128);
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_REQDONE));
          continue;
        }
        const uint32_t last = q.np - 1;
        if (!(ok = waitw(sm, bar(B_PVDONE + last % kPSlots), (last / kPSlots) & 1, p.dev_status) &&
                   waitw(sm, bar(B_STATSFULL), uc & 1, p.dev_status, true)))
          break;
        tc_fence_after();
        const float l = sm.stat_l[r], m = sm.stat_m[r];
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(statsempty_remote);
        const float inv = l == 0.f ? 0.f : 1.f / l;   // (NaN stays NaN)
        const int64_t prow = it.part_row() + kRows * side + r;
        const int rows = it.un.rows - kRows * (int)side;   // of this CTA
        const bool live = r < rows;
        // Columns 256 g .. are rank 2's dims 128 g .. 128 g + 127, then rank 3's, 256 further on.
        if ((warp & 3) * 32 >= rows) {
          // no rows of the unit here
        } else if (q.pages >= 2) {
          // 32 columns at a time through 4 KB of a P slot whose MMAs are complete (the run's last two: one per group), so
          // that rows leave in whole 128-byte lines: stores of 32 lanes to 32 rows took 5 us of LSU time a unit.
          unsigned char *stg = tiles + kPOff + ((q.np - 2 + g) % kPSlots) * kPSlotBytes + (warp & 3) * 4096;
          float *out = p.o_part + (it.part_row() + kRows * (int)side + (warp & 3) * 32) * kDc + 4 * (lane & 7);
          const int left = rows - (warp & 3) * 32 - (lane >> 3);
          uint32_t v[32];
          tmem_ld32(tbase + lane_off + ocol, v);
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<float4 *>(stg + lane * 128 + ((i ^ (lane & 7)) << 4)) =
                  make_float4(__uint_as_float(v[4 * i]) * inv, __uint_as_float(v[4 * i + 1]) * inv,
                              __uint_as_float(v[4 * i + 2]) * inv, __uint_as_float(v[4 * i + 3]) * inv);
            __syncwarp();
            tmem_ld32(tbase + lane_off + ocol + 32 * min(c + 1, 7), v);   // on its way while these are stored
            const int dim = 256 * (c >> 2) + 128 * g + 32 * (c & 3);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int lr = 4 * k + (lane >> 3);
              const float4 y = *reinterpret_cast<const float4 *>(stg + lr * 128 + (((lane & 7) ^ (lr & 7)) << 4));
              if (4 * k < left) *reinterpret_cast<float4 *>(out + (int64_t)lr * kDc + dim) = y;
            }
            __syncwarp();
          }
          tmem_wait_ld();
          fence_proxy_async_smem();   // the slot is written by copies again
        } else {
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t v[32];
            tmem_ld32(tbase + lane_off + ocol + 32 * c, v);
            tmem_wait_ld();
            const int dim = 256 * (c >> 2) + 128 * g + 32 * (c & 3);
            if (live)
#pragma unroll
              for (int i = 0; i < 32; i += 8) {
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(__uint_as_float(v[i + e]) * inv);
                st_global_v8(p.o_part + prow * kDc + dim + i, make_uint4(w[0], w[1], w[2], w[3]),
                             make_uint4(w[4], w[5], w[6], w[7]));
              }
          }
        }
        if (g == 0 && live) p.lse_part[prow] = l > 0.f ? (m + __log2f(l)) * 0.69314718055994531f : -CUDART_INF_F;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          // O has been read: no more than that, so nothing here waits for the stores above (a cluster-scope release
          // did, for 3 us).
          mbar_arrive_cluster_light(ofree2);
          mbar_arrive_cluster_light(ofree3);
        }
        ++uc;
        break;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();   // the pair frees its tensor memory together, after both CTAs' last access
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc2(tbase, 512);
  }
  cluster_sync();   // no CTA leaves while another may still reach its shared memory
}

// The plan by itself, for queries that another kernel than absorb_tc_kernel absorbs.
__global__ void __launch_bounds__(1024) shared_plan_kernel(const SharedPlanArgs a, int in_smem) {
  extern __shared__ int plan_words[];
  grid_dep_launch();
  shared_plan_body(a, in_smem ? plan_words : nullptr);
}

}  // namespace

int shared_clusters_for_device() {
  static std::atomic<int> cached[128];
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {   // no device
    cudaGetLastError();
    return 0;
  }
  if (dev < 0 || dev >= 128) return 0;
  if (const int c = cached[dev].load(std::memory_order_acquire)) return c;
  int ndev = 0;
  if (cudaGetDeviceCount(&ndev) != cudaSuccess || ndev <= 0) {
    cudaGetLastError();
    return 0;
  }
  std::lock_guard<std::mutex> lock(mu);
  if (const int c = cached[dev].load(std::memory_order_acquire)) return c;
  if (cudaFuncSetAttribute(shared_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes)) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(4 * kSharedMaxClusters);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 4;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, shared_attn_kernel, &cfg) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    return 0;
  }
  if (n > kSharedMaxClusters) n = kSharedMaxClusters;
  cached[dev].store(n, std::memory_order_release);
  return n;
}

int launch_shared_plan(const SharedPlanArgs &a, cudaStream_t st) {
  const size_t bytes = shared_plan_words(a.B, a.max_units, a.num_groups) * sizeof(int);
  const bool in_smem = bytes <= 160 * 1024;   // (some 5000 sequences in as many groups; behind that in the workspace)
  static std::atomic<int> cache[kSmemCacheDevs];
  if (in_smem && smem_limit(shared_plan_kernel, bytes, cache) != cudaSuccess) return MLA_ERR_CUDA;
  return launch_pdl(shared_plan_kernel, dim3(1), dim3(1024), in_smem ? bytes : 0, st, a, (int)in_smem) == cudaSuccess
             ? MLA_OK
             : MLA_ERR_CUDA;
}

int launch_shared_attention(const mla_dims &d, int n_q, int max_seqlen, const SharedPlan &pl, const void *q_abs,
                            const CacheView &cache, const int32_t *seqlens, float *o_part, float *lse_part,
                            int *dev_status, cudaStream_t st) {
  const bool tiled = cache.layout == MLA_CACHE_TILED;
  CUtensorMap mc, mpe;
  memset(&mc, 0, sizeof(mc));
  memset(&mpe, 0, sizeof(mpe));
  if (!tiled) {
    const uint64_t rows = (uint64_t)cache.num_blocks * cache.block_size;
    if (!make_tmap_bf16(&mc, cache.c_kv, kDc, rows, (uint64_t)cache.ckv_stride * 2, kPage) ||
        !make_tmap_bf16(&mpe, cache.k_pe, kDr, rows, (uint64_t)cache.kpe_stride * 2, kPage))
      return MLA_ERR_CUDA;
  }
  const int C = shared_clusters_for_device();
  if (C <= 0) return MLA_ERR_CUDA;
  Params p;
  p.shares = pl.shares;
  p.units = pl.units;
  p.q = static_cast<const __nv_bfloat16 *>(q_abs);
  p.block_table = cache.block_table;
  p.max_blocks_per_seq = cache.max_blocks_per_seq;
  p.num_blocks = cache.num_blocks;
  p.block_size = cache.block_size;
  p.H = d.n_heads;
  p.n_q = n_q;
  p.max_seqlen = max_seqlen;
  p.seqlens = seqlens;
  p.own_pages = pl.own_pages;
  p.scale_log2 = default_scale(d) * 1.4426950408889634f;
  p.o_part = o_part;
  p.lse_part = lse_part;
  p.dev_status = dev_status;
  p.tiled = tiled ? static_cast<const unsigned char *>(cache.c_kv) : nullptr;
  p.rows = static_cast<const unsigned char *>(cache.c_kv);
  p.row_bytes = 2 * (int64_t)cache.ckv_stride;
  return launch_pdl(shared_attn_kernel, dim3(4 * C), dim3(kThreads), kSmemBytes, st, mc, mpe, p) == cudaSuccess
             ? MLA_OK
             : MLA_ERR_CUDA;
}

}  // namespace mla
