// Merge of the partials of a decode over shared prefixes, and the per-head up-projection.
//
// Each piece k of a query row carries (O_k normalised by its own sum, lse_k); the row's latent output is
// o_lat = sum_k exp(lse_k - LSE) O_k, LSE = log sum_k exp(lse_k), and out^(s) = o_lat W_UV^(s).
//
// CTA = (head s, 256 / kTpr query rows (b, j), 8 to 64).  The rows' pieces (fp32) are merged straight into the B operand
// of out^T [128 x rows] = W_UV^(s)T . o_lat^T on the tensor cores (W_UV supplies the 128-row M side).  Each merged row
// goes in twice, as the bf16 of its values and the bf16 of what that rounding left; the two products are added in fp32, so
// that the row reaches W_UV with 16 bits instead of 8 (one rounding less in the result: 0.0030 -> 0.0025 of its norm,
// 0.0017 being the rounding of the output itself).  The tile then takes 128 KB, and W_UV (128 KB) does not fit beside
// it: six of its eight 64-row chunks lie in shared memory and two, transposed, in tensor memory (A operand of TS-form
// MMAs), all of them brought in before the kernel waits for the attention.  (Sending the last two after the first two had
// been read took 1.4 to 2.5 us more per tile.)
// Bound by latency: a chain of dependent loads (group, unit, log-sum-exps, pieces), then the MMAs and the stores.  kTpr
// threads per row, all of a row's blocks of two pieces in flight; the fewest rows per CTA with which every CTA is resident
// at once (one per SM), further tiles of a head in the same CTA.  (32 query rows x 16 heads with 8 rows a CTA: the call
// 51 us, with 64 rows a CTA 58.)  11 us behind the attention at 64 rows x 128 heads, 21 at 96 (two tiles a CTA).
#include <cuda.h>
#include <math_constants.h>

#include "shared_tc.cuh"
#include "sm100.cuh"
#include "tmap.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kDc = 512, kDv = 128;
constexpr int kPartRows = kSharedPartRows;
constexpr int kTile = 64;                          // rows of the largest tile
constexpr int kThreads = 256;
constexpr int kChunks = kDc / 64;                  // K chunks of 64 latent dims
constexpr uint32_t kOlChunk = 2 * kTile * 128;     // [64 rounded rows, 64 remainder rows][128 B]
constexpr uint32_t kWChunk = 64 * kDv * 2;         // [2 halves of the output dims][64 latent dims][128 B]
constexpr int kWSmem = 6;                          // chunks of W_UV in shared memory; the others in tensor memory
constexpr uint32_t kWCol = 2 * kTile;              // tensor-memory columns: the product, then 32 per chunk of W_UV^T
constexpr uint32_t kTmemCols = 256;
static_assert(kWCol + (kChunks - kWSmem) * 32 <= kTmemCols, "tensor memory");
constexpr size_t kSmem = 1024 + kChunks * kOlChunk + kWSmem * kWChunk;
static_assert(kSmem <= 232448, "shared memory budget");
constexpr uint64_t kWaitNs = 2000000000ull;

struct Pieces {
  const float *part, *lse;     // rows of 512, their log-sum-exps
  const int2 *unit_parts;      // first partial and number of partials of every unit
  const int2 *seq_group;       // [B]: first unit of the sequence's group, the group's first query row
  int n_q, H, unit_rows;       // unit_rows: query rows of a full unit
};

struct PieceRows {
  int ns = 0;
  int64_t first = 0;
  __device__ __forceinline__ int64_t at(int k) const { return first + (int64_t)k * kPartRows; }
};

// Pieces of query row g = (b, j) of head s.
__device__ __forceinline__ PieceRows piece_rows(const Pieces &pc, int g, int s) {
  PieceRows r;
  const int2 sg = pc.seq_group[g / pc.n_q];
  const int q = g * pc.H + s - sg.y;   // row within the group
  const int2 up = pc.unit_parts[sg.x + q / pc.unit_rows];
  r.first = (int64_t)up.x * kPartRows + q % pc.unit_rows;
  r.ns = up.y;
  return r;
}

// Largest log-sum-exp of a row's pieces and the sum of their weights relative to it, eight loads in flight.
__device__ __forceinline__ void weigh(const Pieces &pc, const PieceRows &pr, float &m, float &sum) {
  m = -CUDART_INF_F;
  for (int k0 = 0; k0 < pr.ns; k0 += 8) {
    float t[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) t[k] = k0 + k < pr.ns ? pc.lse[pr.at(k0 + k)] : -CUDART_INF_F;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = fmaxf(m, t[k]);
  }
  sum = 0.f;
  if (m != -CUDART_INF_F)
    for (int k = 0; k < pr.ns; ++k) sum += __expf(pc.lse[pr.at(k)] - m);
}

// acc[b][0..8) = the merged columns 8 blk(b) .. of a row, kFly pieces' loads at a time.
template <int kBlocks, int kFly, typename Blk>
__device__ __forceinline__ void merge_blocks(const Pieces &pc, const PieceRows &pr, float m, float inv, Blk blk,
                                             float (&acc)[kBlocks][8]) {
#pragma unroll
  for (int i = 0; i < kBlocks; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[i][e] = 0.f;
  for (int k0 = 0; k0 < pr.ns; k0 += kFly) {
    float4 x[kFly][kBlocks][2];
    float w[kFly];
#pragma unroll
    for (int k = 0; k < kFly; ++k) {
      const bool have = k0 + k < pr.ns;
      const int64_t row = pr.at(have ? k0 + k : 0);
#pragma unroll
      for (int i = 0; i < kBlocks; ++i) {
        const float4 *src = reinterpret_cast<const float4 *>(pc.part + row * kDc + 8 * blk(i));
        x[k][i][0] = have ? src[0] : make_float4(0.f, 0.f, 0.f, 0.f);
        x[k][i][1] = have ? src[1] : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      w[k] = have && m != -CUDART_INF_F ? __expf(pc.lse[row] - m) * inv : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kFly; ++k)
#pragma unroll
      for (int i = 0; i < kBlocks; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          acc[i][4 * h] = fmaf(w[k], x[k][i][h].x, acc[i][4 * h]);
          acc[i][4 * h + 1] = fmaf(w[k], x[k][i][h].y, acc[i][4 * h + 1]);
          acc[i][4 * h + 2] = fmaf(w[k], x[k][i][h].z, acc[i][4 * h + 2]);
          acc[i][4 * h + 3] = fmaf(w[k], x[k][i][h].w, acc[i][4 * h + 3]);
        }
  }
}

__device__ __forceinline__ float merged_lse(float m, float sum) { return sum > 0.f ? m + logf(sum) : -CUDART_INF_F; }

template <int kTpr>
__global__ void __launch_bounds__(kThreads, 1)
shared_combine_kernel(const __grid_constant__ CUtensorMap map_w, const __nv_bfloat16 *w_uv, const Pieces pc, int rows,
                      float *lse_out, __nv_bfloat16 *out, int *dev_status) {
  extern __shared__ unsigned char raw[];
  unsigned char *ol = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  unsigned char *wa = ol + kChunks * kOlChunk;
  __shared__ __align__(8) uint64_t bar_w, bar_mma;
  __shared__ uint32_t tmem_slot;
  __shared__ int s_ok;
  const int s = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kR = kThreads / kTpr;         // rows of a tile
  grid_dep_launch();
  // W_UV[s] (an input: no need to wait for the attention).
  if (tid == 0) {
    mbar_init(smem_u32(&bar_w), 1);
    mbar_init(smem_u32(&bar_mma), 1);
    fence_mbar_init();
    tma_prefetch_desc(&map_w);
    mbar_expect_tx(smem_u32(&bar_w), kWSmem * kWChunk);
    for (int kc = 0; kc < kWSmem; ++kc)
      for (int half = 0; half < 2; ++half)
        tma_load_2d(smem_u32(wa + kc * kWChunk + half * (kWChunk / 2)), &map_w, 64 * half, s * kDc + 64 * kc, smem_u32(&bar_w));
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  // Chunk kWSmem + (warp >> 2), transposed: output dim 32 (warp & 3) + lane is this thread's tensor-memory lane, its
  // column c holds latent dims 2 c and 2 c + 1 of the chunk.
  {
    const __nv_bfloat16 *src = w_uv + ((int64_t)s * kDc + 64 * (kWSmem + (warp >> 2))) * kDv + (warp & 3) * 32 + lane;
    uint32_t w[32];
#pragma unroll
    for (int c = 0; c < 32; ++c)
      w[c] = (uint32_t)__bfloat16_as_ushort(src[(2 * c) * kDv]) | ((uint32_t)__bfloat16_as_ushort(src[(2 * c + 1) * kDv]) << 16);
    tmem_st32(tmem + ((uint32_t)((warp & 3) * 32) << 16) + kWCol + 32 * (warp >> 2), w);
    tmem_wait_st();
  }
  grid_dep_wait();   // the plan and the partials
  uint32_t it = 0;   // tiles done
  bool fine = true;  // warp 0: W_UV has arrived
  // This thread's row of the tile, its pieces and their weights; those of the next tile are looked up while the MMAs of
  // this one run.
  const int rr = tid / kTpr, q = tid % kTpr;
  PieceRows pr;
  float m = 0.f, sum = 0.f;
  auto look_up = [&](int g0) {
    pr = g0 + rr < rows ? piece_rows(pc, g0 + rr, s) : PieceRows();
    weigh(pc, pr, m, sum);
  };
  look_up(blockIdx.y * kR);
  for (int g0 = blockIdx.y * kR; g0 < rows; g0 += gridDim.y * kR, ++it) {
    {
      // Row rr of the tile (rows past the end: zero; those past kR stay as they are, they touch only their own columns of
      // the product).  This thread's blocks of 8 columns: kTpr i + q.
      constexpr int kNb = 64 / kTpr, kAtOnce = kNb < 8 ? kNb : 8, kFly = kAtOnce >= 4 ? 2 : 8 / kAtOnce;
      const int g = g0 + rr;
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll 1
      for (int hh = 0; hh < kNb / kAtOnce; ++hh) {
        float acc[kAtOnce][8];
        auto blk = [&](int i) { return kTpr * (kAtOnce * hh + i) + q; };
        merge_blocks<kAtOnce, kFly>(pc, pr, m, inv, blk, acc);
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          uint32_t w[4], z[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            w[e] = pack_bf16x2(acc[i][2 * e], acc[i][2 * e + 1]);
            // A bf16 is the upper half of its fp32.  (The remainder of a value beyond bf16's range is no number, as
            // the value itself is not.)
            z[e] = pack_bf16x2(acc[i][2 * e] - __uint_as_float(w[e] << 16),
                               acc[i][2 * e + 1] - __uint_as_float(w[e] & 0xffff0000u));
          }
          const int cb = blk(i);
          unsigned char *at = ol + (cb >> 3) * kOlChunk + (rr >> 3) * 1024 + (rr & 7) * 128 + (((cb & 7) ^ (rr & 7)) << 4);
          *reinterpret_cast<uint4 *>(at) = make_uint4(w[0], w[1], w[2], w[3]);
          *reinterpret_cast<uint4 *>(at + kTile * 128) = make_uint4(z[0], z[1], z[2], z[3]);
        }
      }
      if (q == 0 && lse_out && g < rows) lse_out[(int64_t)g * pc.H + s] = merged_lse(m, sum);
      fence_proxy_async_smem();   // the tile is read by the MMAs
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) {
      const uint32_t idesc = idesc_bf16_f32(128, 2 * kTile, true, false), idesc_ts = idesc_bf16_f32(128, 2 * kTile, false, false);
      const uint64_t ad = smem_desc_sw128(smem_u32(wa), kWChunk / 2, 1024), bd = smem_desc_sw128(smem_u32(ol), 16, 1024);
      if (it == 0) {
        fine = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar_w), 0, kWaitNs));
        if (!fine && lane == 0) report(dev_status, MLA_ERR_TIMEOUT);
        tc_fence_after();
      }
      if (fine) {
#pragma unroll
        for (int i = 0; i < 4 * (kChunks - kWSmem); ++i)   // 16 latent dims each: 8 columns of W_UV^T
          mma_ts_warp(tmem, tmem + kWCol + 8 * i, bd + (((kWSmem + i / 4) * kOlChunk + (i & 3) * 32) >> 4), idesc_ts, i ? 1u : 0u);
#pragma unroll 1
        for (int kc = 0; kc < kWSmem; ++kc)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ss_warp(tmem, ad + ((kc * kWChunk + kk * 2048) >> 4), bd + ((kc * kOlChunk + kk * 32) >> 4), idesc, 1u);
      }
      tc_commit_warp(smem_u32(&bar_mma));   // (completes also with nothing issued)
      if (lane == 0) s_ok = fine;
    }
    if (g0 + gridDim.y * kR < rows) look_up(g0 + gridDim.y * kR);
    const bool done = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar_mma), it & 1, kWaitNs));
    if (!done && lane == 0) report(dev_status, MLA_ERR_TIMEOUT);
    tc_fence_after();
    // Warp w drains output dims 32 (w & 3) .. of rows 32 (w >> 2) .., the sum of both products, to a [64 x 128] bf16
    // staging tile over the operand.
    __nv_bfloat16 *stg = reinterpret_cast<__nv_bfloat16 *>(ol);
    constexpr int lds = kDv + 8;
    {
      uint32_t v[32], z[32];
      const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 32 * (warp >> 2);
      tmem_ld32(at, v);
      tmem_ld32(at + kTile, z);
      tmem_wait_ld();
      __syncthreads();   // the MMAs are complete: the operand may be overwritten
#pragma unroll
      for (int i = 0; i < 32; ++i)
        stg[(32 * (warp >> 2) + i) * lds + (warp & 3) * 32 + lane] =
            __float2bfloat16_rn(__uint_as_float(v[i]) + __uint_as_float(z[i]));
    }
    tc_fence_before();
    __syncthreads();
    if (done && s_ok)
      for (int c = tid; c < kR * (kDv / 8); c += kThreads) {
        const int rr = c >> 4, q8 = c & 15, g = g0 + rr;
        if (g < rows)
          *reinterpret_cast<uint4 *>(out + ((int64_t)g * pc.H + s) * kDv + q8 * 8) =
              *reinterpret_cast<const uint4 *>(stg + rr * lds + q8 * 8);
      }
    __syncthreads();   // the staged rows have left before the next merge
    tc_fence_after();
  }
  if (warp == 0) {
    // Copies in flight (none unless the wait gave up, or the CTA had no rows) land before the shared memory goes away.
    if (lane == 0 && (!fine || it == 0)) mbar_wait(smem_u32(&bar_w), 0, kWaitNs);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Without W_UV: one warp per (query row, head), the merged row rounded once.
__global__ void __launch_bounds__(kThreads)
shared_merge_kernel(const Pieces pc, int rows, __nv_bfloat16 *o_lat, float *lse_out) {
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (item >= (int64_t)rows * pc.H) return;
  const PieceRows pr = piece_rows(pc, (int)(item / pc.H), (int)(item % pc.H));
  float m, sum, acc[2][8];
  weigh(pc, pr, m, sum);
  merge_blocks<2, 4>(pc, pr, m, sum > 0.f ? 1.f / sum : 0.f, [&](int i) { return 32 * i + lane; }, acc);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = pack_bf16x2(acc[i][2 * e], acc[i][2 * e + 1]);
    *reinterpret_cast<uint4 *>(o_lat + item * kDc + 8 * (32 * i + lane)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (lane == 0 && lse_out) lse_out[item] = merged_lse(m, sum);
}

template <int kTpr>
int launch_as(const CUtensorMap &mw, const void *w_uv, int sms, int rows, const Pieces &pc, void *out, float *lse, int *dev_status,
              cudaStream_t st) {
  static std::atomic<int> smem_set[kSmemCacheDevs];
  if (smem_limit(shared_combine_kernel<kTpr>, kSmem, smem_set) != cudaSuccess) return MLA_ERR_CUDA;
  constexpr int kR = kThreads / kTpr;
  const int tiles = (rows + kR - 1) / kR, per = sms / pc.H > 1 ? sms / pc.H : 1;
  return launch_pdl(shared_combine_kernel<kTpr>, dim3(pc.H, tiles < per ? tiles : per), dim3(kThreads), kSmem, st, mw,
                    static_cast<const __nv_bfloat16 *>(w_uv), pc, rows, lse, static_cast<__nv_bfloat16 *>(out), dev_status) == cudaSuccess
             ? MLA_OK
             : MLA_ERR_CUDA;
}

}  // namespace

int launch_shared_combine(const mla_dims &d, int B, int n_q, const SharedPlan &pl, const float *o_part,
                          const float *lse_part, const void *w_uv, void *out, float *lse, int *dev_status,
                          cudaStream_t st) {
  const int rows = B * n_q, H = d.n_heads;
  const Pieces pc{o_part, lse_part, pl.unit_parts, pl.seq_group, n_q, H, shared_unit_rows(n_q * H)};
  if (!w_uv) {
    const int64_t warps = (int64_t)rows * H;
    const dim3 grid((unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32)));
    return launch_pdl(shared_merge_kernel, grid, dim3(kThreads), 0, st, pc, rows, static_cast<__nv_bfloat16 *>(out), lse) ==
                   cudaSuccess
               ? MLA_OK
               : MLA_ERR_CUDA;
  }
  // W_UV as [H * 512 rows][128] (boxes of 64 rows x 64 columns).
  CUtensorMap mw;
  if (!make_tmap_bf16(&mw, w_uv, kDv, (uint64_t)H * kDc, (uint64_t)kDv * 2, 64)) return MLA_ERR_CUDA;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MLA_ERR_CUDA;
  auto fits = [&](int r) { return (int64_t)H * ((rows + r - 1) / r) <= sms; };
  if (fits(8)) return launch_as<32>(mw, w_uv, sms, rows, pc, out, lse, dev_status, st);
  if (fits(16)) return launch_as<16>(mw, w_uv, sms, rows, pc, out, lse, dev_status, st);
  if (fits(32)) return launch_as<8>(mw, w_uv, sms, rows, pc, out, lse, dev_status, st);
  return launch_as<4>(mw, w_uv, sms, rows, pc, out, lse, dev_status, st);
}

}  // namespace mla
