// linear_split.cu -- tidar_linear_fused for few rows: y = act(x w^T + bias) +
// residual with the reduction split over a thread-block cluster.
//
// With rows in the tens to hundreds the weights are streamed once and what
// bounds the product is how fast they, and the rows that every feature tile
// reads again, come out of HBM and L2.  So the weights are the MMA's A operand
// (256 features over a pair of SMs, tcgen05 cta_group::2), the rows its B operand
// (N = the tile's rows, up to 384 in two MMAs; each SM of the pair holds half of
// them: the rows are read once per 256 features), and the reduction is cut into
// ks ranges, one pair each, to fill the device.  The 2 ks CTAs of a tile are one
// cluster: each leaves its partial sums (fp32, 128 features x the rows) in its own
// shared memory, and CTA (split, half) adds the splits' sums of its share of the
// rows over distributed shared memory, in split order, and writes them with the
// epilogue applied.  No workspace, no second launch, and the sums do not depend
// on timing.
//
// Twelve warps: 0 TMA producer, 1 MMA issuer (the pair's first CTA) and TMEM owner,
// 2..5 move the accumulator from TMEM (lane = feature, column = row) to shared
// memory; all twelve reduce, with up to 16 of their peers' rows in flight a warp (six
// warps with four in flight took 7 us over 136 rows of two splits).  Rows, features
// and the reduction may end anywhere (TMA reads zeros outside).
//
// 272 x 4096 x 4096 with a residual: 16.9 us (0.54 PFLOP/s, 2.4 TB/s; the paired tiles
// of linear_pair.cu 27); 1 x 16384 x 4096: 28.4 us, 4.7 TB/s; 77 x 1000 x 1544: 7.7 to 11 us,
// of which about 7 pass before the first product and after the last (launch,
// cluster, TMEM, the first loads; the exchange of the partial sums).
//
// Every wait is bounded (~1 s): on expiry the CTA records TIDAR_DEVERR_TIMEOUT,
// marks its partial sums invalid (nothing of the tile is written) and still
// meets its cluster at the barriers.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "linear_act.cuh"
#include "pair.cuh"
#include "sm100.cuh"
#include "tc05.cuh"

namespace tidar {

namespace {

constexpr int kThreads = 384;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxStages = 12;
constexpr int kMaxRows = 384;                           // rows of a tile (TMEM columns, shared memory)
constexpr int kMaxSplit = 8;                            // cluster of 16 CTAs
constexpr uint32_t kABytes = 128u * 128u;               // 128 features x 64 bf16
constexpr uint32_t kSmemMax = 225u * 1024u;
constexpr int BAR_FULL = 0;                             // + stage (the pair's first CTA's)
constexpr int BAR_EMPTY = kMaxStages;                   // + stage (each CTA's own)
constexpr int BAR_DONE = 2 * kMaxStages;
constexpr int kNumBars = 2 * kMaxStages + 1;
constexpr uint32_t kTail = kNumBars * 8 + 16;           // barriers, then [0] TMEM base, [1] abort, [2] valid

struct SplitParams {
  int T, K, N;
  int nt, n0, n1;     // rows of a tile, of its first and second MMA (multiples of 32; n1 may be 0)
  int ft;             // feature tiles of 256
  int kb, ks, stages;
  uint32_t stage_bytes;
  const __nv_bfloat16* bias;
  const __nv_bfloat16* residual;
  __nv_bfloat16* y;
  int act;
  unsigned int* err;
};

__device__ __forceinline__ float4 ld_shared_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t idesc(int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((256u >> 4) << 24);
}

// Rows [lo, hi) of the tile at t0, features f0 .. f0+3 of this lane: the sum of up
// to KS splits' partial sums (in split order) and the epilogue.  One warp per row,
// the peers' values of 16 / KS rows in flight before the first is used.
template <int KS>
__device__ __forceinline__ void reduce_rows(const SplitParams& prm, uint32_t sb, int half, int f0, int t0, int lo, int hi,
                                            int warp, int lane) {
  constexpr int U = 16 / KS > 4 ? 4 : 16 / KS;
  const bool vec = prm.N % 4 == 0;                         // rows 8-byte aligned: one access each
  float b4[4] = {0.f, 0.f, 0.f, 0.f};
  if (prm.bias) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (f0 + e < prm.N) b4[e] = __bfloat162float(prm.bias[f0 + e]);
  }
  uint32_t peer[KS];
#pragma unroll
  for (int q = 0; q < KS; ++q) peer[q] = mapa(sb + 16u * (uint32_t)lane, (uint32_t)(2 * min(q, prm.ks - 1) + half));
  for (int tb = lo + warp; tb < hi; tb += kWarps * U) {
    float4 v[U][KS];
    uint2 res[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = tb + kWarps * u;
      if (t < hi) {
#pragma unroll
        for (int q = 0; q < KS; ++q)
          if (q < prm.ks) v[u][q] = KS == 1 ? ld_shared_f32x4(sb + 16u * (uint32_t)lane + 512u * (uint32_t)t)
                                            : ld_cluster_f32x4(peer[q] + 512u * (uint32_t)t);
        if (prm.residual && vec) res[u] = *reinterpret_cast<const uint2*>(prm.residual + (size_t)(t0 + t) * prm.N + f0);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = tb + kWarps * u;
      if (t >= hi) break;
      float o[4] = {v[u][0].x, v[u][0].y, v[u][0].z, v[u][0].w};
#pragma unroll
      for (int q = 1; q < KS; ++q)
        if (q < prm.ks) o[0] += v[u][q].x, o[1] += v[u][q].y, o[2] += v[u][q].z, o[3] += v[u][q].w;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] += b4[e];
      if (prm.act != TIDAR_ACT_NONE) {
        const float4 r = lin_act4(make_float4(o[0], o[1], o[2], o[3]), prm.act);
        o[0] = r.x; o[1] = r.y; o[2] = r.z; o[3] = r.w;
      }
      __nv_bfloat16* y = prm.y + (size_t)(t0 + t) * prm.N + f0;
      if (vec) {
        if (prm.residual) {
          const float2 r0 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&res[u].x));
          const float2 r1 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&res[u].y));
          o[0] += r0.x; o[1] += r0.y; o[2] += r1.x; o[3] += r1.y;
        }
        *reinterpret_cast<uint2*>(y) = make_uint2(tc05::cvt_bf16x2(o[0], o[1]), tc05::cvt_bf16x2(o[2], o[3]));
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (f0 + e < prm.N)
            y[e] = __float2bfloat16_rn(o[e] + (prm.residual ? __bfloat162float(prm.residual[(size_t)(t0 + t) * prm.N + f0 + e]) : 0.f));
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1)
linear_split_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x0,
                    const __grid_constant__ CUtensorMap tm_x1, const SplitParams prm) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int split = (int)rank >> 1, half = (int)rank & 1;
  const uint32_t lead = rank & ~1u;
  const int tile = blockIdx.y, ft = tile % prm.ft, tt = tile / prm.ft;
  const int t0 = tt * prm.nt, nvalid = min(prm.nt, prm.T - t0);
  const int kb0 = (int)((long long)split * prm.kb / prm.ks), nkb = (int)((long long)(split + 1) * prm.kb / prm.ks) - kb0;
  const uint32_t ring = (uint32_t)prm.stages * prm.stage_bytes;
  auto bar = [&](int i) -> uint32_t { return sb + ring + 8u * i; };
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + ring + 8u * kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  if (sb & 1023u) {                // the same window in every CTA of the cluster: they leave together
    if (threadIdx.x == 0) raise_error(prm.err, TIDAR_DEVERR_LAYOUT);
    return;
  }
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < kNumBars; ++i) mbar_init(bar(i), 1u);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    prefetch_tmap(&tm_w);
    prefetch_tmap(&tm_x0);
    prefetch_tmap(&tm_x1);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sb + ring + 8u * kNumBars), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc05::fence_before();
  __syncthreads();
  cluster_sync_all();              // the cluster's barriers are ready
  tc05::fence_after();
  const uint32_t tmem = misc[0];

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    pdl_wait();
    pdl_trigger();
    if (lane == 0) {
      const int f0 = ft * 256 + half * 128;
      const uint32_t full0 = mapa(bar(BAR_FULL), lead);
      // ring position and phase are carried, not divided out: this one thread's
      // instructions are what a slice costs when few rows make its bytes few
      const int x0 = t0 + half * (prm.n0 / 2), x1 = t0 + prm.n0 + half * (prm.n1 / 2);
      const uint32_t off1 = kABytes + (uint32_t)prm.n0 * 64u, tx = 2u * prm.stage_bytes;
      const bool two = prm.n1 > 0;
      uint32_t dst = sb, off = 0, phase = 1;               // phase 1: the first round's stages are free
      int s = 0, issued = 0;
      for (int k = kb0 * 64; issued < nkb; k += 64) {
        if (!wait_bar(bar(BAR_EMPTY) + off, phase, abort_flag, prm.err)) break;
        if (half == 0) mbar_expect_tx(bar(BAR_FULL) + off, tx);
        tma_load_pair(dst, &tm_w, k, f0, full0 + off);
        tma_load_pair(dst + kABytes, &tm_x0, k, x0, full0 + off);
        if (two) tma_load_pair(dst + off1, &tm_x1, k, x1, full0 + off);
        ++issued;
        dst += prm.stage_bytes;
        off += 8;
        if (++s == prm.stages) s = 0, dst = sb, off = 0, phase ^= 1u;
      }
      // drain: the first CTA's barriers count the copies of both
      if (half == 0 && *abort_flag)
        for (int i = max(0, issued - prm.stages); i < issued; ++i)
          wait_quiet(bar(BAR_FULL + i % prm.stages), (uint32_t)((i / prm.stages) & 1));
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    pdl_wait();
    pdl_trigger();
    if (lane == 0 && half == 0) {
      const uint16_t pair = (uint16_t)(3u << lead);
      const uint32_t id0 = idesc(prm.n0), id1 = idesc(prm.n1);
      const bool two = prm.n1 > 0;
      const uint64_t a0 = tc05::desc_k_sw128(sb), step = prm.stage_bytes >> 4, b_off = kABytes >> 4,
                     c_off = (kABytes + (uint32_t)prm.n0 * 64u) >> 4;
      uint64_t a = a0;
      uint32_t off = 0, phase = 0;
      int s = 0;
      for (int i = 0; i < nkb; ++i) {
        if (!wait_bar(bar(BAR_FULL) + off, phase, abort_flag, prm.err)) break;
        tc05::fence_after();
        mma_pair_x4(tmem, a, a + b_off, id0, (uint32_t)i);
        if (two) mma_pair_x4(tmem + (uint32_t)prm.n0, a, a + c_off, id1, (uint32_t)i);
        commit_pair(bar(BAR_EMPTY) + off, pair);
        a += step;
        off += 8;
        if (++s == prm.stages) s = 0, a = a0, off = 0, phase ^= 1u;
      }
      commit_pair(bar(BAR_DONE), pair);   // every MMA issued above is complete
    }
    __syncwarp();
  } else if (warp < 6) {
    // ---------------------------------------------------------------- TMEM -> shared memory
    pdl_wait();
    pdl_trigger();
    const int q4 = warp & 3, f = 32 * q4 + lane;
    if (warp_wait_bar(bar(BAR_DONE), 0, abort_flag, prm.err)) {
      tc05::fence_after();
      float* part = reinterpret_cast<float*>(smem);       // [row][128 features]: the ring is idle
      const uint32_t src = tmem + ((uint32_t)(32 * q4) << 16);
      for (int c = 0; c < nvalid; c += 32) {
        uint32_t r[32];
        tc05::tmem_ld32(src + (uint32_t)c, r);
        tc05::tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (c + e < nvalid) part[(c + e) * 128 + f] = __uint_as_float(r[e]);
      }
    }
  } else {
    pdl_wait();
    pdl_trigger();
  }
  tc05::fence_before();
  __syncthreads();
  if (threadIdx.x == 0) misc[2] = *abort_flag ? 0u : 1u;
  cluster_sync_all();              // every CTA's partial sums and status are in place

  // ------------------------------------------------------------------ reduce + write
  // CTA (split, half): rows [split per, + per) of the tile.
  const int ks = prm.ks, per = (nvalid + ks - 1) / ks;
  const int lo = split * per, hi = min(nvalid, lo + per);
  bool valid = true;
#pragma unroll 4
  for (int r = 0; r < 2 * ks; ++r) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(mapa(sb + ring + 8u * kNumBars + 8u, (uint32_t)r)) : "memory");
    valid = valid && v != 0;
  }
  const int f0 = ft * 256 + half * 128 + 4 * lane;
  if (valid && f0 < prm.N) {
    if (ks == 1) reduce_rows<1>(prm, sb, half, f0, t0, lo, hi, warp, lane);
    else if (ks == 2) reduce_rows<2>(prm, sb, half, f0, t0, lo, hi, warp, lane);
    else if (ks <= 4) reduce_rows<4>(prm, sb, half, f0, t0, lo, hi, warp, lane);
    else reduce_rows<8>(prm, sb, half, f0, t0, lo, hi, warp, lane);
  }
  tc05::fence_before();
  __syncthreads();
  cluster_sync_all();              // no peer reads this CTA's shared memory any more
  if (warp == 1) {
    tc05::fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

cudaError_t smem_attr() {
  static bool set[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorNotSupported;
  if (!set[dev]) {
    e = cudaFuncSetAttribute(linear_split_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMax);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(linear_split_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    set[dev] = true;
  }
  return cudaSuccess;
}

// Clusters of 2 ks CTAs that this device holds at once (every plan takes the
// same shared memory); cached per device.  Without a device: 148 SMs.
int resident(int ks) {
  static int cache[64][kMaxSplit + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) { cudaGetLastError(); return 74 / ks; }
  if (cache[dev][ks]) return cache[dev][ks] - 1;
  int n = 0;
  if (smem_attr() == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * ks, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmemMax;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2 * ks;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, linear_split_kernel, &cfg) != cudaSuccess) n = 0;
  }
  cudaGetLastError();
  cache[dev][ks] = n + 1;
  return n;
}

}  // namespace

LinearSplitPlan plan_linear_split(int T, int K, int N) {
  LinearSplitPlan p{};
  if (T <= 0 || K <= 0 || N <= 0) return p;
  p.ft = (N + 255) / 256;
  const int kb = (K + 63) / 64, least = (T + kMaxRows - 1) / kMaxRows;
  // Row tiles and splits by an estimate in clocks, fitted to measurements: waves of
  // clusters times (the slices of one split at 250 + bytes / 90, a quarter more when
  // the device is full and L2 is shared, + 6000 a CTA, + 55
  // a row that it reduces, + 3000 a further split), and no less than the weights
  // take from HBM.  More row tiles than needed read the weights again, from L2.
  // 272 x 4096 x 4096, row tiles / splits: 1/1 34.0, 1/2 21.9, 1/3 19.3, 1/4 31.2
  // (its clusters of eight take two waves), 2/1 26.1, 2/2 17.3, 2/3 27.4 us.
  double best = 1e300;
  for (int tt = least; tt <= least + 2 && tt <= T; ++tt) {
    const int nt = ((T + tt - 1) / tt + 31) / 32 * 32;
    const uint32_t bytes = kABytes + (uint32_t)nt * 64u;
    const long long tiles = (long long)p.ft * tt;
    for (int ks = 1; ks <= kMaxSplit && ks <= kb; ++ks) {
      const int r = resident(ks);
      if (r <= 0) continue;
      const double waves = (double)((tiles + r - 1) / r);
      const double slice = (250.0 + bytes / 90.0) * (tiles * ks >= 66 ? 1.25 : 1.0);
      const double busy = waves * ((double)((kb + ks - 1) / ks) * slice + 6000.0 + 55.0 * nt / ks + 3000.0 * (ks - 1));
      const double cost = std::max(busy, 5000.0 + (double)N * K * 2.0 / 3000.0);
      if (cost < best - 1e-9) best = cost, p.ks = ks, p.tt = tt, p.nt = nt, p.stage_bytes = bytes;
    }
  }
  p.n0 = p.nt <= 256 ? p.nt : (p.nt / 2 + 31) / 32 * 32;
  p.n1 = p.nt - p.n0;
  p.tt = p.nt ? (T + p.nt - 1) / p.nt : 0;               // rounding may leave the last tile empty
  p.stages = p.stage_bytes ? std::min<int>(kMaxStages, (int)((kSmemMax - kTail) / p.stage_bytes)) : 0;
  p.cost = best;
  p.ok = p.ks > 0 && (long long)p.ft * p.tt <= 65535;
  return p;
}

cudaError_t launch_linear_split(const LinearArgs& a, cudaStream_t s) {
  const LinearSplitPlan p = plan_linear_split(a.T, a.K, a.N);
  if (!p.ok) return cudaErrorNotSupported;
  SplitParams prm{};
  prm.T = a.T; prm.K = a.K; prm.N = a.N;
  prm.nt = p.nt; prm.n0 = p.n0; prm.n1 = p.n1; prm.ft = p.ft;
  prm.kb = (a.K + 63) / 64; prm.ks = p.ks; prm.stages = p.stages; prm.stage_bytes = p.stage_bytes;
  prm.bias = static_cast<const __nv_bfloat16*>(a.bias);
  prm.residual = static_cast<const __nv_bfloat16*>(a.residual);
  prm.y = static_cast<__nv_bfloat16*>(a.y);
  prm.act = a.act;
  prm.err = a.err;
  CUtensorMap tw, tx0, tx1;
  const cuuint64_t str[1] = {(cuuint64_t)a.K * 2};
  const cuuint64_t dx[2] = {(cuuint64_t)a.K, (cuuint64_t)a.T}, dw[2] = {(cuuint64_t)a.K, (cuuint64_t)a.N};
  const cuuint32_t bw[2] = {64, 128}, b0[2] = {64, (cuuint32_t)p.n0 / 2}, b1[2] = {64, (cuuint32_t)(p.n1 ? p.n1 : p.n0) / 2};
  if (!encode(&tw, a.w, 2, dw, str, bw) || !encode(&tx0, a.x, 2, dx, str, b0) || !encode(&tx1, a.x, 2, dx, str, b1))
    return cudaErrorNotSupported;
  cudaError_t e = smem_attr();
  if (e != cudaSuccess) return e;
  return launch_clustered(linear_split_kernel, dim3(2 * p.ks, p.ft * p.tt), dim3(2 * p.ks, 1, 1), kThreads, kSmemMax, s, tw, tx0,
                          tx1, prm);
}

}  // namespace tidar
