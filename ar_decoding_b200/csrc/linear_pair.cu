// linear_pair.cu -- tidar_linear_fused for many rows: y = act(x w^T + bias) +
// residual on pairs of SMs (tcgen05 cta_group::2).
//
// With rows in the thousands the product is bound by the tensor cores, and what
// has to be kept off their back is shared-memory traffic: a 128 x 256 tile on
// one SM reads 48 KB per 64-deep slice for 512 clocks of MMA, more than L2 gives
// 148 SMs at once.  Two SMs sharing a 256 x 256 tile read 32 KB each: every CTA
// holds 128 of the tile's rows of x (A) and 128 of its 256 features of w (B), and
// one MMA of M = 256, N = 256, issued by the first CTA of the pair, reads both
// shared memories and leaves each CTA the accumulator of its own 128 rows (TMEM
// lane = row, column = feature).
//
// Persistent clusters of two CTAs, tiles in groups of eight row tiles (rows
// fastest, so the weights of a feature tile are read from HBM once and its rows
// stay in L2).  Eighteen warps: 0 TMA producer (each CTA loads its own halves and
// counts them on the first CTA's barrier), 1 MMA issuer and TMEM owner, 2..17
// epilogue (a lane quarter and a quarter of the columns each).  Two accumulators of
// 256 columns alternate, so the epilogue of a tile (a thread owns a row: 64
// contiguous bytes a store group) runs under the MMAs of the next.  Rows, features
// and the reduction may end anywhere: TMA reads zeros outside, stores are guarded.
//
// 2048 x 16384 x 4096, bias and tanh GELU: 191 to 201 us in a burst, 1.44 PFLOP/s (0.87 of
// a library product's; 226 to 233 us and 1.2 PFLOP/s in a loop of seconds under the
// power cap, where the library's product alone takes 215).  Without its loads the
// loop takes 167 us: what is left is the 32 KB a slice and SM that come out of L2.
// Tiles of 128 x 256 on single SMs took 454 us.  Eight epilogue warps: 1024 x 4096 x
// 4096 34.6 us, sixteen 32.6.
//
// Every wait is bounded (~1 s): on expiry the CTA records TIDAR_DEVERR_TIMEOUT and
// stops; its peer's waits run out in turn, the first CTA drains the copies of
// both, and the pair meets at the final cluster barrier.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "linear_act.cuh"
#include "pair.cuh"
#include "sm100.cuh"
#include "tc05.cuh"

namespace tidar {

namespace {

constexpr int kEpWarps = 16;
constexpr int kThreads = 32 * (2 + kEpWarps);
constexpr int kTile = 256;                              // rows and features of a pair's tile
constexpr int kStages = 6;
constexpr uint32_t kHalf = 128u * 128u;                 // 128 rows x 64 bf16
constexpr uint32_t kStage = 2 * kHalf;                  // A half, B half
constexpr uint32_t kOffBar = kStages * kStage;
constexpr int BAR_FULL = 0;                             // + stage (the first CTA's are used)
constexpr int BAR_EMPTY = kStages;                      // + stage (each CTA's own)
constexpr int BAR_ACC = 2 * kStages;                    // + buffer: accumulator complete
constexpr int BAR_FREE = 2 * kStages + 2;               // + buffer: accumulator read (the first CTA's)
constexpr int kNumBars = 2 * kStages + 4;
constexpr uint32_t kOffMisc = kOffBar + kNumBars * 8;   // [0] TMEM base, [1] abort flag
// rows that are not 16-byte aligned are written through shared memory: 32 x 32
// values an epilogue warp in two halves, the rows one float apart in banks
constexpr uint32_t kOffTile = kOffMisc + 16;
constexpr uint32_t kSmem = kOffTile + kEpWarps * 32 * 17 * 4;
static_assert(kSmem <= 232448, "shared memory budget");
constexpr int kRowGroup = 8;                            // row tiles that share a sweep over the features

struct PairParams {
  int T, K, N;
  int mt, nt;         // row tiles, feature tiles
  int kb;             // 64-deep slices
  const __nv_bfloat16* bias;
  const __nv_bfloat16* residual;
  __nv_bfloat16* y;
  int act;
  int vec;            // N % 8 == 0: rows of y and residual are 16-byte aligned
  unsigned int* err;
};

constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | ((256u >> 3) << 17) | ((256u >> 4) << 24);

// Tile number -> (row tile, feature tile): groups of kRowGroup row tiles, the
// features in turn, the group's row tiles fastest.
__device__ __forceinline__ void tile_of(const PairParams& p, int tile, int& rt, int& ft) {
  const int per = kRowGroup * p.nt, grp = tile / per, in = tile - grp * per;
  const int rows = min(kRowGroup, p.mt - grp * kRowGroup);
  ft = in / rows;
  rt = grp * kRowGroup + in - ft * rows;
}

__global__ void __launch_bounds__(kThreads, 1)
linear_pair_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                   const PairParams prm) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1, tiles = prm.mt * prm.nt;
  auto bar = [&](int i) -> uint32_t { return sb + kOffBar + 8u * i; };
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  // both CTAs of the pair see the same window alignment, so they leave together
  if (sb & 1023u) {
    if (threadIdx.x == 0) raise_error(prm.err, TIDAR_DEVERR_LAYOUT);
    return;
  }
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < kNumBars; ++i) mbar_init(bar(i), i >= BAR_FREE ? 2u * kEpWarps : 1u);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    prefetch_tmap(&tm_x);
    prefetch_tmap(&tm_w);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sb + kOffMisc), "r"(512u) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc05::fence_before();
  __syncthreads();
  cluster_sync_all();              // both CTAs' barriers are ready
  tc05::fence_after();
  const uint32_t tmem = misc[0];
  pdl_wait();
  pdl_trigger();

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    if (lane == 0) {
      int it = 0, s = 0;           // slices issued, ring position
      uint32_t phase = 1;          // 1: the first round's stages are free
      bool ok = true;
      const uint32_t full0 = mapa(bar(BAR_FULL), 0);
      for (int tile = cluster; ok && tile < tiles; tile += clusters) {
        int rt, ft;
        tile_of(prm, tile, rt, ft);
        const int r0 = rt * kTile + (int)rank * 128, f0 = ft * kTile + (int)rank * 128;
        for (int k = 0; k < prm.kb; ++k, ++it) {
          ok = wait_bar(bar(BAR_EMPTY + s), phase, abort_flag, prm.err);
          if (!ok) break;
          if (rank == 0) mbar_expect_tx(bar(BAR_FULL + s), 2u * kStage);
          const uint32_t full = full0 + 8u * s, dst = sb + (uint32_t)s * kStage;
          tma_load_pair(dst, &tm_x, k * 64, r0, full);
          tma_load_pair(dst + kHalf, &tm_w, k * 64, f0, full);
          if (++s == kStages) s = 0, phase ^= 1u;
        }
      }
      // drain: the first CTA's barriers count the copies of both
      if (rank == 0 && *abort_flag)
        for (int i = max(0, it - kStages); i < it; ++i) wait_quiet(bar(BAR_FULL + i % kStages), (uint32_t)((i / kStages) & 1));
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0 && rank == 0) {
      int s = 0, n = 0;            // ring position, tiles done
      uint32_t phase = 0;
      bool ok = true;
      const uint64_t a0 = tc05::desc_k_sw128(sb);
      for (int tile = cluster; ok && tile < tiles; tile += clusters, ++n) {
        const int buf = n & 1;
        if (n >= 2) ok = wait_bar(bar(BAR_FREE + buf), (uint32_t)((n / 2 - 1) & 1), abort_flag, prm.err);
        if (!ok) break;
        tc05::fence_after();
        const uint32_t d = tmem + (uint32_t)(buf * kTile);
        for (int k = 0; k < prm.kb; ++k) {
          ok = wait_bar(bar(BAR_FULL + s), phase, abort_flag, prm.err);
          if (!ok) break;
          tc05::fence_after();
          const uint64_t a = a0 + (uint64_t)s * (kStage >> 4);
          mma_pair_x4(d, a, a + (kHalf >> 4), kIdesc, (uint32_t)k);
          commit_pair(bar(BAR_EMPTY + s), (uint16_t)3);
          if (++s == kStages) s = 0, phase ^= 1u;
        }
        if (ok) commit_pair(bar(BAR_ACC + buf), (uint16_t)3);
      }
    }
    __syncwarp();                  // this warp releases the tensor memory below, together
  } else {
    // ---------------------------------------------------------------- epilogue
    const int q4 = warp & 3;       // TMEM lane quarter
    constexpr int kCols = kTile / (kEpWarps / 4);
    const int c0 = ((warp - 2) >> 2) * kCols, c1 = c0 + kCols;     // and its share of the columns
    int n = 0;
    for (int tile = cluster; tile < tiles; tile += clusters, ++n) {
      const int buf = n & 1;
      if (!warp_wait_bar(bar(BAR_ACC + buf), (uint32_t)((n / 2) & 1), abort_flag, prm.err)) break;
      tc05::fence_after();
      int rt, ft;
      tile_of(prm, tile, rt, ft);
      const int row = rt * kTile + (int)rank * 128 + 32 * q4 + lane, f0 = ft * kTile;
      const uint32_t src = tmem + ((uint32_t)(32 * q4) << 16) + (uint32_t)(buf * kTile);
      const size_t at = (size_t)row * prm.N + f0;
#pragma unroll 1
      for (int c = c0; c < c1; c += 32) {
        uint32_t acc[32];
        // the stores of the 32 columns before this may have parted the warp (rows past
        // T, features past N), and the load wants it whole
        __syncwarp();
        tc05::tmem_ld32(src + (uint32_t)c, acc);
        tc05::tmem_wait_ld();
        if (c + 32 == c1) {        // this share of the accumulator has been read: the next tile may overwrite it
          tc05::fence_before();
          __syncwarp();
          if (lane == 0) arrive_cluster(mapa(bar(BAR_FREE + buf), 0));
        }
        if (f0 + c >= prm.N) continue;                     // warp-uniform
        if (prm.vec && f0 + c + 32 <= prm.N) {
          if (row < prm.T) {
            __nv_bfloat16* dst = prm.y + at + c;
            const __nv_bfloat16* res = prm.residual ? prm.residual + at + c : nullptr;
            // one copy of the 32 values' code per activation, chosen once
            auto write = [&](auto act) {
#pragma unroll
              for (int e = 0; e < 32; e += 8) {
                float b8[8], r8[8], v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) b8[i] = r8[i] = 0.f;
                if (prm.bias) load_vec<__nv_bfloat16, 8>(prm.bias + f0 + c + e, b8);
                if (res) load_vec<__nv_bfloat16, 8>(res + e, r8);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = lin_act(__uint_as_float(acc[e + i]) + b8[i], decltype(act)::value) + r8[i];
                *reinterpret_cast<uint4*>(dst + e) = make_uint4(tc05::cvt_bf16x2(v[0], v[1]), tc05::cvt_bf16x2(v[2], v[3]),
                                                                tc05::cvt_bf16x2(v[4], v[5]), tc05::cvt_bf16x2(v[6], v[7]));
              }
            };
            switch (prm.act) {
              case TIDAR_ACT_RELU: write(std::integral_constant<int, TIDAR_ACT_RELU>{}); break;
              case TIDAR_ACT_GELU: write(std::integral_constant<int, TIDAR_ACT_GELU>{}); break;
              case TIDAR_ACT_GELU_TANH: write(std::integral_constant<int, TIDAR_ACT_GELU_TANH>{}); break;
              case TIDAR_ACT_SILU: write(std::integral_constant<int, TIDAR_ACT_SILU>{}); break;
              default: write(std::integral_constant<int, TIDAR_ACT_NONE>{});
            }
          }
        } else {
          // a feature a lane, two rows an instruction: 32 contiguous bytes each (a
          // row a thread took 48 us for 1111 x 2049 x 200)
          float* st = reinterpret_cast<float*>(smem + kOffTile) + (warp - 2) * (32 * 17);
          const int rows = min(32, prm.T - (row - lane));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 16; ++e) st[lane * 17 + e] = __uint_as_float(acc[16 * h + e]);
            __syncwarp();
            const int f = f0 + c + 16 * h + (lane & 15);
            if (f < prm.N) {
              const float bias = prm.bias ? __bfloat162float(prm.bias[f]) : 0.f;
              const size_t first = (size_t)(row - lane) * prm.N + f;
#pragma unroll 4
              for (int r = lane >> 4; r < rows; r += 2) {
                const size_t o = first + (size_t)r * prm.N;
                const float v = lin_act(st[r * 17 + (lane & 15)] + bias, prm.act);
                prm.y[o] = __float2bfloat16_rn(v + (prm.residual ? __bfloat162float(prm.residual[o]) : 0.f));
              }
            }
          }
        }
      }
    }
  }
  // No MMA, copy or remote arrival is left when a CTA of the pair exits.  (The producer's
  // warp comes here in two parts; a __syncwarp behind its loop costs 1 % of the large
  // products.)
  tc05::fence_before();
  __syncthreads();
  cluster_sync_apart();
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
    e = cudaFuncSetAttribute(linear_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    set[dev] = true;
  }
  return cudaSuccess;
}

// Pairs this device holds at once (148 SMs: 74); cached per device.
int resident_pairs() {
  static int cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) { cudaGetLastError(); return 0; }
  if (cache[dev]) return cache[dev] - 1;
  int n = 0;
  if (smem_attr() == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, linear_pair_kernel, &cfg) != cudaSuccess) n = 0;
  }
  cudaGetLastError();
  cache[dev] = n + 1;
  return n;
}

}  // namespace

// Clocks that the product takes here, fitted to measurements: waves of tiles times
// their slices (590 clocks each while a few tiles run, 760 when the device is full
// and L2 is shared) + launch, pipeline fill and the last tile's epilogue (longer for
// rows that are not 16-byte aligned).
double linear_pair_cost(int T, int K, int N) {
  const long long tiles = (long long)((T + kTile - 1) / kTile) * ((N + kTile - 1) / kTile);
  const int r = resident_pairs();
  if (r <= 0 || tiles > 0x3fffffffLL) return 1e300;
  return (double)((tiles + r - 1) / r) * ((K + 63) / 64) * (tiles >= 56 ? 760.0 : 590.0) + (N % 8 ? 30000.0 : 16000.0);
}

cudaError_t launch_linear_pair(const LinearArgs& a, cudaStream_t s) {
  PairParams prm{};
  prm.T = a.T; prm.K = a.K; prm.N = a.N;
  prm.mt = (a.T + kTile - 1) / kTile;
  prm.nt = (a.N + kTile - 1) / kTile;
  prm.kb = (a.K + 63) / 64;
  prm.bias = static_cast<const __nv_bfloat16*>(a.bias);
  prm.residual = static_cast<const __nv_bfloat16*>(a.residual);
  prm.y = static_cast<__nv_bfloat16*>(a.y);
  prm.act = a.act;
  prm.vec = a.N % 8 == 0;
  prm.err = a.err;
  CUtensorMap tx, tw;
  const cuuint64_t str[1] = {(cuuint64_t)a.K * 2};
  const cuuint32_t box[2] = {64, 128};
  const cuuint64_t dx[2] = {(cuuint64_t)a.K, (cuuint64_t)a.T}, dw[2] = {(cuuint64_t)a.K, (cuuint64_t)a.N};
  if (!encode(&tx, a.x, 2, dx, str, box) || !encode(&tw, a.w, 2, dw, str, box)) return cudaErrorNotSupported;
  cudaError_t e = smem_attr();
  if (e != cudaSuccess) return e;
  const int pairs = (int)std::min<long long>(resident_pairs(), (long long)prm.mt * prm.nt);
  if (pairs <= 0) return cudaErrorNotSupported;
  return launch_clustered(linear_pair_kernel, dim3(2 * pairs), dim3(2, 1, 1), kThreads, kSmem, s, tx, tw, prm);
}

}  // namespace tidar
