// attn_kv4_dec.cu -- step attention over the 4-bit cache for small query blocks
// (at most 16 packed rows per KV head, e.g. plain decode), bf16, D 128.
//
//   out = softmax(q K^T scale) V over the prefix (K, V = code * scale, kv4.cuh)
//   and the step keys (bf16, zone mask).
//
// The step is a stream of 144 bytes a key and head; at HBM's rate an SM gets a
// key every 6 clocks, so what has to be small is the instructions a key costs.
// Layout of the work: the query rows sit in the MMA N dimension and the cached
// codes in A, both straight out of shared memory in fragment order (that is
// what the page's nibble order is for), so nothing is transposed:
//   S^T (16 keys x 8 rows) = K Q^T.  A lane's 16 bytes of a key row are dims
//     32G + 8t + e of the four groups G.  A pair of codes needs one mask-and-xor
//     to become the bf16 numbers 136 + c; the offset is taken off by starting
//     the accumulator at -136 sum_{d in G} q_d.  Each group has its own
//     accumulator, multiplied by the key's scale of that group in fp32.
//   O^T (16 dims x 8 rows) += V^T P^T.  A lane's 8 bytes of a value row are dims
//     32G + 8(g/2) + g%2 + 2i; the units of two keys are byte-permuted into one
//     word per group, each pair becomes 136 + c, minus 136, times the two keys'
//     scales (exact in bf16; the sums run over the whole prefix here, so an
//     offset in the accumulator would cost its low bits).
// 32 sequences of 512 to 16384 keys, 8 KV heads, 4 or 8 rows a head: 75 to 78 us, 4.0
// TB/s (0.61 of the copy rate; the bf16 cache's kernel 164); one of 8192: 10.9 us in a
// cluster of ten splits (bf16 9.6).  9 to 16 rows a head, two query tiles, whose registers
// (255 a thread) leave eight warps: 16 rows, 4 KV heads 111 us, a third of one tile's
// bytes a second (bf16 149, the tensor-core kernel 233); 12 rows, 2 KV heads 59 (80, 121).
// No pipe is full (issue 60 %, integer 58 %, MMA 22 %; four warps a scheduler, whose
// registers allow no more): a warp's chain of shifts, products and exponentials is
// what a unit takes.  One multiply-add instead of subtract and multiply a value pair
// made it no faster (82 us), nor did multiplies for shifts (104) or 20 warps of 96
// registers (89).
// Both products are exact up to the fp32 accumulation (the scores' partial sums reach
// 143/7 of sum |q||k| by the offset, and round accordingly), so the only rounding besides
// it is p's to bf16: an MMA's operands have one type, V's values are bf16, and the bf16
// cache's step rounds p likewise (2^-8 of each p at most; p in two halves would double
// the products).  MMA row r of a 16-key block is physical key
// (r % 8) / 2 + 4 (r % 2) + 8 (r / 8): the four keys whose values a lane loads
// are then t, t+4, t+8, t+12 and the loads of a warp cover 256 contiguous bytes.
//
// Grid (split, b * Hkv).  Every warp runs its own pipeline: units of 32 keys in
// turn, two slots of shared memory filled by 16-byte asynchronous copies, no
// barrier between warps until the end.  (A producer warp with bulk or tiled
// copies of whole pages could not issue fast enough: 9 KB stages at 2.7 and 3.3
// TB/s with nothing but the copies running.)  The running maximum is only
// raised when a score passes it by 2^8, and only then do the lanes exchange
// maxima.  Warps merge in shared memory; the splits of a prefix merge on chip
// (cluster) or through workspace partials and the finalize launch.
#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"
#include "sm100.cuh"
#include "tc05.cuh"

namespace tidar {

namespace {

using tc05::kStageStride;

// NT 8-row query tiles (1: M <= 8, 2: M <= 16) and the warps that their
// registers leave room for.
template <int NT> struct Kv4Shape {
  static constexpr int kWarps = NT == 1 ? 16 : 8;
  static constexpr int kThreads = 32 * kWarps;
};
constexpr int kSlots = 2;                               // units of 32 keys per warp: one in use, one in flight
constexpr uint32_t kCodes = 32 * 64;                    // 32 keys of 128 dims
constexpr uint32_t kScales = 32 * 8;
constexpr uint32_t kUnit = 2 * (kCodes + kScales);      // K codes, V codes, K scales, V scales
template <int NT> constexpr uint32_t ring_bytes() { return Kv4Shape<NT>::kWarps * kSlots * kUnit; }
// the merge reuses the ring: the staged rows (16-byte aligned, a whole number
// of float4), then the warps' rows, their maxima and sums
constexpr int kXo = 132;
constexpr int kStaged = 16 * (kStageStride + 2);        // floats
static_assert(kStaged % 4 == 0 && kXo % 4 == 0, "rows of float4");
template <int NT> constexpr uint32_t merge_bytes() {
  return 4u * (kStaged + Kv4Shape<NT>::kWarps * 8 * NT * (kXo + 2));
}
template <int NT> constexpr uint32_t smem_bytes() {
  return merge_bytes<NT>() > ring_bytes<NT>() ? merge_bytes<NT>() : ring_bytes<NT>();
}
static_assert(smem_bytes<1>() <= 232448 && smem_bytes<2>() <= 232448, "shared memory budget");

struct Kv4DecParams {
  AttnArgs a;
  float scale_log2;
  int M;              // packed query rows per KV head (R * G <= 16)
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// D = A * B + C with both rows of C equal to (c0, c1).
__device__ __forceinline__ void mma16816_c(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                           uint32_t b1, float c0, float c1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %11, %10, %11};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t sub136_mul(uint32_t x, uint32_t s) {
  const __nv_bfloat162 c = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x), __float2bfloat162_rn(136.f));
  const __nv_bfloat162 v = __hmul2(c, *reinterpret_cast<const __nv_bfloat162*>(&s));
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Physical key of row r (0..15) of a 16-key MMA block.
__device__ __forceinline__ int key_of_row(int r) { return ((r & 7) >> 1) + 4 * (r & 1) + (r & 8); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

template <int NT>
__global__ void __launch_bounds__(Kv4Shape<NT>::kThreads, 1) attn_kv4_dec_kernel(const Kv4DecParams prm) {
  constexpr int kWarps = Kv4Shape<NT>::kWarps;
  constexpr int kRows = 8 * NT;
  constexpr unsigned kAll = 0xffffffffu;
  extern __shared__ __align__(128) uint8_t smem[];
  const AttnArgs& a = prm.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x, g_head = blockIdx.y % a.Hkv;
  pdl_wait();
  pdl_trigger();
  const int b = longest_first(a.seq_lens, a.B, (int)blockIdx.y / a.Hkv);
  int P = a.seq_lens[b];
  const bool len_ok = P >= 0 && P <= a.max_prefix;
  if (!len_ok) {
    if (threadIdx.x == 0 && split == 0) raise_error(a.err, TIDAR_DEVERR_BAD_LEN);
    P = 0;
  }
  const int k0 = split * a.keys_per_split;               // a multiple of 64
  const int kend = min(P, k0 + a.keys_per_split);
  const int units = kend > k0 ? (kend - k0 + 31) / 32 : 0;
  const bool step = split == a.nsplit - 1 && a.step_keys;
  const int32_t* table = a.page_table + (size_t)b * a.max_pages;
  const int ps = a.page_size, lps = 31 - __clz(ps);

  // rows of this CTA's result: normalised O, lse and validity (after the loop)
  float* ost = reinterpret_cast<float*>(smem);
  float* lst = ost + 16 * kStageStride;
  int* wst = reinterpret_cast<int*>(lst + 16);

  // ---- this warp's copies: units warp, warp + kWarps, .. of 32 keys, on one
  // page (or two of 16 rows).  Every lane copies 16-byte pieces: four of K's
  // codes, four of V's, one of a scale row (lanes 0..15 K, 16..31 V).  The page
  // id of the next unit is loaded while this one's copies are issued.
  const size_t page_bytes = kv4_page_bytes(ps, 128);
  const size_t page_stride = (size_t)a.Hkv * page_bytes;
  const uint8_t* kcodes = static_cast<const uint8_t*>(a.k_pages) + (size_t)g_head * page_bytes + 16 * lane;
  const uint8_t* vcodes = static_cast<const uint8_t*>(a.v_pages) + (size_t)g_head * page_bytes + 16 * lane;
  const uint8_t* scales = static_cast<const uint8_t*>(lane < 16 ? a.k_pages : a.v_pages) + (size_t)g_head * page_bytes +
                          (size_t)ps * 64 + 16 * (ps == 16 ? lane & 7 : lane & 15);
  const uint32_t slot0 = smem_u32(smem) + (uint32_t)warp * (kSlots * kUnit) + 16u * lane;
  const int half = ps == 16 ? (lane >> 3) & 1 : 0;        // 16-row pages: the block whose scales this lane copies
  bool bad = false;
  // page of block q of unit u (-1: no key, or no valid page)
  auto load_page = [&](int u, int q) -> int {
    const int key = k0 + 32 * u + 16 * q;
    int pg = -1;
    if (key < kend) {
      pg = table[key >> lps];
      if (pg < 0 || pg >= a.num_pages) pg = -1, bad = true;
    }
    return pg;
  };
  auto load_pages = [&](int u, int (&pg)[2]) {
    pg[0] = load_page(u, 0);
    pg[1] = ps == 16 ? load_page(u, 1) : pg[0];
  };
  // queues unit u's copies into a slot and returns which 16-key blocks it holds
  auto issue = [&](int u, int sl, const int (&pg)[2]) -> int {
    const uint32_t dst = slot0 + (uint32_t)sl * kUnit;
    const uint32_t row = (uint32_t)(k0 + 32 * u) & (uint32_t)(ps - 1);
    if (ps != 16) {
      if (pg[0] < 0) return 0;
      const size_t at = (size_t)pg[0] * page_stride;
      const uint8_t* kc = kcodes + at + row * 64;
      const uint8_t* vc = vcodes + at + row * 64;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        cp_async16(dst + 512 * j, kc + 512 * j);
        cp_async16(dst + kCodes + 512 * j, vc + 512 * j);
      }
      cp_async16(dst + 2 * kCodes, scales + at + row * 8);
      return 3;
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (pg[q] < 0) continue;
      const size_t at = (size_t)pg[q] * page_stride;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        cp_async16(dst + 1024 * q + 512 * j, kcodes + at + 512 * j);
        cp_async16(dst + kCodes + 1024 * q + 512 * j, vcodes + at + 512 * j);
      }
      if (half == q) cp_async16(dst + 2 * kCodes, scales + at);
    }
    return (pg[0] >= 0 ? 1 : 0) | (pg[1] >= 0 ? 2 : 0);
  };
  int pg[2];
  int blocks = 0;                        // two bits per slot in flight, the oldest lowest
#pragma unroll
  for (int i = 0; i < kSlots - 1; ++i) {
    load_pages(warp + i * kWarps, pg);
    blocks |= issue(warp + i * kWarps, i, pg) << (2 * i);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  load_pages(warp + (kSlots - 1) * kWarps, pg);

  {
    const int wid = warp, gq = lane >> 2, cq = lane & 3;
    const float sl2 = prm.scale_log2;
    // Q^T as the B operand: qb[G][nt] = dims 32G + 8cq .. + 7 of row 8nt + gq,
    // two MMA steps of two registers each; qc = -136 times the groups' sums of
    // the two rows that this lane's accumulators belong to
    uint32_t qb[4][NT][4];
    float qc[4][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = 8 * nt + gq;
      const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(a.q) +
                                ((size_t)((size_t)b * a.R + row / a.G) * a.Hq + g_head * a.G + row % a.G) * 128 + 8 * cq;
#pragma unroll
      for (int G = 0; G < 4; ++G) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (row < prm.M) x = *reinterpret_cast<const uint4*>(qp + 32 * G);
        qb[G][nt][0] = x.x; qb[G][nt][1] = x.y; qb[G][nt][2] = x.z; qb[G][nt][3] = x.w;
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&qb[G][nt][e]));
          sum += f.x + f.y;
        }
        sum += __shfl_xor_sync(kAll, sum, 1);
        sum += __shfl_xor_sync(kAll, sum, 2);
        qc[G][nt][0] = -136.f * __shfl_sync(kAll, sum, 8 * cq);
        qc[G][nt][1] = -136.f * __shfl_sync(kAll, sum, 8 * cq + 4);
      }
    }
    float o[8][NT][4];
#pragma unroll
    for (int mt = 0; mt < 8; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) o[mt][nt][0] = o[mt][nt][1] = o[mt][nt][2] = o[mt][nt][3] = 0.f;
    // running maximum (log2 domain), its negative as the exponent's offset (0
    // while there is none), and the raw score past which it is raised
    float m[NT][2], l[NT][2], negm[NT][2], lim[NT][2];
    const float inv_sl2 = 1.f / sl2;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) m[nt][h] = lim[nt][h] = -INFINITY, l[nt][h] = negm[nt][h] = 0.f;

    // Online softmax of KB blocks of 16 keys: sc holds raw scores (-inf where
    // masked) on entry; pb the P^T operands on return.
    auto softmax = [&](auto& sc, auto& pb, auto kb_tag) {
      constexpr int KB = decltype(kb_tag)::value;
      bool up = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float mx = -INFINITY;
#pragma unroll
          for (int kb = 0; kb < KB; ++kb) mx = fmaxf(mx, fmaxf(sc[kb][nt][h], sc[kb][nt][h + 2]));
          up = up || mx > lim[nt][h];
        }
      if (__any_sync(kAll, up)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float mx = -INFINITY;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) mx = fmaxf(mx, fmaxf(sc[kb][nt][h], sc[kb][nt][h + 2]));
            mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 16));
            const float nm = fmaxf(m[nt][h], mx * sl2);
            const float f = m[nt][h] == -INFINITY ? 0.f : ex2(m[nt][h] - nm);
            m[nt][h] = nm;
            negm[nt][h] = nm == -INFINITY ? 0.f : -nm;
            lim[nt][h] = (nm + 8.f) * inv_sl2;
            l[nt][h] *= f;
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
              o[mt][nt][h] *= f;
              o[mt][nt][h + 2] *= f;
            }
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float n0 = negm[nt][0], n1 = negm[nt][1];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          const float p0 = ex2(fmaf(sc[kb][nt][0], sl2, n0)), p1 = ex2(fmaf(sc[kb][nt][1], sl2, n1));
          const float p2 = ex2(fmaf(sc[kb][nt][2], sl2, n0)), p3 = ex2(fmaf(sc[kb][nt][3], sl2, n1));
          l[nt][0] += p0 + p2;
          l[nt][1] += p1 + p3;
          pb[kb][nt][0] = movmatrix_t(tc05::cvt_bf16x2(p0, p1));
          pb[kb][nt][1] = movmatrix_t(tc05::cvt_bf16x2(p2, p3));
        }
      }
    };

    if (step && wid == kWarps - 1) {      // the warp with the fewest units
      // ---- the step keys (R <= 16 rows of k_blk / v_blk), fragments straight
      // from global memory; MMA row r is key_of_row(r)
      float sc[1][NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) sc[0][nt][0] = sc[0][nt][1] = sc[0][nt][2] = sc[0][nt][3] = 0.f;
      const size_t row_el = (size_t)a.Hkv * 128;
      const __nv_bfloat16* kblk = static_cast<const __nv_bfloat16*>(a.k_blk) + (size_t)b * a.R * row_el + g_head * 128;
      const __nv_bfloat16* vblk = static_cast<const __nv_bfloat16*>(a.v_blk) + (size_t)b * a.R * row_el + g_head * 128;
      const int kr[2] = {key_of_row(gq), key_of_row(gq + 8)};
#pragma unroll
      for (int G = 0; G < 4; ++G) {
        uint4 x[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          x[h] = make_uint4(0, 0, 0, 0);
          if (kr[h] < a.R) x[h] = *reinterpret_cast<const uint4*>(kblk + kr[h] * row_el + 32 * G + 8 * cq);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma16816(sc[0][nt], x[0].x, x[1].x, x[0].y, x[1].y, qb[G][nt][0], qb[G][nt][1]);
          mma16816(sc[0][nt], x[0].z, x[1].z, x[0].w, x[1].w, qb[G][nt][2], qb[G][nt][3]);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int rho = min((8 * nt + 2 * cq + (e & 1)) / a.G, a.R - 1), key = kr[e >> 1];
          if (key >= a.R || !step_visible(step_visibility(a.k, rho), key)) sc[0][nt][e] = -INFINITY;
        }
      uint32_t pb[1][NT][2];
      softmax(sc, pb, std::integral_constant<int, 1>{});
#pragma unroll
      for (int G = 0; G < 4; ++G) {
        // dims 32G + 8(g/2) + 0..7 of keys cq, cq + 4, cq + 8, cq + 12; this
        // lane's are those of parity g % 2
        uint4 x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          x[u] = make_uint4(0, 0, 0, 0);
          if (cq + 4 * u < a.R) x[u] = *reinterpret_cast<const uint4*>(vblk + (cq + 4 * u) * row_el + 32 * G + 8 * (gq >> 1));
        }
        const uint32_t sel = (gq & 1) ? 0x7632u : 0x5410u;
        uint32_t v[2][4];                                // [key pair][i]
#pragma unroll
        for (int pr = 0; pr < 2; ++pr) {
          const uint4 lo = x[2 * pr], hi = x[2 * pr + 1];
          v[pr][0] = __byte_perm(lo.x, hi.x, sel); v[pr][1] = __byte_perm(lo.y, hi.y, sel);
          v[pr][2] = __byte_perm(lo.z, hi.z, sel); v[pr][3] = __byte_perm(lo.w, hi.w, sel);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816(o[2 * G + j][nt], v[0][2 * j], v[0][2 * j + 1], v[1][2 * j], v[1][2 * j + 1], pb[0][nt][0], pb[0][nt][1]);
      }
    }

    // ---- the prefix: a unit (32 keys) at a time
    const int krow = key_of_row(gq);
    int sl = 0;
    for (int u = wid; u < units; u += kWarps) {
      // the slot freed last time takes the unit after the ones in flight
      {
        const int nu = u + (kSlots - 1) * kWarps, ns = sl == 0 ? kSlots - 1 : sl - 1;
        blocks |= issue(nu, ns, pg) << (2 * (kSlots - 1));
        asm volatile("cp.async.commit_group;" ::: "memory");
        load_pages(nu + kWarps, pg);
      }
      asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 1) : "memory");
      __syncwarp();
      const int mask = blocks & 3;
      blocks >>= 2;
      const uint8_t* kc = smem + (size_t)warp * (kSlots * kUnit) + (size_t)sl * kUnit;
      const uint8_t* vc = kc + kCodes;
      const uint8_t* ks = vc + kCodes;
      const uint8_t* vs = ks + kScales;
      const int nleft = kend - k0 - 32 * u;              // valid keys of this unit
      float sc[2][NT][4];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        const uint4 ka = *reinterpret_cast<const uint4*>(kc + (16 * kb + krow) * 64 + cq * 16);
        const uint4 kd = *reinterpret_cast<const uint4*>(kc + (16 * kb + 8 + krow) * 64 + cq * 16);
        const uint2 sa = *reinterpret_cast<const uint2*>(ks + (16 * kb + krow) * 8);
        const uint2 sd = *reinterpret_cast<const uint2*>(ks + (16 * kb + 8 + krow) * 8);
        const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wd[4] = {kd.x, kd.y, kd.z, kd.w};
        const float fa[4] = {__uint_as_float(sa.x << 16), __uint_as_float(sa.x & 0xffff0000u),
                             __uint_as_float(sa.y << 16), __uint_as_float(sa.y & 0xffff0000u)};
        const float fd[4] = {__uint_as_float(sd.x << 16), __uint_as_float(sd.x & 0xffff0000u),
                             __uint_as_float(sd.y << 16), __uint_as_float(sd.y & 0xffff0000u)};
#pragma unroll
        for (int G = 0; G < 4; ++G) {
          uint32_t ra[4], rd[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) ra[e] = kv4_offset_codes(wa[G], e), rd[e] = kv4_offset_codes(wd[G], e);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float acc[4];
            mma16816_c(acc, ra[0], rd[0], ra[1], rd[1], qb[G][nt][0], qb[G][nt][1], qc[G][nt][0], qc[G][nt][1]);
            mma16816(acc, ra[2], rd[2], ra[3], rd[3], qb[G][nt][2], qb[G][nt][3]);
            if (G == 0) {
              sc[kb][nt][0] = acc[0] * fa[0]; sc[kb][nt][1] = acc[1] * fa[0];
              sc[kb][nt][2] = acc[2] * fd[0]; sc[kb][nt][3] = acc[3] * fd[0];
            } else {
              sc[kb][nt][0] = fmaf(acc[0], fa[G], sc[kb][nt][0]); sc[kb][nt][1] = fmaf(acc[1], fa[G], sc[kb][nt][1]);
              sc[kb][nt][2] = fmaf(acc[2], fd[G], sc[kb][nt][2]); sc[kb][nt][3] = fmaf(acc[3], fd[G], sc[kb][nt][3]);
            }
          }
        }
      }
      const bool whole = mask == 3 && nleft >= 32;
      if (!whole) {
        // a masked key's value scales may be anything, and 0 times a NaN is not 0
        if (lane >= nleft || !((mask >> (lane >> 4)) & 1))
          *reinterpret_cast<uint2*>(smem + (vs - smem) + lane * 8) = make_uint2(0, 0);
        __syncwarp();
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = 16 * kb + krow + 8 * (e >> 1);
            if (key >= nleft || !((mask >> kb) & 1)) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) sc[kb][nt][e] = -INFINITY;
            }
          }
      }
      uint32_t pb[2][NT][2];
      softmax(sc, pb, std::integral_constant<int, 2>{});
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        uint2 c[4], t[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          c[e] = *reinterpret_cast<const uint2*>(vc + (16 * kb + cq + 4 * e) * 64 + gq * 8);
          t[e] = *reinterpret_cast<const uint2*>(vs + (16 * kb + cq + 4 * e) * 8);
        }
#pragma unroll
        for (int G = 0; G < 4; ++G) {
          const uint32_t sel = (G & 1) ? 0x7632u : 0x5410u;
          uint32_t v[2][4];                              // [key pair][i]
#pragma unroll
          for (int pr = 0; pr < 2; ++pr) {
            const uint32_t w = G < 2 ? __byte_perm(c[2 * pr].x, c[2 * pr + 1].x, sel) : __byte_perm(c[2 * pr].y, c[2 * pr + 1].y, sel);
            const uint32_t sp = G < 2 ? __byte_perm(t[2 * pr].x, t[2 * pr + 1].x, sel) : __byte_perm(t[2 * pr].y, t[2 * pr + 1].y, sel);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[pr][e] = sub136_mul(kv4_offset_codes(w, e), sp);
          }
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma16816(o[2 * G + j][nt], v[0][2 * j], v[0][2 * j + 1], v[1][2 * j], v[1][2 * j + 1], pb[kb][nt][0],
                       pb[kb][nt][1]);
        }
      }
      __syncwarp();                       // every lane has read the slot: it may be refilled
      if (++sl == kSlots) sl = 0;
    }
    if (bad) raise_error(a.err, TIDAR_DEVERR_BAD_PAGE);

    // ---- merge the warps: (max, sum, O) per row through the idle ring
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[nt][h] += __shfl_xor_sync(kAll, l[nt][h], 4);
        l[nt][h] += __shfl_xor_sync(kAll, l[nt][h], 8);
        l[nt][h] += __shfl_xor_sync(kAll, l[nt][h], 16);
      }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();                      // every warp is past its last unit
    float* xo = reinterpret_cast<float*>(smem) + kStaged;             // [warps][kRows][kXo]
    float* xm = xo + kWarps * kRows * kXo;                            // [warps][kRows]
    float* xl = xm + kWarps * kRows;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 8 * nt + 2 * cq + h;
        if (r < prm.M) {
          float* dst = xo + (wid * kRows + r) * kXo + 8 * (gq >> 1) + (gq & 1);
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) {
            dst[32 * (mt >> 1) + 4 * (mt & 1)] = o[mt][nt][h];
            dst[32 * (mt >> 1) + 4 * (mt & 1) + 2] = o[mt][nt][h + 2];
          }
          if (gq == 0) {
            xm[wid * kRows + r] = m[nt][h];
            xl[wid * kRows + r] = l[nt][h];
          }
        }
      }
    __syncthreads();
    for (int r = wid; r < prm.M; r += kWarps) {
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, xm[w * kRows + r]);
      float lt = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = xm[w * kRows + r];
        const float f = mw == -INFINITY ? 0.f : ex2(mw - top);
        const float lw = xl[w * kRows + r];
        const float4 x = *reinterpret_cast<const float4*>(xo + (w * kRows + r) * kXo + 4 * lane);
        // a warp whose scores were NaN has no maximum but a NaN sum: it stays NaN
        if (mw != -INFINITY || lw != 0.f) {
          const float fw = mw == -INFINITY ? 1.f : f;
          lt = fmaf(fw, lw, lt);
          v.x = fmaf(fw, x.x, v.x); v.y = fmaf(fw, x.y, v.y); v.z = fmaf(fw, x.z, v.z); v.w = fmaf(fw, x.w, v.w);
        }
      }
      const bool any = lt != 0.f;                          // NaN counts
      const float inv = any ? 1.f / lt : 0.f;
      *reinterpret_cast<float4*>(ost + r * kStageStride + 4 * lane) = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
      if (lane == 0) {
        lst[r] = any ? (top + log2f(lt)) * 0.69314718055994531f : -INFINITY;
        wst[r] = 1;
      }
    }
  }
  __syncthreads();

  auto out_row = [&](int r) -> long long {
    return ((long long)b * a.R + r / a.G) * a.Hq + g_head * a.G + r % a.G;
  };
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
  if (a.nsplit == 1) {
    tc05::store_rows_bf16(ost, lst, wst, prm.M, out_row, out, a.lse_out);
  } else if (a.cluster_merge) {
    // the splits of one (b, head) are the cluster's CTAs (rank = split): all
    // have staged their rows at the first barrier; the second keeps each CTA's
    // shared memory alive until its peers have read it
    const int ns = a.nsplit, rank = (int)cluster_rank();
    cluster_sync_all();
    const int owned = prm.M > rank ? (prm.M - rank + ns - 1) / ns : 0;
    tc05::merge_rows<1, 8, true>(ost, lst, ns, rank, owned, out_row, out, a.lse_out);
    cluster_sync_all();
  } else {
    const long long stride = (long long)a.B * a.R * a.Hq;
    tc05::store_rows_partial(ost, lst, wst, prm.M, [&](int r) -> long long { return split * stride + out_row(r); }, a.part_o,
                             a.part_lse);
  }

  if (split == 0 && len_ok && (a.nsplit == 1 || a.cluster_merge) && a.append) {
    // draft rows D_1..D_n of this head, quantised: a quad per (row, K or V)
    for (int u0 = warp * 8; u0 < 2 * a.n; u0 += 8 * kWarps) {
      const int u = u0 + (lane >> 2), r = u >> 1, y = lane & 3;
      const bool in = u < 2 * a.n, is_key = !(u & 1);
      const int pos = P + (in ? r : 0);
      const int page = table[pos / ps];
      const bool mapped = page >= 0 && page < a.num_pages;
      if (in && !mapped && y == 0) raise_error(a.err, TIDAR_DEVERR_BAD_PAGE);
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(is_key ? a.k_blk : a.v_blk) +
                                 ((size_t)((size_t)b * a.R + (in ? r : 0)) * a.Hkv + g_head) * 128 + 8 * y;
      float x[4][8];
#pragma unroll
      for (int G = 0; G < 4; ++G) load_vec<__nv_bfloat16, 8>(src + 32 * G, x[G]);
      uint8_t* base = static_cast<uint8_t*>(const_cast<void*>(is_key ? a.k_pages : a.v_pages)) +
                      ((size_t)(mapped ? page : 0) * a.Hkv + g_head) * kv4_page_bytes(ps, 128);
      kv4_store_quad<128, true>(x, is_key, base, ps, pos % ps, in && mapped);
    }
  }
}

template <int NT>
cudaError_t smem_attr() {
  static bool set[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorNotSupported;
  if (!set[dev]) {
    e = cudaFuncSetAttribute(attn_kv4_dec_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<NT>());
    if (e != cudaSuccess) return e;
    set[dev] = true;
  }
  return cudaSuccess;
}

template <int NT>
int resident_clusters_t(int ns) {
  static int cache[64][kMaxCluster + 1];
  if (ns < 1 || ns > kMaxCluster) return 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if (cache[dev][ns]) return cache[dev][ns] - 1;
  int n = 0;
  if (smem_attr<NT>() == cudaSuccess &&
      (ns <= 8 || cudaFuncSetAttribute(attn_kv4_dec_kernel<NT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) ==
                      cudaSuccess)) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ns, 1, 1);
    cfg.blockDim = dim3(Kv4Shape<NT>::kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem_bytes<NT>();
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ns;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, attn_kv4_dec_kernel<NT>, &cfg) != cudaSuccess) n = 0;
  }
  cudaGetLastError();
  cache[dev][ns] = n + 1;
  return n;
}

}  // namespace

int kv4_dec_resident_clusters(int ns, int M) {
  return M <= 8 ? resident_clusters_t<1>(ns) : resident_clusters_t<2>(ns);
}

cudaError_t launch_attn_kv4_dec(const AttnArgs& a, cudaStream_t s) {
  const int M = a.R * a.G;
  if (!a.bf16 || a.D != 128 || M > 16 || a.keys_per_split % 64) return cudaErrorNotSupported;
  Kv4DecParams prm;
  prm.a = a;
  prm.scale_log2 = a.scale * 1.4426950408889634f;
  prm.M = M;
  const bool clu = a.nsplit > 1 && a.cluster_merge;
  if (a.nsplit > 1 && !clu && (!a.part_o || !a.part_lse)) return cudaErrorInvalidValue;
  if (clu && a.nsplit > kMaxCluster) return cudaErrorNotSupported;
  const dim3 grid(a.nsplit, a.B * a.Hkv), cluster(clu ? a.nsplit : 1, 1, 1);
  cudaError_t e = M <= 8 ? smem_attr<1>() : smem_attr<2>();
  if (e != cudaSuccess) return e;
  if (M <= 8)
    return launch_clustered(attn_kv4_dec_kernel<1>, grid, cluster, Kv4Shape<1>::kThreads, smem_bytes<1>(), s, prm);
  return launch_clustered(attn_kv4_dec_kernel<2>, grid, cluster, Kv4Shape<2>::kThreads, smem_bytes<2>(), s, prm);
}

}  // namespace tidar
