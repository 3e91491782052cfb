// kv4.cu -- rows into the 4-bit paged cache and back (layout: kv4.cuh).
//
// kv4_append: row t of k_rows / v_rows [rows][Hkv][D] is quantised and stored
// at slots[t] = page * page_size + row.  Four lanes a (row, head, K or V): each
// brings a quarter of every group, the group maxima meet in two shuffles, and
// each lane writes one chunk (D/8 bytes; 64 contiguous bytes a row and head at
// D = 128).  kv4_gather is the way back, the values exact in bf16 and fp32.
// Both read and write every byte once; the bytes bound them: 8192 rows of 8 heads of
// 128, bf16, stored and read back in 19.0 us, 4.5 TB/s (0.69 of the copy rate; the
// rows of one call fit L2, so part of the time is launch and ramp).
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"

namespace tidar {

namespace {

constexpr int kQThreads = 256;

struct Kv4RowsArgs {
  int rows, Hkv, ps;
  int fill;                    // gather: zeros for rows without a slot
  uint32_t units;              // rows * 2 Hkv, below 2^31
  uint32_t div_mul, div_shift; // u / (2 Hkv) = (u div_mul >> 32) >> div_shift for u < 2^31
  long long nslots;            // num_pages * page_size
  long long k_stride, v_stride;  // elements between rows of k / v
  void* k;
  void* v;
  const int64_t* slots;
  uint8_t* k_pages;
  uint8_t* v_pages;
  unsigned int* err;
};

// Eight consecutive elements as fp32, and back.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    load_vec<T, 8>(p, x);
  } else {
    float a[4], b[4];
    load_vec<T, 4>(p, a);
    load_vec<T, 4>(p + 4, b);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = a[e], x[4 + e] = b[e];
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    __nv_bfloat162 o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(o);
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

template <typename T, int D, bool kStore>
__global__ void __launch_bounds__(kQThreads) kv4_rows_kernel(Kv4RowsArgs a) {
  constexpr int N = D / 32;
  pdl_wait();
  pdl_trigger();
  const int y = (int)threadIdx.x & 3, lps = 31 - __clz(a.ps);
  const size_t page_bytes = kv4_page_bytes(a.ps, D);
  bool bad = false;
  // A unit is one row of one head of K or V, four lanes; heads fastest, so the
  // eight units of a warp are neighbours in the row tensors.  Whole warps loop.
  for (uint32_t u0 = blockIdx.x * (kQThreads / 4) + (threadIdx.x >> 5) * 8; u0 < a.units; u0 += gridDim.x * (kQThreads / 4)) {
    const uint32_t u = u0 + ((threadIdx.x & 31) >> 2);
    const bool in = u < a.units;
    const uint32_t row = in ? __umulhi(u, a.div_mul) >> a.div_shift : 0u;   // u / (2 Hkv)
    const int hv = in ? (int)(u - row * 2u * (uint32_t)a.Hkv) : 0;
    const bool is_key = hv < a.Hkv;
    const int head = is_key ? hv : hv - a.Hkv;
    const long long slot = in ? a.slots[row] : -1;
    const bool live = slot >= 0 && slot < a.nslots;
    if (slot >= a.nslots) bad = true;
    const long long page = live ? slot >> lps : 0;
    const int r = live ? (int)slot & (a.ps - 1) : 0;
    uint8_t* base = (is_key ? a.k_pages : a.v_pages) + (size_t)(page * a.Hkv + head) * page_bytes;
    T* p = static_cast<T*>(is_key ? a.k : a.v) + (size_t)row * (is_key ? a.k_stride : a.v_stride) +
           (size_t)head * D + 8 * y;
    float x[N][8];
    if constexpr (kStore) {
#pragma unroll
      for (int G = 0; G < N; ++G) {
        if (live) {
          load8<T>(p + 32 * G, x[G]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[G][e] = 0.f;
        }
      }
      kv4_store_quad<D, sizeof(T) == 2>(x, is_key, base, a.ps, r, live);
    } else if (live) {
      uint32_t w[N];
      float s[N];
      kv4_load_chunk<D>(base, is_key, a.ps, r, y, w, s);
#pragma unroll
      for (int G = 0; G < N; ++G) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 c = __bfloat1622float2(kv4_codes2(w[G], i));
          x[G][2 * i] = c.x * s[G];
          x[G][2 * i + 1] = c.y * s[G];
        }
        store8<T>(p + 32 * G, x[G]);
      }
    } else if (in && a.fill) {
#pragma unroll
      for (int G = 0; G < N; ++G) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[G][e] = 0.f;
        store8<T>(p + 32 * G, x[G]);
      }
    }
  }
  if (bad) raise_error(a.err, TIDAR_DEVERR_BAD_PAGE);
}

template <bool kStore>
cudaError_t launch_rows(const Kv4RowsArgs& a, int D, bool bf16, cudaStream_t s) {
  const int grid = (int)std::min<uint32_t>((a.units + kQThreads / 4 - 1) / (kQThreads / 4), 148 * 64);
  auto go = [&](auto kernel) { return launch_pdl(kernel, dim3(grid), kQThreads, 0, s, a); };
  if (bf16) return D == 64 ? go(kv4_rows_kernel<__nv_bfloat16, 64, kStore>) : go(kv4_rows_kernel<__nv_bfloat16, 128, kStore>);
  return D == 64 ? go(kv4_rows_kernel<float, 64, kStore>) : go(kv4_rows_kernel<float, 128, kStore>);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Checks shared by the two directions; nothing is queued on failure.
tidar_status prepare(const tidar_kv4_desc* d, const void* k_pages, const void* v_pages, const void* k, const void* v,
                     const int64_t* slots, Kv4RowsArgs& a) {
  if (!d) return TIDAR_ERR_INVALID_ARG;
  if (d->rows < 0 || d->num_kv_heads <= 0 || d->num_pages <= 0 || d->page_size <= 0) return TIDAR_ERR_INVALID_ARG;
  if (d->head_dim != 64 && d->head_dim != 128) return TIDAR_ERR_UNSUPPORTED;
  if (d->page_size != 16 && d->page_size != 32 && d->page_size != 64 && d->page_size != 128)
    return TIDAR_ERR_UNSUPPORTED;
  if (d->dtype != TIDAR_F32 && d->dtype != TIDAR_BF16) return TIDAR_ERR_UNSUPPORTED;
  if (d->rows == 0) return TIDAR_OK;
  if (!k_pages || !v_pages || !k || !v || !slots) return TIDAR_ERR_INVALID_ARG;
  if (!aligned16(k_pages) || !aligned16(v_pages) || !aligned16(k) || !aligned16(v)) return TIDAR_ERR_INVALID_ARG;
  const long long row = (long long)d->num_kv_heads * d->head_dim;
  a.k_stride = d->k_row_stride ? d->k_row_stride : row;
  a.v_stride = d->v_row_stride ? d->v_row_stride : row;
  const int per16 = d->dtype == TIDAR_F32 ? 4 : 8;
  if (a.k_stride < row || a.v_stride < row || a.k_stride % per16 || a.v_stride % per16) return TIDAR_ERR_INVALID_ARG;
  if (d->num_kv_heads > (1 << 24) || (long long)d->rows * 2 * d->num_kv_heads >= (1LL << 31)) return TIDAR_ERR_UNSUPPORTED;
  // Division by n = 2 Hkv: with 2^l >= n > 2^(l-1) and m = ceil(2^(31+l) / n),
  // floor(u m / 2^(31+l)) = floor(u / n) for every u < 2^31 (m n - 2^(31+l) < n <=
  // 2^l, so u times the excess stays below 2^(31+l)); m < 2^32.
  const uint32_t n = 2u * (uint32_t)d->num_kv_heads;
  uint32_t l = 1;
  while ((1u << l) < n) ++l;
  a.units = (uint32_t)d->rows * n;
  a.div_mul = (uint32_t)(((1ULL << (31 + l)) + n - 1) / n);
  a.div_shift = l - 1;
  a.rows = d->rows; a.Hkv = d->num_kv_heads; a.ps = d->page_size; a.fill = d->zero_skipped != 0;
  a.nslots = (long long)d->num_pages * d->page_size;
  a.k = const_cast<void*>(k); a.v = const_cast<void*>(v); a.slots = slots;
  a.k_pages = static_cast<uint8_t*>(const_cast<void*>(k_pages));
  a.v_pages = static_cast<uint8_t*>(const_cast<void*>(v_pages));
  return error_word_status(&a.err);
}

}  // namespace
}  // namespace tidar

extern "C" {

size_t tidar_kv4_page_bytes(int32_t page_size, int32_t head_dim) {
  if (head_dim != 64 && head_dim != 128) return 0;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128) return 0;
  return tidar::kv4_page_bytes(page_size, head_dim);
}

tidar_status tidar_kv4_append(const tidar_kv4_desc* d, void* k_pages, void* v_pages, const void* k_rows,
                              const void* v_rows, const int64_t* slots, tidar_stream_t stream) {
  tidar::Kv4RowsArgs a{};
  const tidar_status st = tidar::prepare(d, k_pages, v_pages, k_rows, v_rows, slots, a);
  if (st != TIDAR_OK || d->rows == 0) return st;
  const cudaError_t e =
      tidar::launch_rows<true>(a, d->head_dim, d->dtype == TIDAR_BF16, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? TIDAR_OK : tidar::cuda_status(e);
}

tidar_status tidar_kv4_gather(const tidar_kv4_desc* d, const void* k_pages, const void* v_pages, const int64_t* slots,
                              void* k_rows, void* v_rows, tidar_stream_t stream) {
  tidar::Kv4RowsArgs a{};
  const tidar_status st = tidar::prepare(d, k_pages, v_pages, k_rows, v_rows, slots, a);
  if (st != TIDAR_OK || d->rows == 0) return st;
  const cudaError_t e =
      tidar::launch_rows<false>(a, d->head_dim, d->dtype == TIDAR_BF16, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? TIDAR_OK : tidar::cuda_status(e);
}

}  // extern "C"
