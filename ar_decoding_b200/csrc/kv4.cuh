// kv4.cuh -- the 4-bit cache page: its layout, the quantiser and the readers
// shared by the kernels that store, read back, evict and attend it.
//
// A row of D dims of one KV head is D/32 groups; group G (dims 32G .. 32G+31)
// has one scale s and 32 codes c in -7..7, and dim d stands for c_d s:
//   s = max|x| / 7 (fp32) rounded to 5 significant bits, c = x / s rounded to
//   the nearest integer, ties to even (exactly: the quotient is never rounded
//   first).
// Five bits of s times three of |c| fit the eight of a bf16, so every value is
// exact in bf16: the attention over this cache is the bf16 attention over the
// values it stands for, whichever kernel reads it.  Rounding s moves the
// largest code's quotient to 7.23 at most, so no code is clipped.
//   max|x| < 2^-120: scale 0, codes 0.
//   max|x| >= 2^126, an infinity or a NaN in the group: scale NaN, codes 0 (the
//   rows that attend such a key come out NaN, as they would from the values).
// A zeroed row (codes and scale 0) stands for zeros.
//
// Page of one head, ps rows: ps rows of D/2 bytes of codes, then ps rows of
// D/32 bf16 scales.  With n = D/32 and dim d = 32 G + 8 y + 2 i + h (y < 4,
// i < 4, h < 2), the code of d is nibble i (lowest first, two's complement) of
// the 16-bit unit
//   y 2n + 2G + h   of a key row,        y 2n + h n + G   of a value row.
// Chunk y of a row (D/8 bytes) so holds dims 8y .. 8y+7 of every group.  A lane
// of an MMA fragment needs a few dims of every group: it gets them in one
// aligned load, and masking a unit pair with 0x000f000f gives two neighbouring
// dims (keys), or one dim of two rows after a byte permute (values), in the
// order in which the fragments want them.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace tidar {

__host__ __device__ constexpr int kv4_code_bytes(int D) { return D / 2; }       // per row
__host__ __device__ constexpr int kv4_scale_bytes(int D) { return D / 16; }     // per row
__host__ __device__ constexpr size_t kv4_page_bytes(int ps, int D) {
  return (size_t)ps * (kv4_code_bytes(D) + kv4_scale_bytes(D));
}

// Scale of a group from the bits of its largest magnitude (compared as
// integers, so a NaN wins over every number).
__device__ __forceinline__ float kv4_scale(uint32_t top) {
  const float m = __uint_as_float(top);
  if (!(m < 8.507059173023462e37f)) return __uint_as_float(0x7fc00000u);        // 2^126
  if (m < 7.523163845262640e-37f) return 0.f;                                   // 2^-120
  uint32_t b = __float_as_uint(__fdiv_rn(m, 7.f));
  b = (b + 0x3ffffu + ((b >> 19) & 1u)) & ~0x7ffffu;
  return __uint_as_float(b);
}

// Nearest integer to x / s, ties to even, in the low bits of the result (two's
// complement).  Adding 1.5 2^23 rounds to an integer whose bits are the low
// mantissa bits.
//   bf16 x: q = x / s correctly rounded (one Newton step on x (1/s): the
//     correction is within a few percent of what it has to be, so a quotient
//     that is representable comes out exactly).  x and s have 8 and 5 bits, so a
//     quotient that is no tie is 2^-13 away from one and stays so.
//   fp32 x: c = round(x (1/s)) is off by at most one, next to a tie; the
//     remainder x - c s is exact, and its comparison with s/2 decides.
template <bool kBf16>
__device__ __forceinline__ uint32_t kv4_code(float x, float s, float rs) {
  constexpr float kRound = 12582912.f;
  if constexpr (kBf16) {
    const float q = x * rs;
    return __float_as_uint(__fadd_rn(fmaf(fmaf(-q, s, x), rs, q), kRound));
  } else {
    const float t = __fadd_rn(x * rs, kRound), c = t - kRound;
    const float r = fmaf(-c, s, x), h = 0.5f * s;
    uint32_t k = __float_as_uint(t);
    if (fabsf(r) > h || (fabsf(r) == h && (k & 1u))) k += r > 0.f ? 1u : ~0u;
    return k;
  }
}

// Eight dims of one group (dims 8y .. 8y+7) as a key-row word: units 2G (even
// dims) and 2G + 1 (odd dims).
template <bool kBf16>
__device__ __forceinline__ uint32_t kv4_pack8(const float (&x)[8], float s) {
  if (!(s > 0.f)) return 0u;                       // scale 0 or NaN
  const float rs = __frcp_rn(s);
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) w |= (kv4_code<kBf16>(x[e], s, rs) & 15u) << (4 * (e >> 1) + 16 * (e & 1));
  return w;
}

// Key-row words (one per group) of a chunk <-> the chunk of a value row.
template <int N>
__device__ __forceinline__ void kv4_key_to_value(const uint32_t (&k)[N], uint32_t (&v)[N]) {
#pragma unroll
  for (int j = 0; j < N / 2; ++j) {
    v[j] = __byte_perm(k[2 * j], k[2 * j + 1], 0x5410);               // even dims of groups 2j, 2j+1
    v[N / 2 + j] = __byte_perm(k[2 * j], k[2 * j + 1], 0x7632);       // odd dims
  }
}
template <int N>
__device__ __forceinline__ void kv4_value_to_key(const uint32_t (&v)[N], uint32_t (&k)[N]) {
#pragma unroll
  for (int j = 0; j < N / 2; ++j) {
    k[2 * j] = __byte_perm(v[j], v[N / 2 + j], 0x5410);
    k[2 * j + 1] = __byte_perm(v[j], v[N / 2 + j], 0x7632);
  }
}

// Pair i of a key-row word (dims 2i, 2i+1 of its eight) as the bf16 numbers
// 136 + c: the nibbles, offset by 8, become the low mantissa bits of 128.  One
// shift and one three-input logic instruction, (x & 0x000f000f) ^ 0x43084308
// (left to the compiler, the two constants cost two instructions).
__device__ __forceinline__ uint32_t kv4_offset_codes(uint32_t w, int i) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(r) : "r"(w >> (4 * i)), "r"(0x000f000fu), "r"(0x43084308u));
  return r;
}
// The same pair as the codes themselves.
__device__ __forceinline__ __nv_bfloat162 kv4_codes2(uint32_t w, int i) {
  const uint32_t b = kv4_offset_codes(w, i);
  return __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&b), __float2bfloat162_rn(136.f));
}

// Quantise and store one row of one head: four consecutive lanes (y = lane & 3)
// each bring the dims 32G + 8y + e, e < 8, of every group G in x[G][e] and
// write chunk y.  All 32 lanes call it; a quad with live = false writes
// nothing.  base: the page's bytes of this head; kBf16: the values are bf16.
template <int D, bool kBf16>
__device__ __forceinline__ void kv4_store_quad(const float (&x)[D / 32][8], bool is_key, uint8_t* base, int ps, int r,
                                               bool live) {
  constexpr int N = D / 32;
  const int y = (int)threadIdx.x & 3;
  uint32_t w[N];
  uint32_t sc[N];
#pragma unroll
  for (int G = 0; G < N; ++G) {
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[G][e]) & 0x7fffffffu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const float s = kv4_scale(top);
    sc[G] = __float_as_uint(s) >> 16;              // exact: 5 significant bits
    w[G] = kv4_pack8<kBf16>(x[G], s);
  }
  if (!live) return;
  uint32_t o[N];
  if (is_key) {
#pragma unroll
    for (int G = 0; G < N; ++G) o[G] = w[G];
  } else {
    kv4_key_to_value<N>(w, o);
  }
  uint8_t* code = base + (size_t)r * kv4_code_bytes(D) + y * (D / 8);
  uint8_t* scale = base + (size_t)ps * kv4_code_bytes(D) + (size_t)r * kv4_scale_bytes(D);
  if constexpr (N == 4) {
    *reinterpret_cast<uint4*>(code) = make_uint4(o[0], o[1], o[2], o[3]);
    if (y == 0) *reinterpret_cast<uint2*>(scale) = make_uint2(sc[0] | (sc[1] << 16), sc[2] | (sc[3] << 16));
  } else {
    *reinterpret_cast<uint2*>(code) = make_uint2(o[0], o[1]);
    if (y == 0) *reinterpret_cast<uint32_t*>(scale) = sc[0] | (sc[1] << 16);
  }
}

// Chunk y of row r as key-row words (one per group) and the row's scales.
template <int D>
__device__ __forceinline__ void kv4_load_chunk(const uint8_t* base, bool is_key, int ps, int r, int y,
                                               uint32_t (&w)[D / 32], float (&s)[D / 32]) {
  constexpr int N = D / 32;
  const uint8_t* code = base + (size_t)r * kv4_code_bytes(D) + y * (D / 8);
  const uint8_t* scale = base + (size_t)ps * kv4_code_bytes(D) + (size_t)r * kv4_scale_bytes(D);
  uint32_t v[N], sw[N / 2];
  if constexpr (N == 4) {
    const uint4 c = *reinterpret_cast<const uint4*>(code);
    const uint2 t = *reinterpret_cast<const uint2*>(scale);
    v[0] = c.x; v[1] = c.y; v[2] = c.z; v[3] = c.w;
    sw[0] = t.x; sw[1] = t.y;
  } else {
    const uint2 c = *reinterpret_cast<const uint2*>(code);
    v[0] = c.x; v[1] = c.y;
    sw[0] = *reinterpret_cast<const uint32_t*>(scale);
  }
  if (is_key) {
#pragma unroll
    for (int G = 0; G < N; ++G) w[G] = v[G];
  } else {
    kv4_value_to_key<N>(v, w);
  }
#pragma unroll
  for (int j = 0; j < N / 2; ++j) {
    s[2 * j] = __uint_as_float(sw[j] << 16);
    s[2 * j + 1] = __uint_as_float(sw[j] & 0xffff0000u);
  }
}

// VPL = D/32 consecutive dims lane VPL .. of one row, as fp32 values: what a
// lane of a warp that splits the head dimension holds.
template <int D>
__device__ __forceinline__ void kv4_load_slice(const uint8_t* base, bool is_key, int ps, int r, int lane,
                                               float (&x)[D / 32]) {
  constexpr int N = D / 32;
  const int d0 = lane * N, G = d0 >> 5, y = (d0 & 31) >> 3, i0 = (d0 & 7) >> 1;
  const uint16_t* row = reinterpret_cast<const uint16_t*>(base + (size_t)r * kv4_code_bytes(D)) + y * 2 * N;
  const uint32_t even = row[is_key ? 2 * G : G], odd = row[is_key ? 2 * G + 1 : N + G];
  const float s = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(base + (size_t)ps * kv4_code_bytes(D))[r * N + G]);
  const uint32_t w = even | (odd << 16);
#pragma unroll
  for (int j = 0; j < N / 2; ++j) {
    const float2 c = __bfloat1622float2(kv4_codes2(w, i0 + j));
    x[2 * j] = c.x * s;
    x[2 * j + 1] = c.y * s;
  }
}

}  // namespace tidar
