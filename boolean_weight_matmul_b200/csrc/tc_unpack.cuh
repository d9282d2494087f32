// Unpacking a weight tile for the tensor cores: one row x 16 columns of W (all
// K kernels) -> 16-bit levels, shared by the prefill GEMM (bf16 levels) and the
// CTA-pair GEMMs (fp16 levels).
//
// An element of the tile is the weight level its K bits select, rounded once:
//     Wt[r][j] = RN_bf16( s_0 a_0 + s_1 a_1 + ... + s_{K-1} a_{K-1} ),
// s_k = +1 for a set bit and -1 for a clear one, a_k the fp16 group scales,
// the sum taken in fp32 in kernel order.  K kernels give at most 2^K levels
// per (row, group) (Paper-Notes page, 关键设计: K Boolean kernels represent
// 2^K weight values), so each level is formed once per (row, group) and the
// per-element work is a selection:
//  * K = 1: the level is +-a_0; one LOP3 applies the sign bit pair.
//  * K = 2: the four levels sit in two registers as bf16; a byte permute
//    (PRMT) whose selector is built from the two bits of each element picks
//    an element pair's levels at once.
//  * K = 3, 4: the levels are sign-symmetric (the level of the complemented
//    bits is the negated level, exactly, since rounding to nearest is
//    symmetric), so only the 2^(K-1) levels with s_0 = +1 are kept: the other
//    bits are replaced by t_k = XNOR(b_k, b_0), a PRMT (two and a select for
//    K = 4) picks M[t], and the sign of b_0 is applied with one LOP3.
// The PRMT selector of columns (2p, 2p+1) needs 2*index in both nibbles of
// each output halfword; index bits sit in a precomputed word Z at 2p+1,
// 2p+2 (column 2p) and 2p+9, 2p+10 (column 2p+1), so the selector is
// ((Z >> 2p) & 0x0606) * 0x11 + 0x1010.

#pragma once

#include "mbok_common.cuh"

namespace mbok {

// bf16 pair (lo, hi), each rounded to nearest even from fp32.
__device__ __forceinline__ uint32_t tc_pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Sign-applied level pair for columns (2i, 2i+1): the level's sign flips
// where the bit of kernel 0 is 0.  u = h | (h << 15) holds bit b at b and at
// 15 + b, so one left shift by 15 - 2i puts bit 2i at 15 and bit 2i+1 at 31.
template <int I>
__device__ __forceinline__ uint32_t tc_signed_pair(uint32_t u, uint32_t lev) {
  const uint32_t s = u << (15 - 2 * I);
  uint32_t r;
  // r = (~s & 0x80008000) ^ lev
  asm("lop3.b32 %0, %1, %2, %3, 0xA6;\n" : "=r"(r) : "r"(s), "r"(0x80008000u), "r"(lev));
  return r;
}

// Index words of 16 columns from two 16-bit planes (A: index bit 0, B:
// index bit 1): z[0] covers columns 0..7, z[1] columns 8..15 (layout above).
__device__ __forceinline__ void tc_index_words(uint32_t A, uint32_t B, uint32_t z[2]) {
  z[0] = ((A & 0x55u) << 1) | ((A & 0xAAu) << 8) | ((B & 0x55u) << 2) | ((B & 0xAAu) << 9);
  z[1] = ((A & 0x5500u) >> 7) | (A & 0xAA00u) | ((B & 0x5500u) >> 6) | ((B & 0xAA00u) << 1);
}

// prmt.b32 in its default mode, where bit 3 of a selector nibble replicates
// the sign (bit 7) of the selected byte (the __byte_perm intrinsic only
// honours the low three bits of each nibble).
__device__ __forceinline__ uint32_t tc_prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;\n" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}

// PRMT selector for column pair I from the index words.
template <int I>
__device__ __forceinline__ uint32_t tc_selector(const uint32_t z[2]) {
  const uint32_t v = (z[I >> 2] >> (2 * (I & 3))) & 0x0606u;
  return v * 0x11u + 0x1010u;
}

// Levels of one (row, group) from its K fp16 scales (kernel order), as fp32:
//   K = 1: v = {a0};
//   K = 2: v = {V0, V1, V2, V3}, V[b0 + 2 b1] = s0 a0 + s1 a1;
//   K = 3: v = {M0 .. M3}, M[t1 + 2 t2] = (a0 + s1 a1) + s2 a2;
//   K = 4: v = {M0 .. M7}, M[t1 + 2 t2 + 4 t3] = ((a0 + s1 a1) + s2 a2) + s3 a3.
template <int K>
__device__ __forceinline__ void tc_level_values(const unsigned char* alpha, int o, int i, float v[8]) {
  float a[K];
#pragma unroll
  for (int k = 0; k < K; ++k)
    a[k] = __half2float(__ushort_as_half(*reinterpret_cast<const uint16_t*>(alpha + (o * K + k) * 16 + 2 * i)));
  if (K == 1) {
    v[0] = a[0];
  } else if (K == 2) {
    const float d = a[0] - a[1], e = a[0] + a[1];
    v[0] = -e; v[1] = d; v[2] = -d; v[3] = e;
  } else {
    const float x = a[0] - a[1], y = a[0] + a[1];
    const float a2 = a[K > 2 ? 2 : 0];
    const float c0 = x - a2, c1 = y - a2, c2 = x + a2, c3 = y + a2;
    if (K == 3) {
      v[0] = c0; v[1] = c1; v[2] = c2; v[3] = c3;
    } else {
      const float a3 = a[K > 3 ? 3 : 0];
      v[0] = c0 - a3; v[1] = c1 - a3; v[2] = c2 - a3; v[3] = c3 - a3;
      v[4] = c0 + a3; v[5] = c1 + a3; v[6] = c2 + a3; v[7] = c3 + a3;
    }
  }
}

// The level registers of one (row, group): P holds the levels rounded once
// to bf16 (low half first; K = 1: (a0, a0)), and, for the split, L holds
// what that rounding left, v - RN_bf16(v) (exact in fp32), rounded to bf16.
// Rounding to nearest is sign-symmetric, so both stay exact negations of the
// complemented levels.
template <int K, bool SPLIT>
__device__ __forceinline__ void tc_levels(const unsigned char* alpha, int o, int i, uint32_t P[4], uint32_t L[4]) {
  float v[8];
  tc_level_values<K>(alpha, o, i, v);
  constexpr int kN = K == 1 ? 1 : (K == 4 ? 8 : 4);
  float hi[8], lo[8];
#pragma unroll
  for (int n = 0; n < kN; ++n) {
    hi[n] = __bfloat162float(__float2bfloat16_rn(v[n]));
    lo[n] = v[n] - hi[n];
  }
  if (K == 1) {
    P[0] = tc_pack_bf16x2(hi[0], hi[0]);
    if (SPLIT) L[0] = tc_pack_bf16x2(lo[0], lo[0]);
  } else {
#pragma unroll
    for (int n = 0; n < kN / 2; ++n) {
      P[n] = tc_pack_bf16x2(hi[2 * n], hi[2 * n + 1]);
      if (SPLIT) L[n] = tc_pack_bf16x2(lo[2 * n], lo[2 * n + 1]);
    }
  }
}

// One row x 16 columns: h[k] = the row's 16 bits of kernel k (column b in
// bit b), P = its levels; out[I] = bf16 pair of columns (2I, 2I+1).
template <int K>
__device__ __forceinline__ void tc_unpack_row(const uint32_t h[K], const uint32_t P[4], uint32_t out[8]) {
  const uint32_t u0 = h[0] | (h[0] << 15);
  if (K == 1) {
#define MBOK_PAIR(I) out[I] = tc_signed_pair<I>(u0, P[0]);
    MBOK_PAIR(0) MBOK_PAIR(1) MBOK_PAIR(2) MBOK_PAIR(3) MBOK_PAIR(4) MBOK_PAIR(5) MBOK_PAIR(6) MBOK_PAIR(7)
#undef MBOK_PAIR
  } else if (K == 2) {
    uint32_t z[2];
    tc_index_words(h[0], h[1], z);
#define MBOK_PAIR(I) out[I] = __byte_perm(P[0], P[1], tc_selector<I>(z));
    MBOK_PAIR(0) MBOK_PAIR(1) MBOK_PAIR(2) MBOK_PAIR(3) MBOK_PAIR(4) MBOK_PAIR(5) MBOK_PAIR(6) MBOK_PAIR(7)
#undef MBOK_PAIR
  } else {
    // t_k = XNOR(b_k, b_0): the bits relative to kernel 0 (only bits 0..15 are read)
    const uint32_t t1 = ~(h[1] ^ h[0]), t2 = ~(h[2 % K] ^ h[0]);
    uint32_t z[2];
    tc_index_words(t1, t2, z);
    if (K == 3) {
#define MBOK_PAIR(I) out[I] = tc_signed_pair<I>(u0, __byte_perm(P[0], P[1], tc_selector<I>(z)));
      MBOK_PAIR(0) MBOK_PAIR(1) MBOK_PAIR(2) MBOK_PAIR(3) MBOK_PAIR(4) MBOK_PAIR(5) MBOK_PAIR(6) MBOK_PAIR(7)
#undef MBOK_PAIR
    } else {
      const uint32_t t3 = ~(h[3 % K] ^ h[0]) & 0xFFFFu;
      const uint32_t u3 = t3 | (t3 << 15);
      // 16-bit masks from bit 15 / bit 31 of the shifted t3 word (sign-replicating permute)
#define MBOK_PAIR(I)                                                           \
  {                                                                            \
    const uint32_t sel = tc_selector<I>(z);                                    \
    const uint32_t lo = __byte_perm(P[0], P[1], sel);                          \
    const uint32_t hi = __byte_perm(P[2], P[3], sel);                          \
    const uint32_t m = tc_prmt(u3 << (15 - 2 * I), 0u, 0xBB99u);               \
    out[I] = tc_signed_pair<I>(u0, (hi & m) | (lo & ~m));                      \
  }
      MBOK_PAIR(0) MBOK_PAIR(1) MBOK_PAIR(2) MBOK_PAIR(3) MBOK_PAIR(4) MBOK_PAIR(5) MBOK_PAIR(6) MBOK_PAIR(7)
#undef MBOK_PAIR
    }
  }
}

// fp16 levels of one (row, group), each a quarter of the level rounded once:
// K fp16 scales sum to at most 4 x 65504, so a quarter never overflows, and a
// level above 2^-12 keeps fp16's 11 bits (smaller ones an absolute 2^-23).
// `zero`: a row that pads the last octet, whose stored scales mean nothing.
constexpr float kLevelScale = 0.25f;
template <int K>
__device__ __forceinline__ void tc_levels_f16(const unsigned char* alpha, int o, int i, bool zero, uint32_t P[4]) {
  float v[8];
  tc_level_values<K>(alpha, o, i, v);
  constexpr int kN = K == 1 ? 1 : (K == 4 ? 8 : 4);
  uint32_t h[8];
#pragma unroll
  for (int n = 0; n < kN; ++n) h[n] = zero ? 0u : uint32_t(__half_as_ushort(__float2half_rn(v[n] * kLevelScale)));
  if (K == 1) {
    P[0] = h[0] | (h[0] << 16);
  } else {
#pragma unroll
    for (int n = 0; n < kN / 2; ++n) P[n] = h[2 * n] | (h[2 * n + 1] << 16);
  }
}

}  // namespace mbok
