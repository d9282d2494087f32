// Products with Boolean weights on CTA pairs (tcgen05 cta_group::2), sm_100a:
//
//  * GATE:  H[t][r] = silu(G) * U,  G = W_gate X^T, U = W_up X^T  (gated
//    feed-forward block; G and U optionally stored for the backward pass);
//  * GRAD:  dX[t][j] = sum over matrices s and rows r of dY_s[t][r] W_s[r][j]
//    (the input gradient of layers that share X).
//
// W = sum_k alpha_k B_k (Paper-Notes page, 方法详解 / 关键设计) is unpacked tile
// by tile in shared memory right before the tensor cores read it, as in the
// prefill GEMM.  What is different:
//
//  * Unpacking bounds the prefill GEMM (its ALU work per weight is shared by
//    256 tokens).  Here a pair of CTAs forms one M = 256 product of up to 512
//    tokens: each CTA unpacks 128 rows of A per 64-deep stage and loads half of
//    the tokens, and the hardware reads both halves: a quarter of the unpacking
//    per product.  Up to 256 tokens, two accumulators alternate and a tile is
//    drained while the next is formed; 512 tokens take all of tensor memory, and
//    the MMAs pause for the drain.  The wider tile is still the faster one where
//    there are tokens for it: with 256 the unpack (about 700 cycles a stage at
//    K = 3 against 512 for the MMAs) and its power draw bound the kernel
//    (LLaMA-7B gate and up, 2048 tokens, input gradient: 451 us against 280).
//  * Levels are fp16, the activations scaled to fp16 per token (scale_rows.cu):
//    the weight's rounding is 2^-11 where bf16's is 2^-8, at the same rate.
//    The token's inverse scale is applied to the fp32 sums.
//  * GATE: a CTA's 128 A rows are 64 gate rows and the same 64 up rows, 16 of
//    each in turn, so that one warp's 32 tensor-memory lanes hold both
//    projections of 16 rows and one exchange across half a warp gates them.
//  * GRAD contracts over rows of W.  Its A is W^T: an unpacked row's 64 columns
//    are a 128-byte line with one k, the M-major form of the same swizzled
//    layout, so the unpack is the same and nothing is transposed.
//
// Per stage: TMA brings this CTA's half of the tokens, completing on the
// leader's `ready` barrier, and the tile's bits and scales, in a ring of their
// own that runs ahead; four unpack warps write A and arrive on the same barrier.
// (One barrier for both: with two, the issuing warp's waits and instructions
// bounded the stages.  16 unpack warps take stages in turn, in four groups: with
// all 16 on every stage the latency of wait, load, store, fence and arrival
// bounded each at about 1 us, whatever the tokens.)  The leader's MMA warp issues
// four tcgen05.mma (M = 256, N <= 256, K = 16) per accumulator and commits the
// stage to both CTAs' `empty` barriers.  Four epilogue warps, one per
// tensor-memory lane quarter, drain finished tiles; the unpack warps join them
// for a CTA's last tile and for every two-accumulator tile.
// Tiles that fill the last wave badly are dealt out as one run of stages, cut into
// equal parts wherever that falls: a pair may begin and end inside a tile, leaves
// such a tile's fp32 sums in the workspace, and a second kernel adds them in order
// (and gates).
// Every mbarrier wait is bounded (1 s): on timeout the CTA records an error
// flag, drains what it issued (bounded) and leaves with the other.
//
// Measured (LLaMA-7B gate and up, K = 3, 4096 columns, with the scaling pass):
//   GATE  2048 tokens 286 us = 1291 TFLOP/s in short runs, 332 us = 1112 under the
//         power limit of long ones (a plain bf16 GEMM of the library: 1632 and
//         1354); tensor pipe 64 % and ALU pipe 72 % busy.  K = 4: 366 to 375 us,
//         bound by the unpack.
//   GATE  256 tokens 62 us, 32 tokens 39 us (81 and 50 at the clocks that calls of
//         2048 tokens leave): the latency of a stage's unpack (32 tokens: ALU 63 %,
//         issue 58 %) and the pipeline's fill.
//   GRAD  2048 tokens 280 .. 300 us, 256 tokens 76 us.
#include "pair_ring.h"
#include "scale_rows.h"
#include "tc_pair.cuh"
#include "tc_unpack.cuh"

namespace mbok {

constexpr int kPairBK = 64;
constexpr int kPairRows = 128;                                // A rows per CTA
constexpr int kPairABytes = kPairRows * kPairBK * 2;          // 16 KB
constexpr int kPairOctets = 8;                                // row octets of a bits box (64 rows)
constexpr int kPairBits = 2 * kPairOctets * MBOK_MAX_K * 64;  // 4 KB: GATE two boxes of 64 bytes, GRAD one of 128
constexpr int kPairAlpha = 2 * kPairOctets * MBOK_MAX_K * 16; // 1 KB
constexpr int kPairWBytes = kPairBits + kPairAlpha;           // one slot of bits and scales
// Rings of A (16 KB a stage) and of this CTA's tokens (64 bytes per token of the
// tile): 4 slots of each for tiles of 512 tokens, 8 and 4 for 256, 8 and 8 from
// 128 down.  With a matrix of four kernels, whose unpack bounds the stages, 6 and
// 3 for 512: 392 -> 373 us (K = 4, 11008 x 2 x 4096, 2048 tokens), where K = 3
// goes 288 -> 295, its tokens arriving late.
// Slots of bits and scales: 6 to 8 (kPairMaxSlots, pair_ring.h).
constexpr int kPairRing = 192 * 1024;
constexpr int kPairBarriers = 512;
constexpr int kPairSmemMax = 226 * 1024;   // of 227 KB, some of it static
constexpr int kPairRings = kPairSmemMax - 1024 - kPairBarriers;
constexpr int kPairGroupWarps = 4;                            // 128 unpack threads per stage
constexpr int kPairUnpackWarps = kPairGroups * kPairGroupWarps;
constexpr int kPairUnpackWarp0 = 3;                           // after the two copy warps and the MMA warp
constexpr int kPairEpiWarp0 = kPairUnpackWarp0 + kPairUnpackWarps;
constexpr int kPairThreads = (kPairEpiWarp0 + 4) * 32;
constexpr unsigned kPairTmemCols = 512;                       // accumulators at columns 0 and 256
constexpr int kPairSums = 2 * kPairRows;                      // sums per token and tile: GATE 128 rows of gate, of up

static __device__ unsigned int g_pair_error;

enum PairMode { kGate, kGrad };

struct PairMat {
  int K, M;
  int stages;   // GRAD: 64-row steps of this matrix
};

struct PairMaps {
  CUtensorMap bits[kMaxMats], alpha[kMaxMats];   // GATE: gate, up
  CUtensorMap act[kMaxMats];                     // GATE: one; GRAD: dY of each matrix
};

struct PairMul {
  uint32_t pow2[8];   // 2^(15 - 2i)
};

struct PairParams {
  PairMat mat[kMaxMats];
  int nmat;
  int M, N, T;
  int n;               // tokens per tile
  int naccs, n_acc;    // accumulators per tile (1 or 2) and tokens in each (multiple of 16, <= 256)
  int slots, xslots, wslots;   // ring slots of A, of tokens, of bits and scales
  int all_drain;       // the unpack warps share in every drain (always with two accumulators)
  int stages;          // per tile
  int row_tiles;       // tiles along W's rows (GATE, 128) or columns (GRAD, 256)
  int ntiles;
  int workers;         // 0: pairs take whole tiles in turn; else the stages of all tiles are cut into this many runs,
  int run, run_rest;   // of `run` + run_rest / workers stages
  uint32_t idesc;
  PairMul mul;
  const float* inverse;   // [T rounded up to 16]
  uint16_t* out;          // H, or dX
  uint16_t* gate;         // GATE: [T][M] or nullptr
  uint16_t* up;
  float* partial;         // sums of tiles that a run begins or ends in: [run][first, last][n tokens][kPairSums]
};

// First stage of run w: w / workers of the stages of all tiles, rounded down.
__device__ __forceinline__ int run_begin(const PairParams& p, int w) {
  return w * p.run + int(unsigned(w * p.run_rest) / unsigned(p.workers));
}

// A pair's items: tiles tile0, tile0 + step, ..., the first from stage k_first,
// the last up to k_last.  (Whole tiles: row tiles vary fastest, so that pairs that
// run together share their tokens.)
struct PairWalk {
  int n, tile0, step, k_first, k_last;
};
struct PairItem {
  int tile, k0, k1;
  int slot;   // of `partial`, or -1: a whole tile
};
__device__ __forceinline__ PairWalk pair_walk(const PairParams& p, int pair, int npairs) {
  PairWalk w;
  if (p.workers == 0) {
    w.n = (p.ntiles - 1 - pair) / npairs + 1;   // at least one
    w.tile0 = pair;
    w.step = npairs;
    w.k_first = 0;
    w.k_last = p.stages;
  } else {
    const int b = run_begin(p, pair), e = run_begin(p, pair + 1);
    w.tile0 = b / p.stages;
    const int last = (e - 1) / p.stages;
    w.n = last - w.tile0 + 1;
    w.step = 1;
    w.k_first = b - w.tile0 * p.stages;
    w.k_last = e - last * p.stages;
  }
  return w;
}
__device__ __forceinline__ PairItem pair_item(const PairParams& p, const PairWalk& w, int pair, int i) {
  PairItem it;
  it.tile = w.tile0 + i * w.step;
  it.k0 = i == 0 ? w.k_first : 0;
  it.k1 = i + 1 == w.n ? w.k_last : p.stages;
  it.slot = it.k1 - it.k0 == p.stages ? -1 : 2 * pair + (i > 0 ? 1 : 0);
  return it;
}

// ---- unpack ----
//
// As tc_unpack_row (an element is the level its K bits select), arranged for
// the two integer pipes: the logic pipe (half rate) bounds the unpack, so
// shifts are multiplications by powers of two on the FMA pipe where they can be
// (factors from the kernel parameters, or the compiler would make them shifts
// again), and one selector word serves two column pairs.
//  * Index word: even columns' index bits (A, B) interleave into P, odd columns'
//    into Q, and z = bytes P0 Q0 P1 Q1, so that byte 2h + e holds the 2-bit
//    indices of the even (e = 0) or odd columns 8h .. 8h + 7.  For p < 4,
//    ((z >> 2p) & 0x03030303) * 0x22 + 0x10101010 is the byte-permute selector of
//    column pair p in its low half and of pair p + 4 in its high half.
//  * Sign word: bit c of the row at bit c (c < 15) and at bit 15 + c; times
//    2^(15 - 2i) it has the signs of columns 2i and 2i + 1 at bits 15 and 31.
// 34 logic operations per 16 columns at K = 3 against 54.

__device__ __forceinline__ uint32_t pair_index_word(uint32_t A, uint32_t B) {
  const uint32_t P = (A & 0x5555u) | ((B + B) & 0xAAAAu);
  const uint32_t Q = ((A >> 1) & 0x5555u) | (B & 0xAAAAu);
  return __byte_perm(P, Q, 0x5140);
}

// lev with each half's sign flipped where the bit of kernel 0 is clear; u = the
// sign word times 2^(15 - 2i).
__device__ __forceinline__ uint32_t pair_sign(uint32_t u, uint32_t lev) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xA6;\n" : "=r"(r) : "r"(u), "r"(0x80008000u), "r"(lev));   // (~u & m) ^ lev
  return r;
}

template <int K>
__device__ __forceinline__ void pair_unpack_row(const uint32_t h[K], const uint32_t P[4], const PairMul& mul,
                                                uint32_t out[8]) {
  const uint32_t u0 = h[0] * 32768u + (h[0] & 0x7FFFu);
  if (K == 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = pair_sign(u0 * mul.pow2[i], P[0]);
    return;
  }
  // K = 2: the index is the two bits; K >= 3: the bits relative to kernel 0
  const uint32_t A = K == 2 ? h[0] : ~(h[1 % K] ^ h[0]), B = K == 2 ? h[1 % K] : ~(h[2 % K] ^ h[0]);
  const uint32_t z = pair_index_word(A, B);
  uint32_t u3 = 0;
  if (K == 4) {
    const uint32_t t3 = ~(h[3 % K] ^ h[0]);
    u3 = (t3 & 0xFFFFu) * 32768u + (t3 & 0x7FFFu);
  }
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const uint32_t two = ((z >> (2 * p)) & 0x03030303u) * 0x22u + 0x10101010u;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = p + 4 * e;
      const uint32_t sel = e == 0 ? two : two >> 16;
      uint32_t lev = __byte_perm(P[0], P[1], sel);
      if (K == 4) {
        const uint32_t up = __byte_perm(P[2], P[3], sel);
        const uint32_t m = tc_prmt(u3 * mul.pow2[i], 0u, 0xBB99u);   // 16-bit masks from bits 15 and 31
        lev = (up & m) | (lev & ~m);
      }
      out[i] = K == 2 ? lev : pair_sign(u0 * mul.pow2[i], lev);
    }
  }
}

// Four units (64 columns) of one row: the row's bits of kernel k and unit u at
// src + k * kstride + u * 16, to the eight swizzled 16-byte chunks of `line`.
// Units are taken in the order u ^ flip.
template <int K>
__device__ __forceinline__ void pair_unpack(const unsigned char* src, int kstride, const uint32_t P[4],
                                            const PairMul& mul, unsigned char* line, int r, int flip) {
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const int u = n ^ flip;
    uint32_t h[K], out[8];
#pragma unroll
    for (int k = 0; k < K; ++k) h[k] = *reinterpret_cast<const uint16_t*>(src + k * kstride + u * 16);
    pair_unpack_row<K>(h, P, mul, out);
    const int c0 = (2 * u) ^ (r & 7), c1 = (2 * u + 1) ^ (r & 7);
    *reinterpret_cast<uint4*>(line + c0 * 16) = make_uint4(out[0], out[1], out[2], out[3]);
    *reinterpret_cast<uint4*>(line + c1 * 16) = make_uint4(out[4], out[5], out[6], out[7]);
  }
}

// GATE: thread gt of a group's 128 unpacks one A row's 64 columns; threads
// 0..63 the gate matrix's rows of this tile, 64..127 the up matrix's.  Row m of
// a matrix is A row 32 (m / 16) + m % 16, + 16 for up.  Eight lanes that store
// together hold eight consecutive rows: distinct chunks.
template <int K>
__device__ __forceinline__ void unpack_gate(const unsigned char* w, unsigned char* a, const PairMul& mul, int gt) {
  const int up = gt >> 6, m = gt & 63;
  const int o = m >> 3, i = m & 7;
  const int r = 32 * (m >> 4) + 16 * up + (m & 15);
  uint32_t P[4];
  tc_levels_f16<K>(w + kPairBits + up * (kPairAlpha / 2), o, i, false, P);
  pair_unpack<K>(w + up * (kPairBits / 2) + o * K * 64 + 2 * i, 64, P, mul, a + r * 128, r, 0);
}

// GRAD: thread gt of a group's 128 unpacks block gt & 1 (64 columns) of row
// gt >> 1 of the stage's 64 rows.  Eight lanes that store together hold four
// rows of both blocks; the second block's units go in the order 2, 3, 0, 1, so
// that its chunks differ from the first's.  Rows at or beyond M are zeros:
// their stored scales mean nothing and could be NaN.
template <int K>
__device__ __forceinline__ void unpack_grad(const unsigned char* w, unsigned char* a, const PairMul& mul, int gt,
                                            int rows) {
  const int r = gt >> 1, b = gt & 1;
  const int o = r >> 3, i = r & 7;
  uint32_t P[4];
  tc_levels_f16<K>(w + kPairBits, o, i, r >= rows, P);
  pair_unpack<K>(w + o * K * 128 + b * 64 + 2 * i, 128, P, mul,
                 a + b * 8192 + r * 128, r, 2 * b);
}

// 16 accumulator columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t v[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
}

// Store n values that this lane holds for row r at tokens t .. t + n - 1 of out
// [T][ld].  With `pairs` (ld even, out 4-byte aligned) lanes 2i and 2i + 1, which
// hold rows r and r + 1, exchange halves: the even lane stores both rows of the
// first n / 2 tokens, the odd lane of the others, as bf16 pairs.
template <int n>
__device__ __forceinline__ void store_rows(bool pairs, uint16_t* out, int ld, int rows, int T, int r, int t,
                                           const float* v, int lane) {
  if (pairs) {
    const bool odd = lane & 1;
    const int r0 = r & ~1, tt = t + (odd ? n / 2 : 0);
    const int live = r0 < rows ? T - tt : 0;   // tokens to store
    uint16_t* at = out + size_t(tt) * ld + r0;
#pragma unroll
    for (int i = 0; i < n / 2; ++i, at += ld) {
      const float other = __shfl_xor_sync(0xffffffffu, odd ? v[i] : v[n / 2 + i], 1);
      const uint32_t two = odd ? tc_pack_bf16x2(other, v[n / 2 + i]) : tc_pack_bf16x2(v[i], other);
      if (i < live) *reinterpret_cast<uint32_t*>(at) = two;
    }
  } else {
    const int live = r < rows ? T - t : 0;
    uint16_t* at = out + size_t(t) * ld + r;
#pragma unroll
    for (int i = 0; i < n; ++i, at += ld)
      if (i < live) *at = __bfloat16_as_ushort(__float2bfloat16_rn(v[i]));
  }
}

// silu(g) u for a bf16 result: g u / (1 + 2^(-g log2 e)) by the approximate
// exponential and reciprocal, a few 2^-22 of the value (and |g| 2^-23), far below
// its step.  Their forms that flush subnormals (the sigmoid's below g = -87 is 0)
// need no range checks: 6 instructions a value, of which a drain has eight per
// lane and 16 tokens.
__device__ __forceinline__ float gated_fast(float g, float u) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(e) : "f"(g * -1.44269504f));
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(1.f + e));
  return g * r * u;
}

// Drain one warp's share of a finished tile whose first accumulator is at
// `tmem`: lane quarter q, chunks of 16 tokens first, first + stride, ...
template <PairMode MODE>
__device__ __forceinline__ void pair_drain(const PairParams& p, uint32_t tmem, const PairItem& it, int rank, int q,
                                           int lane, int first, int stride) {
  const int per = p.n_acc / 16;
  const int t0 = (it.tile / p.row_tiles) * p.n;
  const int rt = it.tile % p.row_tiles;
  const int rows = MODE == kGate ? p.M : p.N;
  const bool pairs = rows % 2 == 0;   // every buffer is 16-byte aligned
  const int r = MODE == kGate ? rt * 128 + rank * 64 + 16 * q + (lane & 15) : rt * 256 + rank * 128 + 32 * q + lane;
  for (int j = first; j < per * p.naccs; j += stride) {
    const int t = t0 + 16 * j;
    if (t >= p.T) break;
    const int col = j < per ? 16 * j : 256 + 16 * (j - per);
    uint32_t w[16];
    tmem_ld16(tmem + (uint32_t(32 * q) << 16) + uint32_t(col), w);
    float v[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 s = *(reinterpret_cast<const float4*>(p.inverse + t) + i);
      v[4 * i] = __uint_as_float(w[4 * i]) * s.x;
      v[4 * i + 1] = __uint_as_float(w[4 * i + 1]) * s.y;
      v[4 * i + 2] = __uint_as_float(w[4 * i + 2]) * s.z;
      v[4 * i + 3] = __uint_as_float(w[4 * i + 3]) * s.w;
    }
    if (it.slot >= 0) {
      float* at = p.partial + (size_t(it.slot) * p.n + 16 * j) * kPairSums +
                  (MODE == kGate ? 128 * (lane >> 4) + rank * 64 + 16 * q + (lane & 15) : rank * 128 + 32 * q + lane);
#pragma unroll
      for (int i = 0; i < 16; ++i) __stcg(at + i * kPairSums, v[i]);
    } else if (MODE == kGrad) {
      store_rows<16>(pairs, p.out, rows, rows, p.T, r, t, v, lane);
    } else {
      const bool low = lane < 16;
      if (p.gate != nullptr) store_rows<16>(pairs, low ? p.gate : p.up, rows, rows, p.T, r, t, v, lane);
      // lanes l and l + 16 hold gate and up of one row: after the exchange the
      // lower lane has both for tokens t .. t + 7, the upper for t + 8 ..
      float h[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float other = __shfl_xor_sync(0xffffffffu, low ? v[8 + i] : v[i], 16);
        h[i] = gated_fast(low ? v[i] : other, low ? other : v[8 + i]);
      }
      store_rows<8>(pairs, p.out, rows, rows, p.T, r, low ? t : t + 8, h, lane);
    }
  }
}

template <PairMode MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
gemm_pair_kernel(const __grid_constant__ PairMaps maps, const __grid_constant__ PairParams p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int x_bytes = p.n_acc / 2 * 128;                    // this CTA's tokens of one accumulator
  const int xslot_bytes = p.naccs * x_bytes;
  unsigned char* xring = smem + p.slots * kPairABytes;
  unsigned char* wring = xring + p.xslots * xslot_bytes;
  uint64_t* wfull = reinterpret_cast<uint64_t*>(wring + p.wslots * kPairWBytes);   // a stage's bits and scales landed
  uint64_t* wempty = wfull + kPairMaxSlots;   // ... and unpacked (both by pair_bits_barrier)
  uint64_t* ready = wempty + kPairMaxSlots;   // leader: both CTAs' tokens landed and their A is unpacked
  uint64_t* empty = ready + kPairMaxSlots;    // the stage's MMAs are done (both CTAs)
  uint64_t* tfull = empty + kPairMaxSlots;    // accumulator b holds a finished tile (both CTAs)
  uint64_t* last_full = tfull + 2;            // the CTA's last tile is finished (completes once; both CTAs)
  uint64_t* tempty = last_full + 1;           // leader: both CTAs drained accumulator b
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);
  __shared__ int s_fail;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = int(pair_rank());
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const PairWalk walk = pair_walk(p, pair, npairs);
  const int n_mine = walk.n;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairMaxSlots; ++s) {
      tc_mbar_init(&wfull[s], 1);
      tc_mbar_init(&wempty[s], kPairGroupWarps);
      tc_mbar_init(&ready[s], 2 * kPairGroupWarps + 1);   // + the leader's expectation of the tokens
      tc_mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc_mbar_init(&tfull[b], 1);
      tc_mbar_init(&tempty[b], 2 * (p.all_drain ? 4 + kPairUnpackWarps : 4));
    }
    tc_mbar_init(last_full, 1);
    s_fail = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
  }
  __syncwarp();
  if (warp == 1) pair_alloc(tmem_slot, kPairTmemCols);
  tc_fence_before();
  pair_sync();   // both CTAs run and their barriers are set up
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  bool ok = true;
  // This grid starts once every CTA of the scaling pass is past its own wait: all
  // that came before that pass is complete, the weights among it, and their copies
  // and unpack run beside it.  Tokens and what is read with the outputs wait for
  // its end (three matrices, 130 and 382 tokens: 12.8 -> 11.7, 48 -> 45 us).

  // Every role walks the stages of all its tiles with a slot index and the
  // parity of the slot's current use.
  if (warp == 0) {
    // ---- token copies ----
    if (elect_lane())
      for (int m = 0; m < (MODE == kGate ? 1 : p.nmat); ++m) prefetch_map(&maps.act[m]);
    pdl_wait();
    // The scale gradients' kernel that may follow reads the scaling pass's copies
    // and nothing that this one writes: it may start on idle SMs.
    pdl_launch();
    const unsigned bytes = unsigned(p.n * kPairBK * 2);   // both CTAs'
    // A stage's tokens arrive on the barrier of its A slot, and their slot is free
    // once the stage xslots before is done (there are at least as many A slots, so
    // that this stage's barrier is then through with its previous use).
    int s = 0, xs = 0, es = 0, g = 0;   // A slot, token slot, A slot of stage g - xslots
    unsigned eph = 0;
    for (int i = 0; i < n_mine && ok; ++i) {
      const PairItem it = pair_item(p, walk, pair, i);
      const int t0 = (it.tile / p.row_tiles) * p.n + rank * (p.n_acc / 2);
      int m = 0, step = it.k0;   // GRAD: matrix and its 64-row step
      if (MODE == kGrad)
        while (step >= p.mat[m].stages) step -= p.mat[m++].stages;
      for (int kb = it.k0; kb < it.k1; ++kb, ++g) {
        if (g >= p.xslots) {
          if (!pair_wait(&empty[es], eph)) { ok = false; break; }
          if (++es == p.slots) { es = 0; eph ^= 1u; }
        }
        const uint32_t bar = pair_leader(&ready[s]);
        const CUtensorMap* map = &maps.act[MODE == kGate ? 0 : m];
        if (elect_lane()) {
          if (rank == 0) tc_arrive_expect_tx(&ready[s], bytes);
          unsigned char* x = xring + xs * xslot_bytes;
          const int k0 = (MODE == kGate ? kb : step) * kPairBK;
          pair_tma_load_2d(x, map, k0, t0, bar);
          if (p.naccs > 1) pair_tma_load_2d(x + x_bytes, map, k0, t0 + p.n_acc, bar);
        }
        __syncwarp();
        if (MODE == kGrad && ++step == p.mat[m].stages) { step = 0; ++m; }
        if (++s == p.slots) s = 0;
        if (++xs == p.xslots) xs = 0;
      }
    }
  } else if (warp == 2) {
    // ---- copies of bits and scales ----
    int s = 0, g = 0;
    for (int i = 0; i < n_mine && ok; ++i) {
      const PairItem it = pair_item(p, walk, pair, i);
      const int rt = it.tile % p.row_tiles;
      int m = 0, step = it.k0;
      if (MODE == kGrad)
        while (step >= p.mat[m].stages) step -= p.mat[m++].stages;
      for (int kb = it.k0; kb < it.k1; ++kb, ++g) {
        // the slot's last stage is unpacked
        const int last = g - p.wslots;
        if (last >= 0 && !pair_wait(&wempty[pair_bits_barrier(last)], pair_bits_parity(last))) { ok = false; break; }
        unsigned char* w = wring + s * kPairWBytes;
        uint64_t* full = &wfull[pair_bits_barrier(g)];
        if (MODE == kGate) {
          const int o = (rt * 128 + rank * 64) / kOctet;
          if (elect_lane()) {
            tc_arrive_expect_tx(full, unsigned(p.mat[0].K + p.mat[1].K) * kPairOctets * (64 + 16));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int K = p.mat[i].K;
              tc_tma_load_2d(w + i * (kPairBits / 2), &maps.bits[i], kb * 64, o * K, full);
              tc_tma_load_2d(w + kPairBits + i * (kPairAlpha / 2), &maps.alpha[i], (kb / 2) * K * kOctet, o, full);
            }
          }
        } else {
          const int K = p.mat[m].K;
          const int j = rt * 256 + rank * 128;
          if (elect_lane()) {
            tc_arrive_expect_tx(full, unsigned(K) * kPairOctets * (128 + 16));
            tc_tma_load_2d(w, &maps.bits[m], j, step * kPairOctets * K, full);
            tc_tma_load_2d(w + kPairBits, &maps.alpha[m], (j / kGroup) * K * kOctet, step * kPairOctets, full);
          }
          if (++step == p.mat[m].stages) { step = 0; ++m; }
        }
        __syncwarp();
        if (++s == p.wslots) s = 0;
      }
    }
  } else if (warp == 1) {
    // ---- MMA issuer: the leader's, for both CTAs ----
    if (rank == 0) {
      constexpr int kAStep = MODE == kGate ? 32 >> 4 : 2048 >> 4;   // 16 k further in A
      const uint32_t base = tc_smem(smem);
      const uint64_t a0 = MODE == kGate ? tc_desc_sw128(base) : tc_desc_sw128_mn(base, 8192);
      const uint64_t x0 = tc_desc_sw128(tc_smem(xring));
      int s = 0, xs = 0;
      unsigned ph = 0;
      for (int i = 0; i < n_mine && ok; ++i) {
        // one accumulator per tile: tiles alternate between two; else all tiles use both
        const int b = p.naccs > 1 ? 0 : i & 1, use = p.naccs > 1 ? i : i >> 1;
        if (use > 0 && !pair_wait(&tempty[b], unsigned(use - 1) & 1u)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d = tmem + uint32_t(b * 256);
        const PairItem it = pair_item(p, walk, pair, i);
        for (int kb = it.k0; kb < it.k1; ++kb) {
          if (!pair_wait(&ready[s], ph)) { ok = false; break; }
          tc_fence_after();
          const uint64_t aoff = uint64_t((s * kPairABytes) >> 4), xoff = uint64_t((xs * xslot_bytes) >> 4);
          if (elect_lane()) {
#pragma unroll
            for (int kk = 0; kk < kPairBK / 16; ++kk) {
              const uint64_t ad = a0 + aoff + uint64_t(kk * kAStep), xd = x0 + xoff + uint64_t(kk * (32 >> 4));
              const uint32_t acc = (kb > it.k0 || kk > 0) ? 1u : 0u;
              pair_mma(d, ad, xd, p.idesc, acc);
              if (p.naccs > 1) pair_mma(d + 256, ad, xd + uint64_t(x_bytes >> 4), p.idesc, acc);
            }
            pair_commit(&empty[s]);
            if (kb + 1 == it.k1) {
              pair_commit(&tfull[b]);
              if (i + 1 == n_mine) pair_commit(last_full);
            }
          }
          __syncwarp();
          if (++s == p.slots) { s = 0; ph ^= 1u; }
          if (++xs == p.xslots) xs = 0;
        }
      }
    }
  } else if (warp < kPairEpiWarp0) {
    // ---- unpack warps: group `grp` takes every fourth stage ----
    const int grp = (warp - kPairUnpackWarp0) / kPairGroupWarps;
    const int gt = threadIdx.x - (kPairUnpackWarp0 + grp * kPairGroupWarps) * 32;
    int s = grp, ws = grp, g = grp, first = grp;   // both rings have at least kPairGroups slots
    unsigned ph = 0;
    for (int i = 0; i < n_mine && ok; ++i) {
      const PairItem it = pair_item(p, walk, pair, i);
      int m = 0, kb = it.k0 + first, step = kb;
      for (; kb < it.k1; kb += kPairGroups, step += kPairGroups, g += kPairGroups) {
        const unsigned char* w = wring + ws * kPairWBytes;
        unsigned char* a = smem + s * kPairABytes;
        // the bits are there, and the slot's previous MMAs are done with its A
        if (!pair_wait(&wfull[pair_bits_barrier(g)], pair_bits_parity(g)) ||
            (g >= p.slots && !pair_wait(&empty[s], ph ^ 1u))) {
          ok = false;
          break;
        }
        if (MODE == kGate) {
          switch (p.mat[gt >> 6].K) {   // the same for a whole warp
            case 1: unpack_gate<1>(w, a, p.mul, gt); break;
            case 2: unpack_gate<2>(w, a, p.mul, gt); break;
            case 3: unpack_gate<3>(w, a, p.mul, gt); break;
            default: unpack_gate<4>(w, a, p.mul, gt); break;
          }
        } else {
          while (step >= p.mat[m].stages) step -= p.mat[m++].stages;
          const int rows = p.mat[m].M - step * kPairBK;
          switch (p.mat[m].K) {
            case 1: unpack_grad<1>(w, a, p.mul, gt, rows); break;
            case 2: unpack_grad<2>(w, a, p.mul, gt, rows); break;
            case 3: unpack_grad<3>(w, a, p.mul, gt, rows); break;
            default: unpack_grad<4>(w, a, p.mul, gt, rows); break;
          }
        }
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");   // generic writes -> tensor core reads
        __syncwarp();
        if (lane == 0) {
          pair_arrive(pair_leader(&ready[s]));
          tc_arrive(&wempty[pair_bits_barrier(g)]);
        }
        if ((s += kPairGroups) >= p.slots) { s -= p.slots; ph ^= 1u; }
        if ((ws += kPairGroups) >= p.wslots) ws -= p.wslots;
      }
      first = kb - it.k1;   // this group's first stage of the next item
      if (!ok) break;
      // Two accumulators: a tile is drained by all warps before the next begins.
      // One, and few stages per tile: behind the next tile's stages.  One, and
      // many stages: only the last tile, on a barrier that completes once (a
      // parity wait on tfull from here could pass on an earlier phase, since these
      // warps do not wait for every tile).
      const bool last = i + 1 == n_mine;
      const int d0 = p.naccs > 1 || (last && !p.all_drain) ? i : p.all_drain ? max(i - 1, 0) : i + 1;
      const int d1 = p.naccs > 1 || last ? i : i - 1;
      if (d0 <= d1) pdl_wait();   // the tokens' scales
      for (int j = d0; j <= d1 && ok; ++j) {
        const int b = p.naccs > 1 ? 0 : j & 1, use = p.naccs > 1 ? j : j >> 1;
        if (!(p.all_drain ? pair_wait(&tfull[b], unsigned(use) & 1u) : pair_wait(last_full, 0u))) { ok = false; break; }
        tc_fence_after();
        pair_drain<MODE>(p, tmem + uint32_t(b * 256), pair_item(p, walk, pair, j), rank, warp & 3, lane,
                         1 + (warp - kPairUnpackWarp0) / 4, 1 + kPairUnpackWarps / 4);
        tc_fence_before();
        __syncwarp();
        if (p.all_drain && lane == 0) pair_arrive(pair_leader(&tempty[b]));
      }
    }
  } else {
    // ---- epilogue: lane quarter warp & 3 ----
    pdl_wait();   // the tokens' scales
    for (int i = 0; i < n_mine; ++i) {
      const int b = p.naccs > 1 ? 0 : i & 1, use = p.naccs > 1 ? i : i >> 1;
      if (!pair_wait(&tfull[b], unsigned(use) & 1u)) { ok = false; break; }
      tc_fence_after();
      const bool shared = p.all_drain || i + 1 == n_mine;   // with the unpack warps: every fifth chunk
      pair_drain<MODE>(p, tmem + uint32_t(b * 256), pair_item(p, walk, pair, i), rank, warp & 3, lane, 0,
                       shared ? 1 + kPairUnpackWarps / 4 : 1);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) pair_arrive(pair_leader(&tempty[b]));
    }
  }

  if (!ok) atomicOr(&s_fail, 1);
  tc_fence_before();
  __syncthreads();
  if (s_fail != 0 && threadIdx.x == 0) {
    atomicOr(&g_pair_error, 1u);
    // copies and MMAs in flight: every barrier but tempty
    tc_drain_barriers(wfull, 4 * kPairMaxSlots + 3);
  }
  __syncthreads();
  __syncwarp();
  pair_sync();   // neither CTA leaves while the other's MMAs or arrivals may reach it
  if (warp == 1) {
    tc_fence_after();
    pair_dealloc(tmem, kPairTmemCols);
  }
}

// dX, or H (and G and U), of the tiles that runs share: block y is the cut at the
// start of run y + 1, and takes the tile that this is the first cut of.  A thread
// adds 4 rows of one token, in the order of the runs.
template <PairMode MODE>
__global__ void __launch_bounds__(256) pair_join_kernel(const __grid_constant__ PairParams p) {
  pdl_launch();
  pdl_wait();
  const int w0 = blockIdx.y, cut = run_begin(p, w0 + 1);
  const int tile = cut / p.stages, begin = tile * p.stages, end = begin + p.stages;
  const int b0 = run_begin(p, w0);
  if (cut == begin || b0 > begin) return;
  int w1 = w0 + 1;   // the tile's last run
  while (run_begin(p, w1 + 1) < end) ++w1;
  constexpr int kRows = MODE == kGate ? kPairSums / 2 : kPairSums;   // of the tile
  constexpr int kPlanes = kPairSums / kRows;
  const int i = blockIdx.x * 256 + threadIdx.x;
  const int tok = i / (kRows / 4), row = i % (kRows / 4) * 4;
  const int t = tile / p.row_tiles * p.n + tok, r = tile % p.row_tiles * kRows + row;
  const int rows = MODE == kGate ? p.M : p.N;
  if (tok >= p.n || t >= p.T || r >= rows) return;
  float sum[kPlanes][4] = {};
  const size_t slot = size_t(p.n) * kPairSums, at = size_t(tok) * kPairSums + row;
  // run w0 ends in this tile (its first tile or a later one), the others begin in it
  const float* first = p.partial + (2 * w0 + (b0 < begin ? 1 : 0)) * slot + at;
  const float* other = p.partial + 2 * w0 * slot + at;
#pragma unroll 4
  for (int w = 0; w <= w1 - w0; ++w) {
    const float* src = w == 0 ? first : other + 2 * w * slot;
#pragma unroll
    for (int m = 0; m < kPlanes; ++m) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(src + m * kRows));
      sum[m][0] += v.x; sum[m][1] += v.y; sum[m][2] += v.z; sum[m][3] += v.w;
    }
  }
  const bool vec = rows % 4 == 0;   // 8-byte aligned, and all four rows there
  auto store = [&](uint16_t* to, const float* v) {
    to += size_t(t) * rows + r;
    if (vec) {
      *reinterpret_cast<uint2*>(to) = make_uint2(tc_pack_bf16x2(v[0], v[1]), tc_pack_bf16x2(v[2], v[3]));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (r + e < rows) to[e] = __bfloat16_as_ushort(__float2bfloat16_rn(v[e]));
    }
  };
  if (MODE == kGrad) {
    store(p.out, sum[0]);
  } else {
    if (p.gate != nullptr) {
      store(p.gate, sum[0]);
      store(p.up, sum[kPlanes - 1]);
    }
    float h[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = gated_fast(sum[0][e], sum[kPlanes - 1][e]);
    store(p.out, h);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

unsigned gemm_pair_error_flags() {
  unsigned v = 0;
  if (cudaMemcpyFromSymbol(&v, g_pair_error, sizeof(v)) != cudaSuccess) return ~0u;
  const unsigned z = 0;
  if (v != 0 && cudaMemcpyToSymbol(g_pair_error, &z, sizeof(z)) != cudaSuccess) return ~0u;
  return v;
}

// Pairs that the device runs at once (queried once per device).
template <PairMode MODE>
static int pair_count() {
  const void* fn = reinterpret_cast<const void*>(gemm_pair_kernel<MODE>);
  static PerDeviceOnce attr_once;
  if (set_smem_attr_once(attr_once, fn, kPairSmemMax) != cudaSuccess) return 0;
  static PerDeviceValue<int> cache;
  return cache.get(current_device(), [fn]() -> int {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kPairThreads);
    cfg.dynamicSmemBytes = kPairSmemMax;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    return cudaOccupancyMaxActiveClusters(&n, fn, &cfg) == cudaSuccess ? n : 0;
  });
}

// Tokens per tile, and runs of stages (0: whole tiles).
struct PairPlan {
  int n, workers;
};

// The tile width (a multiple of 32, at most 512) and the cut that minimise the
// time of kPlanPairs pairs (the plan does not ask the device, so that a
// workspace's size does not depend on it).  In units of one token's MMAs of a
// stage (about 1.1 ns): a stage costs its tokens, and at least the unpack of its
// weights (320 tokens' worth); a launch adds its pipeline's fill (4 stages), an
// item what of its drain is not hidden (1 stage, 12 with two accumulators); runs
// add their sums' way through memory (at 4 TB/s) and a launch (4 us).  Runs that
// cut every tile alike leave one part each, others up to two.  Uncut and cut: dX
// of 9998 x 896, K = 2, 32 tokens 67 and 25 us; gate and up of LLaMA-7B, 32 tokens
// 73 and 52 us, their dX for 256 tokens 185 and 67 us.
constexpr int kPlanPairs = 74;
constexpr int kPairMinRun = 4;   // stages
// With fewer stages per tile than this the four epilogue warps do not keep up
// with one accumulator, and the unpack warps drain too (1818 tokens, 2400 rows, N
// = 128 and 512: 34 -> 21, 37 -> 24 us; at 16 and more no difference).
constexpr int kPairFewStages = 16;
static PairPlan pair_plan(int row_tiles, int stages, int T) {
  PairPlan best = {512, 0};
  double best_cost = -1;
  const int most = T >= 512 ? 512 : (T + 31) / 32 * 32;
  static const int kWidths[] = {512, 448, 416, 384, 352, 320, 288, 256, 224, 192, 160, 128, 96, 64, 32};
  for (const int n : kWidths) {
    if (n > most) continue;
    const long tiles = long(row_tiles) * ((T + n - 1) / n);
    const double stage = n > 320 ? n : 320, drain = n > 256 ? 12 : 1;
    auto consider = [&](double cost, int workers) {
      if (best_cost >= 0 && cost >= best_cost) return;
      best_cost = cost;
      best.n = n;
      best.workers = workers;
    };
    consider(stage * (double((tiles + kPlanPairs - 1) / kPlanPairs) * (stages + drain) + 4), 0);
    if (tiles > 8 * kPlanPairs) continue;
    auto cut = [&](int workers) {
      const double run = double(tiles) * stages / workers;
      if (workers < 2 || run < kPairMinRun) return;
      const double parts = workers % tiles == 0 ? workers : (workers < tiles ? 2.0 * workers : double(workers + tiles));
      const double items = workers % tiles == 0 ? 1 : 2 + double(int(run / stages));
      consider(stage * (run + items * drain + 4) + (parts * n * kPairSums * 8 / 4000.0 + 4000.0) / 1.1, workers);
    };
    for (int k = 2; k * tiles < kPlanPairs; ++k) cut(int(k * tiles));
    cut(kPlanPairs);
  }
  return best;
}

// Sums of the runs' first and last tiles.
static size_t plan_workspace_bytes(const PairPlan& pl) {
  return size_t(2) * pl.workers * pl.n * kPairSums * sizeof(float);
}

template <PairMode MODE>
static cudaError_t launch_pair(const PairMaps& maps, PairParams& p, cudaStream_t stream) {
  const int pairs = pair_count<MODE>();
  if (pairs < 1) return cudaErrorNotSupported;
  const int xslot_bytes = p.n / 2 * 128;
  int most_kernels = 0;
  for (int i = 0; i < p.nmat; ++i) most_kernels = p.mat[i].K > most_kernels ? p.mat[i].K : most_kernels;
  const int slots = (kPairRing - (most_kernels == 4 ? 3 : 4) * xslot_bytes) / kPairABytes;
  p.slots = slots < kPairMaxSlots ? slots : kPairMaxSlots;
  const int xslots = (kPairRing - p.slots * kPairABytes) / xslot_bytes;
  p.xslots = xslots < p.slots ? xslots : p.slots;
  const int ring = p.slots * kPairABytes + p.xslots * xslot_bytes;
  const int wslots = (kPairRings - ring) / kPairWBytes;
  p.wslots = wslots < kPairMaxSlots ? wslots : kPairMaxSlots;
  for (int i = 0; i < 8; ++i) p.mul.pow2[i] = 1u << (15 - 2 * i);
  const int smem = 1024 + ring + p.wslots * kPairWBytes + kPairBarriers;
  if (p.workers > pairs) p.workers = pairs;   // longer runs, whose sums take no more room
  // (the stages of an item, in whole tiles or runs)
  p.all_drain = p.naccs > 1 || (p.workers > 0 ? p.ntiles * p.stages / p.workers : p.stages) < kPairFewStages;
  if (p.workers > 0) {
    p.run = p.ntiles * p.stages / p.workers;
    p.run_rest = p.ntiles * p.stages % p.workers;
  }
  const int items = p.workers > 0 ? p.workers : p.ntiles;
  const int grid = 2 * (items < pairs ? items : pairs);
  const cudaError_t e =
      launch_dependent(gemm_pair_kernel<MODE>, dim3(grid), dim3(kPairThreads), size_t(smem), stream, maps, p);
  if (e != cudaSuccess || p.workers < 2) return e;
  constexpr int kThreadsPerToken = (MODE == kGate ? kPairSums / 2 : kPairSums) / 4;
  return launch_dependent(pair_join_kernel<MODE>, dim3(unsigned((p.n * kThreadsPerToken + 255) / 256), p.workers - 1),
                          dim3(256), 0, stream, p);
}

static void set_plan(PairParams& p, const PairPlan& pl) {
  p.n = pl.n;
  p.naccs = p.n > 256 ? 2 : 1;
  p.n_acc = p.n / p.naccs;   // n is a multiple of 32
  p.ntiles = p.row_tiles * ((p.T + p.n - 1) / p.n);
  p.workers = pl.workers;
}

static size_t up16(size_t n) { return (n + 15) / 16 * 16; }
static size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// ---- gated forward ----

static PairPlan gate_plan(int M, int N, int T) {
  return pair_plan((M + 127) / 128, N / kPairBK, T);
}

// X scaled, the tokens' scales, and the runs' sums.
static size_t gate_sums_offset(int N, int T) { return up256(size_t(T) * N * 2) + up256(up16(T) * sizeof(float)); }
size_t gemm_gated_workspace_bytes(int M, int N, int T) {
  return gate_sums_offset(N, T) + plan_workspace_bytes(gate_plan(M, N, T));
}

cudaError_t launch_gemm_gated(const uint8_t* packed_gate, const uint16_t* alpha_gate, const Shape& gate,
                              const uint8_t* packed_up, const uint16_t* alpha_up, const Shape& up, const uint16_t* X,
                              int T, uint16_t* H, uint16_t* G, uint16_t* U, void* workspace, cudaStream_t stream) {
  uint16_t* xs = static_cast<uint16_t*>(workspace);
  float* inverse = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + up256(size_t(T) * gate.N * 2));
  PairMaps maps;
  PairParams p = {};
  p.nmat = 2;
  p.M = gate.M;
  p.N = gate.N;
  p.T = T;
  p.stages = gate.N / kPairBK;
  p.row_tiles = (gate.M + 127) / 128;
  set_plan(p, gate_plan(gate.M, gate.N, T));
  p.partial = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + gate_sums_offset(gate.N, T));
  p.idesc = tc_idesc_f16(256, p.n_acc, false, false, false);
  p.inverse = inverse;
  p.out = H;
  p.gate = G;
  p.up = U;
  const Shape* shapes[2] = {&gate, &up};
  const uint8_t* packed[2] = {packed_gate, packed_up};
  const uint16_t* alpha[2] = {alpha_gate, alpha_up};
  bool good = make_map(&maps.act[0], CU_TENSOR_MAP_DATA_TYPE_FLOAT16, xs, gate.N, T, uint64_t(gate.N) * 2, kPairBK,
                       p.n_acc / 2, true);
  for (int i = 0; i < 2; ++i) {
    const Shape& s = *shapes[i];
    p.mat[i].K = s.K;
    p.mat[i].M = s.M;
    good = good &&
           make_map(&maps.bits[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, packed[i], s.N, uint64_t(s.O) * s.K, s.N, 64,
                    kPairOctets * s.K, false) &&
           make_map(&maps.alpha[i], CU_TENSOR_MAP_DATA_TYPE_UINT16, alpha[i], uint64_t(s.G) * s.K * kOctet, s.O,
                    uint64_t(s.G) * s.K * kOctet * 2, s.K * kOctet, kPairOctets, false);
  }
  if (!good) return cudaErrorInvalidValue;
  ScaleRows sc = {};
  sc.nseg = 1;
  sc.seg[0].src = X;
  sc.seg[0].dst = xs;
  sc.seg[0].cols = sc.seg[0].ld = gate.N;
  sc.inverse = inverse;
  sc.factor = 1.f / kLevelScale;
  const cudaError_t e = launch_scale_rows(sc, T, stream);
  if (e != cudaSuccess) return e;
  return launch_pair<kGate>(maps, p, stream);
}

// ---- input gradient ----

static PairPlan grad_plan(int nmat, const Shape* shapes, int T) {
  int stages = 0;
  for (int i = 0; i < nmat; ++i) stages += (shapes[i].M + kPairBK - 1) / kPairBK;
  return pair_plan((shapes[0].N + 255) / 256, stages, T);
}

// The runs' sums.
size_t gemm_grad_x_workspace_bytes(int nmat, const Shape* shapes, int T) {
  return plan_workspace_bytes(grad_plan(nmat, shapes, T));
}

// dX from dY_s already scaled to fp16 (rows `ld[s]` apart, zeros beyond M_s)
// with the tokens' inverse scales; workspace as sized by
// gemm_grad_x_workspace_bytes, 16-byte aligned.
cudaError_t launch_gemm_grad_x(int nmat, const uint8_t* const* packed, const uint16_t* const* alpha,
                               const Shape* shapes, const uint16_t* const* dys, const int* ld, const float* inverse,
                               int T, uint16_t* dX, void* workspace, cudaStream_t stream) {
  PairMaps maps;
  PairParams p = {};
  p.nmat = nmat;
  p.N = shapes[0].N;
  p.T = T;
  p.row_tiles = (p.N + 255) / 256;
  for (int i = 0; i < nmat; ++i) {
    p.mat[i].stages = (shapes[i].M + kPairBK - 1) / kPairBK;
    p.stages += p.mat[i].stages;
  }
  set_plan(p, grad_plan(nmat, shapes, T));
  p.partial = static_cast<float*>(workspace);
  p.idesc = tc_idesc_f16(256, p.n_acc, false, true, false);
  p.inverse = inverse;
  p.out = dX;
  bool good = true;
  for (int i = 0; i < nmat; ++i) {
    const Shape& s = shapes[i];
    p.mat[i].K = s.K;
    p.mat[i].M = s.M;
    good = good &&
           make_map(&maps.act[i], CU_TENSOR_MAP_DATA_TYPE_FLOAT16, dys[i], ld[i], T, uint64_t(ld[i]) * 2, kPairBK,
                    p.n_acc / 2, true) &&
           make_map(&maps.bits[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, packed[i], s.N, uint64_t(s.O) * s.K, s.N, 128,
                    kPairOctets * s.K, false) &&
           make_map(&maps.alpha[i], CU_TENSOR_MAP_DATA_TYPE_UINT16, alpha[i], uint64_t(s.G) * s.K * kOctet, s.O,
                    uint64_t(s.G) * s.K * kOctet * 2, s.K * kOctet, kPairOctets, false);
  }
  if (!good) return cudaErrorInvalidValue;
  return launch_pair<kGrad>(maps, p, stream);
}

}  // namespace mbok
