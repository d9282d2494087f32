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
//    tokens: each CTA unpacks 128 rows of A per 64-deep stage, and the pair's
//    tensor cores use every unpacked row for all 512 tokens, twice the tokens
//    per unpacked weight at the same activation traffic (each CTA loads half of
//    the tokens and the hardware reads both halves).
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
// leader's barrier, and the tile's bits and scales, in a ring of their own that
// runs ahead; four unpack warps write A and arrive on the leader's `ready`
// barrier (16 unpack warps in four groups, one per ring slot: with all 16 on
// every stage the latency of wait, load, store, fence and arrival bounded each
// stage at about 1 us, whatever the tokens); the leader's MMA thread issues 4 x (1 or 2) tcgen05.mma
// (M = 256, N <= 256, K = 16) and commits the stage to both CTAs' `empty`
// barriers.  The unpack warps also drain the accumulator (up to 512 columns,
// all of tensor memory) after a tile's last stage: 16 warps, four per lane
// quarter.  Every mbarrier wait is bounded (1 s): on timeout the CTA records an
// error flag, drains what it issued (bounded) and leaves with the other.
#include "scale_rows.h"
#include "tc_pair.cuh"
#include "tc_unpack.cuh"

namespace mbok {

constexpr int kPairStages = 4;
constexpr int kPairBK = 64;
constexpr int kPairRows = 128;                                // A rows per CTA
constexpr int kPairHalf = 128;                                // most tokens per CTA and accumulator
constexpr int kPairXBytes = kPairHalf * kPairBK * 2;          // 16 KB per accumulator
constexpr int kPairABytes = kPairRows * kPairBK * 2;          // 16 KB
constexpr int kPairOctets = 8;                                // row octets of a bits box (64 rows)
constexpr int kPairBits = 2 * kPairOctets * MBOK_MAX_K * 64;  // 4 KB: GATE two boxes of 64 bytes, GRAD one of 128
constexpr int kPairAlpha = 2 * kPairOctets * MBOK_MAX_K * 16; // 1 KB
constexpr int kPairAOff = 2 * kPairXBytes;
constexpr int kPairStageBytes = kPairAOff + kPairABytes;      // 48 KB: tokens and A
constexpr int kPairWStages = 6;                               // a deeper ring for the bits and scales
constexpr int kPairWBytes = kPairBits + kPairAlpha;           // 5 KB
constexpr int kPairWOff = kPairStages * kPairStageBytes;
constexpr int kPairBarOff = kPairWOff + kPairWStages * kPairWBytes;
constexpr int kPairSmem = kPairBarOff + 1024 + 256;
constexpr int kPairUnpackWarps = 16;
constexpr int kPairGroupWarps = kPairUnpackWarps / kPairStages;   // unpack warps per ring slot
constexpr int kPairUnpackWarp0 = 3;                               // after the two copy warps and the MMA warp
constexpr int kPairThreads = (kPairUnpackWarp0 + kPairUnpackWarps) * 32;
constexpr unsigned kPairTmemCols = 512;

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

struct PairParams {
  PairMat mat[kMaxMats];
  int nmat;
  int M, N, T;
  int n_acc, naccs;    // tokens per accumulator (multiple of 16, <= 256), accumulators (1 or 2)
  int stages;          // per tile
  int row_tiles;       // tiles along W's rows (GATE, 128) or columns (GRAD, 256)
  int ntiles;
  uint32_t idesc;
  const float* inverse;   // [T rounded up to 16]
  uint16_t* out;          // H, or dX
  uint16_t* gate;         // GATE: [T][M] or nullptr
  uint16_t* up;
};

// Four units (64 columns) of one row: the row's bits of kernel k and unit u at
// src + k * kstride + u * 16, to the eight swizzled 16-byte chunks of `line`.
// Units are taken in the order u ^ flip.
template <int K>
__device__ __forceinline__ void pair_unpack(const unsigned char* src, int kstride, const uint32_t P[4],
                                            unsigned char* line, int r, int flip) {
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const int u = n ^ flip;
    uint32_t h[K], out[8];
#pragma unroll
    for (int k = 0; k < K; ++k) h[k] = *reinterpret_cast<const uint16_t*>(src + k * kstride + u * 16);
    tc_unpack_row<K>(h, P, out);
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
__device__ __forceinline__ void unpack_gate(const unsigned char* w, unsigned char* a, int gt) {
  const int up = gt >> 6, m = gt & 63;
  const int o = m >> 3, i = m & 7;
  const int r = 32 * (m >> 4) + 16 * up + (m & 15);
  uint32_t P[4];
  tc_levels_f16<K>(w + kPairBits + up * (kPairAlpha / 2), o, i, false, P);
  pair_unpack<K>(w + up * (kPairBits / 2) + o * K * 64 + 2 * i, 64, P, a + r * 128, r, 0);
}

// GRAD: thread gt of a group's 128 unpacks block gt & 1 (64 columns) of row
// gt >> 1 of the stage's 64 rows.  Eight lanes that store together hold four
// rows of both blocks; the second block's units go in the order 2, 3, 0, 1, so
// that its chunks differ from the first's.  Rows at or beyond M are zeros:
// their stored scales mean nothing and could be NaN.
template <int K>
__device__ __forceinline__ void unpack_grad(const unsigned char* w, unsigned char* a, int gt, int rows) {
  const int r = gt >> 1, b = gt & 1;
  const int o = r >> 3, i = r & 7;
  uint32_t P[4];
  tc_levels_f16<K>(w + kPairBits, o, i, r >= rows, P);
  pair_unpack<K>(w + o * K * 128 + b * 64 + 2 * i, 128, P, a + b * 8192 + r * 128, r, 2 * b);
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

// Store n values (n a power of two) that lanes 2i and 2i + 1 hold for rows r
// and r + 1 at tokens t .. t + n - 1 of out [T][ld], ld even and out 4-byte
// aligned: after one exchange per pair of tokens the even lane stores both rows
// of the first half, the odd lane of the second, as bf16 pairs.
template <int n>
__device__ __forceinline__ void store_pairs(uint16_t* out, size_t ld, int rows, int T, int r, int t, const float* v,
                                            int lane) {
  const bool odd = lane & 1;
  const int r0 = r & ~1;
#pragma unroll
  for (int i = 0; i < n / 2; ++i) {
    const float mine = odd ? v[i] : v[n / 2 + i];
    const float other = __shfl_xor_sync(0xffffffffu, mine, 1);
    const float lo = odd ? other : v[i], hi = odd ? v[n / 2 + i] : other;
    const int tt = t + (odd ? n / 2 + i : i);
    if (r0 < rows && tt < T) *reinterpret_cast<uint32_t*>(out + size_t(tt) * ld + r0) = tc_pack_bf16x2(lo, hi);
  }
}

// The same for any ld and alignment.
template <int n>
__device__ __forceinline__ void store_singles(uint16_t* out, size_t ld, int rows, int T, int r, int t, const float* v) {
  if (r >= rows) return;
#pragma unroll
  for (int i = 0; i < n; ++i)
    if (t + i < T) out[size_t(t + i) * ld + r] = __bfloat16_as_ushort(__float2bfloat16_rn(v[i]));
}

template <int n>
__device__ __forceinline__ void store_rows(bool pairs, uint16_t* out, size_t ld, int rows, int T, int r, int t,
                                           const float* v, int lane) {
  if (pairs) store_pairs<n>(out, ld, rows, T, r, t, v, lane);
  else store_singles<n>(out, ld, rows, T, r, t, v);
}

// Drain this warp's share of a finished tile: lane quarter q, chunks of 16
// tokens sub, sub + 4, ...
template <PairMode MODE>
__device__ __forceinline__ void pair_drain(const PairParams& p, uint32_t tmem, int tile, int rank, int q, int sub,
                                           int lane) {
  const int per = p.n_acc / 16;
  const int t0 = (tile / p.row_tiles) * (p.n_acc * p.naccs);
  const int rt = tile % p.row_tiles;
  const int rows = MODE == kGate ? p.M : p.N;
  const size_t ld = size_t(rows);
  const bool pairs = rows % 2 == 0;   // every buffer is 16-byte aligned
  const int r = MODE == kGate ? rt * 128 + rank * 64 + 16 * q + (lane & 15) : rt * 256 + rank * 128 + 32 * q + lane;
  for (int j = sub; j < per * p.naccs; j += kPairUnpackWarps / 4) {
    const int a = j / per, c = j % per;
    const int t = t0 + a * p.n_acc + 16 * c;
    if (t >= p.T) break;
    uint32_t w[16];
    tmem_ld16(tmem + (uint32_t(32 * q) << 16) + uint32_t(a * 256 + 16 * c), w);
    float v[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 s = __ldg(reinterpret_cast<const float4*>(p.inverse + t) + i);
      v[4 * i] = __uint_as_float(w[4 * i]) * s.x;
      v[4 * i + 1] = __uint_as_float(w[4 * i + 1]) * s.y;
      v[4 * i + 2] = __uint_as_float(w[4 * i + 2]) * s.z;
      v[4 * i + 3] = __uint_as_float(w[4 * i + 3]) * s.w;
    }
    if (MODE == kGrad) {
      store_rows<16>(pairs, p.out, ld, rows, p.T, r, t, v, lane);
    } else {
      const bool low = lane < 16;
      if (p.gate != nullptr) store_rows<16>(pairs, low ? p.gate : p.up, ld, rows, p.T, r, t, v, lane);
      // lanes l and l + 16 hold gate and up of one row: after the exchange the
      // lower lane has both for tokens t .. t + 7, the upper for t + 8 ..
      float h[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float other = __shfl_xor_sync(0xffffffffu, low ? v[8 + i] : v[i], 16);
        h[i] = low ? gated(v[i], other) : gated(other, v[8 + i]);
      }
      store_rows<8>(pairs, p.out, ld, rows, p.T, r, low ? t : t + 8, h, lane);
    }
  }
}

template <PairMode MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
gemm_pair_kernel(const __grid_constant__ PairMaps maps, const __grid_constant__ PairParams p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* wfull = reinterpret_cast<uint64_t*>(smem + kPairBarOff);   // bits and scales landed
  uint64_t* wempty = wfull + kPairWStages; // ... and unpacked
  uint64_t* xfull = wempty + kPairWStages; // leader: both CTAs' tokens landed
  uint64_t* ready = xfull + kPairStages;   // leader: both CTAs' A is unpacked
  uint64_t* empty = ready + kPairStages;   // the stage's MMAs are done (both CTAs)
  uint64_t* tfull = empty + kPairStages;   // the accumulator holds a finished tile (both CTAs)
  uint64_t* tempty = tfull + 1;            // leader: both CTAs drained the accumulator
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 1);
  __shared__ int s_fail;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = int(pair_rank());
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairWStages; ++s) {
      tc_mbar_init(&wfull[s], 1);
      tc_mbar_init(&wempty[s], kPairGroupWarps);
    }
    for (int s = 0; s < kPairStages; ++s) {
      tc_mbar_init(&xfull[s], 1);
      tc_mbar_init(&ready[s], 2 * kPairGroupWarps);
      tc_mbar_init(&empty[s], 1);
    }
    tc_mbar_init(tfull, 1);
    tc_mbar_init(tempty, 2 * kPairUnpackWarps);
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

  if (warp == 0) {
    // ---- token copies ----
    const int n_half = p.n_acc / 2;
    const unsigned bytes = unsigned(2 * p.naccs * n_half * kPairBK * 2);   // both CTAs'
    int g = 0;
    for (int tile = pair; tile < p.ntiles && ok; tile += npairs) {
      const int t0 = (tile / p.row_tiles) * (p.n_acc * p.naccs) + rank * n_half;
      int m = 0, step = 0;   // GRAD: matrix and its 64-row step
      for (int kb = 0; kb < p.stages; ++kb, ++g) {
        const int s = g % kPairStages;
        if (g >= kPairStages && !pair_wait(&empty[s], unsigned((g / kPairStages) - 1) & 1u)) { ok = false; break; }
        unsigned char* st = smem + s * kPairStageBytes;
        const uint32_t bar = pair_leader(&xfull[s]);
        const CUtensorMap* map = &maps.act[MODE == kGate ? 0 : m];
        const int x = (MODE == kGate ? kb : step) * kPairBK;
        if (elect_lane()) {
          if (rank == 0) tc_arrive_expect_tx(&xfull[s], bytes);
          pair_tma_load_2d(st, map, x, t0, bar);
          if (p.naccs > 1) pair_tma_load_2d(st + kPairXBytes, map, x, t0 + p.n_acc, bar);
        }
        __syncwarp();
        if (MODE == kGrad && ++step == p.mat[m].stages) { step = 0; ++m; }
      }
    }
  } else if (warp == 2) {
    // ---- copies of bits and scales ----
    int g = 0;
    for (int tile = pair; tile < p.ntiles && ok; tile += npairs) {
      const int rt = tile % p.row_tiles;
      int m = 0, step = 0;
      for (int kb = 0; kb < p.stages; ++kb, ++g) {
        const int s = g % kPairWStages;
        if (g >= kPairWStages && !pair_wait(&wempty[s], unsigned((g / kPairWStages) - 1) & 1u)) { ok = false; break; }
        unsigned char* w = smem + kPairWOff + s * kPairWBytes;
        if (MODE == kGate) {
          const int o = (rt * 128 + rank * 64) / kOctet;
          if (elect_lane()) {
            tc_arrive_expect_tx(&wfull[s], unsigned(p.mat[0].K + p.mat[1].K) * kPairOctets * (64 + 16));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int K = p.mat[i].K;
              tc_tma_load_2d(w + i * (kPairBits / 2), &maps.bits[i], kb * 64, o * K, &wfull[s]);
              tc_tma_load_2d(w + kPairBits + i * (kPairAlpha / 2), &maps.alpha[i], (kb / 2) * K * kOctet, o, &wfull[s]);
            }
          }
        } else {
          const int K = p.mat[m].K;
          const int j = rt * 256 + rank * 128;
          if (elect_lane()) {
            tc_arrive_expect_tx(&wfull[s], unsigned(K) * kPairOctets * (128 + 16));
            tc_tma_load_2d(w, &maps.bits[m], j, step * kPairOctets * K, &wfull[s]);
            tc_tma_load_2d(w + kPairBits, &maps.alpha[m], (j / kGroup) * K * kOctet, step * kPairOctets, &wfull[s]);
          }
          if (++step == p.mat[m].stages) { step = 0; ++m; }
        }
        __syncwarp();
      }
    }
  } else if (warp == 1) {
    // ---- MMA issuer: the leader's, for both CTAs ----
    if (rank == 0) {
      constexpr int kAStep = MODE == kGate ? 32 >> 4 : 2048 >> 4;   // 16 k further in A
      const uint32_t base = tc_smem(smem);
      const uint64_t a0 = MODE == kGate ? tc_desc_sw128(base + kPairAOff) : tc_desc_sw128_mn(base + kPairAOff, 8192);
      const uint64_t x0 = tc_desc_sw128(base);
      int g = 0, i = 0;
      for (int tile = pair; tile < p.ntiles && ok; tile += npairs, ++i) {
        if (i > 0 && !pair_wait(tempty, unsigned(i - 1) & 1u)) { ok = false; break; }
        tc_fence_after();
        for (int kb = 0; kb < p.stages; ++kb, ++g) {
          const int s = g % kPairStages;
          const unsigned ph = unsigned(g / kPairStages) & 1u;
          if (!pair_wait(&xfull[s], ph) || !pair_wait(&ready[s], ph)) { ok = false; break; }
          tc_fence_after();
          const uint64_t off = uint64_t(s * (kPairStageBytes >> 4));
          if (elect_lane()) {
#pragma unroll
            for (int kk = 0; kk < kPairBK / 16; ++kk) {
              const uint64_t ad = a0 + off + uint64_t(kk * kAStep), xd = x0 + off + uint64_t(kk * (32 >> 4));
              const uint32_t acc = (kb > 0 || kk > 0) ? 1u : 0u;
              pair_mma(tmem, ad, xd, p.idesc, acc);
              if (p.naccs > 1) pair_mma(tmem + 256, ad, xd + uint64_t(kPairXBytes >> 4), p.idesc, acc);
            }
            pair_commit(&empty[s]);
            if (kb + 1 == p.stages) pair_commit(tfull);
          }
          __syncwarp();
        }
      }
    }
  } else {
    // ---- unpack warps, which also drain: group s unpacks ring slot s ----
    const int s = (warp - kPairUnpackWarp0) / kPairGroupWarps;
    const int gt = threadIdx.x - (kPairUnpackWarp0 + s * kPairGroupWarps) * 32;
    unsigned char* a = smem + s * kPairStageBytes + kPairAOff;
    const uint32_t my_ready = pair_leader(&ready[s]);
    int g0 = 0, i = 0;   // the tile's first stage, counted over all tiles
    for (int tile = pair; tile < p.ntiles && ok; tile += npairs, g0 += p.stages, ++i) {
      const int first = (s - g0) & (kPairStages - 1);
      int m = 0, step = first;
      for (int kb = first; kb < p.stages; kb += kPairStages, step += kPairStages) {
        const int g = g0 + kb, ws = g % kPairWStages;
        const unsigned char* w = smem + kPairWOff + ws * kPairWBytes;
        // the bits are there, and the slot's previous MMAs are done with its A
        if (!pair_wait(&wfull[ws], unsigned(g / kPairWStages) & 1u) ||
            (g >= kPairStages && !pair_wait(&empty[s], unsigned((g / kPairStages) - 1) & 1u))) {
          ok = false;
          break;
        }
        if (MODE == kGate) {
          switch (p.mat[gt >> 6].K) {   // the same for a whole warp
            case 1: unpack_gate<1>(w, a, gt); break;
            case 2: unpack_gate<2>(w, a, gt); break;
            case 3: unpack_gate<3>(w, a, gt); break;
            default: unpack_gate<4>(w, a, gt); break;
          }
        } else {
          while (step >= p.mat[m].stages) step -= p.mat[m++].stages;
          const int rows = p.mat[m].M - step * kPairBK;
          switch (p.mat[m].K) {
            case 1: unpack_grad<1>(w, a, gt, rows); break;
            case 2: unpack_grad<2>(w, a, gt, rows); break;
            case 3: unpack_grad<3>(w, a, gt, rows); break;
            default: unpack_grad<4>(w, a, gt, rows); break;
          }
        }
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");   // generic writes -> tensor core reads
        __syncwarp();
        if (lane == 0) {
          pair_arrive(my_ready);
          tc_arrive(&wempty[ws]);
        }
      }
      if (!ok) break;
      if (!pair_wait(tfull, unsigned(i) & 1u)) { ok = false; break; }
      tc_fence_after();
      pair_drain<MODE>(p, tmem, tile, rank, warp & 3, (warp - kPairUnpackWarp0) >> 2, lane);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) pair_arrive(pair_leader(tempty));
    }
  }

  if (!ok) atomicOr(&s_fail, 1);
  tc_fence_before();
  __syncthreads();
  if (s_fail != 0 && threadIdx.x == 0) {
    atomicOr(&g_pair_error, 1u);
    // copies and MMAs in flight: every barrier but tempty
    tc_drain_barriers(wfull, 2 * kPairWStages + 3 * kPairStages + 1);
  }
  __syncthreads();
  __syncwarp();
  pair_sync();   // neither CTA leaves while the other's MMAs or arrivals may reach it
  if (warp == 1) {
    tc_fence_after();
    pair_dealloc(tmem, kPairTmemCols);
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
  if (set_smem_attr_once(attr_once, fn, kPairSmem) != cudaSuccess) return 0;
  static PerDeviceValue<int> cache;
  return cache.get(current_device(), [fn]() -> int {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kPairThreads);
    cfg.dynamicSmemBytes = kPairSmem;
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

// Tokens per tile (a multiple of 32, at most 512) that minimises the time of
// the wave-quantised grid; a tile costs its tokens, and at least what unpacking
// its weights costs (about 256 tokens' worth of tensor-core time).
static int pair_token_tile(int row_tiles, int T, int pairs) {
  if (pairs < 1) pairs = 1;
  int best = 512;
  long best_cost = -1;
  const int most = T >= 512 ? 512 : (T + 31) / 32 * 32;
  for (int n = most; n >= 32; n -= 32) {
    const long tiles = long(row_tiles) * ((T + n - 1) / n);
    const long cost = (tiles + pairs - 1) / pairs * (n > 256 ? n : 256);
    if (best_cost < 0 || cost < best_cost) {
      best_cost = cost;
      best = n;
    }
  }
  return best;
}

template <PairMode MODE>
static cudaError_t launch_pair(const PairMaps& maps, PairParams& p, cudaStream_t stream) {
  const int pairs = pair_count<MODE>();
  if (pairs < 1) return cudaErrorNotSupported;
  const int grid = 2 * (p.ntiles < pairs ? p.ntiles : pairs);
  gemm_pair_kernel<MODE><<<grid, kPairThreads, kPairSmem, stream>>>(maps, p);
  return cudaGetLastError();
}

static void set_tokens(PairParams& p, int n) {
  p.naccs = n > 256 ? 2 : 1;
  p.n_acc = n / p.naccs;   // n is a multiple of 32
  p.ntiles = p.row_tiles * ((p.T + n - 1) / n);
}

static size_t up16(size_t n) { return (n + 15) / 16 * 16; }
static size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// ---- gated forward ----

size_t gemm_gated_workspace_bytes(int N, int T) {
  return up256(size_t(T) * N * 2) + up16(T) * sizeof(float);
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
  set_tokens(p, pair_token_tile(p.row_tiles, T, pair_count<kGate>()));
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

// dX from dY_s already scaled to fp16 (rows `ld[s]` apart, zeros beyond M_s)
// with the tokens' inverse scales.
cudaError_t launch_gemm_grad_x(int nmat, const uint8_t* const* packed, const uint16_t* const* alpha,
                               const Shape* shapes, const uint16_t* const* dys, const int* ld, const float* inverse,
                               int T, uint16_t* dX, cudaStream_t stream) {
  PairMaps maps;
  PairParams p = {};
  p.nmat = nmat;
  p.N = shapes[0].N;
  p.T = T;
  p.row_tiles = (p.N + 255) / 256;
  set_tokens(p, pair_token_tile(p.row_tiles, T, pair_count<kGrad>()));
  p.idesc = tc_idesc_f16(256, p.n_acc, false, true, false);
  p.inverse = inverse;
  p.out = dX;
  bool good = true;
  for (int i = 0; i < nmat; ++i) {
    const Shape& s = shapes[i];
    p.mat[i].K = s.K;
    p.mat[i].M = s.M;
    p.mat[i].stages = (s.M + kPairBK - 1) / kPairBK;
    p.stages += p.mat[i].stages;
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
