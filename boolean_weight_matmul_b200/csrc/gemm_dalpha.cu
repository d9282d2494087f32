// Gradients of the group scales of layers that share X, on CTA pairs (sm_100a):
//
//     dalpha_s[k][r][g] = sum_{j in group g} b_k[r][j] C_s[r][j],
//     C_s[r][j] = sum_t dY_s[t][r] X[t][j].
//
// C_s is the gradient of the dense weight, M x N values of which only the
// signed sums over 128-column groups are wanted (K per 128).  So it never
// leaves tensor memory: a pair of CTAs forms 256 x 256 of it (tcgen05
// cta_group::2, M = N = 256, each CTA 128 rows x 256 columns), and the
// epilogue adds each row's 128 columns of a group with the signs of the K
// kernels.
//
//  * Both operands contract over tokens and are stored token-major, so both
//    are M-/N-major tiles, brought by TMA as boxes of 64 tokens x 64 columns
//    with the 128-byte swizzle (16 KB of dY and 16 KB of X per CTA and stage,
//    6 stages); products of bf16 values are exact in the fp32 accumulation.
//  * A CTA's 128 x 256 accumulator is half its tensor memory: two of them
//    alternate, so the signed sums (8 epilogue warps: four lane quarters x two
//    groups) run while the tensor cores fill the other.
//  * Tokens are taken in runs of at most 512, each from a zero accumulator, and
//    the runs' signed sums are added in fp32 registers: the tensor cores' own
//    accumulation truncates, and its error grows with the run (relative error
//    of dalpha at 2048 tokens, 11008 x 4096: 2.6e-7 with runs of 256, 4.8e-7
//    with 512, 1.0e-6 with 1024; fp32 products summed on the CUDA cores 4e-7).
//    Shorter runs repeat the epilogue more often (gate and up of that size, K =
//    3: 331 us with 256, 259 to 268 us = 1375 to 1425 TFLOP/s with 512, tensor
//    pipe 73 % busy; 221 us at K = 1, where the signed sums hide entirely).
//  * With few tiles the tokens are split over several pairs, whose sums land in
//    the workspace ([split][dalpha]) and are added in order by a second kernel:
//    deterministic.
#include "scale_rows.h"
#include "tc_pair.cuh"

namespace mbok {

constexpr int kDaStages = 6;
constexpr int kDaBT = 64;                               // tokens per stage
constexpr int kDaBlock = 64 * kDaBT * 2;                // one box: 64 tokens x 64 columns, 8 KB
constexpr int kDaStageBytes = 4 * kDaBlock;             // two boxes of dY, two of X
constexpr int kDaSmem = kDaStages * kDaStageBytes + 1024 + 256;
constexpr int kDaRunStages = 8;                         // 512 tokens per run
constexpr int kDaEpiWarps = 8;
constexpr int kDaThreads = (2 + kDaEpiWarps) * 32;
constexpr unsigned kDaTmemCols = 512;

static __device__ unsigned int g_dalpha_error;

struct DaMat {
  const uint8_t* packed;
  float* out;          // dalpha, or this matrix's region of split 0 in the workspace
  int K, M, O;
  int row_tiles;       // of 256 rows
  int tile0;           // first tile of this matrix
};

struct DaMaps {
  CUtensorMap x;
  CUtensorMap dy[kMaxMats];
};

struct DaParams {
  DaMat mat[kMaxMats];
  int nmat;
  int N, G;
  int col_tiles;        // of 256 columns
  int ntiles;           // over all matrices
  int splits;
  int stages;           // token stages in all
  size_t split_stride;  // floats between the splits' outputs
  uint32_t idesc;
  int beside;           // follows the input gradient's kernel, of which it needs nothing
};

struct DaItem {
  int m, rt, ct;        // matrix, row tile, column tile
  int s0, s1;           // token stages
  int split;
};

// Item i of the launch: splits vary slowest, row tiles fastest (pairs that run
// together share X columns through L2).
__device__ __forceinline__ DaItem da_item(const DaParams& p, int i) {
  DaItem it;
  it.split = i / p.ntiles;
  const int tile = i % p.ntiles;
  it.m = 0;
  while (it.m + 1 < p.nmat && tile >= p.mat[it.m + 1].tile0) ++it.m;
  const int local = tile - p.mat[it.m].tile0;
  it.rt = local % p.mat[it.m].row_tiles;
  it.ct = local / p.mat[it.m].row_tiles;
  it.s0 = int(long(it.split) * p.stages / p.splits);
  it.s1 = int(long(it.split + 1) * p.stages / p.splits);
  return it;
}

// S[k] += the signed sum over 32 accumulator columns: v[b] enters kernel k with
// a plus where bit b of w[k] is set, taken as twice the sum over the set bits
// minus the sum over all.  A bit test and a predicated add are two instructions
// per element and kernel on two pipes; flipping the sign took three, two of
// them on the logic pipe (K = 3, 2048 tokens: 281 -> 259 us).
__device__ __forceinline__ void add_signed(const uint32_t v[32], const uint32_t w[MBOK_MAX_K], int K,
                                           float S[MBOK_MAX_K]) {
  float t0 = 0.f, t1 = 0.f, t2 = 0.f, t3 = 0.f;
#pragma unroll
  for (int b = 0; b < 32; b += 4) {
    t0 += __uint_as_float(v[b]);
    t1 += __uint_as_float(v[b + 1]);
    t2 += __uint_as_float(v[b + 2]);
    t3 += __uint_as_float(v[b + 3]);
  }
  const float total = (t0 + t1) + (t2 + t3);
#pragma unroll
  for (int k = 0; k < MBOK_MAX_K; ++k) {
    if (k >= K) continue;
    // opaque here: the tests of all kernels' bits, hoisted out of the runs'
    // loop, would not fit the registers
    uint32_t bits = w[k];
    asm volatile("" : "+r"(bits));
    float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
    for (int b = 0; b < 32; b += 4) {
      if (bits & (1u << b)) s0 += __uint_as_float(v[b]);
      if (bits & (2u << b)) s1 += __uint_as_float(v[b + 1]);
      if (bits & (4u << b)) s2 += __uint_as_float(v[b + 2]);
      if (bits & (8u << b)) s3 += __uint_as_float(v[b + 3]);
    }
    S[k] += 2.f * ((s0 + s1) + (s2 + s3)) - total;
  }
}

__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t v[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kDaThreads, 1)
gemm_dalpha_kernel(const __grid_constant__ DaMaps maps, const __grid_constant__ DaParams p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kDaStages * kDaStageBytes);   // leader: both CTAs' copies landed
  uint64_t* empty = full + kDaStages;    // the stage's MMAs are done (both CTAs)
  uint64_t* tfull = empty + kDaStages;   // accumulator b holds a finished run (both CTAs)
  uint64_t* tempty = tfull + 2;          // leader: both CTAs drained accumulator b
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);
  __shared__ int s_fail;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = int(pair_rank());
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int nitems = p.ntiles * p.splits;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kDaStages; ++s) {
      tc_mbar_init(&full[s], 1);
      tc_mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc_mbar_init(&tfull[b], 1);
      tc_mbar_init(&tempty[b], 2 * kDaEpiWarps);
    }
    s_fail = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
  }
  __syncwarp();
  if (warp == 1) pair_alloc(tmem_slot, kDaTmemCols);
  tc_fence_before();
  pair_sync();   // both CTAs run and their barriers are set up
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  bool ok = true;
  // Behind the input gradient's kernel (which starts this one once all before it
  // is complete) this one runs beside it, and waits for it only at its end.
  if (!p.beside) pdl_wait();
  pdl_launch();

  if (warp == 0) {
    // ---- TMA producer: 128 rows of dY^T and half of the tile's columns of X ----
    int g = 0;
    for (int i = pair; i < nitems && ok; i += npairs) {
      const DaItem it = da_item(p, i);
      const int r0 = it.rt * 256 + rank * 128, j0 = it.ct * 256 + rank * 128;
      for (int kb = it.s0; kb < it.s1; ++kb, ++g) {
        const int s = g % kDaStages;
        if (g >= kDaStages && !pair_wait(&empty[s], unsigned((g / kDaStages) - 1) & 1u)) { ok = false; break; }
        unsigned char* st = smem + s * kDaStageBytes;
        const uint32_t bar = pair_leader(&full[s]);
        if (elect_lane()) {
          if (rank == 0) tc_arrive_expect_tx(&full[s], 2 * kDaStageBytes);   // both CTAs' bytes
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            pair_tma_load_2d(st + b * kDaBlock, &maps.dy[it.m], r0 + 64 * b, kb * kDaBT, bar);
            pair_tma_load_2d(st + (2 + b) * kDaBlock, &maps.x, j0 + 64 * b, kb * kDaBT, bar);
          }
        }
        __syncwarp();
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      // ---- MMA issuer, for both CTAs ----
      const uint64_t a0 = tc_desc_sw128_mn(tc_smem(smem), kDaBlock);
      const uint64_t x0 = tc_desc_sw128_mn(tc_smem(smem) + 2 * kDaBlock, kDaBlock);
      int g = 0, run = 0;
      for (int i = pair; i < nitems && ok; i += npairs) {
        const DaItem it = da_item(p, i);
        for (int k0 = it.s0; k0 < it.s1 && ok; k0 += kDaRunStages, ++run) {
          const int k1 = min(k0 + kDaRunStages, it.s1);
          const int b = run & 1;
          // run's buffer was last used by run - 2
          if (run >= 2 && !pair_wait(&tempty[b], unsigned((run >> 1) - 1) & 1u)) { ok = false; break; }
          tc_fence_after();
          for (int kb = k0; kb < k1; ++kb, ++g) {
            const int s = g % kDaStages;
            const unsigned ph = unsigned(g / kDaStages) & 1u;
            if (!pair_wait(&full[s], ph)) { ok = false; break; }
            tc_fence_after();
            const uint64_t off = uint64_t(s * (kDaStageBytes >> 4));
            if (elect_lane()) {
#pragma unroll
              for (int kk = 0; kk < kDaBT / 16; ++kk)
                pair_mma(tmem + uint32_t(b * 256), a0 + off + uint64_t(kk * (2048 >> 4)),
                         x0 + off + uint64_t(kk * (2048 >> 4)), p.idesc, (kb > k0 || kk > 0) ? 1u : 0u);
              pair_commit(&empty[s]);
              if (kb + 1 == k1) pair_commit(&tfull[b]);
            }
            __syncwarp();
          }
        }
      }
    }
  } else {
    // ---- epilogue: lane quarter warp & 3, group (warp - 2) / 4 of the tile's two ----
    const int quarter = warp & 3, gi = (warp - 2) >> 2;
    int run = 0;
    for (int i = pair; i < nitems && ok; i += npairs) {
      const DaItem it = da_item(p, i);
      const DaMat& m = p.mat[it.m];
      const int r = it.rt * 256 + rank * 128 + 32 * quarter + lane;
      const int g = it.ct * 2 + gi;
      const bool live = (r >> 3) < m.O && g < p.G;
      // the row's bits of this group, 32 columns per word
      uint32_t w[4][MBOK_MAX_K];
#pragma unroll
      for (int k = 0; k < MBOK_MAX_K; ++k) {
#pragma unroll
        for (int c = 0; c < 4; ++c) w[c][k] = 0u;
        if (k < m.K && live) {
          const uint8_t* src = m.packed + (size_t(r >> 3) * m.K + k) * p.N + size_t(g) * 128 + 2 * (r & 7);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            w[c][k] = uint32_t(*reinterpret_cast<const uint16_t*>(src + 32 * c)) |
                      (uint32_t(*reinterpret_cast<const uint16_t*>(src + 32 * c + 16)) << 16);
        }
      }
      float S[MBOK_MAX_K] = {0.f, 0.f, 0.f, 0.f};
      for (int k0 = it.s0; k0 < it.s1; k0 += kDaRunStages, ++run) {
        const int b = run & 1;
        if (!pair_wait(&tfull[b], unsigned(run >> 1) & 1u)) { ok = false; break; }
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          tmem_ld32(tmem + (uint32_t(32 * quarter) << 16) + uint32_t(b * 256 + gi * 128 + 32 * c), v);
          add_signed(v, w[c], m.K, S);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) pair_arrive(pair_leader(&tempty[b]));
      }
      if (!ok) break;
      if (live) {
        float* dst = m.out + size_t(it.split) * p.split_stride + (size_t(r >> 3) * p.G + g) * m.K * 8 + (r & 7);
#pragma unroll
        for (int k = 0; k < MBOK_MAX_K; ++k)
          if (k < m.K) dst[k * 8] = r < m.M ? S[k] : 0.f;   // rows that pad the last octet: 0
      }
    }
  }

  if (!ok) atomicOr(&s_fail, 1);
  tc_fence_before();
  __syncthreads();
  if (s_fail != 0 && threadIdx.x == 0) {
    atomicOr(&g_dalpha_error, 1u);
    tc_drain_barriers(full, 2 * kDaStages + 2);   // full, empty and tfull: copies and MMAs in flight
  }
  __syncthreads();
  __syncwarp();
  pair_sync();   // neither CTA leaves while the other's MMAs or arrivals may reach it
  if (warp == 1) {
    tc_fence_after();
    pair_dealloc(tmem, kDaTmemCols);
  }
  if (p.beside) pdl_wait();   // this grid's completion stands for both
}

// out[i] = the splits' sums in order; the matrices' regions follow one another
// in a split, 4 floats per thread.
struct DaJoin {
  float* out[kMaxMats];
  size_t first[kMaxMats + 1];   // in groups of 4 floats
  int nmat;
};

__global__ void __launch_bounds__(256) dalpha_join_kernel(const float* part, size_t split_stride, int splits,
                                                          const __grid_constant__ DaJoin j) {
  pdl_launch();
  pdl_wait();
  const size_t i = size_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= j.first[j.nmat]) return;
  float4 sum = __ldcs(reinterpret_cast<const float4*>(part) + i);
  for (int s = 1; s < splits; ++s) {
    const float4 v = __ldcs(reinterpret_cast<const float4*>(part + s * split_stride) + i);
    sum.x += v.x;
    sum.y += v.y;
    sum.z += v.z;
    sum.w += v.w;
  }
  int m = 0;
  while (m + 1 < j.nmat && i >= j.first[m + 1]) ++m;
  reinterpret_cast<float4*>(j.out[m])[i - j.first[m]] = sum;
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

unsigned gemm_dalpha_error_flags() {
  unsigned v = 0;
  if (cudaMemcpyFromSymbol(&v, g_dalpha_error, sizeof(v)) != cudaSuccess) return ~0u;
  const unsigned z = 0;
  if (v != 0 && cudaMemcpyToSymbol(g_dalpha_error, &z, sizeof(z)) != cudaSuccess) return ~0u;
  return v;
}

static size_t da_elems(const Shape& s) { return size_t(s.O) * kOctet * s.G * s.K; }

// Token splits for `pairs` pairs at once: as many as keep one wave, each of at
// least 4 stages (256 tokens).  The plan goes by the largest device's 74 pairs
// so that a workspace's size does not depend on the device.
constexpr int kDaPlanPairs = 74;
int dalpha_splits(int nmat, const Shape* shapes, int T) {
  long tiles = 0;
  for (int i = 0; i < nmat; ++i) tiles += long((shapes[i].M + 255) / 256) * ((shapes[i].N + 255) / 256);
  const int stages = (T + kDaBT - 1) / kDaBT;
  long splits = tiles >= kDaPlanPairs ? 1 : kDaPlanPairs / tiles;
  if (splits > stages / 4) splits = stages / 4;
  return splits < 1 ? 1 : int(splits);
}

size_t dalpha_workspace_bytes(int nmat, const Shape* shapes, int T) {
  const int splits = dalpha_splits(nmat, shapes, T);
  if (splits == 1) return 0;
  size_t n = 0;
  for (int i = 0; i < nmat; ++i) n += da_elems(shapes[i]);
  return n * splits * sizeof(float);
}

static int da_pair_count() {
  const void* fn = reinterpret_cast<const void*>(gemm_dalpha_kernel);
  static PerDeviceOnce attr_once;
  if (set_smem_attr_once(attr_once, fn, kDaSmem) != cudaSuccess) return 0;
  static PerDeviceValue<int> cache;
  return cache.get(current_device(), [fn]() -> int {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kDaThreads);
    cfg.dynamicSmemBytes = kDaSmem;
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

// dalpha_s for nmat matrices (dY_s bf16 with rows ld[s] apart, a multiple of 8).
// splits: dalpha_splits of these matrices or of a set that holds them;
// beside: the launch before it in the stream is launch_gemm_grad_x's.
// workspace as sized by dalpha_workspace_bytes for that set, 16-byte aligned.
cudaError_t launch_gemm_dalpha(int nmat, const uint8_t* const* packed, const Shape* shapes, const uint16_t* X, int T,
                               const uint16_t* const* dys, const int* ld, float* const* dalpha, int splits,
                               bool beside, void* workspace, cudaStream_t stream) {
  const int pairs = da_pair_count();
  if (pairs < 1) return cudaErrorNotSupported;
  DaMaps maps;
  DaParams p = {};
  p.nmat = nmat;
  p.N = shapes[0].N;
  p.G = shapes[0].G;
  p.col_tiles = (p.N + 255) / 256;
  p.stages = (T + kDaBT - 1) / kDaBT;
  p.splits = splits;
  p.idesc = tc_idesc_f16(256, 256, true, true, true);
  bool good = make_map(&maps.x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, X, p.N, T, uint64_t(p.N) * 2, 64, kDaBT, true);
  DaJoin join = {};
  join.nmat = nmat;
  size_t off = 0;
  for (int i = 0; i < nmat; ++i) {
    const Shape& s = shapes[i];
    DaMat& m = p.mat[i];
    m.packed = packed[i];
    m.K = s.K;
    m.M = s.M;
    m.O = s.O;
    m.row_tiles = (s.M + 255) / 256;
    m.tile0 = p.ntiles;
    m.out = p.splits == 1 ? dalpha[i] : static_cast<float*>(workspace) + off;
    join.out[i] = dalpha[i];
    join.first[i] = off / 4;
    off += da_elems(s);
    p.ntiles += m.row_tiles * p.col_tiles;
    good = good && make_map(&maps.dy[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dys[i], s.M, T, uint64_t(ld[i]) * 2, 64,
                            kDaBT, true);
  }
  join.first[nmat] = off / 4;
  p.split_stride = off;
  if (!good) return cudaErrorInvalidValue;
  const long items = long(p.ntiles) * p.splits;
  const int grid = 2 * int(items < pairs ? items : pairs);
  p.beside = beside ? 1 : 0;
  const cudaError_t e =
      launch_dependent(gemm_dalpha_kernel, dim3(grid), dim3(kDaThreads), size_t(kDaSmem), stream, maps, p);
  if (e != cudaSuccess || p.splits == 1) return e;
  return launch_dependent(dalpha_join_kernel, dim3(unsigned((off / 4 + 255) / 256)), dim3(256), 0, stream,
                          static_cast<const float*>(workspace), off, p.splits, join);
}

}  // namespace mbok
