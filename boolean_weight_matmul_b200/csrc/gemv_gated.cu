// Gated decode  h[b] = silu(W_gate x[b]) * (W_up x[b])  for 2..16 vectors on the
// tensor cores, and the choice between this form and the lookup form (one
// vector, gemv_lut.cu).
//
// A gated feed-forward block reads x once for two projections and uses them only
// as this product, so neither is stored.  As in gemv_mma.cu each kernel's dot
// product over a 128-column group is an exact MMA, scaled per group in fp32; the
// rest is arranged for the instruction count, which bounds this size:
//
//  * Bits as they are.  A single set bit of an fp16 word is a power of two, exact
//    for the tensor cores: bits 5 .. 9 are the subnormals 2^-19 .. 2^-15, bits 10,
//    11 and 12 are 2^-14, 2^-13 and 2^-11.  Column i of a row's 16 is bit i of
//    its halfword, so with bytes 0 and 1 in the two halves of a word (one byte
//    permute), five bits up, the fragment word of columns (i, i + 8) is one AND
//    with 0x00200020 << i.  The activations carry the inverse factor (2^8 .. 1)
//    and S, a power of two per warp and vector that puts the largest finite |x|
//    below 2^7 (exact for bf16 values down to 2^-23 of the largest, off by at most
//    2^-31 of it below).  With T the sum over set bits and X the sum over all
//    columns (an MMA with every bit set, once per group), the +-1 sum is 2 T - X.
//    Building +-1 words took a logic and a multiply-add instruction each and more
//    around them: 23 instructions per MMA, 35.8 us for two to eight vectors
//    (LLaMA-7B gate and up, K = 3) against 27.1.
//    The five bits up are for accuracy: products are aligned for their sum as if a
//    subnormal had a leading one, so a subnormal's product is cut off 2^z too
//    early, z its leading zeros.  With the bits left at 0 .. 7 (z up to 10) h was
//    off by 1.8e-6 of its norm (fp32 activations 5e-6); at 5 .. 12 by 1.0e-7.
//  * Persistent CTAs.  A warp owns at most two 128-column groups and keeps their
//    activations in registers as MMA fragments for all rows it meets; it streams
//    the bits and scales of its columns for one row octet after another through
//    a private shared-memory ring (cp.async, two to four steps ahead).
//  * A step is two row octets (the MMA's 16 rows) with every plane (matrix,
//    kernel) of gate and up, K_gate + K_up in all: what a step costs besides its
//    MMAs is spread over as many as the columns give.
//  * The P warps that share a step's rows (a row group; small N has several per
//    CTA) leave their columns' sums in a double-buffered shared-memory array; each
//    adds, gates and stores its share of a step's outputs, in a fixed order, one
//    step later, when the sums have long arrived (with a barrier per step 30 % of
//    the time passed outside the MMAs).  With
//    more columns than one CTA's warps cover (N > 5120, or 4096 for more than 8
//    fragment columns) CTAs take slabs of columns and a second small launch adds
//    the slabs through the workspace.
//  * fp32 activations are split into three fp16 parts (three columns), exact as
//    above.
// An infinite activation makes its vector's outputs NaN (0 x infinity in T).
// Measured in a graph: LLaMA-7B gate and up (K = 3) 27.1 us for 2 to 8 vectors,
// 41.1 us for 16; LLaMA-13B (K = 4 and 2, 5120 columns) 38.9 us for 7, of which 17 us
// are the MMAs and their ANDs (each about 8 cycles of its pipe per MMA), 3.6 us
// the copies' instructions, 3.6 us the joined sums.  All forms spill registers (44 to
// 244 bytes of stores a thread, 92 to 352 of loads).
#include "lut_common.cuh"
#include "tc_common.cuh"

namespace mbok {

cudaError_t launch_gemv_lut_gated(const uint8_t*, const uint16_t*, const Shape&, const uint8_t*, const uint16_t*,
                                  const Shape&, const void*, bool, void*, bool, void*, cudaStream_t, bool);
size_t gemv_gated_lut_workspace_bytes(const Shape&);

constexpr float kGdProduct = 2048.f;         // x S over the product of a set bit and its activation
constexpr int kGdMaxDepth = 4;               // steps in flight per warp: as many as fit, at least 2
constexpr int kGdSmemMax = 227 * 1024, kGdStatic = 1024;   // of which static (barriers)
constexpr int kGdGroups = 2;                 // groups per warp
constexpr int kGdUnits = kGdGroups * kUnitsPerGroup;
constexpr int kGdPlaneBytes = 2 * kGdUnits * 16;             // one plane's bits of a step: [octet][unit][8 rows]
constexpr int kGdScaleBytes = 2 * kGdGroups * 16;            // one plane's scales of a step: [octet][group][8 rows]
// Warps per CTA: with one 8-column tile of vectors up to 20 (96 registers), with
// two up to 16 (128 registers).
template <int NT>
struct GdGeom {
  static constexpr int kMaxWarps = NT == 1 ? 20 : 16;
  static constexpr int kRed = 2 * 16 * 8 * NT + 2;          // floats per warp: [gate, up][row][column], padded
  static constexpr int kConst = (kGdGroups + 1) * 8 * NT;   // floats per warp: X of each group, 1 / S
};
// Shared memory of one warp besides its ring: two buffers of sums and constants.
template <int NT>
constexpr int gd_warp_bytes() { return (2 * GdGeom<NT>::kRed + GdGeom<NT>::kConst) * 4; }

static __device__ unsigned int g_gemv_gated_error;

struct GatedMmaParams {
  const uint8_t* packed[2];   // gate, up
  const uint16_t* alpha[2];
  Shape s[2];
  const void* x;              // [batch][N] bf16 or fp32
  void* h;                    // [batch][M]
  float* partial;             // several slabs: [slab][gate, up][batch][M]
  int h_bf16;
  int batch, per, nchunk;     // vectors, in chunks of `per` (fewer in the last)
  int nslab, slab_groups;     // column slabs, groups in each (fewer in the last)
  int parts, row_groups;      // warps per row group, row groups per CTA
  int stage_bytes, depth;
  int weights_static;
};

__device__ __forceinline__ void gd_mma(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same from zero.
__device__ __forceinline__ void gd_mma0(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// The fragment word of columns (I, I + 8) from a row's 16 bits, 0..7 at bits 5..12
// and 8..15 at bits 21..28.
template <int I>
__device__ __forceinline__ uint32_t gd_word(uint32_t u) { return u & (0x00200020u << I); }

// d (from zero where FIRST) += 64 columns of two planes' rows (their bits u0, u1)
// times the fragments b.
template <int NT, bool FIRST>
__device__ __forceinline__ void gd_chunk(float d[NT][4], uint32_t u0, uint32_t u1, const uint32_t b[NT][8]) {
#define MBOK_GD_STEP(J, MMA)                                                                                \
  _Pragma("unroll") for (int nt = 0; nt < NT; ++nt)                                                         \
      MMA(d[nt], gd_word<2 * J>(u0), gd_word<2 * J>(u1), gd_word<2 * J + 1>(u0), gd_word<2 * J + 1>(u1),    \
          b[nt][2 * J], b[nt][2 * J + 1]);
  if (FIRST) {
    MBOK_GD_STEP(0, gd_mma0)
  } else {
    MBOK_GD_STEP(0, gd_mma)
  }
  MBOK_GD_STEP(1, gd_mma)
  MBOK_GD_STEP(2, gd_mma)
  MBOK_GD_STEP(3, gd_mma)
#undef MBOK_GD_STEP
}

// Part `part` (0 = high) of the three-way fp16 split of v.
__device__ __forceinline__ float gd_part(float v, int part) {
  const float h = __half2float(__float2half_rn(v));
  if (part == 0) return h;
  const float r = __fsub_rn(v, h);
  const float m = __half2float(__float2half_rn(r));
  return part == 1 ? m : __fsub_rn(r, m);
}

// The 16 activations of unit q of vector vec: raw words (8 for bf16, 16 for
// fp32); zeros at or beyond vector `end`.
template <bool XF32>
struct GdUnit {
  uint32_t w[XF32 ? 16 : 8];

  __device__ __forceinline__ void load(const GatedMmaParams& p, int vec, int end, int q) {
    constexpr int kWords = XF32 ? 16 : 8;
    if (vec >= end) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = 0u;
      return;
    }
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint32_t*>(p.x) +
                                                      (size_t(vec) * p.s[0].N + q * kUnit) / (XF32 ? 1 : 2));
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      const uint4 v = src[i];
      w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
    }
  }
  __device__ __forceinline__ float at(int i) const {
    if (XF32) return __uint_as_float(w[i]);
    return (i & 1) ? __uint_as_float(w[i >> 1] & 0xFFFF0000u) : __uint_as_float(w[i >> 1] << 16);
  }
  // The larger of m and the finite magnitudes, as fp32 bits.
  __device__ __forceinline__ uint32_t high(uint32_t m) const {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t a = __float_as_uint(at(i)) & 0x7FFFFFFFu;
      if (a < 0x7F800000u) m = max(m, a);
    }
    return m;
  }
  // Fragments: column i (and i + 8) times scale over (kGdProduct times bit 5 + i).
  __device__ __forceinline__ void fragment(float scale, int part, uint32_t b[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float f = i < 7 ? float(1 << (8 - i)) : 1.f;
      float lo, hi;
      if (XF32) {
        lo = gd_part(at(i) * scale, part) * f;
        hi = gd_part(at(i + 8) * scale, part) * f;
      } else {
        // the value scaled first: scale * f overflows where the vector is tiny
        lo = at(i) * scale * f;
        hi = at(i + 8) * scale * f;
      }
      const __half2 h = __floats2half2_rn(lo, hi);
      b[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
};

// Copy the bits (every plane, this warp's ng groups from g0) and scales of
// octets 2 step and 2 step + 1 into a stage; one commit group.  A second octet
// beyond the last is not copied (its rows are not stored).
__device__ __forceinline__ void gd_issue(const GatedMmaParams& p, int step, int g0, int ng, unsigned char* st,
                                         int lane) {
  const int K0 = p.s[0].K, np = K0 + p.s[1].K;
  // half a warp per octet, a lane per unit
  const int oi = lane >> 4, u = lane & 15, o = 2 * step + oi;
  if (o < p.s[0].O) {
    if (u < ng * kUnitsPerGroup) {
      unsigned char* dst = st + (oi * kGdUnits + u) * 16;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int K = p.s[m].K;
        const uint8_t* src = p.packed[m] + unit_offset(p.s[m], o, 0, g0 * kUnitsPerGroup + u);
        for (int k = 0; k < K; ++k, dst += kGdPlaneBytes, src += size_t(p.s[m].Q) * 16) cp_async16(dst, src);
      }
    }
    // scales: lane u takes plane u / 2, group u % 2
    if (u < 2 * np && (u & 1) < ng) {
      const int plane = u >> 1, g = u & 1;
      const int m = plane < K0 ? 0 : 1, k = plane - (m != 0 ? K0 : 0);
      cp_async16(st + np * kGdPlaneBytes + plane * kGdScaleBytes + (oi * kGdGroups + g) * 16,
                 p.alpha[m] + alpha_offset(p.s[m], o, g0 + g, k));
    }
  }
  cp_async_commit();
}

// Part `part`'s share of one step's outputs (rows row0 .. row0 + 15) from the sums
// of a row group's parts at `all` (and hi + mid + lo of fp32), added in a fixed
// order: gated and stored, or stored for the other slabs.  With many parts four
// lanes share an output, every fourth part each.
template <int NT, bool XF32>
__device__ __forceinline__ void gd_add(const GatedMmaParams& p, const float* all, int row0, int slab, int vec0,
                                       int nb, int part, int lane) {
  using G = GdGeom<NT>;
  const int M = p.s[0].M;
  const int share = p.parts >= 8 ? 4 : 1, sub = lane & (share - 1);
#pragma unroll 1
  for (int item0 = part * (32 / share); item0 < nb * 16; item0 += p.parts * (32 / share)) {
    const int item = item0 + lane / share;   // share 1: the last round may have idle lanes
    const bool live = item < nb * 16;
    const int vec = live ? item >> 4 : 0, r = item & 15;
    float total[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      float sum[XF32 ? 3 : 1];
#pragma unroll
      for (int q = 0; q < (XF32 ? 3 : 1); ++q) {
        const float* at = all + (m * 16 + r) * 8 * NT + (XF32 ? 3 * vec + q : vec);
        sum[q] = 0.f;
        for (int w = sub; w < p.parts; w += share) sum[q] += at[w * G::kRed];
        if (share > 1) {
          sum[q] += __shfl_xor_sync(0xffffffffu, sum[q], 1);
          sum[q] += __shfl_xor_sync(0xffffffffu, sum[q], 2);
        }
      }
      total[m] = XF32 ? (sum[0] + sum[XF32 ? 1 : 0]) + sum[XF32 ? 2 : 0] : sum[0];
    }
    if (!live || sub != 0 || row0 + r >= M) continue;
    if (p.nslab == 1) {
      store_act(p.h, p.h_bf16 != 0, size_t(vec0 + vec) * M + row0 + r, gated(total[0], total[1]));
    } else {
      float* out = p.partial + (size_t(slab) * 2 * p.batch + vec0 + vec) * M + row0 + r;
      __stcg(out, total[0]);
      __stcg(out + size_t(p.batch) * M, total[1]);
    }
  }
}

template <int NT, bool XF32>
__global__ void __launch_bounds__(GdGeom<NT>::kMaxWarps * 32, 1)
gemv_gated_kernel(const __grid_constant__ GatedMmaParams p) {
  using G = GdGeom<NT>;
  extern __shared__ __align__(128) unsigned char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gq = lane >> 2, t = lane & 3;   // fragment row and column thread
  const int rg = warp / p.parts, part = warp % p.parts;
  const int workers = p.parts * p.row_groups;
  // this CTA's slab and chunk of vectors, and its place among their CTAs
  const int cells = p.nslab * p.nchunk, cell = int(blockIdx.x) % cells, cta = int(blockIdx.x) / cells;
  const int chunk = p.nchunk == 1 ? 0 : cell / p.nslab, slab = cell - chunk * p.nslab;
  const int vec0 = chunk * p.per, nb = min(p.per, p.batch - vec0);
  const int ctas = (int(gridDim.x) - cell + cells - 1) / cells;
  // this warp's groups: part of the slab's, as equal as whole groups allow
  const int sg0 = slab * p.slab_groups, sg = min(p.slab_groups, p.s[0].G - sg0);
  const int g0 = sg0 + part * sg / p.parts, ng = sg0 + (part + 1) * sg / p.parts - g0;
  const int np = p.s[0].K + p.s[1].K;
  const int O = p.s[0].O;
  unsigned char* ring = smem + warp * p.depth * p.stage_bytes;
  float* red = reinterpret_cast<float*>(smem + workers * p.depth * p.stage_bytes);   // [2][worker][kRed]
  float* consts = red + 2 * workers * G::kRed + warp * G::kConst;
  __shared__ __align__(8) uint64_t sums_full[GdGeom<1>::kMaxWarps][2], sums_free[GdGeom<1>::kMaxWarps][2];
  const int steps = (O + 1) / 2;
  const int first = cta * p.row_groups + rg, stride = ctas * p.row_groups;
  const int n_mine = first < steps ? (steps - 1 - first) / stride + 1 : 0;

  if (threadIdx.x == 0) {
    for (int r = 0; r < p.row_groups; ++r)
      for (int b = 0; b < 2; ++b) {
        tc_mbar_init(&sums_full[r][b], p.parts);
        tc_mbar_init(&sums_free[r][b], p.parts);
      }
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  __syncthreads();
  if (p.weights_static) {
    for (int i = 0; i < p.depth; ++i) {
      if (i < n_mine) gd_issue(p, first + i * stride, g0, ng, ring + i * p.stage_bytes, lane);
      else cp_async_commit();
    }
  }
  allow_dependents();
  // x, the workspace and (unless static) the weights may be written by the
  // previous grid
  grid_dependency_wait();
  uint32_t b[kGdGroups][2][NT][8];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int n = gq + 8 * nt, vec = XF32 ? n / 3 : n;
    GdUnit<XF32> x[kGdGroups][2];
    uint32_t high = 0u;   // the largest finite magnitude of the vector in this warp's columns
#pragma unroll
    for (int g = 0; g < kGdGroups; ++g)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        x[g][c].load(p, vec0 + vec, g < ng ? vec0 + nb : 0, (g0 + g) * kUnitsPerGroup + 4 * c + t);
        high = x[g][c].high(high);
      }
    high = max(high, __shfl_xor_sync(0xffffffffu, high, 1));
    high = max(high, __shfl_xor_sync(0xffffffffu, high, 2));
    // S = 2^e, e = 6 - floor(log2 high): at most 2^126 (tiny vectors), 1 for zeros
    const int e = high == 0u ? 0 : min(133 - int(high >> 23), 126);
    const float scale = __uint_as_float(uint32_t(127 + e) << 23);
#pragma unroll
    for (int g = 0; g < kGdGroups; ++g)
#pragma unroll
      for (int c = 0; c < 2; ++c) x[g][c].fragment(scale, n % 3, b[g][c][nt]);
    // 1 / S of the column; accumulator columns are 2t and 2t + 1
    if (t == 0) consts[(kGdGroups * NT + nt) * 8 + gq] = __uint_as_float(uint32_t(127 - e) << 23);
  }
  // X of each group and column: every bit set (row 0 of the product)
#pragma unroll
  for (int g = 0; g < kGdGroups; ++g) {
    float d[NT][4];
    gd_chunk<NT, true>(d, 0x1FE01FE0u, 0u, b[g][0]);
    gd_chunk<NT, false>(d, 0x1FE01FE0u, 0u, b[g][1]);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      if (gq == 0)
        *reinterpret_cast<float2*>(consts + (g * NT + nt) * 8 + 2 * t) =
            make_float2(d[nt][0] * kGdProduct, d[nt][1] * kGdProduct);
  }
  __syncwarp();
  if (!p.weights_static) {
    for (int i = 0; i < p.depth; ++i) {
      if (i < n_mine) gd_issue(p, first + i * stride, g0, ng, ring + i * p.stage_bytes, lane);
      else cp_async_commit();
    }
  }

  bool ok = true;
  for (int i = 0, slot = 0; i < n_mine; ++i) {
    const int step = first + i * stride;
    unsigned char* st = ring + slot * p.stage_bytes;
    // the step has landed (this lane's copies)
    if (p.depth == 4) cp_async_wait<3>();
    else if (p.depth == 3) cp_async_wait<2>();
    else cp_async_wait<1>();
    __syncwarp();   // ... and every lane's
    // gate, up: rows gq of both octets, columns 2t and 2t + 1 of each tile (as the accumulators)
    float y[2][NT][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) y[m][nt][0] = y[m][nt][1] = y[m][nt][2] = y[m][nt][3] = 0.f;
#pragma unroll
    for (int g = 0; g < kGdGroups; ++g) {
      if (g >= ng) break;
      const unsigned char* bits = st + g * (kUnitsPerGroup * 16) + 16 * t + 2 * gq;
      const unsigned char* scales = st + np * kGdPlaneBytes + g * 16 + 2 * gq;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int K = p.s[m].K;
#pragma unroll 2
        for (int k = 0; k < K; ++k, bits += kGdPlaneBytes, scales += kGdScaleBytes) {
          float d[NT][4];
          uint32_t u[2][2];
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int oi = 0; oi < 2; ++oi)
              u[c][oi] = __byte_perm(*reinterpret_cast<const uint16_t*>(bits + oi * kGdUnits * 16 + 64 * c), 0u, 0x4140) * 32u;
          gd_chunk<NT, true>(d, u[0][0], u[0][1], b[g][0]);
          gd_chunk<NT, false>(d, u[1][0], u[1][1], b[g][1]);
          // the +-1 sums 2 T - X times the plane's group scales
#pragma unroll
          for (int oi = 0; oi < 2; ++oi) {
            const float a = __half2float(
                __ushort_as_half(*reinterpret_cast<const uint16_t*>(scales + oi * kGdGroups * 16)));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const float2 X = *reinterpret_cast<const float2*>(consts + (g * NT + nt) * 8 + 2 * t);
              y[m][nt][2 * oi] = fmaf(a, fmaf(2.f * kGdProduct, d[nt][2 * oi], -X.x), y[m][nt][2 * oi]);
              y[m][nt][2 * oi + 1] = fmaf(a, fmaf(2.f * kGdProduct, d[nt][2 * oi + 1], -X.y), y[m][nt][2 * oi + 1]);
            }
          }
        }
      }
    }
    __syncwarp();   // every lane is done with the stage
    if (i + p.depth < n_mine) gd_issue(p, step + p.depth * stride, g0, ng, st, lane);
    else cp_async_commit();
    if (++slot == p.depth) slot = 0;
    // this warp's sums: [buffer][warp][gate, up][column][row]
    const int buf = i & 1;
    if (i >= 2 && ok && !tc_wait(&sums_free[rg][buf], unsigned(i / 2 - 1) & 1u)) ok = false;
    float* mine = red + (buf * workers + warp) * G::kRed;   // 8-byte aligned
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float2 back = *reinterpret_cast<const float2*>(consts + (kGdGroups * NT + nt) * 8 + 2 * t);
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int oi = 0; oi < 2; ++oi)
          *reinterpret_cast<float2*>(mine + (m * 16 + 8 * oi + gq) * 8 * NT + 8 * nt + 2 * t) =
              make_float2(y[m][nt][2 * oi] * back.x, y[m][nt][2 * oi + 1] * back.y);
    }
    __syncwarp();
    if (lane == 0) tc_arrive(&sums_full[rg][buf]);
    // this warp's share of step i - 1 (and at the end of the last step)
    for (int j = i > 0 ? i - 1 : i; j <= (i + 1 < n_mine ? i - 1 : i); ++j) {
      if (ok && !tc_wait(&sums_full[rg][j & 1], unsigned(j / 2) & 1u)) ok = false;
      if (!ok) continue;   // nothing more is stored
      gd_add<NT, XF32>(p, red + ((j & 1) * workers + rg * p.parts) * G::kRed, (first + j * stride) * 2 * kOctet, slab,
                       vec0, nb, part, lane);
      __syncwarp();
      if (lane == 0) tc_arrive(&sums_free[rg][j & 1]);
    }
  }
  if (!ok) atomicOr(&g_gemv_gated_error, 1u);
  cp_async_wait<0>();
}

// h from the slabs' sums ([slab][gate, up][n], n = nb * M), in slab order.
__global__ void __launch_bounds__(256) gemv_gated_combine_kernel(const float* __restrict__ partial, void* h,
                                                                 int h_bf16, size_t n, int nslab) {
  allow_dependents();
  grid_dependency_wait();
  const size_t i = size_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n) return;
  float g = 0.f, u = 0.f;
  for (int s = 0; s < nslab; ++s) {
    g += __ldcg(partial + size_t(2 * s) * n + i);
    u += __ldcg(partial + size_t(2 * s + 1) * n + i);
  }
  store_act(h, h_bf16 != 0, i, gated(g, u));
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// Chunks of vectors (one takes two 8-column tiles at most), as equal as can be, and
// the fragment columns of one.  Chunks run side by side in one launch: their CTAs
// share the weights through L2, and few rows leave SMs for all (one launch after
// another against side by side, fp32, equal chunks: 6 vectors, 70 rows, N = 1664 31
// and 16 us; LLaMA-7B gate and up, 6 vectors 87 and 80, 16 vectors 175 and 145; 5 and
// 1 vectors one after another, the last on one tile, 76).  Each chunk streams all
// weights, so that the time steps with their number: LLaMA-7B, fp32, 3 to 5 vectors
// 44 us, 6 to 10 80, 11 to 15 115, 16 145.
static int gd_chunks(bool x_f32, int batch) { return x_f32 ? (batch + 4) / 5 : (batch + 15) / 16; }
static int gd_columns(bool x_f32, int nb) { return x_f32 ? 3 * nb : nb; }

struct GdPlan {
  int nslab, slab_groups, parts, row_groups;
};

// Slabs of as many groups as one CTA's warps take, two groups per warp; with few
// groups several row groups per CTA.
static GdPlan gd_plan(int groups, int max_warps) {
  GdPlan pl;
  const int most = kGdGroups * max_warps;
  pl.nslab = (groups + most - 1) / most;
  pl.slab_groups = (groups + pl.nslab - 1) / pl.nslab;
  pl.nslab = (groups + pl.slab_groups - 1) / pl.slab_groups;
  pl.parts = (pl.slab_groups + kGdGroups - 1) / kGdGroups;
  pl.row_groups = max_warps / pl.parts;
  if (pl.row_groups > 8) pl.row_groups = 8;
  return pl;
}

static int gd_max_warps(int columns) { return columns <= 8 ? GdGeom<1>::kMaxWarps : GdGeom<2>::kMaxWarps; }

// One vector: the lookup kernel's partial sums; more: the slabs' sums (0 with one
// slab).
size_t gemv_gated_workspace_bytes(const Shape& s, int batch) {
  if (batch == 1) return gemv_gated_lut_workspace_bytes(s);
  size_t most = 0;
  for (int f32 = 0; f32 < 2; ++f32) {   // the call may bring either type
    const int chunks = gd_chunks(f32 != 0, batch), per = (batch + chunks - 1) / chunks;
    const GdPlan pl = gd_plan(s.G, gd_max_warps(gd_columns(f32 != 0, per)));
    const size_t bytes = pl.nslab > 1 ? size_t(pl.nslab) * 2 * batch * s.M * sizeof(float) : 0;
    if (bytes > most) most = bytes;
  }
  return most;
}

template <int NT, bool XF32>
static cudaError_t launch_gd(GatedMmaParams& p, cudaStream_t stream) {
  using G = GdGeom<NT>;
  const GdPlan pl = gd_plan(p.s[0].G, G::kMaxWarps);
  p.nslab = pl.nslab;
  p.slab_groups = pl.slab_groups;
  p.parts = pl.parts;
  p.row_groups = pl.row_groups;
  p.stage_bytes = (p.s[0].K + p.s[1].K) * (kGdPlaneBytes + kGdScaleBytes);
  const int workers = pl.parts * pl.row_groups;
  const int red_bytes = workers * gd_warp_bytes<NT>();
  p.depth = (kGdSmemMax - kGdStatic - red_bytes) / (workers * p.stage_bytes);
  if (p.depth > kGdMaxDepth) p.depth = kGdMaxDepth;
  static_assert(G::kMaxWarps * (2 * 2 * MBOK_MAX_K * (kGdPlaneBytes + kGdScaleBytes) + gd_warp_bytes<NT>()) <=
                    kGdSmemMax - kGdStatic,
                "two steps and the sums fit one CTA");
  auto fn = gemv_gated_kernel<NT, XF32>;
  static PerDeviceOnce attr_once;   // the attribute is per device context
  const cudaError_t ae = set_smem_attr_once(attr_once, reinterpret_cast<const void*>(fn), kGdSmemMax - kGdStatic);
  if (ae != cudaSuccess) return ae;
  const int steps = (p.s[0].O + 1) / 2;
  const int per_slab = (steps + pl.row_groups - 1) / pl.row_groups;   // CTAs that have a step to begin with
  const int cells = pl.nslab * p.nchunk;
  int ctas = device_sm_count() / cells;
  if (ctas < 1) ctas = 1;
  if (ctas > per_slab) ctas = per_slab;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas * cells);
  cfg.blockDim = dim3(workers * 32);
  cfg.dynamicSmemBytes = size_t(workers * p.depth * p.stage_bytes + red_bytes);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, fn, p);
  if (e != cudaSuccess) return e;
  if (pl.nslab > 1) {
    const size_t n = size_t(p.batch) * p.s[0].M;
    cudaLaunchConfig_t c2 = {};
    c2.gridDim = dim3(unsigned((n + 255) / 256));
    c2.blockDim = dim3(256);
    c2.stream = stream;
    c2.attrs = attr;
    c2.numAttrs = 1;
    e = cudaLaunchKernelEx(&c2, gemv_gated_combine_kernel, static_cast<const float*>(p.partial), p.h, p.h_bf16, n,
                           pl.nslab);
    if (e != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

// h[b] for b < batch (x: [batch][N], h: [batch][M]); workspace as sized by
// gemv_gated_workspace_bytes.
cudaError_t launch_gemv_gated(const uint8_t* packed_gate, const uint16_t* alpha_gate, const Shape& gate,
                              const uint8_t* packed_up, const uint16_t* alpha_up, const Shape& up, const void* x,
                              bool x_f32, int batch, void* h, bool h_bf16, void* workspace, cudaStream_t stream,
                              bool weights_static) {
  if (batch == 1)
    return launch_gemv_lut_gated(packed_gate, alpha_gate, gate, packed_up, alpha_up, up, x, x_f32, h, h_bf16,
                                 workspace, stream, weights_static);
  GatedMmaParams p = {};
  p.packed[0] = packed_gate;
  p.packed[1] = packed_up;
  p.alpha[0] = alpha_gate;
  p.alpha[1] = alpha_up;
  p.s[0] = gate;
  p.s[1] = up;
  p.x = x;
  p.h = h;
  p.h_bf16 = h_bf16 ? 1 : 0;
  p.partial = static_cast<float*>(workspace);
  p.batch = batch;
  p.per = (batch + gd_chunks(x_f32, batch) - 1) / gd_chunks(x_f32, batch);
  p.nchunk = (batch + p.per - 1) / p.per;
  p.weights_static = weights_static ? 1 : 0;
  if (gd_columns(x_f32, p.per) <= 8) return x_f32 ? launch_gd<1, true>(p, stream) : launch_gd<1, false>(p, stream);
  return x_f32 ? launch_gd<2, true>(p, stream) : launch_gd<2, false>(p, stream);
}

// Reads and clears the kernel's error flag; ~0u if the read itself failed.
unsigned gemv_gated_error_flags() {
  unsigned v = 0;
  if (cudaMemcpyFromSymbol(&v, g_gemv_gated_error, sizeof(v)) != cudaSuccess) return ~0u;
  const unsigned z = 0;
  if (v != 0 && cudaMemcpyToSymbol(g_gemv_gated_error, &z, sizeof(z)) != cudaSuccess) return ~0u;
  return v;
}

}  // namespace mbok
