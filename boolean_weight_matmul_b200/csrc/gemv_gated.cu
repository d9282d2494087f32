// Gated decode  h[b] = silu(W_gate x[b]) * (W_up x[b])  for 2..16 vectors on the
// tensor cores, and the choice between this form and the lookup form (one
// vector, gemv_lut.cu).
//
// A gated feed-forward block reads x once for two projections and uses them only
// as this product, so neither is stored.  Each +-1 dot product of a kernel's
// 128-column group is an exact bf16 MMA, scaled per group in fp32, as in
// gemv_mma.cu (signs built in registers from the bits: one logic and one
// multiply-add instruction per pair); the arrangement differs:
//
//  * Persistent CTAs.  A warp owns at most two 128-column groups and keeps their
//    activations in registers as MMA fragments for all rows it meets; it streams
//    the bits and scales of its columns for one row octet after another through
//    a private shared-memory ring (cp.async, four octets ahead).  Loading the
//    fragments anew for every 16-row tile, on CTAs that lived for one tile, left
//    the tensor and logic pipes idle two thirds of the time (two to eight
//    vectors, LLaMA-7B gate and up, K = 3: 38.9 us).
//  * An MMA's 16 rows are the 8 rows of an octet twice: the planes (matrix,
//    kernel) of gate and up, K_gate + K_up in all, are taken two at a time, one
//    in rows 0..7 and one in rows 8..15, so matrices with different K waste
//    nothing (at most half an MMA).  Both halves of a fragment belong to the same
//    octet row of the same thread.
//  * The P warps that share a row octet (a row group; small N has several per
//    CTA) add their columns' sums through a double-buffered shared-memory array,
//    one barrier per octet, in warp order; two warps gate and store while the
//    others go on.  With more columns than one CTA's warps cover (N > 5120, or
//    4096 for more than 8 fragment columns) CTAs take slabs of columns and a
//    second small launch adds the slabs through the workspace.
//  * fp32 activations are split exactly into three bf16 parts (three columns).
// What bounds it: the logic pipe.  An MMA's four fragment words take 4 logic
// operations at half rate, about 10 cycles of a quarter SM with the unpacking of
// the halfwords, against 8 for the MMA.
#include "lut_common.cuh"

namespace mbok {

cudaError_t launch_gemv_lut_gated(const uint8_t*, const uint16_t*, const Shape&, const uint8_t*, const uint16_t*,
                                  const Shape&, const void*, bool, void*, bool, void*, cudaStream_t, bool);
size_t gemv_gated_lut_workspace_bytes(const Shape&);

constexpr int kGdDepth = 4;                  // octets in flight per warp
constexpr int kGdGroups = 2;                 // groups per warp
constexpr int kGdUnits = kGdGroups * kUnitsPerGroup;
constexpr int kGdPlaneBytes = kGdUnits * 16;                 // one plane's bits of an octet
constexpr int kGdAlphaBytes = kGdGroups * MBOK_MAX_K * 16;   // one matrix's scales of an octet
// Warps per CTA: with one 8-column tile of vectors up to 20 (96 registers), with
// two up to 16 (128 registers).
template <int NT>
struct GdGeom {
  static constexpr int kMaxWarps = NT == 1 ? 20 : 16;
  static constexpr int kRed = 2 * 8 * NT * 8;   // floats per warp: [gate, up][column][row]
};

struct GatedMmaParams {
  const uint8_t* packed[2];   // gate, up
  const uint16_t* alpha[2];
  Shape s[2];
  const void* x;              // [nb][N] bf16 or fp32
  void* h;                    // [nb][M]
  float* partial;             // several slabs: [slab][gate, up][nb][M]
  int h_bf16;
  int nb;                     // vectors in this launch
  int nslab, slab_groups;     // column slabs, groups in each (fewer in the last)
  int parts, row_groups;      // warps per row group, row groups per CTA
  int stage_bytes;
  int weights_static;
  uint32_t mul[8];            // 2^(15 - 2i): sign_pair factors
};

// Bits P and P + 1 of a halfword as a bf16 pair of signs; u = h | h << 15 (see
// gemv_mma.cu: a logic operation and a multiply-add on the FMA pipe).
template <int P>
__device__ __forceinline__ uint32_t gd_sign_pair(uint32_t u, const uint32_t* mul) {
  constexpr uint32_t kMask = 0x80008000u >> (15 - P);
  return (~u & kMask) * mul[P / 2] + 0x3F803F80u;
}

__device__ __forceinline__ void gd_mma(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Part `part` (0 = high) of the exact three-way bf16 split of v.
__device__ __forceinline__ uint32_t gd_part(float v, int part) {
  auto rn = [](float f) { return uint32_t(__bfloat16_as_ushort(__float2bfloat16_rn(f))); };
  const uint32_t h = rn(v);
  if (part == 0) return h;
  const float r = __fsub_rn(v, __uint_as_float(h << 16));
  const uint32_t m = rn(r);
  return part == 1 ? m : rn(__fsub_rn(r, __uint_as_float(m << 16)));
}

// The 16 activations of unit q in fragment column n as 8 bf16 pairs: vector n,
// or part n % 3 of vector n / 3; zeros beyond the launch's vectors.
template <bool XF32>
__device__ __forceinline__ void gd_load_b(const GatedMmaParams& p, int n, int q, uint32_t b[8]) {
  const int vec = XF32 ? n / 3 : n;
  if (vec >= p.nb) {
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = 0u;
    return;
  }
  if (!XF32) {
    const uint4* src =
        reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x) + size_t(vec) * p.s[0].N + q * kUnit);
    const uint4 v0 = src[0], v1 = src[1];
    b[0] = v0.x; b[1] = v0.y; b[2] = v0.z; b[3] = v0.w;
    b[4] = v1.x; b[5] = v1.y; b[6] = v1.z; b[7] = v1.w;
  } else {
    const int part = n - 3 * vec;
    const float4* src =
        reinterpret_cast<const float4*>(static_cast<const float*>(p.x) + size_t(vec) * p.s[0].N + q * kUnit);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = src[i];
      b[2 * i] = gd_part(v.x, part) | (gd_part(v.y, part) << 16);
      b[2 * i + 1] = gd_part(v.z, part) | (gd_part(v.w, part) << 16);
    }
  }
}

// Copy octet o's bits (every plane, this warp's ng groups from g0) and scales
// into a stage; one commit group.
__device__ __forceinline__ void gd_issue(const GatedMmaParams& p, int o, int g0, int ng, unsigned char* st, int lane) {
  const int K0 = p.s[0].K, np = K0 + p.s[1].K;
  const int per = ng * kUnitsPerGroup;   // 8 or 16 chunks per plane
  const int shift = ng > 1 ? 4 : 3;
  for (int c = lane; c < np * per; c += 32) {
    const int plane = c >> shift, u = c & (per - 1);
    const int m = plane < K0 ? 0 : 1, k = plane - (m != 0 ? K0 : 0);
    cp_async16(st + plane * kGdPlaneBytes + u * 16, p.packed[m] + unit_offset(p.s[m], o, k, g0 * kUnitsPerGroup + u));
  }
  // scales: [group][kernel][8 rows], contiguous for the warp's groups
  unsigned char* sa = st + np * kGdPlaneBytes;
  const int n0 = ng * K0, n1 = ng * p.s[1].K;
  if (lane < n0) cp_async16(sa + lane * 16, p.alpha[0] + alpha_offset(p.s[0], o, g0, 0) + lane * 8);
  else if (lane - n0 < n1)
    cp_async16(sa + kGdAlphaBytes + (lane - n0) * 16, p.alpha[1] + alpha_offset(p.s[1], o, g0, 0) + (lane - n0) * 8);
  cp_async_commit();
}

template <int NT, bool XF32>
__global__ void __launch_bounds__(GdGeom<NT>::kMaxWarps * 32, 1)
gemv_gated_kernel(const __grid_constant__ GatedMmaParams p) {
  using G = GdGeom<NT>;
  extern __shared__ __align__(128) unsigned char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gq = lane >> 2, t = lane & 3;   // fragment row and column thread
  const int rg = warp / p.parts, part = warp % p.parts;
  const int slab = int(blockIdx.x) % p.nslab, cta = int(blockIdx.x) / p.nslab;
  const int ctas = (int(gridDim.x) - slab + p.nslab - 1) / p.nslab;   // CTAs of this slab
  // this warp's groups: part of the slab's, as equal as whole groups allow
  const int sg0 = slab * p.slab_groups, sg = min(p.slab_groups, p.s[0].G - sg0);
  const int g0 = sg0 + part * sg / p.parts, ng = sg0 + (part + 1) * sg / p.parts - g0;
  const int K0 = p.s[0].K, np = K0 + p.s[1].K;
  const int O = p.s[0].O, M = p.s[0].M;
  unsigned char* ring = smem + warp * kGdDepth * p.stage_bytes;
  const int warps = p.parts * p.row_groups;
  float* red = reinterpret_cast<float*>(smem + warps * kGdDepth * p.stage_bytes);   // [2][warp][kRed]
  const int first = cta * p.row_groups + rg, stride = ctas * p.row_groups;
  const int n_mine = first < O ? (O - 1 - first) / stride + 1 : 0;

  if (p.weights_static) {
#pragma unroll
    for (int i = 0; i < kGdDepth; ++i) {
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
  for (int g = 0; g < kGdGroups; ++g)
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (g < ng) {
          gd_load_b<XF32>(p, gq + 8 * nt, (g0 + g) * kUnitsPerGroup + 4 * c + t, b[g][c][nt]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) b[g][c][nt][i] = 0u;
        }
      }
  if (!p.weights_static) {
#pragma unroll
    for (int i = 0; i < kGdDepth; ++i) {
      if (i < n_mine) gd_issue(p, first + i * stride, g0, ng, ring + i * p.stage_bytes, lane);
      else cp_async_commit();
    }
  }

  for (int i = 0; i < n_mine; ++i) {
    const int o = first + i * stride;
    unsigned char* st = ring + (i % kGdDepth) * p.stage_bytes;
    cp_async_wait<kGdDepth - 1>();   // octet i has landed (this lane's copies)
    __syncwarp();                    // ... and every lane's
    const unsigned char* sa = st + np * kGdPlaneBytes;
    float y[2][NT][2];               // gate, up: row gq, columns 2t and 2t + 1 of each tile
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) y[m][nt][0] = y[m][nt][1] = 0.f;
#pragma unroll
    for (int g = 0; g < kGdGroups; ++g) {
      if (g >= ng) break;
      for (int q = 0; q < np; q += 2) {
        const bool two = q + 1 < np;   // the last of an odd number of planes stands alone
        float d[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) d[nt][0] = d[nt][1] = d[nt][2] = d[nt][3] = 0.f;
        const unsigned char* bits = st + q * kGdPlaneBytes + g * (kUnitsPerGroup * 16) + 16 * t + 2 * gq;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint32_t h0 = *reinterpret_cast<const uint16_t*>(bits + 64 * c);
          const uint32_t h1 = two ? *reinterpret_cast<const uint16_t*>(bits + kGdPlaneBytes + 64 * c) : 0u;
          const uint32_t v0 = h0 | (h0 << 15), v1 = h1 | (h1 << 15);
#define MBOK_GD_STEP(J)                                                                                            \
  {                                                                                                                \
    const uint32_t a0 = gd_sign_pair<4 * J>(v0, p.mul), a1 = gd_sign_pair<4 * J>(v1, p.mul);                       \
    const uint32_t a2 = gd_sign_pair<4 * J + 2>(v0, p.mul), a3 = gd_sign_pair<4 * J + 2>(v1, p.mul);               \
    _Pragma("unroll") for (int nt = 0; nt < NT; ++nt)                                                              \
        gd_mma(d[nt], a0, a1, a2, a3, b[g][c][nt][2 * J], b[g][c][nt][2 * J + 1]);                                 \
  }
          MBOK_GD_STEP(0)
          MBOK_GD_STEP(1)
          MBOK_GD_STEP(2)
          MBOK_GD_STEP(3)
#undef MBOK_GD_STEP
        }
        // scale the planes' rows by the group's scales
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (e == 1 && !two) break;
          const int plane = q + e;
          const int m = plane < K0 ? 0 : 1, k = plane - (m != 0 ? K0 : 0);
          const float a = __half2float(__ushort_as_half(*reinterpret_cast<const uint16_t*>(
              sa + m * kGdAlphaBytes + (g * p.s[m].K + k) * 16 + 2 * gq)));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (m == 0) {
              y[0][nt][0] = __fmaf_rn(a, d[nt][2 * e], y[0][nt][0]);
              y[0][nt][1] = __fmaf_rn(a, d[nt][2 * e + 1], y[0][nt][1]);
            } else {
              y[1][nt][0] = __fmaf_rn(a, d[nt][2 * e], y[1][nt][0]);
              y[1][nt][1] = __fmaf_rn(a, d[nt][2 * e + 1], y[1][nt][1]);
            }
          }
        }
      }
    }
    __syncwarp();   // every lane is done with the stage
    if (i + kGdDepth < n_mine) gd_issue(p, o + kGdDepth * stride, g0, ng, st, lane);
    else cp_async_commit();
    // the row group's sums meet: [buffer][warp][gate, up][column][row]
    float* buf = red + (i & 1) * (warps * G::kRed);
    float* mine = buf + warp * G::kRed;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) mine[(m * 8 * NT + 8 * nt + 2 * t + e) * 8 + gq] = y[m][nt][e];
    asm volatile("bar.sync %0, %1;\n" ::"r"(1 + rg), "r"(p.parts * 32) : "memory");
    // thread (vector, row): the parts in warp order (and hi + mid + lo of fp32)
    const float* all = buf + rg * p.parts * G::kRed;
    for (int item = part * 32 + lane; item < p.nb * 8; item += p.parts * 32) {
      const int vec = item >> 3, r = item & 7;
      const int row = o * kOctet + r;
      if (row >= M) continue;
      float total[2];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        float sum[XF32 ? 3 : 1];
#pragma unroll
        for (int q = 0; q < (XF32 ? 3 : 1); ++q) {
          const float* at = all + (m * 8 * NT + (XF32 ? 3 * vec + q : vec)) * 8 + r;
          sum[q] = 0.f;
          for (int w = 0; w < p.parts; ++w) sum[q] += at[w * G::kRed];
        }
        total[m] = XF32 ? (sum[0] + sum[XF32 ? 1 : 0]) + sum[XF32 ? 2 : 0] : sum[0];
      }
      if (p.nslab == 1) {
        store_act(p.h, p.h_bf16 != 0, size_t(vec) * M + row, gated(total[0], total[1]));
      } else {
        float* out = p.partial + (size_t(slab) * 2 * p.nb + vec) * M + row;
        __stcg(out, total[0]);
        __stcg(out + size_t(p.nb) * M, total[1]);
      }
    }
  }
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

// Vectors per launch (two 8-column tiles) and fragment columns they take.
static int gd_vectors(bool x_f32) { return x_f32 ? 5 : 16; }
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
  if (pl.row_groups > 8) pl.row_groups = 8;   // a named barrier each
  return pl;
}

static int gd_max_warps(int columns) { return columns <= 8 ? GdGeom<1>::kMaxWarps : GdGeom<2>::kMaxWarps; }

// One vector: the lookup kernel's partial sums; more: the slabs' sums of the
// launch with the most (0 with one slab).
size_t gemv_gated_workspace_bytes(const Shape& s, int batch) {
  if (batch == 1) return gemv_gated_lut_workspace_bytes(s);
  size_t most = 0;
  for (int f32 = 0; f32 < 2; ++f32) {   // the call may bring either type
    const int nb = batch < gd_vectors(f32 != 0) ? batch : gd_vectors(f32 != 0);
    for (int n = 1; n <= nb; ++n) {     // the last launch may have fewer vectors
      const GdPlan pl = gd_plan(s.G, gd_max_warps(gd_columns(f32 != 0, n)));
      if (pl.nslab > 1) {
        const size_t bytes = size_t(pl.nslab) * 2 * n * s.M * sizeof(float);
        if (bytes > most) most = bytes;
      }
    }
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
  p.stage_bytes = (p.s[0].K + p.s[1].K) * kGdPlaneBytes + 2 * kGdAlphaBytes;
  constexpr int kStageMax = 2 * MBOK_MAX_K * kGdPlaneBytes + 2 * kGdAlphaBytes;
  constexpr int kSmemMax = G::kMaxWarps * (kGdDepth * kStageMax + 2 * G::kRed * 4);
  static_assert(kSmemMax <= 227 * 1024, "the ring and the sums fit one CTA");
  auto fn = gemv_gated_kernel<NT, XF32>;
  static PerDeviceOnce attr_once;   // the attribute is per device context
  const cudaError_t ae = set_smem_attr_once(attr_once, reinterpret_cast<const void*>(fn), kSmemMax);
  if (ae != cudaSuccess) return ae;
  const int warps = pl.parts * pl.row_groups;
  const int per_slab = (p.s[0].O + pl.row_groups - 1) / pl.row_groups;   // CTAs that have an octet to begin with
  int ctas = device_sm_count() / pl.nslab;
  if (ctas < 1) ctas = 1;
  if (ctas > per_slab) ctas = per_slab;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas * pl.nslab);
  cfg.blockDim = dim3(warps * 32);
  cfg.dynamicSmemBytes = size_t(warps) * (kGdDepth * p.stage_bytes + 2 * G::kRed * 4);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, fn, p);
  if (e != cudaSuccess) return e;
  if (pl.nslab > 1) {
    const size_t n = size_t(p.nb) * p.s[0].M;
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
  const int per_launch = gd_vectors(x_f32);
  const size_t x_elem = x_f32 ? 4 : 2, h_elem = h_bf16 ? 2 : 4;
  for (int b0 = 0; b0 < batch; b0 += per_launch) {
    GatedMmaParams p = {};
    p.packed[0] = packed_gate;
    p.packed[1] = packed_up;
    p.alpha[0] = alpha_gate;
    p.alpha[1] = alpha_up;
    p.s[0] = gate;
    p.s[1] = up;
    p.x = static_cast<const char*>(x) + size_t(b0) * gate.N * x_elem;
    p.h = static_cast<char*>(h) + size_t(b0) * gate.M * h_elem;
    p.h_bf16 = h_bf16 ? 1 : 0;
    p.partial = static_cast<float*>(workspace);
    p.nb = batch - b0 < per_launch ? batch - b0 : per_launch;
    p.weights_static = weights_static ? 1 : 0;
    for (int i = 0; i < 8; ++i) p.mul[i] = 1u << (15 - 2 * i);
    const bool one = gd_columns(x_f32, p.nb) <= 8;
    const cudaError_t e = one ? (x_f32 ? launch_gd<1, true>(p, stream) : launch_gd<1, false>(p, stream))
                              : (x_f32 ? launch_gd<2, true>(p, stream) : launch_gd<2, false>(p, stream));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace mbok
