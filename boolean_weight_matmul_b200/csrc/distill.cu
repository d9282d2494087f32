// Distillation loss against a teacher's top logits, and its gradient.
//
// Per token t, with temperature tau, the student's logits z over V entries and
// the teacher's listed entries (c_i, v_i), i < top (the method fine-tunes a
// converted model by a KL loss on the logits of its full-precision teacher:
// Italian technical summary 2C, KD):
//     p_i   = exp(v_i / tau) / sum over the listed entries of exp(v / tau),
//     lse   = log sum_j exp(z_j / tau),     log q_j = z_j / tau - lse,
//     loss  = w sum_i p_i (log p_i - log q_{c_i}),
//     dz_j  = grad w / tau (q_j - sum over i with c_i = j of p_i).
//
// What bounds it: memory.  The floor reads each logit once and writes each
// gradient once.  So a row stays in registers between the sum that gives lse
// and the gradient that needs it: 512 threads hold 8 vectors of 16 bytes each
// (32768 bf16 or 16384 fp32 logits per CTA), all loads of a row issued before
// the first is used, and a row wider than one CTA is cut over a cluster of 2,
// 4 or 8, whose (max, sum) pairs meet in distributed shared memory.  Each
// thread keeps a running (max, sum) pair of its own; one block step merges
// them.  Warp 0 meanwhile forms the teacher's softmax from the list.  The
// listed entries' logits are gathered before anything is written, so dz may be
// the logits themselves.  Listed entries are few: their gradient is written
// over the dense pass's after a block barrier, with the p of equal indices
// added in list order.
//
// Sums, maxima and the softmax are fp32.  z / tau is taken in base 2: the
// factor log2(e) / tau is carried as two floats for fp32 logits, so that the
// exponent's error stays below the rounding of the result; bf16 gradients do
// not need the second one.
#include <cooperative_groups.h>

#include "mbok_common.cuh"

namespace mbok {

namespace cg = cooperative_groups;

constexpr int kDistillThreads = 512;
constexpr int kDistillWarps = kDistillThreads / 32;
constexpr int kDistillVecs = 8;                                       // 16-byte vectors per thread
constexpr int kDistillCtaVecs = kDistillThreads * kDistillVecs;       // per CTA
constexpr int kDistillMaxCluster = 8;
constexpr float kNegInf = -INFINITY;

struct DistillParams {
  const void* z;
  size_t ld;
  const float* teacher;     // [T][top]
  const int* index;         // [T][top]
  const float* weight;      // [T] or nullptr (1)
  const float* grad;        // [T] (backward) or nullptr (1)
  const float* lse_in;      // [T] (backward)
  float* loss;
  float* lse;
  void* dz;
  size_t ld_dz;
  int V, top;
  int slices;               // CTAs per row
  float inv_temp;           // 1 / tau
  float c2_hi, c2_lo;       // log2(e) / tau
};

template <bool F32>
struct DistillType {
  static constexpr int kVec = F32 ? 4 : 8;
  static constexpr int kBytes = F32 ? 4 : 2;
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.f32 %0, %1;\n" : "=f"(r) : "f"(x));
  return r;
}

// 2^((z - ref) log2(e) / tau) for ref = the running maximum.  Minus infinity
// (a masked logit) times a negative c2_lo would be NaN: it becomes the lowest
// finite value, whose power is 0 as well.
template <bool F32>
__device__ __forceinline__ float exp_gap(float z, float ref, const DistillParams& p) {
  float d = z - ref;
  if (!F32) return ex2(d * p.c2_hi);
  d = d == kNegInf ? -3.4028235e38f : d;
  return ex2(fmaf(d, p.c2_lo, d * p.c2_hi));
}

// Element i of a 16-byte vector as fp32.
template <bool F32>
__device__ __forceinline__ float vec_get(const uint4& v, int i) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if (F32) return __uint_as_float(w[i]);
  return (i & 1) ? __uint_as_float(w[i >> 1] & 0xFFFF0000u) : __uint_as_float(w[i >> 1] << 16);
}

// A row as 16-byte vectors: vector q holds elements q * kVec - a .. + kVec - 1,
// a = the row's start within its 16-byte line, in elements.  Only whole vectors
// inside the row are accessed as vectors; elements outside read as -infinity.
struct RowView {
  int a, nvec, V;
};

template <bool F32>
__device__ __forceinline__ RowView row_view(const void* row, int V) {
  using D = DistillType<F32>;
  RowView r;
  r.a = int(reinterpret_cast<uintptr_t>(row) & 15u) / D::kBytes;
  r.V = V;
  r.nvec = (r.a + V + D::kVec - 1) / D::kVec;
  return r;
}

template <bool F32>
__device__ __forceinline__ uint4 load_vec(const void* row, const RowView& r, int q) {
  using D = DistillType<F32>;
  const int e0 = q * D::kVec - r.a;
  const char* base = static_cast<const char*>(row) + ptrdiff_t(e0) * D::kBytes;
  if (e0 >= 0 && e0 + D::kVec <= r.V) {
    return __ldcs(reinterpret_cast<const uint4*>(base));
  }
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (F32) {
      const int e = e0 + i;
      w[i] = (e >= 0 && e < r.V) ? reinterpret_cast<const uint32_t*>(base)[i] : 0xFF800000u;
    } else {
      uint32_t h[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int e = e0 + 2 * i + j;
        h[j] = (e >= 0 && e < r.V) ? reinterpret_cast<const uint16_t*>(base)[2 * i + j] : 0xFF80u;
      }
      w[i] = h[0] | (h[1] << 16);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Store the gradients g[0 .. kVec) of vector q: one 16-byte store where the
// gradient's row lies like the logits' row (`aligned`) and the vector is whole.
template <bool F32>
__device__ __forceinline__ void store_vec(void* drow, const RowView& r, int q, bool aligned, const float* g) {
  using D = DistillType<F32>;
  const int e0 = q * D::kVec - r.a;
  char* base = static_cast<char*>(drow) + ptrdiff_t(e0) * D::kBytes;
  if (aligned && e0 >= 0 && e0 + D::kVec <= r.V) {
    uint4 v;
    if (F32) {
      v = make_uint4(__float_as_uint(g[0]), __float_as_uint(g[1]), __float_as_uint(g[2]), __float_as_uint(g[3]));
    } else {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(g[2 * i % D::kVec], g[(2 * i + 1) % D::kVec]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
      v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __stcs(reinterpret_cast<uint4*>(base), v);
    return;
  }
#pragma unroll
  for (int i = 0; i < D::kVec; ++i) {
    const int e = e0 + i;
    if (e < 0 || e >= r.V) continue;
    if (F32) reinterpret_cast<float*>(base)[i] = g[i];
    else reinterpret_cast<__nv_bfloat16*>(base)[i] = __float2bfloat16_rn(g[i]);
  }
}

template <bool F32>
__device__ __forceinline__ float load_elem(const void* row, int e) {
  if (F32) return static_cast<const float*>(row)[e];
  return bf16_bits_to_float(static_cast<const uint16_t*>(row)[e]);
}

// The listed entries of a row in shared memory.
struct TeacherSmem {
  int idx[MBOK_DISTILL_MAX_TOP];     // -1 where the entry is not used
  float z[MBOK_DISTILL_MAX_TOP];     // the student's logit there
  float p[MBOK_DISTILL_MAX_TOP];
  float logp[MBOK_DISTILL_MAX_TOP];
  int some;                          // the row has a used entry
};

// Warp 0: the teacher's softmax over the entries of row t whose index lies in
// [0, V) and whose logit is above -infinity; the gathered student logits.
template <bool F32>
__device__ __forceinline__ void teacher_softmax(const DistillParams& p, size_t t, const void* row, TeacherSmem& s,
                                                int lane) {
  const float* tv = p.teacher + t * p.top;
  const int* ti = p.index + t * p.top;
  float high = kNegInf;
  for (int i = lane; i < p.top; i += 32) {
    const int e = ti[i];
    const float v = tv[i];
    const bool used = e >= 0 && e < p.V && v != kNegInf;
    s.idx[i] = used ? e : -1;
    s.p[i] = v;
    s.z[i] = used ? load_elem<F32>(row, e) : 0.f;
    if (used) high = fmaxf(high, v);
  }
  int any = 0;
  for (int i = lane; i < p.top; i += 32) any |= s.idx[i] >= 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, o));
  any = __any_sync(0xffffffffu, any);
  float total = 0.f;
  for (int i = lane; i < p.top; i += 32)
    if (s.idx[i] >= 0) total += expf((s.p[i] - high) * p.inv_temp);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const float log_total = logf(total), inv_total = 1.f / total;
  for (int i = lane; i < p.top; i += 32) {
    if (s.idx[i] < 0) continue;
    const float gap = (s.p[i] - high) * p.inv_temp;
    s.p[i] = expf(gap) * inv_total;
    s.logp[i] = gap - log_total;
  }
  if (lane == 0) s.some = any;
}

// Warp 0: sum_i p_i (log p_i - log q_i) from the row's maximum m and the
// logarithm of its sum, log q = (z - m) / tau - log_sum.  The two logarithms
// are subtracted entry by entry: their sums over the list are each far larger
// than the loss of a student that is close to its teacher.
__device__ __forceinline__ float listed_loss(const DistillParams& p, const TeacherSmem& s, float m, float log_sum,
                                             int lane) {
  float sum = 0.f;
  for (int i = lane; i < p.top; i += 32) {
    if (s.idx[i] < 0) continue;
    const float prob = s.p[i];
    // an entry of probability 0 adds nothing, whatever the student's logit
    if (prob != 0.f) sum += prob * (s.logp[i] - ((s.z[i] - m) * p.inv_temp - log_sum));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// Merge two (max, sum) pairs; a pair without a finite logit keeps its sum as
// it is (0, or NaN from a NaN logit).
template <bool F32>
__device__ __forceinline__ void merge(float& m, float& s, float m2, float s2, const DistillParams& p) {
  const float hi = fmaxf(m, m2);
  s = (m == kNegInf ? s : s * exp_gap<F32>(m, hi, p)) + (m2 == kNegInf ? s2 : s2 * exp_gap<F32>(m2, hi, p));
  m = hi;
}

// Zeros for the vectors of a row that has no weight.
template <bool F32>
__device__ __forceinline__ void zero_row(void* drow, const RowView& r, int q0, int q1, bool aligned) {
  const float g[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int q = q0 + int(threadIdx.x); q < q1; q += kDistillThreads) store_vec<F32>(drow, r, q, aligned, g);
}

// The listed entries of this CTA's vectors [q0, q1): dz = scale (q - p), with
// the p of equal indices added in list order by the first of them.
template <bool F32, class Q>
__device__ __forceinline__ void patch_listed(const DistillParams& p, const TeacherSmem& s, void* drow,
                                             const RowView& r, int q0, int q1, float scale, Q prob_of) {
  using D = DistillType<F32>;
  for (int i = threadIdx.x; i < p.top; i += kDistillThreads) {
    const int e = s.idx[i];
    if (e < 0) continue;
    const int q = (e + r.a) / D::kVec;
    if (q < q0 || q >= q1) continue;
    float sum = 0.f;
    bool first = true;
    for (int j = 0; j < p.top; ++j) {
      if (s.idx[j] != e) continue;
      if (j < i) { first = false; break; }
      sum += s.p[j];
    }
    if (!first) continue;
    const float g = scale * (prob_of(s.z[i]) - sum);
    if (F32) static_cast<float*>(drow)[e] = g;
    else static_cast<__nv_bfloat16*>(drow)[e] = __float2bfloat16_rn(g);
  }
}

// Loss, lse and (WRITE) the gradient with grad = 1: one cluster per row.
// Without WRITE a CTA may pass over its slice in several chunks.
template <bool F32, bool WRITE>
__global__ void __launch_bounds__(kDistillThreads, 2) distill_row_kernel(const __grid_constant__ DistillParams p) {
  using D = DistillType<F32>;
  __shared__ TeacherSmem teach;
  __shared__ float2 warp_pair[kDistillWarps];
  __shared__ float2 cta_pair[kDistillMaxCluster];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t t = blockIdx.x / unsigned(p.slices);
  const int slice = int(blockIdx.x % unsigned(p.slices));
  const void* row = static_cast<const char*>(p.z) + t * p.ld * D::kBytes;
  void* drow = WRITE ? static_cast<char*>(p.dz) + t * p.ld_dz * D::kBytes : nullptr;
  const RowView r = row_view<F32>(row, p.V);
  const int per = (r.nvec + p.slices - 1) / p.slices;
  const int q0 = min(slice * per, r.nvec), q1 = min(q0 + per, r.nvec);
  const bool aligned = WRITE && ((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(drow)) & 15u) == 0;
  const float w = p.weight != nullptr ? p.weight[t] : 1.f;

  // the row's CTAs have all started once this barrier's wait returns (below,
  // before the first access to another CTA's shared memory)
  if (p.slices > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory");

  uint4 v[kDistillVecs];
  float m = kNegInf, s = 0.f;
  if (w != 0.f) {
    for (int c0 = q0; c0 < q1; c0 += kDistillCtaVecs) {
#pragma unroll
      for (int i = 0; i < kDistillVecs; ++i) {
        const int q = c0 + i * kDistillThreads + int(threadIdx.x);
        if (q < q1) v[i] = load_vec<F32>(row, r, q);
        else v[i] = F32 ? make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u)
                        : make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
      }
      if (c0 == q0 && warp == 0) teacher_softmax<F32>(p, t, row, teach, lane);
      float cm = kNegInf;
#pragma unroll
      for (int i = 0; i < kDistillVecs; ++i)
#pragma unroll
        for (int j = 0; j < D::kVec; ++j) cm = fmaxf(cm, vec_get<F32>(v[i], j));
      const float ref = cm == kNegInf ? 0.f : cm;
      float cs = 0.f;
#pragma unroll
      for (int i = 0; i < kDistillVecs; ++i) {
        if (c0 + i * kDistillThreads >= q1) break;   // nothing from here on, for the whole block
#pragma unroll
        for (int j = 0; j < D::kVec; ++j) cs += exp_gap<F32>(vec_get<F32>(v[i], j), ref, p);
      }
      if (c0 == q0) {
        m = cm;
        s = cs;
      } else {
        merge<F32>(m, s, cm, cs, p);
      }
    }
    if (q0 >= q1 && warp == 0) teacher_softmax<F32>(p, t, row, teach, lane);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
      merge<F32>(m, s, m2, s2, p);
    }
    if (lane == 0) warp_pair[warp] = make_float2(m, s);
  }
  __syncthreads();
  if (w != 0.f) {
    const float2 pr = warp_pair[lane % kDistillWarps];
    m = lane < kDistillWarps ? pr.x : kNegInf;
    s = lane < kDistillWarps ? pr.y : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
      merge<F32>(m, s, m2, s2, p);
    }
  }
  if (p.slices > 1) {
    // every CTA of the row gets every pair; nothing remote is touched after the barrier
    cg::cluster_group cluster = cg::this_cluster();
    asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory");
    if (threadIdx.x < unsigned(p.slices))
      *cluster.map_shared_rank(&cta_pair[slice], int(threadIdx.x)) = make_float2(m, s);
    cluster.sync();
    m = cta_pair[0].x;
    s = cta_pair[0].y;
    for (int i = 1; i < p.slices; ++i) merge<F32>(m, s, cta_pair[i].x, cta_pair[i].y, p);
  }
  const bool used = w != 0.f && teach.some != 0;
  if (!used) {
    // no weight, or nothing listed: no loss and no gradient, whatever the logits
    if (slice == 0 && threadIdx.x == 0) {
      p.loss[t] = 0.f;
      p.lse[t] = 0.f;
    }
    if (WRITE) zero_row<F32>(drow, r, q0, q1, aligned);
    return;
  }
  if (m == kNegInf) s = NAN;   // no logit above -infinity: the row has no distribution
  if (slice == 0 && warp == 0) {
    const float log_sum = logf(s);
    const float sum = listed_loss(p, teach, m, log_sum, lane);
    if (lane == 0) {
      p.loss[t] = w * sum;
      p.lse[t] = fmaf(m, p.inv_temp, log_sum);
    }
  }
  if (WRITE) {
    const float scale = w * p.inv_temp, inv = 1.f / s, qs = scale * inv;
#pragma unroll
    for (int i = 0; i < kDistillVecs; ++i) {
      const int q = q0 + i * kDistillThreads + int(threadIdx.x);
      if (q >= q1) break;
      float g[D::kVec];
#pragma unroll
      for (int j = 0; j < D::kVec; ++j) g[j] = qs * exp_gap<F32>(vec_get<F32>(v[i], j), m, p);
      store_vec<F32>(drow, r, q, aligned, g);
    }
    __syncthreads();
    patch_listed<F32>(p, teach, drow, r, q0, q1, scale, [&](float z) { return exp_gap<F32>(z, m, p) * inv; });
  }
}

// The gradient from a forward pass's lse: slices of a row are independent.
template <bool F32>
__global__ void __launch_bounds__(kDistillThreads, 2) distill_grad_kernel(const __grid_constant__ DistillParams p) {
  using D = DistillType<F32>;
  __shared__ TeacherSmem teach;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t t = blockIdx.x / unsigned(p.slices);
  const int slice = int(blockIdx.x % unsigned(p.slices));
  const void* row = static_cast<const char*>(p.z) + t * p.ld * D::kBytes;
  void* drow = static_cast<char*>(p.dz) + t * p.ld_dz * D::kBytes;
  const RowView r = row_view<F32>(row, p.V);
  const int per = (r.nvec + p.slices - 1) / p.slices;
  const int q0 = min(slice * per, r.nvec), q1 = min(q0 + per, r.nvec);
  const bool aligned = ((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(drow)) & 15u) == 0;
  const float w = (p.weight != nullptr ? p.weight[t] : 1.f) * (p.grad != nullptr ? p.grad[t] : 1.f);
  if (w == 0.f) {
    zero_row<F32>(drow, r, q0, q1, aligned);
    return;
  }
  uint4 v[kDistillVecs];
#pragma unroll
  for (int i = 0; i < kDistillVecs; ++i) {
    const int q = q0 + i * kDistillThreads + int(threadIdx.x);
    if (q < q1) v[i] = load_vec<F32>(row, r, q);
  }
  if (warp == 0) teacher_softmax<F32>(p, t, row, teach, lane);
  const float lse = p.lse_in[t];
  __syncthreads();   // the list is ready, and its logits are read before any gradient is written
  if (teach.some == 0) {
    zero_row<F32>(drow, r, q0, q1, aligned);
    return;
  }
  // q = 2^(z c2 - lse log2 e), both factors as two floats
  const float scale = w * p.inv_temp;
  constexpr float kLog2eHi = 1.44269502f, kLog2eLo = 1.92596299e-8f;
  const float l_hi = lse * kLog2eHi;
  const float l_lo = fmaf(lse, kLog2eHi, -l_hi) + lse * kLog2eLo;
  auto prob = [&](float z) {
    if (F32) z = z == kNegInf ? -3.4028235e38f : z;
    const float x = fmaf(z, p.c2_hi, -l_hi);
    return ex2(F32 ? x + fmaf(z, p.c2_lo, -l_lo) : x - l_lo);
  };
#pragma unroll
  for (int i = 0; i < kDistillVecs; ++i) {
    const int q = q0 + i * kDistillThreads + int(threadIdx.x);
    if (q >= q1) break;
    float g[D::kVec];
#pragma unroll
    for (int j = 0; j < D::kVec; ++j) g[j] = scale * prob(vec_get<F32>(v[i], j));
    store_vec<F32>(drow, r, q, aligned, g);
  }
  __syncthreads();
  patch_listed<F32>(p, teach, drow, r, q0, q1, scale, prob);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// Vectors of the widest row (a row may start anywhere in a 16-byte line).
static int max_vecs(int V, bool f32) {
  const int vec = f32 ? 4 : 8;
  return (V + vec - 1 + vec - 1) / vec;
}

template <bool F32, bool WRITE>
static cudaError_t launch_row(const DistillParams& p, int T, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(T) * unsigned(p.slices));
  cfg.blockDim = dim3(kDistillThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(p.slices);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, distill_row_kernel<F32, WRITE>, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

static DistillParams distill_params(const void* z, size_t ld, int V, const float* teacher, const int* index, int top,
                                    float temperature, const float* weight) {
  DistillParams p = {};
  p.z = z;
  p.ld = ld;
  p.V = V;
  p.teacher = teacher;
  p.index = index;
  p.top = top;
  p.weight = weight;
  p.inv_temp = 1.f / temperature;
  const double c2 = 1.4426950408889634 / double(temperature);
  p.c2_hi = float(c2);
  p.c2_lo = float(c2 - double(p.c2_hi));
  return p;
}

cudaError_t launch_distill_backward(const void* z, bool f32, int T, int V, size_t ld, const float* teacher,
                                    const int* index, int top, float temperature, const float* weight,
                                    const float* lse, const float* grad, void* dz, size_t ld_dz,
                                    cudaStream_t stream) {
  DistillParams p = distill_params(z, ld, V, teacher, index, top, temperature, weight);
  p.lse_in = lse;
  p.grad = grad;
  p.dz = dz;
  p.ld_dz = ld_dz;
  const int vecs = max_vecs(V, f32);
  p.slices = (vecs + kDistillCtaVecs - 1) / kDistillCtaVecs;
  // few rows: more slices, down to one vector per thread
  while (long(T) * p.slices < 2L * device_sm_count() && vecs / (2 * p.slices) >= kDistillThreads) p.slices *= 2;
  const unsigned grid = unsigned(T) * unsigned(p.slices);
  if (f32) distill_grad_kernel<true><<<grid, kDistillThreads, 0, stream>>>(p);
  else distill_grad_kernel<false><<<grid, kDistillThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_distill_loss(const void* z, bool f32, int T, int V, size_t ld, const float* teacher,
                                const int* index, int top, float temperature, const float* weight, float* loss,
                                float* lse, void* dz, size_t ld_dz, cudaStream_t stream) {
  DistillParams p = distill_params(z, ld, V, teacher, index, top, temperature, weight);
  p.loss = loss;
  p.lse = lse;
  p.dz = dz;
  p.ld_dz = ld_dz;
  const int vecs = max_vecs(V, f32);
  p.slices = 1;
  while (p.slices < kDistillMaxCluster &&
         (vecs > p.slices * kDistillCtaVecs ||
          (long(T) * p.slices < 2L * device_sm_count() && vecs / (2 * p.slices) >= kDistillThreads)))
    p.slices *= 2;
  const bool fits = vecs <= p.slices * kDistillCtaVecs;
  if (dz != nullptr && fits)
    return f32 ? launch_row<true, true>(p, T, stream) : launch_row<false, true>(p, T, stream);
  const cudaError_t e = f32 ? launch_row<true, false>(p, T, stream) : launch_row<false, false>(p, T, stream);
  if (e != cudaSuccess || dz == nullptr) return e;
  // a row wider than a cluster holds: the gradient reads it again
  return launch_distill_backward(z, f32, T, V, ld, teacher, index, top, temperature, weight, lse, nullptr, dz, ld_dz,
                                 stream);
}

}  // namespace mbok
