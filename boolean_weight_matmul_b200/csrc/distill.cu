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
// What bounds it: memory.  The floor reads each logit from DRAM once and writes
// each gradient once.  A CTA takes a row (or, with few rows, a slice of one: a
// cluster of 2, 4 or 8 CTAs per row whose (max, sum) pairs meet in distributed
// shared memory): 256 threads pass over it for lse, then again for the
// gradient, which finds the row in L2 (five CTAs per SM hold rows of about 50 MB
// in flight on the whole GPU at V = 32000 bf16, L2 is 126 MB).  Keeping the row
// in registers between the passes instead left two CTAs per SM, too few to hide
// one's loads behind the other's arithmetic: 2048 x 32000 bf16 took 109 us against
// 74.  Apart (1024 x 32000 fp32) loss and gradient take 67 us, 5.8 TB/s.  All three
// kernels start while the preceding grid ends (72 and 61 us without).
// Each thread keeps a running (max, sum) pair of its own; one block step merges
// them.  A ninth warp meanwhile forms the teacher's softmax from the list and
// gathers the listed logits before any of them is written over, so dz may be the
// logits themselves.  Listed entries are few: their gradient is written over the dense
// pass's after a block barrier, with the p of equal indices added in list order.
//
// Arithmetic.  Everything runs in base 2, and a running sum is kept as
// sum 2^((z - m) c), c = log2(e) / tau, for a reference m, the largest logit.  The
// difference is taken first: it is exact near m, and the exponent is right, and
// never above 0, wherever the logits lie.  (A multiply-add of z and the rounded m c,
// one operation less, is off by that rounding: beyond 2^31 its power is an infinity,
// also in a thread whose logits are all masked by a large negative number.  2048 x
// 32000 bf16, loss alone: 27.8 us by multiply-adds, 29.0 by differences.)
// lse = m / tau + ln sum.  Sums, maxima and the softmax are fp32.  The gradient
// from a given lse, and the row ring, take multiply-adds: their reference is of
// moderate size, or the row's result is limited by lse's own rounding anyway.
#include <cooperative_groups.h>

#include <cfloat>
#include <cmath>

#include "tc_common.cuh"

namespace mbok {

namespace cg = cooperative_groups;

constexpr int kDistillThreads = 256;                                  // that pass over the row
constexpr int kDistillWarps = kDistillThreads / 32;
constexpr int kDistillBlock = kDistillThreads + 32;                   // and the teacher's warp
constexpr int kDistillCtas = 5;                                       // per SM
constexpr int kDistillVecs = 4;                                       // 16-byte vectors in flight per thread
constexpr int kDistillChunk = kDistillThreads * kDistillVecs;         // vectors per step of a CTA
constexpr int kDistillMaxCluster = 8;
constexpr float kNegInf = -INFINITY;
constexpr float kLn2 = 0.693147182f;   // ln 2 rounded

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
  float c2;                 // log2(e) / tau rounded
  float c2_hi, c2_lo;       // ... and as a sum; c2_lo > 0
};

template <bool F32>
struct DistillType {
  static constexpr int kVec = F32 ? 4 : 8;
  static constexpr int kBytes = F32 ? 4 : 2;
};

// 2^x; results below 2^-126 are 0 (without that the instruction needs three
// more around it, which bounded the kernel: 78 us at 2048 x 32000 bf16).
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
  return r;
}

// (z - m) log2(e) / tau, m finite.
__device__ __forceinline__ float exponent(float z, float m, const DistillParams& p) { return (z - m) * p.c2; }
__device__ __forceinline__ float exp_from(float z, float m, const DistillParams& p) { return ex2(exponent(z, m, p)); }

// z log2(e) / tau - r, for |r| far below 2^24.  fp32 logits: log2(e) / tau as two
// floats, so that the exponent's error stays at its rounding; bf16 gradients do not
// need the second one.  c2_lo is positive, so that a logit of minus infinity
// (masked) gives that and not NaN.
template <bool F32>
__device__ __forceinline__ float exponent_near(float z, float r, const DistillParams& p) {
  const float y = fmaf(z, p.c2_hi, -r);
  return F32 ? fmaf(z, p.c2_lo, y) : y;
}

// Whether a row whose largest logit is m has a distribution: not if all are
// masked (by -infinity or the type's lowest value), nor where m log2(e) / tau
// overflows.
template <bool F32>
__device__ __forceinline__ bool has_distribution(float m, const DistillParams& p) {
  const float lowest = F32 ? -FLT_MAX : __uint_as_float(0xFF7F0000u);
  return m > lowest && fabsf(m * p.c2) < INFINITY;
}

// Natural logarithm of a sum that refers to the largest logit m.
__device__ __forceinline__ float lse_of(float m, float log2_sum, const DistillParams& p) {
  return fmaf(m, p.inv_temp, log2_sum * kLn2);
}

// Element i of a 16-byte vector as fp32.
template <bool F32>
__device__ __forceinline__ float vec_get(const uint4& v, int i) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if (F32) return __uint_as_float(w[i]);
  return (i & 1) ? __uint_as_float(w[i >> 1] & 0xFFFF0000u) : __uint_as_float(w[i >> 1] << 16);
}

// A row as 16-byte vectors: vector q holds elements q * kVec - a .. + kVec - 1,
// a = the row's start within its 16-byte line, in elements.  Vectors qb <= q < qe
// lie inside the row and are accessed whole; the row's ends element by element
// (functions of their own, so that the loops stay short), elements outside read
// as -infinity.
struct RowView {
  const void* row;
  const uint4* vec;   // vector 0 (its first a elements lie before the row)
  int a, qb, qe, nvec, V;
};

template <bool F32>
__device__ __forceinline__ RowView row_view(const void* row, int V) {
  using D = DistillType<F32>;
  RowView r;
  r.row = row;
  const unsigned off = unsigned(reinterpret_cast<uintptr_t>(row)) & 15u;
  r.vec = reinterpret_cast<const uint4*>(static_cast<const char*>(row) - off);
  r.a = int(off) / D::kBytes;
  r.qb = off != 0 ? 1 : 0;
  r.qe = (r.a + V) / D::kVec;
  r.nvec = (r.a + V + D::kVec - 1) / D::kVec;
  r.V = V;
  return r;
}

template <bool F32>
__device__ __noinline__ uint4 load_edge(const void* row, int e0, int V) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (F32) {
      const int e = e0 + i;
      w[i] = (e >= 0 && e < V) ? static_cast<const uint32_t*>(row)[e] : 0xFF800000u;
    } else {
      uint32_t h[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int e = e0 + 2 * i + j;
        h[j] = (e >= 0 && e < V) ? static_cast<const uint16_t*>(row)[e] : 0xFF80u;
      }
      w[i] = h[0] | (h[1] << 16);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool F32>
__device__ __forceinline__ uint4 load_vec(const RowView& r, int q) {
  if (q >= r.qb && q < r.qe) return __ldcs(r.vec + q);
  return load_edge<F32>(r.row, q * DistillType<F32>::kVec - r.a, r.V);
}

// The gradients v (packed as the row) of vector q, element by element.
template <bool F32>
__device__ __noinline__ void store_edge(void* drow, int e0, int V, uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < DistillType<F32>::kVec; ++i) {
    const int e = e0 + i;
    if (e < 0 || e >= V) continue;
    if (F32) static_cast<uint32_t*>(drow)[e] = w[i % 4];
    else static_cast<uint16_t*>(drow)[e] = uint16_t(w[i / 2 % 4] >> (16 * (i & 1)));
  }
}

// A row of gradients: its vectors, where it lies in its line like the logits'
// row (`vec`, else nullptr), and its elements.
struct GradView {
  void* row;
  uint4* vec;
};

template <bool F32>
__device__ __forceinline__ GradView grad_view(void* drow, const RowView& r) {
  GradView d;
  d.row = drow;
  const unsigned off = unsigned(reinterpret_cast<uintptr_t>(drow)) & 15u;
  d.vec = int(off) == r.a * DistillType<F32>::kBytes
              ? reinterpret_cast<uint4*>(static_cast<char*>(drow) - off)
              : nullptr;
  return d;
}

// Gradients g[0 .. kVec) rounded to the row's type, as one vector.
template <bool F32>
__device__ __forceinline__ uint4 pack_vec(const float* g) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (F32) {
      w[i] = __float_as_uint(g[i]);
    } else {
      const __nv_bfloat162 b = __floats2bfloat162_rn(g[2 * i], g[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool F32>
__device__ __forceinline__ void store_vec(const GradView& d, const RowView& r, int q, const float* g) {
  const uint4 v = pack_vec<F32>(g);
  if (d.vec != nullptr && q >= r.qb && q < r.qe) __stcs(d.vec + q, v);
  else store_edge<F32>(d.row, q * DistillType<F32>::kVec - r.a, r.V, v);
}

template <bool F32>
__device__ __forceinline__ float load_elem(const void* row, int e) {
  if (F32) return static_cast<const float*>(row)[e];
  return bf16_bits_to_float(static_cast<const uint16_t*>(row)[e]);
}

// The listed entries of a row in shared memory; the indices padded with -1 to a
// multiple of 4.
struct Teacher {
  unsigned char* at;   // 16-byte aligned
  int top4;            // entries, padded
  __device__ __forceinline__ int& idx(int i) const { return reinterpret_cast<int*>(at)[i]; }   // -1: not used
  __device__ __forceinline__ float& z(int i) const { return reinterpret_cast<float*>(at)[top4 + i]; }   // its logit
  __device__ __forceinline__ float& p(int i) const { return reinterpret_cast<float*>(at)[2 * top4 + i]; }
  __device__ __forceinline__ float& logp(int i) const { return reinterpret_cast<float*>(at)[3 * top4 + i]; }
  // p summed over the entries with this index; -1 at all but the first of them
  __device__ __forceinline__ float& sum(int i) const { return reinterpret_cast<float*>(at)[4 * top4 + i]; }
  __device__ __forceinline__ int& some() const { return reinterpret_cast<int*>(at)[5 * top4]; }   // any used entry
};
// Bytes of one Teacher (a multiple of 16).
__host__ __device__ constexpr int teacher_bytes(int top) { return 20 * ((top + 3) / 4 * 4) + 16; }
__device__ __forceinline__ Teacher teacher_at(unsigned char* at, int top) { return Teacher{at, (top + 3) & ~3}; }

// One warp: the teacher's softmax over the entries of row t whose index lies in
// [0, V) and whose logit is above -infinity; the gathered student logits.
template <bool F32>
__device__ __forceinline__ void teacher_softmax(const DistillParams& p, size_t t, const void* row, const Teacher& s,
                                                int lane) {
  const float* tv = p.teacher + t * p.top;
  const int* ti = p.index + t * p.top;
  float high = kNegInf;
  int any = 0;
  if (lane < s.top4 - p.top) s.idx(p.top + lane) = -1;
  // Four entries per lane at a time: all indices are under way before the first
  // is used, then all logits (one after another, these loads from memory took
  // most of a row's time on the SM).
  for (int i0 = lane; i0 < p.top; i0 += 128) {
    int e[4];
    float v[4], z[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int i = i0 + 32 * n;
      e[n] = i < p.top ? ti[i] : -1;
      v[n] = i < p.top ? tv[i] : kNegInf;
    }
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      if (!(e[n] >= 0 && e[n] < p.V && v[n] != kNegInf)) e[n] = -1;
      z[n] = e[n] >= 0 ? load_elem<F32>(row, e[n]) : kNegInf;
    }
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int i = i0 + 32 * n;
      if (i < p.top) {
        s.idx(i) = e[n];
        s.p(i) = v[n];
        s.z(i) = z[n];
      }
      if (e[n] >= 0) {
        high = fmaxf(high, v[n]);
        any = 1;
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, o));
  any = __any_sync(0xffffffffu, any);
  float total = 0.f;
  for (int i = lane; i < p.top; i += 32)
    if (s.idx(i) >= 0) total += expf((s.p(i) - high) * p.inv_temp);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const float log_total = logf(total), inv_total = 1.f / total;
  for (int i = lane; i < p.top; i += 32) {
    if (s.idx(i) < 0) continue;
    const float gap = (s.p(i) - high) * p.inv_temp;
    s.p(i) = expf(gap) * inv_total;
    s.logp(i) = gap - log_total;
  }
  if (lane == 0) s.some() = any;
  __syncwarp();
  // Is an index given again?  Indices are compared four at a time; only where
  // one is are the probabilities looked at, in list order.
  for (int i = lane; i < p.top; i += 32) {
    const int e = s.idx(i);
    float sum = -1.f;
    if (e >= 0) {
      int same = 0;
      const int4* list = reinterpret_cast<const int4*>(s.at);
#pragma unroll 4
      for (int j = 0; j < s.top4 / 4; ++j) {
        const int4 c = list[j];
        same += (c.x == e) + (c.y == e) + (c.z == e) + (c.w == e);
      }
      sum = s.p(i);
      if (same > 1) {
        sum = 0.f;
        bool first = true;
        for (int j = 0; j < p.top; ++j) {
          if (s.idx(j) != e) continue;
          if (j < i) first = false;
          sum += s.p(j);
        }
        if (!first) sum = -1.f;
      }
    }
    s.sum(i) = sum;
  }
}

// One warp: sum_i p_i (log p_i - log q_i) from log2 of the row's sum and the
// exponents that refer to it, exponent_of(z).  The two logarithms are subtracted entry by entry: their sums over
// the list are each far larger than the loss of a student that is close to its
// teacher.
template <class Y>
__device__ __forceinline__ float listed_loss(const DistillParams& p, const Teacher& s, float log2_sum, Y exponent_of,
                                             int lane) {
  float sum = 0.f;
  for (int i = lane; i < p.top; i += 32) {
    if (s.idx(i) < 0) continue;
    const float prob = s.p(i);
    const float log2_q = exponent_of(s.z(i)) - log2_sum;
    // an entry of probability 0 adds nothing, whatever the student's logit
    if (prob != 0.f) sum += prob * fmaf(-log2_q, kLn2, s.logp(i));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// Merge two (reference, sum) pairs; a pair without a logit above -infinity keeps
// its sum as it is (0, or NaN from a NaN logit).
__device__ __forceinline__ void merge(float& m, float& s, float m2, float s2, const DistillParams& p) {
  const float hi = fmaxf(m, m2);
  s = (m == kNegInf ? s : s * exp_from(m, hi, p)) + (m2 == kNegInf ? s2 : s2 * exp_from(m2, hi, p));
  m = hi;
}

// The largest of n vectors' logits (NaN ignored; -infinity if there is none).
template <bool F32, int n>
__device__ __forceinline__ float vecs_max(const uint4* v) {
  if constexpr (F32) {
    float m = kNegInf;
#pragma unroll
    for (int i = 0; i < n; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) m = fmaxf(m, vec_get<true>(v[i], j));
    return m;
  } else {
    const uint32_t none = 0xFF80FF80u;
    __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162*>(&none);
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&w[j]));
    }
    return fmaxf(__low2float(m), __high2float(m));
  }
}

// Zeros for the vectors of a row that has no weight.
template <bool F32>
__device__ __forceinline__ void zero_row(const GradView& d, const RowView& r, int q0, int q1) {
  const float g[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int q = q0 + int(threadIdx.x); q < q1; q += kDistillBlock) store_vec<F32>(d, r, q, g);
}

// Entry i of the list in vectors [q0, q1), if it is the first with its index:
// its gradient scale (q - p).  Returns the element, or -1.
template <bool F32, class Q>
__device__ __forceinline__ int listed_grad(const Teacher& s, const RowView& r, int q0, int q1, int i, float scale,
                                           Q prob_of, float& grad) {
  const float sum = s.sum(i);
  if (sum == -1.f) return -1;   // not used, or not the first (a NaN probability is)
  const int e = s.idx(i);
  const int q = (e + r.a) / DistillType<F32>::kVec;
  if (q < q0 || q >= q1) return -1;
  grad = scale * (prob_of(s.z(i)) - sum);
  return e;
}

template <bool F32>
__device__ __forceinline__ void store_elem(void* row, int e, float g) {
  if (F32) static_cast<float*>(row)[e] = g;
  else static_cast<__nv_bfloat16*>(row)[e] = __float2bfloat16_rn(g);
}

template <bool F32, class Q>
__device__ __forceinline__ void patch_listed(const DistillParams& p, const Teacher& s, void* drow, const RowView& r,
                                             int q0, int q1, float scale, Q prob_of) {
  for (int i = threadIdx.x; i < p.top; i += kDistillBlock) {
    float g;
    const int e = listed_grad<F32>(s, r, q0, q1, i, scale, prob_of, g);
    if (e >= 0) store_elem<F32>(drow, e, g);
  }
}

// The vectors c0 + i * kDistillThreads + threadIdx.x < q1 of a row; others read
// as -infinity.
template <bool F32>
__device__ __forceinline__ void load_chunk(const RowView& r, int c0, int q1, uint4 v[kDistillVecs]) {
#pragma unroll
  for (int i = 0; i < kDistillVecs; ++i) {
    const int q = c0 + i * kDistillThreads + int(threadIdx.x);
    const uint32_t none = F32 ? 0xFF800000u : 0xFF80FF80u;
    v[i] = q < q1 ? load_vec<F32>(r, q) : make_uint4(none, none, none, none);
  }
}

// Store prob(logit) * scale for the vectors of a chunk.
template <bool F32, class Q>
__device__ __forceinline__ void store_chunk(const GradView& d, const RowView& r, int c0, int q1,
                                            const uint4 v[kDistillVecs], Q value) {
  using D = DistillType<F32>;
#pragma unroll
  for (int i = 0; i < kDistillVecs; ++i) {
    const int q = c0 + i * kDistillThreads + int(threadIdx.x);
    if (q >= q1) break;
    float g[D::kVec];
#pragma unroll
    for (int j = 0; j < D::kVec; ++j) g[j] = value(vec_get<F32>(v[i], j));
    store_vec<F32>(d, r, q, g);
  }
}

// Loss, lse and (WRITE) the gradient with grad = 1: a cluster of p.slices CTAs
// per row.
template <bool F32, bool WRITE>
__global__ void __launch_bounds__(kDistillBlock, kDistillCtas)
distill_row_kernel(const __grid_constant__ DistillParams p) {
  using D = DistillType<F32>;
  __shared__ __align__(16) unsigned char teach_smem[teacher_bytes(MBOK_DISTILL_MAX_TOP)];
  __shared__ float2 warp_pair[kDistillWarps];
  __shared__ float2 cta_pair[kDistillMaxCluster];
  const Teacher teach = teacher_at(teach_smem, p.top);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t t = blockIdx.x / unsigned(p.slices);
  const int slice = int(blockIdx.x % unsigned(p.slices));
  const void* row = static_cast<const char*>(p.z) + t * p.ld * D::kBytes;
  void* drow = WRITE ? static_cast<char*>(p.dz) + t * p.ld_dz * D::kBytes : nullptr;
  const RowView r = row_view<F32>(row, p.V);
  const int per = (r.nvec + p.slices - 1) / p.slices;
  const int q0 = min(slice * per, r.nvec), q1 = min(q0 + per, r.nvec);
  const GradView d = grad_view<F32>(drow, r);
  pdl_wait();   // nothing is read or written before the preceding grid is complete

  // the row's CTAs have all started once this barrier's wait returns (below,
  // before the first access to another CTA's shared memory)
  if (p.slices > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory");

  const float w = p.weight != nullptr ? p.weight[t] : 1.f;
  float ref = kNegInf, s = 0.f;
  if (warp == kDistillWarps) {
    if (w != 0.f) teacher_softmax<F32>(p, t, row, teach, lane);
  } else {
    for (int c0 = q0; c0 < q1; c0 += kDistillChunk) {
      uint4 v[kDistillVecs];
      load_chunk<F32>(r, c0, q1, v);
      if (w == 0.f) break;   // the first loads did not wait for the weight
      // rescale the running sum where the reference grows
      const float top = vecs_max<F32, kDistillVecs>(v);
      if (top > ref) {
        s *= exp_from(ref, top, p);   // 0 x 0 the first time
        ref = top;
      }
      const float from = ref == kNegInf ? 0.f : ref;
#pragma unroll
      for (int i = 0; i < kDistillVecs; ++i)
#pragma unroll
        for (int j = 0; j < D::kVec; ++j) s += exp_from(vec_get<F32>(v[i], j), from, p);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float r2 = __shfl_xor_sync(0xffffffffu, ref, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
      merge(ref, s, r2, s2, p);
    }
    if (lane == 0) warp_pair[warp] = make_float2(ref, s);
  }
  __syncthreads();
  {
    const float2 pr = warp_pair[lane % kDistillWarps];
    ref = pr.x;
    s = pr.y;
#pragma unroll
    for (int o = kDistillWarps / 2; o > 0; o >>= 1) {
      const float r2 = __shfl_xor_sync(0xffffffffu, ref, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
      merge(ref, s, r2, s2, p);
    }
  }
  if (p.slices > 1) {
    // every CTA of the row gets every pair; nothing remote is touched after the barrier
    cg::cluster_group cluster = cg::this_cluster();
    asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory");
    if (threadIdx.x < unsigned(p.slices))
      *cluster.map_shared_rank(&cta_pair[slice], int(threadIdx.x)) = make_float2(ref, s);
    cluster.sync();
    ref = cta_pair[0].x;
    s = cta_pair[0].y;
    for (int i = 1; i < p.slices; ++i) merge(ref, s, cta_pair[i].x, cta_pair[i].y, p);
  }
  // The next grid may start from here on: started with this one, its CTAs filled
  // the SMs unevenly where a grid is less than a wave (82 x 5591 fp32: 7.6 us, from
  // here 5.5; 64 x 128000 bf16 4 % less).
  pdl_launch();
  const bool used = w != 0.f && teach.some() != 0;
  if (!used) {
    // no weight, or nothing listed: no loss and no gradient, whatever the logits
    if (slice == 0 && threadIdx.x == 0) {
      p.loss[t] = 0.f;
      p.lse[t] = 0.f;
    }
    if (WRITE) zero_row<F32>(d, r, q0, q1);
    return;
  }
  if (!has_distribution<F32>(ref, p)) s = NAN;
  if (slice == 0 && warp == kDistillWarps) {
    const float log2_sum = log2f(s);
    const float sum = listed_loss(p, teach, log2_sum, [&](float z) { return exponent(z, ref, p); }, lane);
    if (lane == 0) {
      p.loss[t] = w * sum;
      p.lse[t] = lse_of(ref, log2_sum, p);
    }
  }
  if (WRITE) {
    const float scale = w * p.inv_temp, inv = 1.f / s, qs = scale * inv;
    if (warp < kDistillWarps) {
      for (int c0 = q0; c0 < q1; c0 += kDistillChunk) {
        uint4 v[kDistillVecs];
        load_chunk<F32>(r, c0, q1, v);
        store_chunk<F32>(d, r, c0, q1, v, [&](float z) { return qs * exp_from(z, ref, p); });
      }
    }
    __syncthreads();
    patch_listed<F32>(p, teach, drow, r, q0, q1, scale, [&](float z) { return exp_from(z, ref, p) * inv; });
  }
}

// The gradient from a forward pass's lse: slices of a row are independent.
template <bool F32>
__global__ void __launch_bounds__(kDistillBlock, kDistillCtas)
distill_grad_kernel(const __grid_constant__ DistillParams p) {
  using D = DistillType<F32>;
  __shared__ __align__(16) unsigned char teach_smem[teacher_bytes(MBOK_DISTILL_MAX_TOP)];
  const Teacher teach = teacher_at(teach_smem, p.top);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t t = blockIdx.x / unsigned(p.slices);
  const int slice = int(blockIdx.x % unsigned(p.slices));
  const void* row = static_cast<const char*>(p.z) + t * p.ld * D::kBytes;
  void* drow = static_cast<char*>(p.dz) + t * p.ld_dz * D::kBytes;
  const RowView r = row_view<F32>(row, p.V);
  const int per = (r.nvec + p.slices - 1) / p.slices;
  const int q0 = min(slice * per, r.nvec), q1 = min(q0 + per, r.nvec);
  const GradView d = grad_view<F32>(drow, r);
  pdl_launch();
  pdl_wait();
  uint4 v[kDistillVecs];
  if (warp < kDistillWarps) load_chunk<F32>(r, q0, q1, v);   // not waiting for the weight
  const float weight = p.weight != nullptr ? p.weight[t] : 1.f;
  const float w = weight * (p.grad != nullptr ? p.grad[t] : 1.f);
  const float lse = p.lse_in[t];
  if (weight == 0.f || w == 0.f) {   // a weight of 0 also masks a gradient that is no number
    zero_row<F32>(d, r, q0, q1);
    return;
  }
  if (warp == kDistillWarps) teacher_softmax<F32>(p, t, row, teach, lane);
  __syncthreads();   // the list is ready, and its logits are read before any gradient is written
  if (teach.some() == 0) {
    zero_row<F32>(d, r, q0, q1);
    return;
  }
  // q = 2^(z c2 - lse log2 e), both factors as two floats
  const float scale = w * p.inv_temp;
  constexpr float kLog2eHi = 1.44269502f, kLog2eLo = 1.92596299e-8f;
  const float l_hi = lse * kLog2eHi;
  const float l_lo = fmaf(lse, kLog2eHi, -l_hi) + lse * kLog2eLo;
  const float l = l_hi + l_lo;   // bf16: one float is enough
  auto prob = [&](float z) {
    return ex2(F32 ? fmaf(z, p.c2_hi, -l_hi) + fmaf(z, p.c2_lo, -l_lo) : fmaf(z, p.c2_hi, -l));
  };
  if (warp < kDistillWarps) {
    for (int c0 = q0; c0 < q1; c0 += kDistillChunk) {
      if (c0 > q0) load_chunk<F32>(r, c0, q1, v);
      store_chunk<F32>(d, r, c0, q1, v, [&](float z) { return scale * prob(z); });
    }
  }
  __syncthreads();
  patch_listed<F32>(p, teach, drow, r, q0, q1, scale, prob);
}

// ---- many rows that fit shared memory three times: the row stays on the SM ----
//
// One CTA per SM walks rows blockIdx.x, + gridDim.x, ...; a ring of three slots
// holds them.  A slot's copy warp brings a row's whole vectors in by one bulk
// copy, waits until its gradient stands in the same slot, sends that out by one
// bulk copy and goes on to the slot's next row.  24 warps pass over one row at a
// time, so that of three slots two are always in transfer; four warps prepare
// the lists of the rows ahead, one writes the listed entries' gradients and the
// loss behind them.  DRAM reads, writes and arithmetic of different rows thus
// overlap all the time, which rows on independent CTAs do not: those start
// together and stay in step.
//
// The reference of a row's sum is not its maximum but that of 32 vectors spread over
// it, which the slot's copy warp finds, rounded to a whole exponent: any reference
// serves from which no term overflows and no exponent is so large that its rounding
// counts, and with it the pass needs no maxima, no rescaling and no list.  Whole
// exponents are exact to add, so that the sum is then taken to one in [1, 2) and
// every further exponent refers to that: rounded where it is small, wherever the
// logits lie.  Where the sum leaves 2^-32 .. 2^32 (exponents of up to 32, rounded by
// 2^-20) or is NaN, the row is summed again from its maximum.  (From 0, without a
// maximum, exponents of rows at 69 were off by 2^-18 and losses by 4e-6.)
// Only the last step needs the list: it is long in coming for the first row.
// 2048 x 32000 bf16, loss and gradient: 59.5 us, 4.4 TB/s of logits and gradients
// (two passes on independent CTAs: 74 us).  The exponentials' pipe is 52 % busy, the
// issue slots 65 %: a row's two passes and their barriers take as long as its copies.
//
// In place: a slot is copied out behind its list (done), and a row's ends, which no
// copy moves, are written by the warp that waits for the list (the row warps, which
// do not, would overwrite listed logits that a list warp has yet to gather).
constexpr int kRingSlots = 3;
constexpr int kRingRowWarps = 24;
constexpr int kRingRowThreads = kRingRowWarps * 32;
constexpr int kRingLists = 4;   // lists, and warps that prepare them
constexpr int kRingListWarp0 = kRingRowWarps;
constexpr int kRingEndWarp = kRingListWarp0 + kRingLists;
constexpr int kRingCopyWarp0 = kRingEndWarp + 1;
constexpr int kRingThreads = (kRingCopyWarp0 + kRingSlots) * 32;
constexpr int kRingSmemMax = 224 * 1024;
constexpr float kRingFarthest = 0x1p20f;   // references' magnitude: whole numbers, exact to add

static __device__ unsigned int g_distill_error;

struct RingParams {
  DistillParams d;
  int T;
  int slot_bytes;   // multiple of 128
};

// Barrier of the row warps alone.
__device__ __forceinline__ void row_sync() { asm volatile("bar.sync 1, %0;\n" ::"n"(kRingRowThreads) : "memory"); }

// Sum (or maximum) of x over the row warps, in a fixed order.
template <bool MAX>
__device__ __forceinline__ float row_reduce(float x, float* warp_val, int warp, int lane) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float y = __shfl_xor_sync(0xffffffffu, x, o);
    x = MAX ? fmaxf(x, y) : x + y;
  }
  if (lane == 0) warp_val[warp] = x;
  row_sync();
  float all = warp_val[0];
#pragma unroll
  for (int w = 1; w < kRingRowWarps; ++w) all = MAX ? fmaxf(all, warp_val[w]) : all + warp_val[w];
  return all;
}

// Vector q of a row: from its slot, the row's ends from memory.
template <bool F32>
__device__ __forceinline__ uint4 ring_vec(const RowView& r, const uint4* vecs, int q) {
  return q >= r.qb && q < r.qe ? vecs[q] : load_edge<F32>(r.row, q * DistillType<F32>::kVec - r.a, r.V);
}

// Put the gradients g of vector q in its slot; where the gradients' rows lie
// otherwise than the logits' (never in place), in memory.  The row's ends follow
// with the listed entries.
template <bool F32>
__device__ __forceinline__ void ring_put(const RowView& r, const GradView& d, uint4* vecs, int q, const float* g) {
  if (d.vec == nullptr) store_edge<F32>(d.row, q * DistillType<F32>::kVec - r.a, r.V, pack_vec<F32>(g));
  else if (q >= r.qb && q < r.qe) vecs[q] = pack_vec<F32>(g);
}

// One warp: the reference of a row's first sum, the largest logit among 32 vectors
// spread over the row, as a whole exponent; 0 if all are masked.
template <bool F32>
__device__ __forceinline__ float ring_reference(const DistillParams& p, const RowView& r, const uint4* vecs, int lane) {
  float y = kNegInf;
  if (r.qe > r.qb) {
    const uint4 v = vecs[r.qb + lane * (r.qe - r.qb) / 32];
    y = rintf(vecs_max<F32, 1>(&v) * p.c2_hi);
  }
  const int high = __reduce_max_sync(0xffffffffu, int(fminf(fmaxf(y, -kRingFarthest), kRingFarthest)));
  return high == int(-kRingFarthest) ? 0.f : float(high);
}

// The row warps' two passes for a row summed from its maximum m, a function of its
// own: rare, and beside the others it would lengthen their loops.
template <bool F32>
__device__ __noinline__ float ring_sum_from(const DistillParams& p, RowView r, const uint4* vecs, float m) {
  float s0 = 0.f, s1 = 0.f;
  for (int q = threadIdx.x; q < r.nvec; q += kRingRowThreads) {
    const uint4 v = ring_vec<F32>(r, vecs, q);
#pragma unroll
    for (int j = 0; j < DistillType<F32>::kVec; j += 2) {
      s0 += exp_from(vec_get<F32>(v, j), m, p);
      s1 += exp_from(vec_get<F32>(v, j + 1), m, p);
    }
  }
  return s0 + s1;
}
template <bool F32>
__device__ __noinline__ void ring_grad_from(const DistillParams& p, RowView r, GradView d, uint4* vecs, float m,
                                            float qs) {
  for (int q = threadIdx.x; q < r.nvec; q += kRingRowThreads) {
    const uint4 v = ring_vec<F32>(r, vecs, q);
    float g[DistillType<F32>::kVec];
#pragma unroll
    for (int j = 0; j < DistillType<F32>::kVec; ++j) g[j] = qs * exp_from(vec_get<F32>(v, j), m, p);
    ring_put<F32>(r, d, vecs, q, g);
  }
}

template <bool F32>
__global__ void __launch_bounds__(kRingThreads, 1) distill_ring_kernel(const __grid_constant__ RingParams rp) {
  using D = DistillType<F32>;
  const DistillParams& p = rp.d;
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ __align__(8) uint64_t full[kRingSlots];     // a slot's row landed
  __shared__ __align__(8) uint64_t ready[kRingSlots];    // ... and its reference is found
  __shared__ __align__(8) uint64_t dense[kRingSlots];    // its dense gradient stands in the slot
  __shared__ __align__(8) uint64_t done[kRingSlots];     // ... and its listed entries
  __shared__ __align__(8) uint64_t lfull[kRingLists], lempty[kRingLists];   // a list is ready, is read
  __shared__ __align__(16) float warp_val[3][kRingRowWarps];
  __shared__ float row_from[kRingSlots];                 // the first sum's reference
  __shared__ float4 row_sum[kRingSlots];                 // reference, sum, weight, whether summed from the maximum
  __shared__ int s_fail;                                 // a wait gave up: no row is copied out any more
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tbytes = teacher_bytes(p.top);
  unsigned char* lists = ring + kRingSlots * rp.slot_bytes;
  const int nrows = (rp.T - 1 - int(blockIdx.x)) / int(gridDim.x) + 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kRingSlots; ++s) {
      tc_mbar_init(&full[s], 1);
      tc_mbar_init(&ready[s], 1);
      tc_mbar_init(&dense[s], kRingRowWarps);
      tc_mbar_init(&done[s], 1);
    }
    for (int k = 0; k < kRingLists; ++k) {
      tc_mbar_init(&lfull[k], 1);
      tc_mbar_init(&lempty[k], 1);
    }
    s_fail = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
  }
  __syncthreads();
  pdl_launch();
  pdl_wait();
  auto row_of = [&](int i) { return size_t(blockIdx.x) + size_t(i) * gridDim.x; };
  auto logits_of = [&](size_t t) {
    return static_cast<const void*>(static_cast<const char*>(p.z) + t * p.ld * D::kBytes);
  };
  auto grads_of = [&](size_t t) { return static_cast<void*>(static_cast<char*>(p.dz) + t * p.ld_dz * D::kBytes); };
  auto weight_of = [&](size_t t) { return p.weight != nullptr ? p.weight[t] : 1.f; };
  auto list_of = [&](int i) { return teacher_at(lists + i % kRingLists * tbytes, p.top); };
  bool ok = true;
  auto failed = [&]() {
    *reinterpret_cast<volatile int*>(&s_fail) = 1;
    ok = false;
  };

  if (warp < kRingRowWarps) {
    // ---- the rows (a wait that gave up is not waited for again, but the warps
    // keep to their barriers; what they still write stays within the outputs, which
    // are undefined then) ----
    const int gt = threadIdx.x;
    float w = weight_of(row_of(0));
    for (int i = 0; i < nrows; ++i) {
      const size_t t = row_of(i);
      const int s = i % kRingSlots;
      uint4* vecs = reinterpret_cast<uint4*>(ring + s * rp.slot_bytes);
      const RowView r = row_view<F32>(logits_of(t), p.V);
      const GradView d = grad_view<F32>(grads_of(t), r);
      const float next_w = i + 1 < nrows ? weight_of(row_of(i + 1)) : 0.f;
      auto vec_at = [&](int q) { return ring_vec<F32>(r, vecs, q); };
      if (ok && !tc_wait(&ready[s], unsigned(i / kRingSlots) & 1u)) failed();
      const bool used = w != 0.f;
      float s0 = 0.f, s1 = 0.f, from = row_from[s];
      for (int q = gt; used && q < r.nvec; q += kRingRowThreads) {
        const uint4 v = vec_at(q);
#pragma unroll
        for (int j = 0; j < D::kVec; j += 2) {
          s0 += ex2(exponent_near<F32>(vec_get<F32>(v, j), from, p));
          s1 += ex2(exponent_near<F32>(vec_get<F32>(v, j + 1), from, p));
        }
      }
      float ref = from, sum = row_reduce<false>(used ? s0 + s1 : 1.f, warp_val[i & 1], warp, lane);
      const bool far = !(sum > 0x1p-32f && sum < 0x1p32f);   // the same for all; a NaN is far
      if (!far) {   // the sum in [1, 2)
        const uint32_t bits = __float_as_uint(sum);
        ref += float(int(bits >> 23) - 127);
        sum = __uint_as_float((bits & 0x007FFFFFu) | 0x3F800000u);
      } else {   // from the row's maximum
        float m = kNegInf;
        for (int q = gt; q < r.nvec; q += kRingRowThreads) {
          const uint4 v = vec_at(q);
#pragma unroll
          for (int j = 0; j < D::kVec; ++j) m = fmaxf(m, vec_get<F32>(v, j));
        }
        ref = row_reduce<true>(m, warp_val[2], warp, lane);
        row_sync();   // warp_val[i & 1] is read
        sum = row_reduce<false>(has_distribution<F32>(ref, p) ? ring_sum_from<F32>(p, r, vecs, ref) : NAN,
                                warp_val[i & 1], warp, lane);
      }
      if (gt == 0) row_sum[s] = make_float4(ref, sum, w, far ? 1.f : 0.f);
      const float inv = 1.f / sum, qs = w * p.inv_temp * inv;
      // the gradient in the row's place; an unused row's is 0 whatever its logits
      if (far) ring_grad_from<F32>(p, r, d, vecs, ref, qs);
      for (int q = gt; !far && q < r.nvec; q += kRingRowThreads) {
        float g[D::kVec];
        if (used) {
          const uint4 v = vec_at(q);
#pragma unroll
          for (int j = 0; j < D::kVec; ++j) g[j] = qs * ex2(exponent_near<F32>(vec_get<F32>(v, j), ref, p));
        } else {
#pragma unroll
          for (int j = 0; j < D::kVec; ++j) g[j] = 0.f;
        }
        ring_put<F32>(r, d, vecs, q, g);
      }
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");   // generic writes -> bulk copy
      __syncwarp();
      if (lane == 0) tc_arrive(&dense[s]);
      w = next_w;
    }
  } else if (warp < kRingEndWarp) {
    // ---- the lists of the rows ahead, one warp per list ----
    const int b = warp - kRingListWarp0;
    for (int i = b, u = 0; i < nrows; i += kRingLists, ++u) {
      if (u > 0 && !tc_wait(&lempty[b], unsigned(u - 1) & 1u)) {
        failed();
        break;
      }
      const size_t t = row_of(i);
      if (weight_of(t) != 0.f) teacher_softmax<F32>(p, t, logits_of(t), list_of(i), lane);
      __syncwarp();
      if (lane == 0) tc_arrive(&lfull[b]);
    }
  } else if (warp == kRingEndWarp) {
    // ---- loss, lse and the listed entries' gradients ----
    for (int i = 0; i < nrows; ++i) {
      const size_t t = row_of(i);
      const int s = i % kRingSlots;
      if (!tc_wait(&lfull[i % kRingLists], unsigned(i / kRingLists) & 1u) ||
          !tc_wait(&dense[s], unsigned(i / kRingSlots) & 1u)) {
        failed();
        break;
      }
      const RowView r = row_view<F32>(logits_of(t), p.V);
      const GradView d = grad_view<F32>(grads_of(t), r);
      const Teacher teach = list_of(i);
      const float4 rs = row_sum[s];
      const float ref = rs.x, w = rs.z;
      const bool far = rs.w != 0.f;
      auto y_of = [&](float z) { return far ? exponent(z, ref, p) : exponent_near<F32>(z, ref, p); };
      uint4* vecs = reinterpret_cast<uint4*>(ring + s * rp.slot_bytes);
      const bool used = w != 0.f && teach.some() != 0;
      const float inv = 1.f / rs.y, scale = w * p.inv_temp;
      if (d.vec != nullptr) {
        // the row's ends, an element a lane: before the first whole vector, behind the last
        const int head = r.qb == 0 ? 0 : min(D::kVec - r.a, r.V), tail = max(head, r.qe * D::kVec - r.a);
        const int e = lane < head ? lane : tail + lane - head;
        if (e < r.V)
          store_elem<F32>(d.row, e, used ? scale * inv * ex2(y_of(load_elem<F32>(r.row, e))) : 0.f);
        __syncwarp();   // listed entries among them are written after
      }
      if (used) {
        const float log2_sum = log2f(rs.y);
        for (int n = lane; n < p.top; n += 32) {
          float g;
          const int e = listed_grad<F32>(teach, r, 0, r.nvec, n, scale,
                                         [&](float z) { return ex2(y_of(z)) * inv; }, g);
          if (e < 0) continue;
          const int q = (e + r.a) / D::kVec;
          if (d.vec != nullptr && q >= r.qb && q < r.qe) store_elem<F32>(vecs, e + r.a, g);
          else store_elem<F32>(d.row, e, g);
        }
        const float kl = listed_loss(p, teach, log2_sum, y_of, lane);
        if (lane == 0) {
          p.loss[t] = w * kl;
          p.lse[t] = far ? lse_of(ref, log2_sum, p) : (ref + log2_sum) * kLn2;
        }
      } else {
        // no weight (the row warps wrote zeros), or nothing listed
        if (lane == 0) {
          p.loss[t] = 0.f;
          p.lse[t] = 0.f;
        }
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        for (int q = lane; w != 0.f && q < r.nvec; q += 32) {
          if (d.vec == nullptr) store_edge<F32>(d.row, q * D::kVec - r.a, r.V, zero);
          else if (q >= r.qb && q < r.qe) vecs[q] = zero;
        }
      }
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        tc_arrive(&done[s]);
        tc_arrive(&lempty[i % kRingLists]);
      }
    }
  } else {
    // ---- a slot's copies (its first lane), and its row's reference ----
    const int s = warp - kRingCopyWarp0;
    unsigned char* slot = ring + s * rp.slot_bytes;
    float w = s < nrows ? weight_of(row_of(s)) : 0.f;
    for (int i = s, u = 0; i < nrows; i += kRingSlots, ++u) {
      const size_t t = row_of(i);
      const RowView r = row_view<F32>(logits_of(t), p.V);
      const GradView d = grad_view<F32>(grads_of(t), r);
      const uint32_t bytes = r.qe > r.qb ? uint32_t(r.qe - r.qb) * 16 : 0u;
      const bool wanted = bytes > 0 && w != 0.f;
      if (lane == 0) {
        tc_arrive_expect_tx(&full[s], wanted ? bytes : 0u);
        if (wanted)
          asm volatile(
              "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
                  tc_smem(slot + r.qb * 16)),
              "l"(r.vec + r.qb), "r"(bytes), "r"(tc_smem(&full[s]))
              : "memory");
      }
      if (i + kRingSlots < nrows) w = weight_of(row_of(i + kRingSlots));
      if (!tc_wait(&full[s], unsigned(u) & 1u)) failed();
      __syncwarp();
      const float from = wanted ? ring_reference<F32>(p, r, reinterpret_cast<const uint4*>(slot), lane) : 0.f;
      if (lane == 0) {
        row_from[s] = from;
        tc_arrive(&ready[s]);
      }
      if (!tc_wait(&done[s], unsigned(u) & 1u)) failed();
      if (__any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&s_fail) != 0)) break;
      if (lane == 0 && bytes > 0 && d.vec != nullptr) {
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n" ::"l"(d.vec + r.qb),
                     "r"(tc_smem(slot + r.qb * 16)), "r"(bytes)
                     : "memory");
        asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
        // the slot may be filled again once the copy has read it
        asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory");
      }
      __syncwarp();
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory");
  }
  if (!ok) {
    // record it, and let this CTA's copies in land (bounded) before it leaves
    atomicOr(&g_distill_error, 1u);
    for (int s = 0; s < kRingSlots; ++s) {
      (void)tc_wait(&full[s], 0u, kTcDrainNs);
      (void)tc_wait(&full[s], 1u, kTcDrainNs);
    }
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// CTAs per row: one, and with few rows more (a power of two, at most `most`)
// until every SM has its five or a CTA's slice is one step.
static int row_slices(int T, int V, bool f32, int most) {
  const int vec = f32 ? 4 : 8;
  const int vecs = (V + vec - 1 + vec - 1) / vec;   // a row may start anywhere in a 16-byte line
  int slices = 1;
  while (slices < most && long(T) * slices < long(kDistillCtas) * device_sm_count() &&
         vecs > slices * kDistillChunk)
    slices *= 2;
  return slices;
}

template <bool F32, bool WRITE>
static cudaError_t launch_row(const DistillParams& p, int T, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(T) * unsigned(p.slices));
  cfg.blockDim = dim3(kDistillBlock);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(p.slices);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, distill_row_kernel<F32, WRITE>, p);
}

// Bytes of a ring slot: the row's vectors wherever it starts in its line.
static int ring_slot_bytes(int V, bool f32) {
  const long vec = f32 ? 4 : 8;
  const long bytes = (V + vec - 1 + vec - 1) / vec * 16;
  return bytes > kRingSmemMax ? kRingSmemMax : int((bytes + 127) / 128 * 128);
}
constexpr int kRingMinRows = 4;   // rows per SM from which the ring kernel is taken

template <bool F32>
static cudaError_t launch_ring(const DistillParams& d, int T, int slot, int smem, cudaStream_t stream) {
  auto fn = distill_ring_kernel<F32>;
  static PerDeviceOnce attr_once;   // the attribute is per device context
  const cudaError_t ae = set_smem_attr_once(attr_once, reinterpret_cast<const void*>(fn), kRingSmemMax);
  if (ae != cudaSuccess) return ae;
  RingParams rp;
  rp.d = d;
  rp.T = T;
  rp.slot_bytes = slot;
  const int sms = device_sm_count();
  return launch_dependent(fn, dim3(unsigned(T < sms ? T : sms)), dim3(kRingThreads), size_t(smem), stream, rp);
}

// Reads and clears the ring kernel's error flag; ~0u if the read itself failed.
unsigned distill_error_flags() {
  unsigned v = 0;
  if (cudaMemcpyFromSymbol(&v, g_distill_error, sizeof(v)) != cudaSuccess) return ~0u;
  const unsigned z = 0;
  if (v != 0 && cudaMemcpyToSymbol(g_distill_error, &z, sizeof(z)) != cudaSuccess) return ~0u;
  return v;
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
  // rounded down, and below c2 also where fp32 holds it: c2_lo stays positive
  p.c2 = p.c2_hi = float(c2);
  if (double(p.c2_hi) >= c2) p.c2_hi = nextafterf(p.c2_hi, 0.f);
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
  p.slices = row_slices(T, V, f32, 1 << 20);
  return launch_dependent(f32 ? distill_grad_kernel<true> : distill_grad_kernel<false>,
                          dim3(unsigned(T) * unsigned(p.slices)), dim3(kDistillBlock), 0, stream, p);
}

cudaError_t launch_distill_loss(const void* z, bool f32, int T, int V, size_t ld, const float* teacher,
                                const int* index, int top, float temperature, const float* weight, float* loss,
                                float* lse, void* dz, size_t ld_dz, cudaStream_t stream) {
  DistillParams p = distill_params(z, ld, V, teacher, index, top, temperature, weight);
  p.loss = loss;
  p.lse = lse;
  p.dz = dz;
  p.ld_dz = ld_dz;
  if (dz != nullptr) {
    const int slot = ring_slot_bytes(V, f32);
    const int smem = kRingSlots * slot + kRingLists * teacher_bytes(top);
    if (T >= kRingMinRows * device_sm_count() && smem <= kRingSmemMax)
      return f32 ? launch_ring<true>(p, T, slot, smem, stream) : launch_ring<false>(p, T, slot, smem, stream);
  }
  p.slices = row_slices(T, V, f32, kDistillMaxCluster);
  if (dz != nullptr) return f32 ? launch_row<true, true>(p, T, stream) : launch_row<false, true>(p, T, stream);
  return f32 ? launch_row<true, false>(p, T, stream) : launch_row<false, false>(p, T, stream);
}

}  // namespace mbok
