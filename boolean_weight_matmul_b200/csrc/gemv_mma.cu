// The plain form of the tensor-core GEMV (kernel and notes: gemv_mma.cuh) and
// the self-check of its bounded waits.
#include "gemv_mma.cuh"

namespace mbok {

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

template <int K, int NT, bool XF32, int MINB, bool DEEP>
static cudaError_t launch_mma_k(const GemvMmaParams& p, cudaStream_t stream) {
  auto fn = gemv_mma_kernel<K, NT, XF32, MINB, DEEP, false>;
  using G = MmaGeom<K, NT, XF32, DEEP>;
  static PerDeviceOnce attr_once;   // the attribute is per device context
  const cudaError_t ae = set_smem_attr_once(attr_once, reinterpret_cast<const void*>(fn), G::kSmem);
  if (ae != cudaSuccess) return ae;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.s.O + 1) / 2);
  cfg.blockDim = dim3(kMmaThreads);
  cfg.dynamicSmemBytes = G::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

template <int K, bool DEEP>
static cudaError_t launch_mma_nt_d(const GemvMmaParams& p, bool x_f32, cudaStream_t stream) {
  const int cols = x_f32 ? 3 * p.nb : p.nb;
  const bool big_grid = (p.s.O + 1) / 2 >= 3 * device_sm_count();
  if (cols <= 8) {
    if (big_grid)
      return x_f32 ? launch_mma_k<K, 1, true, 3, DEEP>(p, stream) : launch_mma_k<K, 1, false, 3, DEEP>(p, stream);
    return x_f32 ? launch_mma_k<K, 1, true, 2, DEEP>(p, stream) : launch_mma_k<K, 1, false, 2, DEEP>(p, stream);
  }
  constexpr int kMinB2 = K >= 3 ? 1 : 2;
  return x_f32 ? launch_mma_k<K, 2, true, kMinB2, DEEP>(p, stream)
               : launch_mma_k<K, 2, false, kMinB2, DEEP>(p, stream);
}

template <int K>
static cudaError_t launch_mma_nt(const GemvMmaParams& p, bool x_f32, cudaStream_t stream) {
  const int slices = (p.s.N + MmaGeom<K, 1, false>::kCols - 1) / MmaGeom<K, 1, false>::kCols;
  return slices >= kMmaDeepMinSlices ? launch_mma_nt_d<K, true>(p, x_f32, stream)
                                     : launch_mma_nt_d<K, false>(p, x_f32, stream);
}

// Self-check of the bounded waits: one warp waits, with the kernels' own wait
// helper, on an mbarrier that nothing completes; when the wait gives up it
// records the same flag a stuck copy would.
__global__ void wait_timeout_probe_kernel(unsigned long long limit_ns) {
  __shared__ __align__(8) uint64_t bar;
  if (threadIdx.x == 0) mm_bar_init(&bar, 1);
  __syncwarp();
  asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  __syncwarp();
  const bool done = __all_sync(0xffffffffu, mm_wait(&bar, 0u, limit_ns));
  if (!done && threadIdx.x == 0) atomicOr(&g_gemv_mma_error, 1u);
}

cudaError_t launch_wait_timeout_probe(unsigned timeout_us, cudaStream_t stream) {
  wait_timeout_probe_kernel<<<1, 32, 0, stream>>>(1000ull * timeout_us);
  return cudaGetLastError();
}

// Reads and clears the kernel's error flag; ~0u if the read itself failed.
unsigned gemv_mma_error_flags() {
  unsigned v = 0;
  if (cudaMemcpyFromSymbol(&v, g_gemv_mma_error, sizeof(v)) != cudaSuccess) return ~0u;
  const unsigned z = 0;
  if (v != 0 && cudaMemcpyToSymbol(g_gemv_mma_error, &z, sizeof(z)) != cudaSuccess) return ~0u;
  return v;
}

// Y[b] = W X[b] for b < batch (x: [batch][N], y: [batch][M]); launches cover
// up to 16 bf16 or 5 fp32 vectors each.
cudaError_t launch_gemv_mma(const uint8_t* packed, const uint16_t* alpha, const Shape& s,
                            const void* x, bool x_f32, int batch, float* y, cudaStream_t stream,
                            bool weights_static) {
  const int per_launch = x_f32 ? (8 * kMaxNT) / 3 : 8 * kMaxNT;
  const size_t x_elem = x_f32 ? 4 : 2;
  for (int b0 = 0; b0 < batch; b0 += per_launch) {
    GemvMmaParams p = {};
    p.packed = packed;
    p.alpha = alpha;
    p.x = static_cast<const char*>(x) + size_t(b0) * s.N * x_elem;
    p.y = y + size_t(b0) * s.M;
    p.s = s;
    p.nb = batch - b0 < per_launch ? batch - b0 : per_launch;
    p.weights_static = weights_static ? 1 : 0;
    for (int i = 0; i < 8; ++i) p.mul[i] = 1u << (15 - 2 * i);
    cudaError_t e;
    switch (s.K) {
      case 1: e = launch_mma_nt<1>(p, x_f32, stream); break;
      case 2: e = launch_mma_nt<2>(p, x_f32, stream); break;
      case 3: e = launch_mma_nt<3>(p, x_f32, stream); break;
      default: e = launch_mma_nt<4>(p, x_f32, stream); break;
    }
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace mbok
