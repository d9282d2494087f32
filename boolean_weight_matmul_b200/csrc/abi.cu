// C ABI of the MBOK library: argument checks on the host, then launches on
// the caller's stream.  Nothing here allocates, synchronises or keeps state
// beyond cached kernel attributes.
#include <atomic>
#include <cmath>

#include "mbok_common.cuh"

namespace mbok {
cudaError_t launch_pack_bits(const int8_t*, const Shape&, uint8_t*, cudaStream_t);
cudaError_t launch_pack_alpha(const uint16_t*, const Shape&, uint16_t*, cudaStream_t);
cudaError_t launch_residual_binarize(const float*, const Shape&, uint8_t*, __half*, float*,
                                     cudaStream_t);
cudaError_t launch_refit_alpha(const float*, const uint8_t*, const Shape&, __half*, cudaStream_t);
size_t svid_workspace_bytes(int, int);
cudaError_t launch_svid_binarize(const float*, const Shape&, int, uint8_t*, __half*, __half*, float*, void*,
                                 cudaStream_t);
cudaError_t launch_gemv_lut(const uint8_t*, const uint16_t*, const Shape&, const void*, bool,
                            float*, void*, cudaStream_t, bool);
cudaError_t launch_gemv_lut4(const uint8_t*, const uint16_t*, const Shape&, const void*, bool, float*,
                             cudaStream_t, bool);
bool gemv_lut4_supported(const Shape&);
unsigned gemv_lut4_error_flags();
size_t gemv_lut_workspace_bytes(const Shape&);
size_t gemv_svid_workspace_bytes(const Shape&);
cudaError_t launch_gemv_svid(const uint8_t*, const uint16_t*, const uint16_t*, const Shape&, const void*, bool,
                             float*, void*, cudaStream_t, bool);
unsigned gemv_mma_error_flags();
cudaError_t launch_wait_timeout_probe(unsigned, cudaStream_t);
cudaError_t launch_gemv_mma(const uint8_t*, const uint16_t*, const Shape&, const void*, bool, int,
                            float*, cudaStream_t, bool);
cudaError_t launch_gemv(const uint8_t*, const uint16_t*, const Shape&, const void*, bool, int, float*,
                        void*, cudaStream_t);

cudaError_t launch_gemv_lut_multi(int, const uint8_t* const*, const uint16_t* const*, const int*, const int*, int,
                                  const void*, bool, float*, void*, cudaStream_t, bool);
size_t gemv_multi_workspace_bytes(int, const int*, const int*, int);

size_t gemv_gated_workspace_bytes(const Shape&, int);
cudaError_t launch_gemv_gated(const uint8_t*, const uint16_t*, const Shape&, const uint8_t*, const uint16_t*,
                              const Shape&, const void*, bool, int, void*, bool, void*, cudaStream_t, bool);
cudaError_t launch_gated_backward(const uint16_t*, const uint16_t*, const uint16_t*, size_t, uint16_t*, uint16_t*,
                                  uint16_t*, cudaStream_t);
size_t gemm_gated_workspace_bytes(int, int, int);
cudaError_t launch_gemm_gated(const uint8_t*, const uint16_t*, const Shape&, const uint8_t*, const uint16_t*,
                              const Shape&, const uint16_t*, int, uint16_t*, uint16_t*, uint16_t*, void*,
                              cudaStream_t);
size_t gemm_backward_workspace_bytes(int, const Shape*, int);
cudaError_t launch_gemm_backward(int, const uint8_t* const*, const uint16_t* const*, const Shape*, const uint16_t*,
                                 int, const uint16_t* const*, uint16_t*, float* const*, void*, cudaStream_t);
unsigned gemv_gated_error_flags();
unsigned gemm_pair_error_flags();
unsigned gemm_dalpha_error_flags();
unsigned distill_error_flags();
cudaError_t launch_distill_loss(const void*, bool, int, int, size_t, const float*, const int*, int, float,
                                const float*, float*, float*, void*, size_t, cudaStream_t);
cudaError_t launch_distill_backward(const void*, bool, int, int, size_t, const float*, const int*, int, float,
                                    const float*, const float*, const float*, void*, size_t, cudaStream_t);

cudaError_t launch_gemm_tc(const uint8_t*, const uint16_t*, const Shape&, const uint16_t*, int,
                           uint16_t*, bool, cudaStream_t);
unsigned gemm_error_flags();

// Process-wide kernel choice of mbok_gemv / mbok_gemv_noalloc (atomic: host
// threads may set and read it concurrently; a call reads it once).
std::atomic<int> gemv_kernel_choice{MBOK_GEMV_AUTO};
// Process-wide: GEMV weights may be read before the grid dependency wait
// (see mbok_gemv_set_static_weights).
std::atomic<bool> gemv_weights_static{true};

// One decode GEMV call with kernel choice `choice` (MBOK_GEMV_*): a
// lookup-table kernel once per vector -- 512-column slabs with 8-bit tables
// and a combine launch, or, when asked for, whole rows with 4-bit tables in
// one launch where they fit one CTA (N <= 10240) -- or the tensor-core kernel
// over the whole batch.  The slab kernel is the default lookup kernel: on B200
// it measured faster at the LLaMA shapes (the whole-row kernel saves the
// combine launch but does twice the lookups).
cudaError_t launch_gemv(const uint8_t* packed, const uint16_t* alpha, const Shape& s, const void* x,
                        bool x_f32, int batch, float* y, void* workspace, cudaStream_t stream, int choice,
                        bool weights_static) {
  bool tensor = batch > 1;
  if (choice == MBOK_GEMV_LOOKUP || choice == MBOK_GEMV_LOOKUP_SLABS || choice == MBOK_GEMV_LOOKUP_ROWS)
    tensor = false;
  if (choice == MBOK_GEMV_TENSOR) tensor = true;
  if (tensor) return launch_gemv_mma(packed, alpha, s, x, x_f32, batch, y, stream, weights_static);
  const bool rows = choice == MBOK_GEMV_LOOKUP_ROWS && gemv_lut4_supported(s);
  const size_t xbytes = x_f32 ? 4 : 2;
  for (int b = 0; b < batch; ++b) {
    const void* xb = static_cast<const char*>(x) + size_t(b) * s.N * xbytes;
    const cudaError_t e =
        rows ? launch_gemv_lut4(packed, alpha, s, xb, x_f32, y + size_t(b) * s.M, stream, weights_static)
             : launch_gemv_lut(packed, alpha, s, xb, x_f32, y + size_t(b) * s.M, workspace, stream, weights_static);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// The same with the process-wide choices (mbok_gemv_set_kernel,
// mbok_gemv_set_static_weights), read once.
cudaError_t launch_gemv(const uint8_t* packed, const uint16_t* alpha, const Shape& s, const void* x,
                        bool x_f32, int batch, float* y, void* workspace, cudaStream_t stream) {
  return launch_gemv(packed, alpha, s, x, x_f32, batch, y, workspace, stream,
                     gemv_kernel_choice.load(std::memory_order_relaxed),
                     gemv_weights_static.load(std::memory_order_relaxed));
}
}  // namespace mbok

using namespace mbok;

namespace {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Whether two buffers share memory (NULL shares none).
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a != nullptr && b != nullptr && x < y + nb && y < x + na;
}

inline cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

// Common shape checks; returns MBOK_OK or the first failing status.
int check_shape(int K, int M, int N) {
  if (K < 1 || K > MBOK_MAX_K) return MBOK_ERR_INVALID_ARG;
  if (M < 1 || N < MBOK_GROUP || N % MBOK_GROUP != 0) return MBOK_ERR_SHAPE;
  // keep every grid dimension and 32-bit unit index in range
  if (M > (1 << 22) || N > (1 << 20)) return MBOK_ERR_SHAPE;
  return MBOK_OK;
}

constexpr int kMaxTokens = 1 << 23;   // as mbok_gemm
constexpr int kMaxRows = 1 << 22;     // as check_shape

inline bool is_dtype(int d) { return d == MBOK_F32 || d == MBOK_BF16; }
inline size_t dtype_bytes(int d) { return d == MBOK_F32 ? 4 : 2; }

inline int from_cuda(cudaError_t e) { return e == cudaSuccess ? MBOK_OK : MBOK_ERR_CUDA; }

}  // namespace

extern "C" {

const char* mbok_status_string(int status) {
  switch (status) {
    case MBOK_OK: return "ok";
    case MBOK_ERR_INVALID_ARG: return "invalid argument";
    case MBOK_ERR_SHAPE: return "unsupported shape";
    case MBOK_ERR_ALIGN: return "misaligned pointer";
    case MBOK_ERR_UNSUPPORTED: return "unsupported option";
    case MBOK_ERR_CUDA: return "CUDA launch error";
    case MBOK_ERR_WORKSPACE: return "workspace missing or too small";
    case MBOK_ERR_SCRATCH_LIMIT: return "problem exceeds the built-in scratch of mbok_gemv_noalloc";
    default: return "unknown status";
  }
}

int mbok_layout_version(void) { return MBOK_LAYOUT_VERSION; }

size_t mbok_packed_bytes(int K, int M, int N) {
  if (check_shape(K, M, N) != MBOK_OK) return 0;
  const Shape s = make_shape(K, M, N);
  return size_t(s.O) * K * N;
}

size_t mbok_alpha_elems(int K, int M, int N) {
  if (check_shape(K, M, N) != MBOK_OK) return 0;
  const Shape s = make_shape(K, M, N);
  return size_t(s.O) * kOctet * s.G * K;
}

size_t mbok_gemv_workspace_bytes(int K, int M, int N, int batch) {
  if (check_shape(K, M, N) != MBOK_OK || batch < 1 || batch > MBOK_MAX_BATCH) return 0;
  return gemv_lut_workspace_bytes(make_shape(K, M, N));
}

int mbok_pack_bits(const int8_t* signs, int K, int M, int N, uint32_t* packed, void* stream) {
  const int st = check_shape(K, M, N);
  if (st != MBOK_OK) return st;
  if (signs == nullptr || packed == nullptr) return MBOK_ERR_INVALID_ARG;
  if (!aligned(signs, 16) || !aligned(packed, 16)) return MBOK_ERR_ALIGN;
  return from_cuda(launch_pack_bits(signs, make_shape(K, M, N), reinterpret_cast<uint8_t*>(packed),
                                    as_stream(stream)));
}

int mbok_pack_alpha(const uint16_t* alpha_mgk, int K, int M, int N, uint16_t* alpha_out,
                    void* stream) {
  const int st = check_shape(K, M, N);
  if (st != MBOK_OK) return st;
  if (alpha_mgk == nullptr || alpha_out == nullptr) return MBOK_ERR_INVALID_ARG;
  if (!aligned(alpha_mgk, 16) || !aligned(alpha_out, 16)) return MBOK_ERR_ALIGN;
  return from_cuda(launch_pack_alpha(alpha_mgk, make_shape(K, M, N), alpha_out, as_stream(stream)));
}

int mbok_residual_binarize(const float* W, int M, int N, int K, int group, uint32_t* packed,
                           uint16_t* alpha, float* residual, void* stream) {
  const int st = check_shape(K, M, N);
  if (st != MBOK_OK) return st;
  if (group != MBOK_GROUP) return MBOK_ERR_UNSUPPORTED;
  if (W == nullptr || packed == nullptr || alpha == nullptr) return MBOK_ERR_INVALID_ARG;
  if (!aligned(W, 16) || !aligned(packed, 16) || !aligned(alpha, 16) ||
      (residual != nullptr && !aligned(residual, 16)))
    return MBOK_ERR_ALIGN;
  const Shape s = make_shape(K, M, N);
  if (s.O > 65535) return MBOK_ERR_SHAPE;
  return from_cuda(launch_residual_binarize(W, s, reinterpret_cast<uint8_t*>(packed),
                                            reinterpret_cast<__half*>(alpha), residual,
                                            as_stream(stream)));
}

size_t mbok_svid_workspace_bytes(int M, int N) {
  if (check_shape(1, M, N) != MBOK_OK) return 0;
  return svid_workspace_bytes(M, N);
}

int mbok_svid_binarize(const float* W, int M, int N, int K, int iters, uint32_t* packed, uint16_t* s_in,
                       uint16_t* s_out, float* residual, void* workspace, size_t workspace_bytes, void* stream) {
  const int st = check_shape(K, M, N);
  if (st != MBOK_OK) return st;
  if (iters < 1 || iters > 1000) return MBOK_ERR_INVALID_ARG;
  if (W == nullptr || packed == nullptr || s_in == nullptr || s_out == nullptr || residual == nullptr)
    return MBOK_ERR_INVALID_ARG;
  if (!aligned(W, 16) || !aligned(packed, 16) || !aligned(s_in, 2) || !aligned(s_out, 2) || !aligned(residual, 16))
    return MBOK_ERR_ALIGN;
  if (workspace == nullptr || workspace_bytes < svid_workspace_bytes(M, N) || !aligned(workspace, 16))
    return MBOK_ERR_WORKSPACE;
  return from_cuda(launch_svid_binarize(W, make_shape(K, M, N), iters, reinterpret_cast<uint8_t*>(packed),
                                        reinterpret_cast<__half*>(s_in), reinterpret_cast<__half*>(s_out), residual,
                                        workspace, as_stream(stream)));
}

int mbok_refit_alpha(const float* W, const uint32_t* packed, int K, int M, int N, int group, uint16_t* alpha,
                     void* stream) {
  const int st = check_shape(K, M, N);
  if (st != MBOK_OK) return st;
  if (group != MBOK_GROUP) return MBOK_ERR_UNSUPPORTED;
  if (W == nullptr || packed == nullptr || alpha == nullptr) return MBOK_ERR_INVALID_ARG;
  if (!aligned(W, 16) || !aligned(packed, 16) || !aligned(alpha, 16)) return MBOK_ERR_ALIGN;
  const Shape s = make_shape(K, M, N);
  if (s.O > 65535) return MBOK_ERR_SHAPE;
  return from_cuda(launch_refit_alpha(W, reinterpret_cast<const uint8_t*>(packed), s,
                                      reinterpret_cast<__half*>(alpha), as_stream(stream)));
}

int mbok_gemv_ex(const uint32_t* packed, const uint16_t* alpha, int K, int M, int N, int group,
                 const void* x, int x_dtype, int batch, float* y, void* workspace, size_t workspace_bytes,
                 int kernel, int weights_static, void* stream) {
  const int st = check_shape(K, M, N);
  if (st != MBOK_OK) return st;
  if (group != MBOK_GROUP) return MBOK_ERR_UNSUPPORTED;
  if (packed == nullptr || alpha == nullptr || x == nullptr || y == nullptr)
    return MBOK_ERR_INVALID_ARG;
  if (x_dtype != MBOK_F32 && x_dtype != MBOK_BF16) return MBOK_ERR_INVALID_ARG;
  if (batch < 1 || batch > MBOK_MAX_BATCH) return MBOK_ERR_INVALID_ARG;
  if (kernel < MBOK_GEMV_AUTO || kernel > MBOK_GEMV_LOOKUP_ROWS) return MBOK_ERR_INVALID_ARG;
  if (weights_static != 0 && weights_static != 1) return MBOK_ERR_INVALID_ARG;
  if (!aligned(packed, 16) || !aligned(alpha, 16) || !aligned(x, 16) || !aligned(y, 4))
    return MBOK_ERR_ALIGN;
  const Shape s = make_shape(K, M, N);
  const size_t need = gemv_lut_workspace_bytes(s);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 16)))
    return MBOK_ERR_WORKSPACE;
  return from_cuda(launch_gemv(reinterpret_cast<const uint8_t*>(packed), alpha, s, x, x_dtype == MBOK_F32,
                               batch, y, workspace, as_stream(stream), kernel, weights_static == 1));
}

int mbok_gemv(const uint32_t* packed, const uint16_t* alpha, int K, int M, int N, int group,
              const void* x, int x_dtype, int batch, float* y, void* workspace,
              size_t workspace_bytes, void* stream) {
  return mbok_gemv_ex(packed, alpha, K, M, N, group, x, x_dtype, batch, y, workspace, workspace_bytes,
                      gemv_kernel_choice.load(std::memory_order_relaxed),
                      gemv_weights_static.load(std::memory_order_relaxed) ? 1 : 0, stream);
}

// Argument checks of the multi-matrix GEMV's shape arrays; MBOK_OK or the
// first failing status, and the total row count in *rows.
static int check_multi(int nseg, const int* K, const int* M, int N, long long* rows) {
  if (nseg < 1 || nseg > 8 || K == nullptr || M == nullptr) return MBOK_ERR_INVALID_ARG;
  long long total = 0;
  for (int i = 0; i < nseg; ++i) {
    const int st = check_shape(K[i], M[i], N);
    if (st != MBOK_OK) return st;
    total += M[i];
  }
  if (total > (1 << 22)) return MBOK_ERR_SHAPE;
  *rows = total;
  return MBOK_OK;
}

size_t mbok_gemv_multi_workspace_bytes(int nseg, const int* K, const int* M, int N) {
  long long rows = 0;
  if (check_multi(nseg, K, M, N, &rows) != MBOK_OK) return 0;
  return gemv_multi_workspace_bytes(nseg, K, M, N);
}

int mbok_gemv_multi(int nseg, const uint32_t* const* packed, const uint16_t* const* alpha, const int* K,
                    const int* M, int N, int group, const void* x, int x_dtype, int batch, float* y,
                    void* workspace, size_t workspace_bytes, void* stream) {
  long long rows = 0;
  const int st = check_multi(nseg, K, M, N, &rows);
  if (st != MBOK_OK) return st;
  if (group != MBOK_GROUP) return MBOK_ERR_UNSUPPORTED;
  if (packed == nullptr || alpha == nullptr || x == nullptr || y == nullptr) return MBOK_ERR_INVALID_ARG;
  if (x_dtype != MBOK_F32 && x_dtype != MBOK_BF16) return MBOK_ERR_INVALID_ARG;
  if (batch < 1 || batch > MBOK_MAX_BATCH) return MBOK_ERR_INVALID_ARG;
  for (int i = 0; i < nseg; ++i) {
    if (packed[i] == nullptr || alpha[i] == nullptr) return MBOK_ERR_INVALID_ARG;
    if (!aligned(packed[i], 16) || !aligned(alpha[i], 16)) return MBOK_ERR_ALIGN;
  }
  if (!aligned(x, 16) || !aligned(y, 4)) return MBOK_ERR_ALIGN;
  const size_t need = gemv_multi_workspace_bytes(nseg, K, M, N);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 16)))
    return MBOK_ERR_WORKSPACE;
  const uint8_t* p8[8];
  for (int i = 0; i < nseg; ++i) p8[i] = reinterpret_cast<const uint8_t*>(packed[i]);
  const size_t xbytes = (x_dtype == MBOK_F32) ? 4 : 2;
  for (int b = 0; b < batch; ++b) {
    const void* xb = static_cast<const char*>(x) + size_t(b) * N * xbytes;
    const cudaError_t e = launch_gemv_lut_multi(nseg, p8, alpha, K, M, N, xb, x_dtype == MBOK_F32,
                                                y + size_t(b) * size_t(rows), workspace, as_stream(stream),
                                                gemv_weights_static.load(std::memory_order_relaxed));
    if (e != cudaSuccess) return MBOK_ERR_CUDA;
  }
  return MBOK_OK;
}

size_t mbok_gemv_gated_workspace_bytes(int K_gate, int K_up, int M, int N, int batch) {
  if (check_shape(K_gate, M, N) != MBOK_OK || check_shape(K_up, M, N) != MBOK_OK) return 0;
  if (batch < 1 || batch > MBOK_MAX_BATCH) return 0;
  return gemv_gated_workspace_bytes(make_shape(K_gate, M, N), batch);
}

int mbok_gemv_gated(const uint32_t* packed_gate, const uint16_t* alpha_gate, int K_gate, const uint32_t* packed_up,
                    const uint16_t* alpha_up, int K_up, int M, int N, int group, const void* x, int x_dtype, int batch,
                    void* h, int h_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_shape(K_gate, M, N);
  if (st == MBOK_OK) st = check_shape(K_up, M, N);
  if (st != MBOK_OK) return st;
  if (group != MBOK_GROUP) return MBOK_ERR_UNSUPPORTED;
  if (packed_gate == nullptr || alpha_gate == nullptr || packed_up == nullptr || alpha_up == nullptr ||
      x == nullptr || h == nullptr)
    return MBOK_ERR_INVALID_ARG;
  if (!is_dtype(x_dtype) || !is_dtype(h_dtype)) return MBOK_ERR_INVALID_ARG;
  if (batch < 1 || batch > MBOK_MAX_BATCH) return MBOK_ERR_INVALID_ARG;
  if (!aligned(packed_gate, 16) || !aligned(alpha_gate, 16) || !aligned(packed_up, 16) || !aligned(alpha_up, 16) ||
      !aligned(x, 16) || !aligned(h, dtype_bytes(h_dtype)))
    return MBOK_ERR_ALIGN;
  const Shape gate = make_shape(K_gate, M, N), up = make_shape(K_up, M, N);
  const size_t need = gemv_gated_workspace_bytes(gate, batch);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 16)))
    return MBOK_ERR_WORKSPACE;
  if (overlap(h, size_t(batch) * M * dtype_bytes(h_dtype), x, size_t(batch) * N * dtype_bytes(x_dtype)))
    return MBOK_ERR_INVALID_ARG;
  return from_cuda(launch_gemv_gated(reinterpret_cast<const uint8_t*>(packed_gate), alpha_gate, gate,
                                     reinterpret_cast<const uint8_t*>(packed_up), alpha_up, up, x,
                                     x_dtype == MBOK_F32, batch, h, h_dtype == MBOK_BF16, workspace,
                                     as_stream(stream), gemv_weights_static.load(std::memory_order_relaxed)));
}

int mbok_gated_backward(const uint16_t* dH, const uint16_t* gate, const uint16_t* up, int T, int M, uint16_t* dgate,
                        uint16_t* dup, uint16_t* H, void* stream) {
  if (T < 1 || T > kMaxTokens || M < 1 || M > kMaxRows) return MBOK_ERR_SHAPE;
  const size_t n = size_t(T) * size_t(M);
  if (n > (size_t(1) << 42)) return MBOK_ERR_SHAPE;   // keeps the grid in range
  if (dH == nullptr || gate == nullptr || up == nullptr || dgate == nullptr || dup == nullptr)
    return MBOK_ERR_INVALID_ARG;
  if (!aligned(dH, 16) || !aligned(gate, 16) || !aligned(up, 16) || !aligned(dgate, 16) || !aligned(dup, 16) ||
      !aligned(H, 16))
    return MBOK_ERR_ALIGN;
  if (overlap(dgate, n * 2, dup, n * 2) || overlap(dgate, n * 2, H, n * 2) || overlap(dup, n * 2, H, n * 2))
    return MBOK_ERR_INVALID_ARG;
  for (const uint16_t* out : {dgate, dup, H})
    for (const uint16_t* in : {dH, gate, up})
      if (out != in && overlap(out, n * 2, in, n * 2)) return MBOK_ERR_INVALID_ARG;
  return from_cuda(launch_gated_backward(dH, gate, up, n, dgate, dup, H, as_stream(stream)));
}

size_t mbok_gemm_gated_workspace_bytes(int M, int N, int T) {
  if (check_shape(1, M, N) != MBOK_OK || T < 1 || T > kMaxTokens) return 0;
  return gemm_gated_workspace_bytes(M, N, T);
}

int mbok_gemm_gated(const uint32_t* packed_gate, const uint16_t* alpha_gate, int K_gate, const uint32_t* packed_up,
                    const uint16_t* alpha_up, int K_up, int M, int N, int group, const uint16_t* X, int T, uint16_t* H,
                    uint16_t* gate, uint16_t* up, void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_shape(K_gate, M, N);
  if (st == MBOK_OK) st = check_shape(K_up, M, N);
  if (st != MBOK_OK) return st;
  if (group != MBOK_GROUP) return MBOK_ERR_UNSUPPORTED;
  if (T < 1 || T > kMaxTokens) return MBOK_ERR_SHAPE;
  if (packed_gate == nullptr || alpha_gate == nullptr || packed_up == nullptr || alpha_up == nullptr ||
      X == nullptr || H == nullptr || (gate == nullptr) != (up == nullptr))
    return MBOK_ERR_INVALID_ARG;
  if (!aligned(packed_gate, 16) || !aligned(alpha_gate, 16) || !aligned(packed_up, 16) || !aligned(alpha_up, 16) ||
      !aligned(X, 16) || !aligned(H, 16) || !aligned(gate, 16) || !aligned(up, 16))
    return MBOK_ERR_ALIGN;
  if (workspace == nullptr || workspace_bytes < gemm_gated_workspace_bytes(M, N, T) || !aligned(workspace, 256))
    return MBOK_ERR_WORKSPACE;
  const size_t bytes = size_t(T) * M * 2;
  if (overlap(H, bytes, gate, bytes) || overlap(H, bytes, up, bytes) || overlap(gate, bytes, up, bytes))
    return MBOK_ERR_INVALID_ARG;
  return from_cuda(launch_gemm_gated(reinterpret_cast<const uint8_t*>(packed_gate), alpha_gate,
                                     make_shape(K_gate, M, N), reinterpret_cast<const uint8_t*>(packed_up), alpha_up,
                                     make_shape(K_up, M, N), X, T, H, gate, up, workspace, as_stream(stream)));
}

size_t mbok_gemm_backward_workspace_bytes(int nseg, const int* K, const int* M, int N, int T) {
  long long rows = 0;
  if (check_multi(nseg, K, M, N, &rows) != MBOK_OK || T < 1 || T > kMaxTokens) return 0;
  Shape shapes[8];
  for (int i = 0; i < nseg; ++i) shapes[i] = make_shape(K[i], M[i], N);
  return gemm_backward_workspace_bytes(nseg, shapes, T);
}

int mbok_gemm_backward(int nseg, const uint32_t* const* packed, const uint16_t* const* alpha, const int* K,
                       const int* M, int N, int group, const uint16_t* X, int T, const uint16_t* const* dY,
                       uint16_t* dX, float* const* dalpha, void* workspace, size_t workspace_bytes, void* stream) {
  long long rows = 0;
  const int st = check_multi(nseg, K, M, N, &rows);
  if (st != MBOK_OK) return st;
  if (group != MBOK_GROUP) return MBOK_ERR_UNSUPPORTED;
  if (T < 1 || T > kMaxTokens) return MBOK_ERR_SHAPE;
  if (packed == nullptr || alpha == nullptr || dY == nullptr) return MBOK_ERR_INVALID_ARG;
  Shape shapes[8];
  const uint8_t* p8[8];
  bool any = false;
  for (int i = 0; i < nseg; ++i) {
    if (packed[i] == nullptr || alpha[i] == nullptr || dY[i] == nullptr) return MBOK_ERR_INVALID_ARG;
    if (!aligned(packed[i], 16) || !aligned(alpha[i], 16) || !aligned(dY[i], 16)) return MBOK_ERR_ALIGN;
    if (dalpha != nullptr && dalpha[i] != nullptr) {
      if (!aligned(dalpha[i], 16)) return MBOK_ERR_ALIGN;
      any = true;
    }
    shapes[i] = make_shape(K[i], M[i], N);
    p8[i] = reinterpret_cast<const uint8_t*>(packed[i]);
  }
  if (dX == nullptr && !any) return MBOK_ERR_INVALID_ARG;   // nothing asked for
  if (any && X == nullptr) return MBOK_ERR_INVALID_ARG;
  if (!aligned(X, 16) || !aligned(dX, 16)) return MBOK_ERR_ALIGN;
  if (workspace == nullptr || workspace_bytes < gemm_backward_workspace_bytes(nseg, shapes, T) ||
      !aligned(workspace, 256))
    return MBOK_ERR_WORKSPACE;
  // the scales' gradients read X and dY while dX is written
  const size_t x_bytes = size_t(T) * N * 2;
  if (any && overlap(dX, x_bytes, X, x_bytes)) return MBOK_ERR_INVALID_ARG;
  for (int i = 0; i < nseg; ++i)
    if (any && overlap(dX, x_bytes, dY[i], size_t(T) * M[i] * 2)) return MBOK_ERR_INVALID_ARG;
  // and are written while those are read; a matrix given twice has two gradients:
  // they are not added up
  for (int i = 0; any && i < nseg; ++i) {
    const size_t bytes = mbok_alpha_elems(K[i], M[i], N) * 4;
    if (overlap(dalpha[i], bytes, dX, x_bytes) || overlap(dalpha[i], bytes, X, x_bytes)) return MBOK_ERR_INVALID_ARG;
    for (int j = 0; j < nseg; ++j)
      if (overlap(dalpha[i], bytes, dY[j], size_t(T) * M[j] * 2) ||
          (j < i && overlap(dalpha[i], bytes, dalpha[j], mbok_alpha_elems(K[j], M[j], N) * 4)))
        return MBOK_ERR_INVALID_ARG;
  }
  return from_cuda(launch_gemm_backward(nseg, p8, alpha, shapes, X, T, dY, dX, dalpha, workspace, as_stream(stream)));
}

// Checks common to the distillation calls.
static int check_distill(const void* logits, int dtype, int T, int V, size_t ld, const float* teacher,
                         const int32_t* index, int top, float temperature) {
  if (!is_dtype(dtype)) return MBOK_ERR_INVALID_ARG;
  if (T < 1 || T > kMaxTokens || V < 1 || V > MBOK_DISTILL_MAX_VOCAB || ld < size_t(V)) return MBOK_ERR_SHAPE;
  if (logits == nullptr || teacher == nullptr || index == nullptr) return MBOK_ERR_INVALID_ARG;
  if (top < 1 || top > MBOK_DISTILL_MAX_TOP) return MBOK_ERR_INVALID_ARG;
  if (!(temperature >= 1.f / 1024.f && temperature <= 1024.f)) return MBOK_ERR_INVALID_ARG;   // NaN too
  if (!aligned(logits, 16) || !aligned(teacher, 4) || !aligned(index, 4)) return MBOK_ERR_ALIGN;
  return MBOK_OK;
}

int mbok_distill_loss(const void* logits, int dtype, int T, int V, size_t ld, const float* teacher,
                      const int32_t* index, int top, float temperature, const float* weight, float* loss, float* lse,
                      void* dlogits, size_t ld_dlogits, void* stream) {
  const int st = check_distill(logits, dtype, T, V, ld, teacher, index, top, temperature);
  if (st != MBOK_OK) return st;
  if (loss == nullptr || lse == nullptr) return MBOK_ERR_INVALID_ARG;
  if (dlogits != nullptr && ld_dlogits < size_t(V)) return MBOK_ERR_SHAPE;
  if (dlogits == logits && ld_dlogits != ld) return MBOK_ERR_SHAPE;   // in place: the same rows
  if (!aligned(weight, 4) || !aligned(loss, 4) || !aligned(lse, 4) || !aligned(dlogits, 16)) return MBOK_ERR_ALIGN;
  if (overlap(loss, size_t(T) * 4, lse, size_t(T) * 4)) return MBOK_ERR_INVALID_ARG;
  return from_cuda(launch_distill_loss(logits, dtype == MBOK_F32, T, V, ld, teacher, index, top, temperature, weight,
                                       loss, lse, dlogits, ld_dlogits, as_stream(stream)));
}

int mbok_distill_backward(const void* logits, int dtype, int T, int V, size_t ld, const float* teacher,
                          const int32_t* index, int top, float temperature, const float* weight, const float* lse,
                          const float* grad, void* dlogits, size_t ld_dlogits, void* stream) {
  const int st = check_distill(logits, dtype, T, V, ld, teacher, index, top, temperature);
  if (st != MBOK_OK) return st;
  if (lse == nullptr || dlogits == nullptr) return MBOK_ERR_INVALID_ARG;
  if (ld_dlogits < size_t(V)) return MBOK_ERR_SHAPE;
  if (dlogits == logits && ld_dlogits != ld) return MBOK_ERR_SHAPE;
  if (!aligned(weight, 4) || !aligned(lse, 4) || !aligned(grad, 4) || !aligned(dlogits, 16)) return MBOK_ERR_ALIGN;
  return from_cuda(launch_distill_backward(logits, dtype == MBOK_F32, T, V, ld, teacher, index, top, temperature,
                                           weight, lse, grad, dlogits, ld_dlogits, as_stream(stream)));
}

int mbok_gemv_set_static_weights(int on) {
  if (on != 0 && on != 1) return MBOK_ERR_INVALID_ARG;
  gemv_weights_static.store(on == 1, std::memory_order_relaxed);
  return MBOK_OK;
}

int mbok_gemv_set_kernel(int kernel) {
  if (kernel < MBOK_GEMV_AUTO || kernel > MBOK_GEMV_LOOKUP_ROWS) return MBOK_ERR_INVALID_ARG;
  gemv_kernel_choice.store(kernel, std::memory_order_relaxed);
  return MBOK_OK;
}

size_t mbok_gemv_svid_workspace_bytes(int K, int M, int N, int batch) {
  if (check_shape(K, M, N) != MBOK_OK || batch < 1 || batch > MBOK_MAX_BATCH) return 0;
  return gemv_svid_workspace_bytes(make_shape(K, M, N));
}

int mbok_gemv_svid(const uint32_t* packed, const uint16_t* s_in, const uint16_t* s_out, int K, int M, int N,
                   const void* x, int x_dtype, int batch, float* y, void* workspace, size_t workspace_bytes,
                   void* stream) {
  const int st = check_shape(K, M, N);
  if (st != MBOK_OK) return st;
  if (packed == nullptr || s_in == nullptr || s_out == nullptr || x == nullptr || y == nullptr)
    return MBOK_ERR_INVALID_ARG;
  if (x_dtype != MBOK_F32 && x_dtype != MBOK_BF16) return MBOK_ERR_INVALID_ARG;
  if (batch < 1 || batch > MBOK_MAX_BATCH) return MBOK_ERR_INVALID_ARG;
  if (!aligned(packed, 16) || !aligned(s_in, 16) || !aligned(s_out, 2) || !aligned(x, 16) || !aligned(y, 4))
    return MBOK_ERR_ALIGN;
  const Shape s = make_shape(K, M, N);
  const size_t need = gemv_svid_workspace_bytes(s);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 16)))
    return MBOK_ERR_WORKSPACE;
  const size_t xbytes = (x_dtype == MBOK_F32) ? 4 : 2;
  for (int b = 0; b < batch; ++b) {
    const void* xb = static_cast<const char*>(x) + size_t(b) * N * xbytes;
    const cudaError_t e = launch_gemv_svid(reinterpret_cast<const uint8_t*>(packed), s_in, s_out, s, xb,
                                           x_dtype == MBOK_F32, y + size_t(b) * M, workspace, as_stream(stream),
                                           gemv_weights_static.load(std::memory_order_relaxed));
    if (e != cudaSuccess) return MBOK_ERR_CUDA;
  }
  return MBOK_OK;
}

int mbok_check_wait_timeout(unsigned timeout_us, void* stream) {
  if (timeout_us < 1 || timeout_us > 1000000) return MBOK_ERR_INVALID_ARG;
  return from_cuda(launch_wait_timeout_probe(timeout_us, as_stream(stream)));
}

int mbok_read_device_errors(unsigned* flags) {
  if (flags == nullptr) return MBOK_ERR_INVALID_ARG;
  if (cudaDeviceSynchronize() != cudaSuccess) return MBOK_ERR_CUDA;
  const unsigned g = gemv_lut4_error_flags();
  const unsigned m = gemm_error_flags();
  const unsigned t = gemv_mma_error_flags();
  const unsigned d = gemv_gated_error_flags();
  const unsigned p = gemm_pair_error_flags();
  const unsigned a = gemm_dalpha_error_flags();
  const unsigned l = distill_error_flags();
  if (g == ~0u || m == ~0u || t == ~0u || d == ~0u || p == ~0u || a == ~0u || l == ~0u) return MBOK_ERR_CUDA;
  *flags = (g ? 1u : 0u) | (m ? 2u : 0u) | ((t | d) ? 4u : 0u) | ((p | a) ? 8u : 0u) | (l ? 16u : 0u);
  return MBOK_OK;
}

int mbok_gemm_ex(const uint32_t* packed, const uint16_t* alpha, int K, int M, int N, int group,
                 const uint16_t* X, int T, uint16_t* Y, int precision, void* stream) {
  const int st = check_shape(K, M, N);
  if (st != MBOK_OK) return st;
  if (group != MBOK_GROUP) return MBOK_ERR_UNSUPPORTED;
  if (T < 1 || T > (1 << 23)) return MBOK_ERR_SHAPE;
  if (packed == nullptr || alpha == nullptr || X == nullptr || Y == nullptr)
    return MBOK_ERR_INVALID_ARG;
  if (precision < MBOK_GEMM_AUTO || precision > MBOK_GEMM_SPLIT) return MBOK_ERR_INVALID_ARG;
  if (!aligned(packed, 16) || !aligned(alpha, 16) || !aligned(X, 16) || !aligned(Y, 16))
    return MBOK_ERR_ALIGN;
  const bool split = precision == MBOK_GEMM_SPLIT || (precision == MBOK_GEMM_AUTO && N <= MBOK_GEMM_SPLIT_MAX_N);
  return from_cuda(launch_gemm_tc(reinterpret_cast<const uint8_t*>(packed), alpha, make_shape(K, M, N), X,
                                  T, Y, split, as_stream(stream)));
}

int mbok_gemm(const uint32_t* packed, const uint16_t* alpha, int K, int M, int N, int group,
              const uint16_t* X, int T, uint16_t* Y, void* stream) {
  return mbok_gemm_ex(packed, alpha, K, M, N, group, X, T, Y, MBOK_GEMM_AUTO, stream);
}

}  // extern "C"
