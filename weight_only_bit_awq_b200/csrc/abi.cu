// C ABI entry points of libawq_b200.so (declared in include/awq.h): argument
// checks, workspace layout, dispatch between the GEMV and GEMM paths.
#include <cfloat>
#include <cmath>
#include <mutex>

#include "awq_internal.cuh"
#include "sm100_ptx.cuh"

namespace awq {

namespace {
// One thread waits, through the kernels' bounded-wait helper, on an mbarrier
// phase that nothing will ever complete; the wait gives up after `limit_ns`
// and records AWQ_ERR_TIMEOUT in the status word.
__global__ void bounded_wait_probe_kernel(uint32_t* status, uint64_t limit_ns) {
  __shared__ __align__(8) uint64_t barrier;
  __shared__ uint32_t abort_flag;
  const uint32_t bar = ptx::smem_u32(&barrier);
  ptx::mbar_init(bar, 1);
  abort_flag = 0;
  ptx::fence_mbarrier_init();
  ptx::wait_bar(bar, 0, &abort_flag, status, limit_ns);
}
}  // namespace

namespace {
constexpr int kMaxDevices = 64;
DeviceInfo g_info[kMaxDevices];
std::once_flag g_once[kMaxDevices];

constexpr int64_t kMaxK = int64_t(1) << 22;
constexpr int64_t kMaxN = int64_t(1) << 22;
constexpr int64_t kMaxM = int64_t(1) << 24;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return an && bn && a0 < b0 + bn && b0 < a0 + an;
}

awq_status check_kn(int64_t K, int64_t N, int group) {
  if (K <= 0 || N <= 0) return AWQ_ERR_SHAPE;
  if (group != 128 && group != 64 && group != 32) return AWQ_ERR_UNSUPPORTED;
  if (K % kKPerBlock != 0 || K % group != 0 || N % kRowsPerBlock != 0) return AWQ_ERR_SHAPE;
  if (K > kMaxK || N > kMaxN) return AWQ_ERR_UNSUPPORTED;
  return AWQ_OK;
}

awq_status check_device() {
  const DeviceInfo& d = device_info();
  if (d.device < 0 || d.cc_major != 10) return AWQ_ERR_UNSUPPORTED;
  return AWQ_OK;
}

struct LinearArgs {
  const void *x, *qweight, *scales, *zeros;
  void* y;
  int64_t M, K, N;
  int group;
  void* workspace;
  size_t ws_bytes;
};

awq_status check_linear(const LinearArgs& a) {
  if (a.M < 0) return AWQ_ERR_SHAPE;
  awq_status st = check_kn(a.K, a.N, a.group);
  if (st != AWQ_OK) return st;
  if (a.M > kMaxM) return AWQ_ERR_UNSUPPORTED;
  // x and y may be null for an empty batch (nothing is read or written).
  if ((a.M > 0 && (!a.x || !a.y)) || !a.qweight || !a.scales || !a.zeros || !a.workspace)
    return AWQ_ERR_INVALID_ARG;
  if (!aligned16(a.x) || !aligned16(a.qweight) || !aligned16(a.scales) || !aligned16(a.zeros) ||
      !aligned16(a.y) || !aligned16(a.workspace))
    return AWQ_ERR_ALIGNMENT;
  const size_t ybytes = (size_t)a.M * a.N * 2;
  const size_t ng = (size_t)(a.K / a.group);
  if (overlap(a.y, ybytes, a.x, (size_t)a.M * a.K * 2) || overlap(a.y, ybytes, a.qweight, (size_t)a.K * a.N / 2) ||
      overlap(a.y, ybytes, a.scales, ng * a.N * 2) || overlap(a.y, ybytes, a.zeros, ng * a.N / 2) ||
      overlap(a.y, ybytes, a.workspace, a.ws_bytes))
    return AWQ_ERR_INVALID_ARG;
  if (a.ws_bytes < awq_workspace_bytes(a.M, a.K, a.N, a.group)) return AWQ_ERR_WORKSPACE;
  return AWQ_OK;
}

inline uint32_t* status_word(void* ws) { return static_cast<uint32_t*>(ws); }

}  // namespace

const DeviceInfo& device_info() {
  static DeviceInfo none;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return none;
  }
  std::call_once(g_once[dev], [dev] {
    DeviceInfo& d = g_info[dev];
    int v = 0;
    if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess) d.sm_count = v;
    cudaDeviceGetAttribute(&d.cc_major, cudaDevAttrComputeCapabilityMajor, dev);
    cudaDeviceGetAttribute(&d.cc_minor, cudaDevAttrComputeCapabilityMinor, dev);
    if (cudaDeviceGetAttribute(&v, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) == cudaSuccess) d.smem_optin = v;
    d.device = dev;
  });
  return g_info[dev];
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    else
      cudaGetLastError();
  });
  return fn;
}

}  // namespace awq

using namespace awq;

namespace {

int sm_count_or_default() {
  int dev = -1, n = 0;
  if (cudaGetDevice(&dev) == cudaSuccess && cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess &&
      n > 0)
    return n;
  cudaGetLastError();
  return 148;
}

awq_status gemv_impl(const LinearArgs& a, cudaStream_t stream) {
  const GemvPlan p = plan_gemv(a.M, a.K, a.N, a.group, device_info().sm_count);
  cudaError_t e = launch_gemv(static_cast<const __half*>(a.x), static_cast<const uint32_t*>(a.qweight),
                              static_cast<const __half*>(a.scales), static_cast<const uint8_t*>(a.zeros),
                              static_cast<__half*>(a.y), a.M, a.K, a.N, a.workspace, p, stream);
  return e == cudaSuccess ? AWQ_OK : AWQ_ERR_CUDA;
}

awq_status gemm_impl(const LinearArgs& a, cudaStream_t stream) {
  const GemmPlan p = plan_gemm(a.M, a.K, a.N, device_info().sm_count);
  cudaError_t e = launch_gemm(static_cast<const __half*>(a.x), static_cast<const uint32_t*>(a.qweight),
                              static_cast<const __half*>(a.scales), static_cast<const uint8_t*>(a.zeros),
                              static_cast<__half*>(a.y), a.M, a.K, a.N, a.group, p, a.workspace, stream);
  return e == cudaSuccess ? AWQ_OK : AWQ_ERR_CUDA;
}

// Dispatch of awq_linear between the decode GEMV and the tensor-core GEMM,
// from measurements on B200 (CUDA graphs, rotating weights, LLaMA-3-8B and
// LLaMA-2-70B decode layers at M = 4 .. 64): the GEMV is faster on every layer
// up to M = 16; at M = 24 and 32 the GEMM is faster on layers with at least
// as many 128-channel tiles as SMs (gate_up: 54.6 against 76.4 us at M = 32
// on LLaMA-3-8B, 195.6 against 256.3 us on 70B) and slower on the narrower
// ones, which leave most SMs without a tile.
constexpr int kGemvAlwaysM = 16;

bool linear_uses_gemv(int64_t M, int64_t N, int sm_count) {
  return M <= kGemvAlwaysM || (M <= AWQ_GEMV_MAX_M && (N + 127) / 128 < sm_count);
}

// Shared checks of the norm and the SiLU: `in` inputs, `out` outputs.
struct Span {
  const void* p;
  size_t bytes;
};

awq_status check_spans(const Span* in, int n_in, const Span* out, int n_out) {
  for (int i = 0; i < n_in; ++i)
    if (!in[i].p) return AWQ_ERR_INVALID_ARG;
  for (int i = 0; i < n_out; ++i)
    if (!out[i].p) return AWQ_ERR_INVALID_ARG;
  for (int i = 0; i < n_in; ++i)
    if (!aligned16(in[i].p)) return AWQ_ERR_ALIGNMENT;
  for (int i = 0; i < n_out; ++i)
    if (!aligned16(out[i].p)) return AWQ_ERR_ALIGNMENT;
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (overlap(out[i].p, out[i].bytes, in[j].p, in[j].bytes)) return AWQ_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return AWQ_ERR_INVALID_ARG;
  }
  return AWQ_OK;
}

awq_status rmsnorm_impl(const void* x, const void* residual, const void* weight, float eps, void* h, void* y, void* x8,
                        void* sx, bool fp8, int64_t M, int64_t K, void* stream) {
  if (M < 0 || K <= 0 || K % 8 != 0) return AWQ_ERR_SHAPE;
  if (K > kMaxK || M > kMaxM) return AWQ_ERR_UNSUPPORTED;
  if (!(eps >= 0.f && eps <= FLT_MAX) || (residual == nullptr) != (h == nullptr)) return AWQ_ERR_INVALID_ARG;
  if (M == 0) return AWQ_OK;
  const size_t n = (size_t)M * K;
  const Span in[3] = {{x, 2 * n}, {weight, (size_t)K * 2}, {residual, 2 * n}};
  const Span out[2] = {{fp8 ? x8 : y, fp8 ? n : 2 * n}, {sx, (size_t)M * 4}};
  awq_status st = check_spans(in, residual ? 3 : 2, out, fp8 ? 2 : 1);
  if (st != AWQ_OK) return st;
  if (h) {
    if (!aligned16(h)) return AWQ_ERR_ALIGNMENT;
    // every thread reads its elements of x and residual before it writes the same ones of h
    if ((h != x && overlap(h, 2 * n, x, 2 * n)) || (h != residual && overlap(h, 2 * n, residual, 2 * n)) ||
        overlap(h, 2 * n, weight, (size_t)K * 2) || overlap(h, 2 * n, out[0].p, out[0].bytes) ||
        (fp8 && overlap(h, 2 * n, sx, (size_t)M * 4)))
      return AWQ_ERR_INVALID_ARG;
  }
  if ((st = check_device()) != AWQ_OK) return st;
  cudaError_t e = launch_rmsnorm(static_cast<const __half*>(x), static_cast<const __half*>(residual),
                                 static_cast<const __half*>(weight), eps, static_cast<__half*>(h),
                                 static_cast<__half*>(y), static_cast<uint8_t*>(x8), static_cast<float*>(sx), M, K,
                                 static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? AWQ_OK : AWQ_ERR_CUDA;
}

awq_status silu_impl(const void* gate_up, void* y, void* x8, void* sx, bool fp8, int64_t M, int64_t F, void* stream) {
  if (M < 0 || F <= 0 || F % 8 != 0) return AWQ_ERR_SHAPE;
  if (F > kMaxK || M > kMaxM || M * F > int64_t(1) << 40) return AWQ_ERR_UNSUPPORTED;
  if (M == 0) return AWQ_OK;
  const size_t n = (size_t)M * F;
  const Span in[1] = {{gate_up, 4 * n}};
  const Span out[2] = {{fp8 ? x8 : y, fp8 ? n : 2 * n}, {sx, (size_t)M * 4}};
  awq_status st = check_spans(in, 1, out, fp8 ? 2 : 1);
  if (st != AWQ_OK) return st;
  if ((st = check_device()) != AWQ_OK) return st;
  cudaError_t e = launch_silu_mul(static_cast<const __half*>(gate_up), static_cast<__half*>(y),
                                  static_cast<uint8_t*>(x8), static_cast<float*>(sx), M, F,
                                  static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? AWQ_OK : AWQ_ERR_CUDA;
}

constexpr int kMaxHeads = 4096;
// |q . k| <= 128 * 65504 * 448 * 2^31 < 2^63: with it no score comes near 2^99,
// below which the attention kernel takes a row's keys for none.
constexpr float kMaxScale = 0x1p32f;

awq_status check_kv8_sizes(int64_t rows, int64_t seqs, int64_t q_heads, int64_t heads, int64_t head_dim) {
  if (rows < 0 || seqs < 0 || q_heads <= 0 || heads <= 0 || q_heads % heads != 0) return AWQ_ERR_SHAPE;
  if (head_dim != 64 && head_dim != 128) return AWQ_ERR_UNSUPPORTED;
  if (rows > kMaxM || seqs > int64_t(1) << 20 || q_heads > kMaxHeads || seqs * heads > int64_t(1) << 24 ||
      rows * q_heads > 0x7FFFFFFF)
    return AWQ_ERR_UNSUPPORTED;
  return AWQ_OK;
}

// The cache and batch of a call, checked, as the kernels take them.
awq_status check_kv8(const awq_kv8_cache* cache, const awq_kv8_batch* batch, int64_t q_heads, const void* workspace,
                     size_t ws_bytes, Kv8Cache* c, Kv8Batch* b) {
  if (!cache || !batch) return AWQ_ERR_INVALID_ARG;
  awq_status st = check_kv8_sizes(batch->rows, batch->seqs, q_heads, cache->heads, cache->head_dim);
  if (st != AWQ_OK) return st;
  if (cache->blocks < 0 || batch->table_width < 0) return AWQ_ERR_SHAPE;
  const int bs = cache->block_tokens;
  if (bs != 16 && bs != 32 && bs != 64 && bs != 128) return AWQ_ERR_UNSUPPORTED;
  if (cache->blocks > 0x7FFFFFFF || cache->blocks * cache->heads * bs > 0x7FFFFFFF || batch->table_width > (int64_t(1) << 28) / bs) return AWQ_ERR_UNSUPPORTED;
  *b = Kv8Batch{};
  if (batch->rows == 0 || batch->seqs == 0) return AWQ_OK;  // nothing is read or written: pointers may be null
  if (!cache->k || !cache->v || !cache->k_exp || !cache->v_exp || !batch->starts || !batch->lens || !batch->table || !workspace)
    return AWQ_ERR_INVALID_ARG;
  if (cache->blocks == 0 || batch->table_width == 0) return AWQ_ERR_SHAPE;
  if (!aligned16(cache->k) || !aligned16(cache->v) || !aligned16(workspace) ||
      ((reinterpret_cast<uintptr_t>(batch->starts) | reinterpret_cast<uintptr_t>(batch->lens) |
        reinterpret_cast<uintptr_t>(batch->table)) & 3u) != 0)
    return AWQ_ERR_ALIGNMENT;
  if (ws_bytes < awq_kv8_workspace_bytes(batch->rows, batch->seqs, (int)q_heads, cache->heads, cache->head_dim))
    return AWQ_ERR_WORKSPACE;
  *c = Kv8Cache{static_cast<uint8_t*>(cache->k), static_cast<uint8_t*>(cache->v), static_cast<int8_t*>(cache->k_exp),
                static_cast<int8_t*>(cache->v_exp), cache->blocks, cache->heads, cache->head_dim};
  *b = Kv8Batch{static_cast<const int*>(batch->starts), static_cast<const int*>(batch->lens),
                static_cast<const int*>(batch->table), (int)batch->seqs, (int)batch->rows, (int)batch->table_width, bs};
  const Span parts[5] = {{c->k, (size_t)c->blocks * c->heads * bs * c->head_dim},
                         {c->v, (size_t)c->blocks * c->heads * bs * c->head_dim},
                         {c->k_exp, (size_t)c->blocks * c->heads},
                         {c->v_exp, (size_t)c->blocks * c->heads},
                         {workspace, ws_bytes}};
  const Span lists[3] = {{b->starts, (size_t)(b->seqs + 1) * 4},
                         {b->lens, (size_t)b->seqs * 4},
                         {b->table, (size_t)b->seqs * b->table_width * 4}};
  for (int i = 0; i < 5; ++i) {
    for (int j = 0; j < i; ++j)
      if (overlap(parts[i].p, parts[i].bytes, parts[j].p, parts[j].bytes)) return AWQ_ERR_INVALID_ARG;
    for (int j = 0; j < 3; ++j)
      if (overlap(parts[i].p, parts[i].bytes, lists[j].p, lists[j].bytes)) return AWQ_ERR_INVALID_ARG;
  }
  return AWQ_OK;
}

// Bytes from the first element of a strided matrix to its last.
size_t row_bytes(int64_t rows, int64_t stride, int64_t width) { return (size_t)((rows - 1) * stride + width) * 2; }

// Whether [p, p + bytes) touches the cache or the batch's lists.
bool kv8_overlap(const Kv8Cache& c, const Kv8Batch& b, const void* p, size_t bytes) {
  const size_t codes = (size_t)c.blocks * c.heads * b.block_tokens * c.head_dim, exps = (size_t)c.blocks * c.heads;
  return overlap(p, bytes, c.k, codes) || overlap(p, bytes, c.v, codes) || overlap(p, bytes, c.k_exp, exps) ||
         overlap(p, bytes, c.v_exp, exps) || overlap(p, bytes, b.starts, (size_t)(b.seqs + 1) * 4) ||
         overlap(p, bytes, b.lens, (size_t)b.seqs * 4) || overlap(p, bytes, b.table, (size_t)b.seqs * b.table_width * 4);
}

}  // namespace

extern "C" {

awq_status awq_packed_size(int64_t K, int64_t N, int group, awq_packed_sizes* out) {
  if (!out) return AWQ_ERR_INVALID_ARG;
  awq_status st = check_kn(K, N, group);
  if (st != AWQ_OK) return st;
  out->qweight_bytes = (size_t)K * (size_t)N / 2;
  out->scales_bytes = (size_t)(K / group) * (size_t)N * 2;
  out->zeros_bytes = (size_t)(K / group) * (size_t)N / 2;
  return AWQ_OK;
}

size_t awq_workspace_bytes(int64_t M, int64_t K, int64_t N, int group) {
  if (M < 0 || check_kn(K, N, group) != AWQ_OK || M > kMaxM) return 0;
  size_t need = kWsHeaderBytes;
  if (M >= 1 && M <= AWQ_GEMV_MAX_M) {
    const GemvPlan p = plan_gemv(M, K, N, group, sm_count_or_default());
    if (p.ws_bytes > need) need = p.ws_bytes;
  } else if (M > AWQ_GEMV_MAX_M) {
    const GemmPlan p = plan_gemm(M, K, N, sm_count_or_default());
    if (p.ws_bytes > need) need = p.ws_bytes;
  }
  return need;
}

awq_status awq_workspace_init(void* workspace, size_t ws_bytes, void* stream) {
  if (!workspace || ws_bytes < kWsHeaderBytes) return AWQ_ERR_INVALID_ARG;
  if (!aligned16(workspace)) return AWQ_ERR_ALIGNMENT;
  return cudaMemsetAsync(workspace, 0, ws_bytes, static_cast<cudaStream_t>(stream)) == cudaSuccess ? AWQ_OK
                                                                                                   : AWQ_ERR_CUDA;
}

awq_status awq_pack(const void* w, int64_t K, int64_t N, int group, void* qweight, void* scales, void* zeros,
                    void* workspace, size_t ws_bytes, void* stream) {
  awq_status st = check_kn(K, N, group);
  if (st != AWQ_OK) return st;
  if (!w || !qweight || !scales || !zeros || !workspace) return AWQ_ERR_INVALID_ARG;
  if (!aligned16(w) || !aligned16(qweight) || !aligned16(scales) || !aligned16(zeros) || !aligned16(workspace))
    return AWQ_ERR_ALIGNMENT;
  const size_t wb = (size_t)K * N * 2, ng = (size_t)(K / group);
  if (overlap(w, wb, qweight, (size_t)K * N / 2) || overlap(w, wb, scales, ng * N * 2) ||
      overlap(w, wb, zeros, ng * N / 2) || overlap(qweight, (size_t)K * N / 2, scales, ng * N * 2) ||
      overlap(qweight, (size_t)K * N / 2, zeros, ng * N / 2) || overlap(scales, ng * N * 2, zeros, ng * N / 2))
    return AWQ_ERR_INVALID_ARG;
  if (ws_bytes < kWsHeaderBytes) return AWQ_ERR_WORKSPACE;
  if ((st = check_device()) != AWQ_OK) return st;
  cudaError_t e = launch_pack(static_cast<const __half*>(w), K, N, group, static_cast<uint32_t*>(qweight),
                              static_cast<__half*>(scales), static_cast<uint8_t*>(zeros), status_word(workspace),
                              static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? AWQ_OK : AWQ_ERR_CUDA;
}

awq_status awq_dequant(const void* qweight, const void* scales, const void* zeros, int64_t K, int64_t N, int group,
                       void* w_out, void* stream) {
  awq_status st = check_kn(K, N, group);
  if (st != AWQ_OK) return st;
  if (!w_out || !qweight || !scales || !zeros) return AWQ_ERR_INVALID_ARG;
  if (!aligned16(w_out) || !aligned16(qweight) || !aligned16(scales) || !aligned16(zeros)) return AWQ_ERR_ALIGNMENT;
  const size_t wb = (size_t)K * N * 2, ng = (size_t)(K / group);
  if (overlap(w_out, wb, qweight, (size_t)K * N / 2) || overlap(w_out, wb, scales, ng * N * 2) ||
      overlap(w_out, wb, zeros, ng * N / 2))
    return AWQ_ERR_INVALID_ARG;
  if ((st = check_device()) != AWQ_OK) return st;
  cudaError_t e = launch_dequant(static_cast<const uint32_t*>(qweight), static_cast<const __half*>(scales),
                                 static_cast<const uint8_t*>(zeros), K, N, group, static_cast<__half*>(w_out),
                                 static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? AWQ_OK : AWQ_ERR_CUDA;
}

awq_status awq_w4a16_gemv(const void* x, const void* qweight, const void* scales, const void* zeros, void* y,
                          int64_t M, int64_t K, int64_t N, int group, void* workspace, size_t ws_bytes,
                          void* stream) {
  LinearArgs a{x, qweight, scales, zeros, y, M, K, N, group, workspace, ws_bytes};
  awq_status st = check_linear(a);
  if (st != AWQ_OK) return st;
  if (M > AWQ_GEMV_MAX_M) return AWQ_ERR_UNSUPPORTED;
  if (M == 0) return AWQ_OK;
  if ((st = check_device()) != AWQ_OK) return st;
  return gemv_impl(a, static_cast<cudaStream_t>(stream));
}

awq_status awq_w4a16_gemm(const void* x, const void* qweight, const void* scales, const void* zeros, void* y,
                          int64_t M, int64_t K, int64_t N, int group, void* workspace, size_t ws_bytes,
                          void* stream) {
  LinearArgs a{x, qweight, scales, zeros, y, M, K, N, group, workspace, ws_bytes};
  awq_status st = check_linear(a);
  if (st != AWQ_OK) return st;
  if (M == 0) return AWQ_OK;
  if ((st = check_device()) != AWQ_OK) return st;
  return gemm_impl(a, static_cast<cudaStream_t>(stream));
}

awq_status awq_linear(const void* x, const void* qweight, const void* scales, const void* zeros, void* y, int64_t M,
                      int64_t K, int64_t N, int group, void* workspace, size_t ws_bytes, void* stream) {
  LinearArgs a{x, qweight, scales, zeros, y, M, K, N, group, workspace, ws_bytes};
  awq_status st = check_linear(a);
  if (st != AWQ_OK) return st;
  if (M == 0) return AWQ_OK;
  if ((st = check_device()) != AWQ_OK) return st;
  if (linear_uses_gemv(M, N, device_info().sm_count)) return gemv_impl(a, static_cast<cudaStream_t>(stream));
  return gemm_impl(a, static_cast<cudaStream_t>(stream));
}

int awq_linear_gemv_limit(void) { return kGemvAlwaysM; }

awq_status awq_fp8_row_exponents(const void* scales, int64_t K, int64_t N, int group, void* e_out, void* stream) {
  awq_status st = check_kn(K, N, group);
  if (st != AWQ_OK) return st;
  if (!scales || !e_out) return AWQ_ERR_INVALID_ARG;
  if (!aligned16(scales)) return AWQ_ERR_ALIGNMENT;
  if (overlap(e_out, (size_t)N, scales, (size_t)(K / group) * N * 2)) return AWQ_ERR_INVALID_ARG;
  if ((st = check_device()) != AWQ_OK) return st;
  cudaError_t e = launch_fp8_row_exponents(static_cast<const __half*>(scales), K, N, group,
                                           static_cast<int8_t*>(e_out), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? AWQ_OK : AWQ_ERR_CUDA;
}

awq_status awq_fp8_quantize_x(const void* x, int64_t M, int64_t K, void* x8, void* sx, void* stream) {
  if (M < 0 || K <= 0) return AWQ_ERR_SHAPE;
  if (K % kKPerBlock != 0) return AWQ_ERR_SHAPE;
  if (K > kMaxK || M > kMaxM) return AWQ_ERR_UNSUPPORTED;
  if (M == 0) return AWQ_OK;
  if (!x || !x8 || !sx) return AWQ_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(x8) || !aligned16(sx)) return AWQ_ERR_ALIGNMENT;
  const size_t xb = (size_t)M * K * 2, x8b = (size_t)M * K, sxb = (size_t)M * 4;
  if (overlap(x, xb, x8, x8b) || overlap(x, xb, sx, sxb) || overlap(x8, x8b, sx, sxb)) return AWQ_ERR_INVALID_ARG;
  awq_status st = check_device();
  if (st != AWQ_OK) return st;
  cudaError_t e = launch_fp8_quantize_x(static_cast<const __half*>(x), M, K, static_cast<uint8_t*>(x8),
                                        static_cast<float*>(sx), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? AWQ_OK : AWQ_ERR_CUDA;
}

awq_status awq_dequant_fp8(const void* qweight, const void* scales, const void* zeros, const void* row_exp,
                           int64_t K, int64_t N, int group, void* w8_out, void* stream) {
  awq_status st = check_kn(K, N, group);
  if (st != AWQ_OK) return st;
  if (!w8_out || !qweight || !scales || !zeros || !row_exp) return AWQ_ERR_INVALID_ARG;
  if (!aligned16(w8_out) || !aligned16(qweight) || !aligned16(scales) || !aligned16(zeros)) return AWQ_ERR_ALIGNMENT;
  const size_t wb = (size_t)K * N, ng = (size_t)(K / group);
  if (overlap(w8_out, wb, qweight, (size_t)K * N / 2) || overlap(w8_out, wb, scales, ng * N * 2) ||
      overlap(w8_out, wb, zeros, ng * N / 2) || overlap(w8_out, wb, row_exp, (size_t)N))
    return AWQ_ERR_INVALID_ARG;
  if ((st = check_device()) != AWQ_OK) return st;
  cudaError_t e = launch_dequant_fp8(static_cast<const uint32_t*>(qweight), static_cast<const __half*>(scales),
                                     static_cast<const uint8_t*>(zeros), static_cast<const int8_t*>(row_exp), K, N,
                                     group, static_cast<uint8_t*>(w8_out), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? AWQ_OK : AWQ_ERR_CUDA;
}

awq_status awq_w4a8_gemm(const void* x8, const void* sx, const void* qweight, const void* scales, const void* zeros,
                         const void* row_exp, void* y, int64_t M, int64_t K, int64_t N, int group, void* workspace,
                         size_t ws_bytes, void* stream) {
  if (M < 0) return AWQ_ERR_SHAPE;
  awq_status st = check_kn(K, N, group);
  if (st != AWQ_OK) return st;
  if (M > kMaxM) return AWQ_ERR_UNSUPPORTED;
  if ((M > 0 && (!x8 || !sx || !y)) || !qweight || !scales || !zeros || !row_exp || !workspace)
    return AWQ_ERR_INVALID_ARG;
  if (!aligned16(x8) || !aligned16(sx) || !aligned16(qweight) || !aligned16(scales) || !aligned16(zeros) ||
      !aligned16(y) || !aligned16(workspace))
    return AWQ_ERR_ALIGNMENT;
  const size_t ybytes = (size_t)M * N * 2, ng = (size_t)(K / group);
  if (overlap(y, ybytes, x8, (size_t)M * K) || overlap(y, ybytes, sx, (size_t)M * 4) ||
      overlap(y, ybytes, qweight, (size_t)K * N / 2) || overlap(y, ybytes, scales, ng * N * 2) ||
      overlap(y, ybytes, zeros, ng * N / 2) || overlap(y, ybytes, row_exp, (size_t)N) ||
      overlap(y, ybytes, workspace, ws_bytes))
    return AWQ_ERR_INVALID_ARG;
  if (ws_bytes < kWsHeaderBytes) return AWQ_ERR_WORKSPACE;
  if (M == 0) return AWQ_OK;
  if ((st = check_device()) != AWQ_OK) return st;
  cudaError_t e = launch_gemm_fp8(static_cast<const uint8_t*>(x8), static_cast<const float*>(sx),
                                  static_cast<const uint32_t*>(qweight), static_cast<const __half*>(scales),
                                  static_cast<const uint8_t*>(zeros), static_cast<const int8_t*>(row_exp),
                                  static_cast<__half*>(y), M, K, N, group, status_word(workspace),
                                  static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? AWQ_OK : AWQ_ERR_CUDA;
}

awq_status awq_rmsnorm(const void* x, const void* residual, const void* weight, float eps, void* h, void* y, int64_t M,
                       int64_t K, void* stream) {
  return rmsnorm_impl(x, residual, weight, eps, h, y, nullptr, nullptr, false, M, K, stream);
}

awq_status awq_rmsnorm_fp8(const void* x, const void* residual, const void* weight, float eps, void* h, void* x8,
                           void* sx, int64_t M, int64_t K, void* stream) {
  return rmsnorm_impl(x, residual, weight, eps, h, nullptr, x8, sx, true, M, K, stream);
}

awq_status awq_silu_mul(const void* gate_up, void* y, int64_t M, int64_t F, void* stream) {
  return silu_impl(gate_up, y, nullptr, nullptr, false, M, F, stream);
}

awq_status awq_silu_mul_fp8(const void* gate_up, void* x8, void* sx, int64_t M, int64_t F, void* stream) {
  return silu_impl(gate_up, nullptr, x8, sx, true, M, F, stream);
}

size_t awq_kv8_workspace_bytes(int64_t rows, int64_t seqs, int q_heads, int heads, int head_dim) {
  if (check_kv8_sizes(rows, seqs, q_heads, heads, head_dim) != AWQ_OK) return 0;
  return kv8_workspace_bytes(head_dim, sm_count_or_default());
}

awq_status awq_kv8_append(const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                          const awq_kv8_cache* cache, const awq_kv8_batch* batch, void* workspace, size_t ws_bytes,
                          void* stream) {
  Kv8Cache c;
  Kv8Batch b;
  awq_status st = check_kv8(cache, batch, cache ? cache->heads : 0, workspace, ws_bytes, &c, &b);
  if (st != AWQ_OK) return st;
  if (b.rows == 0) return AWQ_OK;
  const int64_t width = (int64_t)c.heads * c.head_dim;
  if (k_stride < width || v_stride < width || k_stride % 8 != 0 || v_stride % 8 != 0) return AWQ_ERR_SHAPE;
  if (!k || !v) return AWQ_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v)) return AWQ_ERR_ALIGNMENT;
  const size_t kbytes = row_bytes(b.rows, k_stride, width), vbytes = row_bytes(b.rows, v_stride, width);
  if (kv8_overlap(c, b, k, kbytes) || kv8_overlap(c, b, v, vbytes) || overlap(k, kbytes, workspace, ws_bytes) ||
      overlap(v, vbytes, workspace, ws_bytes))
    return AWQ_ERR_INVALID_ARG;
  if ((st = check_device()) != AWQ_OK) return st;
  cudaError_t e = launch_kv8_append(static_cast<const __half*>(k), static_cast<const __half*>(v), k_stride, v_stride, c, b,
                                    status_word(workspace), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? AWQ_OK : AWQ_ERR_CUDA;
}

awq_status awq_kv8_attention(const void* q, int64_t q_stride, int q_heads, float scale, const awq_kv8_cache* cache,
                             const awq_kv8_batch* batch, void* y, void* workspace, size_t ws_bytes, void* stream) {
  Kv8Cache c;
  Kv8Batch b;
  awq_status st = check_kv8(cache, batch, q_heads, workspace, ws_bytes, &c, &b);
  if (st != AWQ_OK) return st;
  if (b.rows == 0) return AWQ_OK;
  const int64_t width = (int64_t)q_heads * c.head_dim;
  if (q_stride < width || q_stride % 8 != 0) return AWQ_ERR_SHAPE;
  if (!(scale >= -FLT_MAX && scale <= FLT_MAX)) return AWQ_ERR_INVALID_ARG;
  if (fabsf(scale) > kMaxScale) return AWQ_ERR_UNSUPPORTED;
  if (!q || !y) return AWQ_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(y)) return AWQ_ERR_ALIGNMENT;
  const size_t ybytes = (size_t)b.rows * width * 2, qbytes = row_bytes(b.rows, q_stride, width);
  if (kv8_overlap(c, b, y, ybytes) || overlap(y, ybytes, q, qbytes) || overlap(y, ybytes, workspace, ws_bytes) ||
      overlap(q, qbytes, workspace, ws_bytes))
    return AWQ_ERR_INVALID_ARG;
  if ((st = check_device()) != AWQ_OK) return st;
  cudaError_t e = launch_kv8_attention(static_cast<const __half*>(q), q_stride, q_heads, scale, c, b,
                                       static_cast<__half*>(y), workspace, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? AWQ_OK : AWQ_ERR_CUDA;
}

int awq_linear_path(int64_t M, int64_t K, int64_t N, int group) {
  if (M <= 0 || M > kMaxM || check_kn(K, N, group) != AWQ_OK) return 0;
  const int sms = sm_count_or_default();
  if (linear_uses_gemv(M, N, sms)) return 1;
  return plan_gemm(M, K, N, sms).pair ? 3 : 2;
}

int awq_linear_launches(int64_t M, int64_t K, int64_t N, int group) {
  if (M <= 0 || M > kMaxM || check_kn(K, N, group) != AWQ_OK) return 0;
  const int sms = sm_count_or_default();
  if (!linear_uses_gemv(M, N, sms)) return plan_gemm(M, K, N, sms).stream_k ? 2 : 1;
  return plan_gemv(M, K, N, group, sms).has_split ? 2 : 1;
}

awq_status awq_check_bounded_wait(void* workspace, size_t ws_bytes, uint32_t limit_us, void* stream) {
  if (!workspace || limit_us == 0 || limit_us > 1000000) return AWQ_ERR_INVALID_ARG;
  if (!aligned16(workspace)) return AWQ_ERR_ALIGNMENT;
  if (ws_bytes < kWsHeaderBytes) return AWQ_ERR_WORKSPACE;
  awq_status st = check_device();
  if (st != AWQ_OK) return st;
  bounded_wait_probe_kernel<<<1, 1, 0, static_cast<cudaStream_t>(stream)>>>(status_word(workspace),
                                                                             (uint64_t)limit_us * 1000);
  return cudaGetLastError() == cudaSuccess ? AWQ_OK : AWQ_ERR_CUDA;
}

awq_status awq_get_status(void* workspace, void* stream) {
  if (!workspace) return AWQ_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(s) != cudaSuccess) return AWQ_ERR_CUDA;
  uint32_t word = 0;
  if (cudaMemcpy(&word, workspace, sizeof(word), cudaMemcpyDeviceToHost) != cudaSuccess) return AWQ_ERR_CUDA;
  if (word != 0 && cudaMemset(workspace, 0, sizeof(word)) != cudaSuccess) return AWQ_ERR_CUDA;
  return static_cast<awq_status>(word);
}

const char* awq_status_string(awq_status status) {
  switch (status) {
    case AWQ_OK: return "AWQ_OK";
    case AWQ_ERR_INVALID_ARG: return "AWQ_ERR_INVALID_ARG: null pointer, overlapping buffers or bad workspace";
    case AWQ_ERR_SHAPE: return "AWQ_ERR_SHAPE: need M >= 0, K > 0, N > 0, K % 128 == 0, N % 16 == 0";
    case AWQ_ERR_ALIGNMENT: return "AWQ_ERR_ALIGNMENT: every pointer must be 16-byte aligned";
    case AWQ_ERR_WORKSPACE: return "AWQ_ERR_WORKSPACE: workspace smaller than awq_workspace_bytes()";
    case AWQ_ERR_UNSUPPORTED: return "AWQ_ERR_UNSUPPORTED: group not 32, 64 or 128, size above a limit, or no sm_100 device";
    case AWQ_ERR_CUDA: return "AWQ_ERR_CUDA: a CUDA call or kernel launch failed";
    case AWQ_ERR_TIMEOUT: return "AWQ_ERR_TIMEOUT: a bounded wait on the device expired";
    case AWQ_ERR_NONFINITE: return "AWQ_ERR_NONFINITE: awq_pack met an inf or NaN weight";
    case AWQ_ERR_BOUNDS: return "AWQ_ERR_BOUNDS: a bad block number, row start or length of a cache batch, or a failed index check of the debug build";
  }
  return "unknown awq_status";
}

}  // extern "C"
