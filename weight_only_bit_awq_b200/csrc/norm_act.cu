// The elementwise steps around a decoder layer's 4-bit linear layers:
// awq_rmsnorm(_fp8) and awq_silu_mul(_fp8).
//
//   h = x + residual,  y = h * rsqrt(sum_k h^2 / K + eps) * w       (rmsnorm)
//   y = g / (1 + 2^(-g log2 e)) * u,  gate_up row = [g | u]         (silu_mul)
//   fp16:  y rounded once;   fp8:  sx = max_k|y| / 448, x8 = e4m3(y / sx)
//
// All sums and products are fp32; y is rounded once, to the output's type.
// Both are bound by HBM (8 or 7 bytes an element for the norm with a
// residual, 6 or 5 for the SiLU) and, at a few rows, by the launch.
//
// A row that needs a sum or a maximum is held in registers by one CTA: every
// element is read once, between the load and the store there is one block
// reduction. The norm's E4M3 form needs no second one: with m = max_k|h w|,
// y / sx = h w 448 / m whatever the root mean square is.
#include <cuda_fp8.h>

#include <atomic>

#include "awq_internal.cuh"
#include "sm100_ptx.cuh"

namespace awq {
namespace {

constexpr float kE4m3Max = 448.0f;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}
// The codes of v * f; all zero (not minus zero) for f = 0, the factor of a row of zeros.
__device__ __forceinline__ uint2 codes8(float (&v)[8], float f) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] *= f;
  return f == 0.f ? make_uint2(0, 0) : make_uint2(e4m3x4(v[0], v[1], v[2], v[3]), e4m3x4(v[4], v[5], v[6], v[7]));
}
__device__ __forceinline__ float2 h2f(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
__device__ __forceinline__ uint32_t f2h(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const float2 a = h2f(v.x), b = h2f(v.y), c = h2f(v.z), d = h2f(v.w);
  f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y, f[4] = c.x, f[5] = c.y, f[6] = d.x, f[7] = d.y;
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(f2h(f[0], f[1]), f2h(f[2], f[3]), f2h(f[4], f[5]), f2h(f[6], f[7]));
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Largest |v| as the bits of fp32: a NaN is above infinity, infinity above
// every number, so the maximum also tells a row that is not finite.
__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Maximum that is NaN when an operand is one.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Sum of `s` (kSum) and maximum of `m` (kMax) over the CTA; `red` holds two
// buffers that alternate from row to row, so one barrier a row is enough.
template <bool kSum, bool kMax>
__device__ __forceinline__ void block_reduce(float& s, uint32_t& m, uint2* red, int parity) {
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  auto warp_reduce = [&]() {
    if (kMax) m = __reduce_max_sync(0xffffffffu, m);
    if (kSum) {
#pragma unroll
      for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    }
  };
  warp_reduce();
  red += 32 * parity;
  if (lane == 0) red[threadIdx.x >> 5] = make_uint2(__float_as_uint(s), m);
  __syncthreads();
  const uint2 v = lane < warps ? red[lane] : make_uint2(0, 0);
  s = __uint_as_float(v.x);
  m = v.y;
  warp_reduce();
}

// Vector c of the n of a row, and of the `all` of the matrix at `at`. (Here is no
// status word: the debug build's checks skip the access, and so leave a wrong
// output in place of a fault.)
__device__ __forceinline__ bool inside(int c, int n, [[maybe_unused]] int64_t at, [[maybe_unused]] int64_t all) {
  return c < n && AWQ_CHECK(in_range(at, 1, all), nullptr);
}
// Vector i of the dynamic shared memory.
__device__ __forceinline__ bool in_ahead([[maybe_unused]] int i) {
  return AWQ_CHECK(in_range(16 * (int64_t)i, 16, dynamic_smem_bytes()), nullptr);
}

struct NormArgs {
  const __half *x, *residual, *w;
  __half *h, *y;
  uint8_t* x8;
  float* sx;
  float eps, inv_k;  // inv_k: 1 / K
  int64_t M;
  int K8;  // 8-element vectors of a row
};

// The row factor of y (fp16 output) or of the codes (E4M3 output, where the
// row's scale is stored too); m: largest |h w|. A row with an infinity or a NaN
// has a sum that is not finite, under a weight that is one m is not: then y, or
// sx, is not finite either.
template <bool kFp8>
__device__ __forceinline__ float norm_factor(const NormArgs& a, int64_t row, float sum, uint32_t m) {
  const float rs = rsqrtf(sum * a.inv_k + a.eps), mx = __uint_as_float(m);
  if (!kFp8) return rs;
  if (threadIdx.x == 0) a.sx[row] = sum - sum == 0.f ? mx * rs * (1.f / kE4m3Max) : sum - sum;
  return mx > 0.f ? kE4m3Max / mx : 0.f;
}

// One CTA a row at a time, the row in V vectors of 8 per thread. The weights are
// read for each row (from L1) rather than kept. kWide: more than 512 threads;
// with 32 registers a thread two such CTAs fit an SM (517 x 14848 to fp16 7.5
// against 9.9 us with one, 4096 x 11008 to E4M3 50.2 against 60.1, x 14848 73.5
// against 72.2; narrower CTAs lose by that limit: 8192 x 8192 to E4M3 78.2
// against 72.0).
// With four vectors a thread there is one CTA on an SM, so nothing would be
// loaded while it computes: there the next row's inputs are copied to shared
// memory meanwhile, by the threads that will use them, so that needs no barrier
// (2048 x 28672 to E4M3: 66.6 against 71.5 us; 8192 wide 80.9 against 73.1).
template <int V, bool kRes, bool kFp8, bool kWide>
__global__ void __launch_bounds__(kWide ? 1024 : 512, V <= 2 ? 2 : 1) rmsnorm_kernel(const NormArgs a) {
  constexpr bool kAhead = V == 4;
  extern __shared__ uint4 ahead[];  // [V][x, residual][thread]
  __shared__ uint2 red[64];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int NT = blockDim.x, tid = threadIdx.x;
  constexpr int kIn = kRes ? 2 : 1;
  const uint4 *x = reinterpret_cast<const uint4*>(a.x), *residual = reinterpret_cast<const uint4*>(a.residual);
  auto copy = [&](int64_t row) {
    if (row >= a.M) return;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * NT + tid;
      if (!inside(c, a.K8, row * a.K8 + c, a.M * a.K8) || !in_ahead((kIn * i + kIn - 1) * NT + tid)) continue;
      ptx::cp_async_16(ptx::smem_u32(ahead + kIn * i * NT + tid), x + row * a.K8 + c);
      if (kRes) ptx::cp_async_16(ptx::smem_u32(ahead + (kIn * i + 1) * NT + tid), residual + row * a.K8 + c);
    }
  };
  if (kAhead) copy(blockIdx.x);
  int parity = 0;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, parity ^= 1) {
    const int64_t base = row * a.K8;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 vx[V], vr[V];
    if (kAhead) asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * NT + tid;
      const bool live = inside(c, a.K8, base + c, a.M * a.K8) && (!kAhead || in_ahead((kIn * i + kIn - 1) * NT + tid));
      vx[i] = !live ? zero : kAhead ? ahead[kIn * i * NT + tid] : x[base + c];
      if (kRes) vr[i] = !live ? zero : kAhead ? ahead[(kIn * i + 1) * NT + tid] : residual[base + c];
    }
    if (kAhead) copy(row + gridDim.x);
    float h[V][8], sum = 0.f, most = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * NT + tid;
      unpack8(vx[i], h[i]);
      if (kRes) {
        float r[8];
        unpack8(vr[i], r);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] += r[j];
        if (inside(c, a.K8, base + c, a.M * a.K8)) reinterpret_cast<uint4*>(a.h)[base + c] = pack8(h[i]);
      }
      float wf[8];
      if (kFp8) unpack8(c < a.K8 ? __ldg(reinterpret_cast<const uint4*>(a.w) + c) : zero, wf);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sum = fmaf(h[i][j], h[i][j], sum);
        if (kFp8) {
          h[i][j] *= wf[j];
          most = max_nan(most, fabsf(h[i][j]));
        }
      }
    }
    uint32_t mx = __float_as_uint(most);  // order as their bits, a NaN (of x, the residual or the weights) above all
    block_reduce<true, kFp8>(sum, mx, red, parity);
    const float f = norm_factor<kFp8>(a, row, sum, mx);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * NT + tid;
      if (!inside(c, a.K8, base + c, a.M * a.K8)) continue;
      if (kFp8) {
        reinterpret_cast<uint2*>(a.x8)[base + c] = codes8(h[i], f);
      } else {
        float wf[8];
        unpack8(__ldg(reinterpret_cast<const uint4*>(a.w) + c), wf);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] *= f * wf[j];
        reinterpret_cast<uint4*>(a.y)[base + c] = pack8(h[i]);
      }
    }
  }
}

// Rows too long for the registers of one CTA: read twice (the second time
// mostly from L2). A thread reads again only what it read itself, so h may
// still be x or the residual.
template <bool kRes, bool kFp8>
__global__ void __launch_bounds__(1024) rmsnorm_long_kernel(const NormArgs a) {
  __shared__ uint2 red[64];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  int parity = 0;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, parity ^= 1) {
    const int64_t base = row * a.K8;
    float h[8], r[8], wf[8], sum = 0.f;
    uint32_t mx = 0;
    for (int c = threadIdx.x; inside(c, a.K8, base + c, a.M * a.K8); c += blockDim.x) {
      unpack8(reinterpret_cast<const uint4*>(a.x)[base + c], h);
      if (kRes) unpack8(reinterpret_cast<const uint4*>(a.residual)[base + c], r);
      unpack8(reinterpret_cast<const uint4*>(a.w)[c], wf);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (kRes) h[j] += r[j];
        sum = fmaf(h[j], h[j], sum);
        if (kFp8) mx = max(mx, mag(h[j] * wf[j]));
      }
    }
    block_reduce<true, kFp8>(sum, mx, red, parity);
    const float f = norm_factor<kFp8>(a, row, sum, mx);
    for (int c = threadIdx.x; inside(c, a.K8, base + c, a.M * a.K8); c += blockDim.x) {
      unpack8(reinterpret_cast<const uint4*>(a.x)[base + c], h);
      if (kRes) {
        unpack8(reinterpret_cast<const uint4*>(a.residual)[base + c], r);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] += r[j];
        reinterpret_cast<uint4*>(a.h)[base + c] = pack8(h);
      }
      unpack8(reinterpret_cast<const uint4*>(a.w)[c], wf);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] *= wf[j];
      if (kFp8) {
        reinterpret_cast<uint2*>(a.x8)[base + c] = codes8(h, f);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] *= f;
        reinterpret_cast<uint4*>(a.y)[base + c] = pack8(h);
      }
    }
  }
}

struct SiluArgs {
  const __half* gu;
  __half* y;
  uint8_t* x8;
  float* sx;
  int64_t M;
  int F8;
  int row_ctas;  // CTAs of a row (fp16 output)
};

__device__ __forceinline__ void silu8(const uint4& vg, const uint4& vu, float (&y)[8]) {
  float u[8];
  unpack8(vg, y);
  unpack8(vu, u);
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = y[j] * rcp(1.f + ex2(-kLog2e * y[j])) * u[j];  // 1 / inf is 0
}

// fp16 output: no reduction, a CTA takes blockDim * V vectors of one row (V = 2:
// 8192 x 14336 100.9 us, against 105.6 with one and 100.1 with four).
template <int V>
__global__ void __launch_bounds__(256) silu_mul_kernel(const SiluArgs a) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int64_t row = blockIdx.x / (unsigned)a.row_ctas;
  const int c0 = (int)(blockIdx.x - row * a.row_ctas) * blockDim.x * V + threadIdx.x;
  const uint4* g = reinterpret_cast<const uint4*>(a.gu) + row * 2 * a.F8;
  uint4 vg[V], vu[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = c0 + i * blockDim.x;
    if (inside(c, a.F8, row * 2 * a.F8 + a.F8 + c, a.M * 2 * a.F8)) vg[i] = g[c], vu[i] = g[a.F8 + c];
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = c0 + i * blockDim.x;
    if (!inside(c, a.F8, row * a.F8 + c, a.M * a.F8)) break;
    float y[8];
    silu8(vg[i], vu[i], y);
    reinterpret_cast<uint4*>(a.y)[row * a.F8 + c] = pack8(y);
  }
}

// Stores sx of a row whose largest |y| is m (bits), and returns the codes'
// factor 1 / sx. Below 2^-100 that factor would overflow fp32:
// such a row counts as zero (a y below 2^-25 is zero in fp16 too).
__device__ __forceinline__ float silu_factor(const SiluArgs& a, int64_t row, uint32_t m) {
  const float mx = m < __float_as_uint(0x1p-100f) ? 0.f : __uint_as_float(m);
  if (threadIdx.x == 0) a.sx[row] = mx * (1.f / kE4m3Max);  // infinity and NaN stay
  return mx > 0.f ? kE4m3Max / mx : 0.f;
}

// E4M3 output: one CTA a row at a time, the row in registers. With four vectors
// a thread there is one CTA on an SM, so nothing would be loaded while it
// computes: there the next row's inputs are copied to shared memory meanwhile,
// by the threads that will use them, so that needs no barrier (2048 x 28672:
// 46.8 against 55.4 us; with two CTAs, at 14336, it changed nothing).
template <int V>
__global__ void __launch_bounds__(1024) silu_mul_fp8_kernel(const SiluArgs a) {
  constexpr bool kAhead = V == 4;
  extern __shared__ uint4 ahead[];  // [V][g, u][thread]
  __shared__ uint2 red[64];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int NT = blockDim.x, tid = threadIdx.x;
  auto copy = [&](int64_t row, int i) {
    const int c = i * NT + tid;
    const uint4* g = reinterpret_cast<const uint4*>(a.gu) + row * 2 * a.F8;
    if (row < a.M && inside(c, a.F8, row * 2 * a.F8 + a.F8 + c, a.M * 2 * a.F8) && in_ahead((2 * i + 1) * NT + tid)) {
      ptx::cp_async_16(ptx::smem_u32(ahead + 2 * i * NT + tid), g + c);
      ptx::cp_async_16(ptx::smem_u32(ahead + (2 * i + 1) * NT + tid), g + a.F8 + c);
    }
  };
  if (kAhead) {
#pragma unroll
    for (int i = 0; i < V; ++i) copy(blockIdx.x, i);
  }
  int parity = 0;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, parity ^= 1) {
    const uint4* g = reinterpret_cast<const uint4*>(a.gu) + row * 2 * a.F8;
    float y[V][8], none = 0.f;
    uint32_t mx = 0;
    uint4 vg[V], vu[V];
    if (kAhead) {
      asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = i * NT + tid;
        const bool live = inside(c, a.F8, row * 2 * a.F8 + a.F8 + c, a.M * 2 * a.F8);
        vg[i] = live ? g[c] : make_uint4(0, 0, 0, 0);
        vu[i] = live ? g[a.F8 + c] : make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (kAhead) {
        const bool live = i * NT + tid < a.F8 && in_ahead((2 * i + 1) * NT + tid);
        vg[i] = live ? ahead[2 * i * NT + tid] : make_uint4(0, 0, 0, 0);
        vu[i] = live ? ahead[(2 * i + 1) * NT + tid] : make_uint4(0, 0, 0, 0);
        copy(row + gridDim.x, i);
      }
      silu8(vg[i], vu[i], y[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) mx = max(mx, mag(y[i][j]));
    }
    block_reduce<false, true>(none, mx, red, parity);
    const float f = silu_factor(a, row, mx);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * NT + tid;
      if (inside(c, a.F8, row * a.F8 + c, a.M * a.F8)) reinterpret_cast<uint2*>(a.x8)[row * a.F8 + c] = codes8(y[i], f);
    }
  }
}

// E4M3 output of rows too long for the registers of one CTA: read twice.
__global__ void __launch_bounds__(1024) silu_mul_fp8_long_kernel(const SiluArgs a) {
  __shared__ uint2 red[64];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  int parity = 0;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, parity ^= 1) {
    const uint4* g = reinterpret_cast<const uint4*>(a.gu) + row * 2 * a.F8;
    float y[8], none = 0.f;
    uint32_t mx = 0;
    for (int c = threadIdx.x; inside(c, a.F8, row * 2 * a.F8 + a.F8 + c, a.M * 2 * a.F8); c += blockDim.x) {
      silu8(g[c], g[a.F8 + c], y);
#pragma unroll
      for (int j = 0; j < 8; ++j) mx = max(mx, mag(y[j]));
    }
    block_reduce<false, true>(none, mx, red, parity);
    const float f = silu_factor(a, row, mx);
    for (int c = threadIdx.x; inside(c, a.F8, row * 2 * a.F8 + a.F8 + c, a.M * 2 * a.F8); c += blockDim.x) {
      silu8(g[c], g[a.F8 + c], y);
      reinterpret_cast<uint2*>(a.x8)[row * a.F8 + c] = codes8(y, f);
    }
  }
}

// Vectors per thread for rows of n: the fewest that 1024 threads hold (fp16
// output, 8192 rows: 4096 wide 43.1 us with one against 45.9 with two, 8192
// wide 82.8 against 89.4; a single row of 4096 1.74 against 2.08). With E4M3
// output, whose second half is longer, two from 2048 wide on (8192 rows of 4096:
// the norm 37.2 against 48.6 us with one, the SiLU 27.8 against 31.1; four
// instead of two for 14336: 104 against 97.5).
int row_vectors(int n, bool fp8) {
  if (n <= (fp8 ? 256 : 1024)) return 1;
  return n <= 2048 ? 2 : 4;
}
// Threads of a CTA that holds a row of n vectors, V per thread.
int row_threads(int n, int V) { return (n + 32 * V - 1) / (32 * V) * 32; }

template <typename Args>
cudaError_t launch_rows(void (*kernel)(Args), const Args& a, unsigned ctas, int threads, cudaStream_t stream,
                        size_t smem = 0) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

// CTAs that walk M rows: as many as fit the SMs at once by 2048 threads each. The
// two kernels with four vectors a thread fit one: the SiLU gets that many
// (2048 x 28672: 46.8 against 49.6 us, 4000 x 18944 64.2 against 67.3), the norm,
// for which a second set of shorter walks is as good or better, as many as others
// (2000 x 20480 to fp16 55.3 against 58.7, 2048 x 28672 to E4M3 65.9 against 66.4).
unsigned row_ctas(int64_t M, int threads) {
  const int64_t fit = (int64_t)device_info().sm_count * (2048 / threads);
  return (unsigned)(M < fit ? M : fit);
}

// Allows a kernel more than 48 KB of dynamic shared memory, once per device;
// `set` has one bit per device.
template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes, std::atomic<uint64_t>& set) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return cudaErrorInvalidDevice;
  if (set.load(std::memory_order_acquire) >> dev & 1) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) set.fetch_or(uint64_t(1) << dev, std::memory_order_acq_rel);
  return e;
}

template <int V, bool kRes, bool kFp8, bool kWide>
cudaError_t launch_norm_v(const NormArgs& a, int threads, cudaStream_t stream) {
  auto kernel = rmsnorm_kernel<V, kRes, kFp8, kWide>;
  if (V < 4) return launch_rows(kernel, a, row_ctas(a.M, threads), threads, stream);
  static std::atomic<uint64_t> set{0};
  constexpr size_t kRowBytes = (size_t)V * (kRes ? 2 : 1) * 16;  // per thread
  cudaError_t e = allow_smem(kernel, kRowBytes * 1024, set);
  return e != cudaSuccess ? e : launch_rows(kernel, a, row_ctas(a.M, threads), threads, stream, kRowBytes * threads);
}

template <bool kRes, bool kFp8>
cudaError_t launch_norm(const NormArgs& a, cudaStream_t stream) {
  if (a.K8 > 4096) return launch_rows(rmsnorm_long_kernel<kRes, kFp8>, a, row_ctas(a.M, 1024), 1024, stream);
  const int V = row_vectors(a.K8, kFp8);
  const int t = row_threads(a.K8, V);
  if (V == 4) return launch_norm_v<4, kRes, kFp8, true>(a, t, stream);
  if (V == 2)
    return t > 512 ? launch_norm_v<2, kRes, kFp8, true>(a, t, stream) : launch_norm_v<2, kRes, kFp8, false>(a, t, stream);
  return t > 512 ? launch_norm_v<1, kRes, kFp8, true>(a, t, stream) : launch_norm_v<1, kRes, kFp8, false>(a, t, stream);
}

}  // namespace

cudaError_t launch_rmsnorm(const __half* x, const __half* residual, const __half* w, float eps, __half* h, __half* y,
                           uint8_t* x8, float* sx, int64_t M, int64_t K, cudaStream_t stream) {
  const NormArgs a{x, residual, w, h, y, x8, sx, eps, 1.f / (float)K, M, (int)(K / 8)};
  if (residual) return x8 ? launch_norm<true, true>(a, stream) : launch_norm<true, false>(a, stream);
  return x8 ? launch_norm<false, true>(a, stream) : launch_norm<false, false>(a, stream);
}

cudaError_t launch_silu_mul(const __half* gate_up, __half* y, uint8_t* x8, float* sx, int64_t M, int64_t F,
                            cudaStream_t stream) {
  SiluArgs a{gate_up, y, x8, sx, M, (int)(F / 8), 0};
  if (x8) {
    if (a.F8 > 4096) return launch_rows(silu_mul_fp8_long_kernel, a, row_ctas(M, 1024), 1024, stream);
    const int V = row_vectors(a.F8, true);
    const int t = row_threads(a.F8, V);
    if (V == 1) return launch_rows(silu_mul_fp8_kernel<1>, a, row_ctas(M, t), t, stream);
    if (V == 2) return launch_rows(silu_mul_fp8_kernel<2>, a, row_ctas(M, t), t, stream);
    static std::atomic<uint64_t> set{0};
    cudaError_t e = allow_smem(silu_mul_fp8_kernel<4>, (size_t)4 * 32 * 1024, set);
    if (e != cudaSuccess) return e;
    // registers leave room for one CTA on an SM
    return launch_rows(silu_mul_fp8_kernel<4>, a, row_ctas(M, 2048), t, stream, (size_t)4 * 32 * t);
  }
  constexpr int V = 2;
  const int parts = (a.F8 + 256 * V - 1) / (256 * V);
  const int t = row_threads((a.F8 + parts - 1) / parts, V);
  a.row_ctas = (a.F8 + t * V - 1) / (t * V);
  const int64_t ctas = M * a.row_ctas;
  if (ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  return launch_rows(silu_mul_kernel<V>, a, (unsigned)ctas, t, stream);
}

}  // namespace awq
