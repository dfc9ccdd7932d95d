// The 8-bit key/value cache: awq_kv8_append and awq_kv8_attention.
//
// The cache is paged. A block holds `block_tokens` tokens of every kv head;
// one head of a block is one contiguous run of E4M3 codes with one exponent:
//   value = code * 2^e,   e = the smallest integer with amax <= 448 * 2^e
// (the power-of-two form the library's W4A8 weights have). Powers of two make
// both uses exact: a code times 2^e is exact in fp16 arithmetic up to fp32
// accumulation, and when a later token of a block raises e, the codes that
// are there are multiplied by 2^(e_old - e_new), which rounds only those that
// become E4M3 subnormals.
#include <cuda_fp8.h>

#include <atomic>

#include "awq_internal.cuh"
#include "sm100_ptx.cuh"

namespace awq {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr float kLog2e = 1.4426950408889634f;

// ---------------------------------------------------------------------------
// the batch: who owns which rows, and where work item `u` lies
// ---------------------------------------------------------------------------

struct Seq {
  int row0, tokens, len;  // first new row, new tokens, cached tokens (the new ones included)
};

// Sequence b, its bounds clamped to the buffers (a clamp is reported).
__device__ __forceinline__ Seq load_seq(const Kv8Batch& bt, int b, uint32_t* status) {
  const int s0 = bt.starts[b], s1 = bt.starts[b + 1], len = bt.lens[b];
  const int cap = bt.table_width * bt.block_tokens;
  Seq s;
  s.row0 = min(max(s0, 0), bt.rows);
  s.tokens = min(max(s1, s.row0), bt.rows) - s.row0;
  s.len = min(max(len, 0), cap);
  if (s.row0 != s0 || s.row0 + s.tokens != s1 || s.len != len) record_status(status, AWQ_ERR_BOUNDS);
  return s;
}

// The items of all sequences, one after another: items(b) of them belong to
// sequence b. Every thread of the CTA calls this; `total` is their sum, and
// for item u (u < total) `b` its sequence and `base` the sequence's first.
template <typename Items>
__device__ __forceinline__ int64_t total_items(int B, const Items& items, int64_t* scan /* [kWarps + 1] */,
                                               int64_t& before) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (B + kThreads - 1) / kThreads;
  int64_t mine = 0;
  for (int b = tid * per; b < min(B, (tid + 1) * per); ++b) mine += items(b);
  int64_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) scan[warp] = inc;
  __syncthreads();
  int64_t total = 0;
  before = inc - mine;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  return total;
}

struct Place {
  int b;
  int64_t base;
};

// Sequence of item u < total; `before` is this thread's from total_items.
template <typename Items>
__device__ __forceinline__ Place find_item(int B, const Items& items, int64_t before, int64_t u, Place* shared) {
  const int per = (B + kThreads - 1) / kThreads;
  int64_t at = before;
  for (int b = threadIdx.x * per; b < min(B, (int)(threadIdx.x + 1) * per); ++b) {
    const int64_t n = items(b);
    if (u >= at && u < at + n) *shared = Place{b, at};
    at += n;
  }
  __syncthreads();
  return *shared;
}

// ---------------------------------------------------------------------------
// E4M3
// ---------------------------------------------------------------------------

// Two codes (low byte first) as exact fp16 values; a NaN code stays NaN.
__device__ __forceinline__ uint32_t codes_to_h2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}
__device__ __forceinline__ uint32_t lo_h2(uint32_t w) { return codes_to_h2((uint16_t)w); }
__device__ __forceinline__ uint32_t hi_h2(uint32_t w) { return codes_to_h2((uint16_t)(w >> 16)); }
__device__ __forceinline__ float2 h2f(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
__device__ __forceinline__ uint32_t f2h(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t code2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Smallest e with |v| <= 448 2^e for the fp16 magnitude bits of a finite v:
// v = 1.m 2^x in fp32, 448 = 1.75 * 2^8. Zero needs the least, -32 (what
// 2^-24, the smallest fp16, needs).
__device__ __forceinline__ int needed_exponent(uint32_t mag) {
  if (mag == 0) return -32;
  const uint32_t f = __float_as_uint(__half2float(__ushort_as_half((unsigned short)mag)));
  return (int)(f >> 23) - 127 - 8 + ((f & 0x7FFFFFu) > 0x600000u);
}

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------

// One CTA per (block that gets new tokens, kv head, K or V). The block's new
// rows stay in registers between the maximum and the conversion, so they are
// read once. Bound by HBM for prompts (2 bytes read, 1 written an element),
// by the launch for single tokens.
template <int kIter>  // 16-byte pieces of a block's rows per thread: block_tokens * D / 1024
__global__ void __launch_bounds__(kThreads) kv8_append_kernel(const __half* __restrict__ knew,
                                                              const __half* __restrict__ vnew, int64_t k_stride,
                                                              int64_t v_stride, Kv8Cache cache, Kv8Batch bt,
                                                              uint32_t* status) {
  __shared__ int64_t scan[kWarps];
  __shared__ Place place;
  __shared__ uint32_t wmax[kWarps];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int bs = bt.block_tokens, D = cache.head_dim;
  // blocks of sequence b that get new tokens
  auto items = [&](int b) -> int64_t {
    const Seq s = load_seq(bt, b, status);
    const int first = max(s.len - s.tokens, 0);
    return first < s.len && s.tokens > 0 ? (s.len - 1) / bs - first / bs + 1 : 0;
  };
  int64_t before;
  const int64_t total = total_items(bt.seqs, items, scan, before);
  const int64_t u = blockIdx.x;
  if (u >= total) return;
  const Place p = find_item(bt.seqs, items, before, u, &place);
  const Seq s = load_seq(bt, p.b, status);
  const int past = s.len - s.tokens;  // position of the first new row (rows at negative positions have no place)
  const int j = max(past, 0) / bs + (int)(u - p.base);
  const int blk = bt.table[(int64_t)p.b * bt.table_width + j];
  if (blk < 0 || blk >= cache.blocks) {
    if (threadIdx.x == 0) record_status(status, AWQ_ERR_BOUNDS);
    return;
  }
  const int h = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  const int lo = max(max(past, 0) - j * bs, 0), hi = min(s.len - j * bs, bs);  // new rows of the block
  const int pieces = D / 8, rows_per_pass = kThreads / pieces;
  const int r0 = threadIdx.x / pieces, c = threadIdx.x % pieces;
  const __half* src = (is_v ? vnew : knew) + (int64_t)h * D + 8 * c;
  const int64_t stride = is_v ? v_stride : k_stride;
  const int64_t row0 = (int64_t)s.row0 + (int64_t)j * bs - past;  // source row of the block's token 0

  uint4 x[kIter];
  uint32_t mag = 0;
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int r = r0 + i * rows_per_pass;
    x[i] = r >= lo && r < hi ? *reinterpret_cast<const uint4*>(src + (row0 + r) * stride) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t a = w[q] & 0x7FFFu, b = (w[q] >> 16) & 0x7FFFu;
      if (a < 0x7C00u) mag = max(mag, a);  // infinities and NaN become NaN codes and set no scale
      if (b < 0x7C00u) mag = max(mag, b);
    }
  }
  mag = __reduce_max_sync(0xffffffffu, mag);
  if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = mag;
  int8_t* exps = (is_v ? cache.v_exp : cache.k_exp) + (int64_t)blk * cache.heads + h;
  const int e_old = lo > 0 ? (int)*exps : -128;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) mag = max(mag, wmax[w]);
  const int e = max(needed_exponent(mag), e_old);
  if (threadIdx.x == 0) *exps = (int8_t)e;
  uint8_t* dst = (is_v ? cache.v : cache.k) + ((int64_t)blk * cache.heads + h) * bs * D + 8 * c;
  const float inv = ldexpf(1.f, -e);
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int r = r0 + i * rows_per_pass;
    if (r < lo || r >= hi) continue;
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint32_t o[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float2 f = h2f(w[q]);
      f.x = fabsf(f.x) <= 65504.f ? f.x * inv : NAN;  // exact; the conversion would saturate an infinity
      f.y = fabsf(f.y) <= 65504.f ? f.y * inv : NAN;
      o[q] = code2(f.x, f.y);
    }
    *reinterpret_cast<uint2*>(dst + (int64_t)r * D) = make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
  }
  if (e > e_old && lo > 0) {  // the codes that were there, under the larger exponent
    const float down = ldexpf(1.f, e_old - e);
    for (int r = r0; r < lo; r += rows_per_pass) {
      uint2* at = reinterpret_cast<uint2*>(dst + (int64_t)r * D);
      const uint2 v = *at;
      const float2 a = h2f(lo_h2(v.x)), b = h2f(hi_h2(v.x)), d = h2f(lo_h2(v.y)), f = h2f(hi_h2(v.y));
      *at = make_uint2(code2(a.x * down, a.y * down) | (code2(b.x * down, b.y * down) << 16),
                       code2(d.x * down, d.y * down) | (code2(f.x * down, f.y * down) << 16));
    }
  }
}

// ---------------------------------------------------------------------------
// attention
// ---------------------------------------------------------------------------

// S^T = K q^T and O^T = V^T P^T with mma.sync m16n8k16: the keys (of S) and
// the head's channels (of O) are the MMA's 16 rows, the query rows its 8
// columns, so the few rows of a generation step (query heads that share a kv
// head, times new tokens) waste half as much as they would as the 16-row
// operand. Codes become exact fp16 in registers; the products are exact, the
// sums fp32.
//
// Bound by HBM: every code is read once, 4 flops a code and row. So each lane
// copies exactly the codes that its own MMA fragments hold, 16 bytes at a
// time with cp.async into its own part of a ring in shared memory: no
// barrier, no bank conflict, no lane waits for another.
//
// Softmax in one pass, in powers of two. With x = scale log2(e) q.k and the V
// exponent e of a key's block, the weight kept for a key is
// p = 2^(x + e - M + 15), M the running maximum of x + e: V's codes then need
// no scaling, p uses fp16's range down to 2^-39 of the largest, and
// l = sum p 2^-e is the denominator in the same unit. p is rounded to fp16
// (2^-11 relative) for the second MMA; l sums the unrounded p.
constexpr float kPOffset = 15.f;

// The group of units that starts in a CTA's range and ends in a later one's.
struct Kv8Fix {
  int valid, row0, rows, tile0, head, last_cta, pad0, pad1;
};

struct AttnArgs {
  const __half* q;
  int64_t q_stride;
  __half* out;
  int group;          // query heads per kv head
  float scale_log2;   // softmax scale times log2 e
  float* partial;     // [ctas][2][slot]
  int slot;           // floats of a slot: rows * (D + 2)
  Kv8Fix* fix;        // [ctas]
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// Copies that write zeros when !ok (then nothing is read).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(ok ? 8 : 0) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// D: head dimension; SUB: 16-key subtiles of a warp's step; NT: column tiles
// of 8 query rows. A unit of work is 4 warps x 16 SUB keys of one (sequence,
// kv head, row tile).
template <int D, int SUB, int NT>
struct Attn {
  static constexpr int kRows = 8 * NT;
  static constexpr int kKeys = kWarps * 16 * SUB;             // keys of a unit
  static constexpr int kStages = 3;
  static constexpr int kStageBytes = SUB * 32 * D;            // per warp: 16 keys, K and V
  static constexpr int kMergeBytes = kWarps * kRows * (D + 4) * 4 + kWarps * kRows * 8;
  static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
  static constexpr int kSmem = kRingBytes > kMergeBytes ? kRingBytes : kMergeBytes;
  static constexpr int kSlot = kRows * (D + 2);
  static constexpr int kCtasPerSm = NT == 1 ? 4 : 3;          // 128 or 168 registers a thread
};

template <int D, int SUB, int NT>
__global__ void __launch_bounds__(kThreads, Attn<D, SUB, NT>::kCtasPerSm)
    kv8_attention_kernel(const AttnArgs a, const Kv8Cache cache, const Kv8Batch bt, uint32_t* status) {
  using L = Attn<D, SUB, NT>;
  constexpr int KS = D / 16;     // k-steps of S
  constexpr int MT = D / 16;     // channel tiles of O
  constexpr int KH = D / 64;     // 64-byte halves of a key
  extern __shared__ __align__(16) char smem[];
  __shared__ int64_t scan[kWarps];
  __shared__ Place place;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int bs = bt.block_tokens, shift = __ffs(bs) - 1;
  auto row_tiles = [&](const Seq& s) { return ((int64_t)s.tokens * a.group + L::kRows - 1) / L::kRows; };
  // a sequence with no keys still has one (empty) unit per row tile: its rows are zero
  auto key_tiles = [&](const Seq& s) { return max((s.len + L::kKeys - 1) / L::kKeys, 1); };
  auto items = [&](int b) -> int64_t {
    const Seq s = load_seq(bt, b, status);
    return row_tiles(s) * key_tiles(s) * cache.heads;
  };
  int64_t before;
  const int64_t total = total_items(bt.seqs, items, scan, before);
  const int64_t ctas = total < (int64_t)gridDim.x ? total : (int64_t)gridDim.x;
  if (tid == 0) a.fix[blockIdx.x].valid = 0;
  if ((int64_t)blockIdx.x >= ctas) return;
  auto first_unit = [&](int64_t c) { return total / ctas * c + total % ctas * c / ctas; };
  int64_t u = first_unit(blockIdx.x);
  const int64_t u1 = first_unit((int64_t)blockIdx.x + 1);
  Place p = find_item(bt.seqs, items, before, u, &place);

  const uint32_t ring = ptx::smem_u32(smem) + warp * (L::kStages * L::kStageBytes) + lane * 16;

  while (u < u1) {
    Seq s = load_seq(bt, p.b, status);
    int64_t n_seq = row_tiles(s) * key_tiles(s) * cache.heads;
    while (u >= p.base + n_seq) {
      p.base += n_seq;
      s = load_seq(bt, ++p.b, status);
      n_seq = row_tiles(s) * key_tiles(s) * cache.heads;
    }
    const int tiles = key_tiles(s);
    const int64_t in_seq = u - p.base, group_no = in_seq / tiles;
    const int tile0 = (int)(in_seq - group_no * tiles);
    const int h = (int)(group_no / row_tiles(s));
    const int row_tile = (int)(group_no - (int64_t)h * row_tiles(s));
    const int n = (int)(u1 - u < tiles - tile0 ? u1 - u : tiles - tile0);
    const int rows = s.tokens * a.group, r0 = row_tile * L::kRows;
    const int past = s.len - s.tokens;

    // ---- this segment's query rows as B fragments: k = channels of the lane's K bytes
    uint32_t qf[NT][KS][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = r0 + 8 * nt + g;
      const __half* q = a.q + (int64_t)(s.row0 + r / a.group) * a.q_stride + ((int64_t)h * a.group + r % a.group) * D + 16 * t;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint2 v = make_uint2(0, 0);
        if (r < rows) v = *reinterpret_cast<const uint2*>(q + 64 * (ks / 4) + 4 * (ks % 4));
        qf[nt][ks][0] = v.x;
        qf[nt][ks][1] = v.y;
      }
    }
    int limit[NT][2];  // keys that the lane's two rows of each column tile see
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) limit[nt][c] = past + (r0 + 8 * nt + 2 * t + c) / a.group + 1;
    const int least = past + r0 / a.group + 1;  // keys that every row sees

    float o[NT][MT][4], M[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < MT; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
      M[nt][0] = M[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }

    // Blocks and exponents of the next 32 subtiles of this warp, one per lane.
    const int* table = bt.table + (int64_t)p.b * bt.table_width;
    auto key_of = [&](int sub) { return (tile0 + sub / SUB) * L::kKeys + warp * 16 * SUB + (sub % SUB) * 16; };
    int blk = -1, exps = 0, exps_prev = 0;
    auto load_info = [&](int sub0) {
      const int sub = sub0 + lane, key = key_of(sub);
      exps_prev = exps;
      blk = -1;
      exps = 0;
      if (sub < n * SUB && key < s.len) {
        blk = table[key >> shift];
        if (blk < 0 || blk >= cache.blocks) {
          record_status(status, AWQ_ERR_BOUNDS);
          blk = -1;
        } else {
          const int64_t at = (int64_t)blk * cache.heads + h;
          exps = (uint8_t)cache.k_exp[at] | ((uint8_t)cache.v_exp[at] << 8);
        }
      }
    };
    auto issue = [&](int step) {
      if (step < n) {
        if ((step * SUB) % 32 == 0) load_info(step * SUB);
        const uint32_t dst = ring + (step % L::kStages) * L::kStageBytes;
#pragma unroll
        for (int sb = 0; sb < SUB; ++sb) {
          const int sub = step * SUB + sb, key = key_of(sub);
          const int id = __shfl_sync(0xffffffffu, blk, sub & 31);
          const int64_t at = (((int64_t)max(id, 0) * cache.heads + h) * bs + (key & (bs - 1))) * D;
          const int live = id < 0 ? 0 : s.len - key;  // keys of the subtile that exist
          const uint32_t d0 = dst + sb * (32 * D);
#pragma unroll
          for (int rh = 0; rh < 2; ++rh)
#pragma unroll
            for (int kh = 0; kh < KH; ++kh) {
              const bool ok = 8 * rh + g < live;
              copy16(d0 + (rh * KH + kh) * 512, cache.k + at + (ok ? (8 * rh + g) * D : 0) + 64 * kh + 16 * t, ok);
            }
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const int kn = 2 * t + (kk & 1) + 8 * (kk >> 1);
            const bool ok = kn < live;
            if (D == 128)
              copy16(d0 + 16 * D + kk * 512, cache.v + at + (ok ? kn * D : 0) + 16 * g, ok);
            else
              copy8(d0 + 16 * D + (kk >> 1) * 512 + (kk & 1) * 8, cache.v + at + (ok ? kn * D : 0) + 8 * g, ok);
          }
        }
      }
      copy_commit();
    };

#pragma unroll
    for (int i = 0; i < L::kStages - 1; ++i) issue(i);
    for (int step = 0; step < n; ++step) {
      issue(step + L::kStages - 1);
      copy_wait<L::kStages - 1>();
      const uint32_t src = ring + (step % L::kStages) * L::kStageBytes;

      // S^T of the step's subtiles, as x + e_v (masked keys: -inf)
      float x[SUB][NT][4], inv_ev[SUB];
#pragma unroll
      for (int sb = 0; sb < SUB; ++sb) {
        uint4 kw[2][KH];
#pragma unroll
        for (int rh = 0; rh < 2; ++rh)
#pragma unroll
          for (int kh = 0; kh < KH; ++kh) kw[rh][kh] = lds16(src + sb * (32 * D) + (rh * KH + kh) * 512);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) x[sb][nt][0] = x[sb][nt][1] = x[sb][nt][2] = x[sb][nt][3] = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const uint4 &ka = kw[0][ks / 4], &kb = kw[1][ks / 4];
          const uint32_t wa = ks % 4 == 0 ? ka.x : ks % 4 == 1 ? ka.y : ks % 4 == 2 ? ka.z : ka.w;
          const uint32_t wb = ks % 4 == 0 ? kb.x : ks % 4 == 1 ? kb.y : ks % 4 == 2 ? kb.z : kb.w;
          const uint32_t a0 = lo_h2(wa), a1 = lo_h2(wb), a2 = hi_h2(wa), a3 = hi_h2(wb);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(x[sb][nt], a0, a1, a2, a3, qf[nt][ks][0], qf[nt][ks][1]);
        }
        const int sub = step * SUB + sb, key = key_of(sub);
        // the issuing side is up to kStages - 1 steps ahead: it may have loaded the next 32 already
        const int ahead = min(step + L::kStages - 1, n - 1) * SUB / 32;
        const int e2 = __shfl_sync(0xffffffffu, sub / 32 == ahead ? exps : exps_prev, sub & 31);
        const float ks2 = a.scale_log2 * __int_as_float(((int)(int8_t)e2 + 127) << 23);
        const int ev = (int8_t)(e2 >> 8);
        inv_ev[sb] = __int_as_float((127 - ev) << 23);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) x[sb][nt][c] = fmaf(x[sb][nt][c], ks2, (float)ev);
        if (key + 16 > least) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (key + g + 8 * (c >> 1) >= min(limit[nt][c & 1], s.len)) x[sb][nt][c] = -INFINITY;
        }
      }

      // running maximum over keys (rows of S^T: the lanes' g)
      float Mn[NT][2];
      bool grew = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float m = M[nt][c];
#pragma unroll
          for (int sb = 0; sb < SUB; ++sb) m = fmaxf(m, fmaxf(x[sb][nt][c], x[sb][nt][c + 2]));
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
          Mn[nt][c] = m;
          grew |= m > M[nt][c];
        }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float f[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            f[c] = Mn[nt][c] == -INFINITY ? 0.f : ex2(M[nt][c] - Mn[nt][c]);
            l[nt][c] *= f[c];
            M[nt][c] = Mn[nt][c];
          }
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            o[nt][i][0] *= f[0], o[nt][i][1] *= f[1];
            o[nt][i][2] *= f[0], o[nt][i][3] *= f[1];
          }
        }
      }

#pragma unroll
      for (int sb = 0; sb < SUB; ++sb) {
        uint32_t pf[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float pr[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float m = M[nt][c & 1] == -INFINITY ? 0.f : M[nt][c & 1];
            pr[c] = ex2(x[sb][nt][c] - m + kPOffset);
            l[nt][c & 1] = fmaf(pr[c], inv_ev[sb], l[nt][c & 1]);
          }
          pf[nt][0] = transpose8x8(f2h(pr[0], pr[1]));
          pf[nt][1] = transpose8x8(f2h(pr[2], pr[3]));
        }
        const uint32_t vsrc = src + sb * (32 * D) + 16 * D;
        uint32_t vw[4][MT / 2];  // the lane's channels of keys 2t, 2t+1, 2t+8, 2t+9
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          if (D == 128) {
            const uint4 v = lds16(vsrc + kk * 512);
            vw[kk][0] = v.x, vw[kk][1] = v.y, vw[kk][MT / 2 - 2] = v.z, vw[kk][MT / 2 - 1] = v.w;
          } else {
            const uint2 v = lds8(vsrc + (kk >> 1) * 512 + (kk & 1) * 8);
            vw[kk][0] = v.x, vw[kk][1] = v.y;
          }
        }
        // Where some rows do not see all 16 keys, a NaN code must reach only
        // the rows that see it: 0 * NaN in the MMA would reach all. Such codes
        // are taken out and their channels of the rows that see them set to NaN here.
        const int key = key_of(step * SUB + sb);
        if (least < s.len && key + 16 > least) {
          uint32_t nan[4][MT / 2], any = 0;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int w = 0; w < MT / 2; ++w) {
              nan[kk][w] = ((vw[kk][w] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;  // 0x80 in bytes that are 0x7F or 0xFF
              any |= nan[kk][w];
            }
          if (__any_sync(0xffffffffu, any)) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
#pragma unroll
              for (int w = 0; w < MT / 2; ++w) {
                vw[kk][w] &= ~((nan[kk][w] >> 7) * 0xFFu);
#pragma unroll 1
                for (int tt = 0; tt < 4; ++tt) {  // the four lanes that share this lane's channels
                  const uint32_t m = __shfl_sync(0xffffffffu, nan[kk][w], (lane & ~3) | tt);
                  const int at = key + 2 * tt + (kk & 1) + 8 * (kk >> 1);
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int b = 0; b < 4; ++b)
#pragma unroll
                      for (int c = 0; c < 2; ++c)
                        if ((m >> (8 * b + 7) & 1) && at < limit[nt][c]) o[nt][2 * w + (b >> 1)][2 * (b & 1) + c] = NAN;
                }
              }
          }
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const uint32_t sel = i & 1 ? 0x7362u : 0x5140u;
          const uint32_t p01 = __byte_perm(vw[0][i / 2], vw[1][i / 2], sel);
          const uint32_t p23 = __byte_perm(vw[2][i / 2], vw[3][i / 2], sel);
          const uint32_t a0 = lo_h2(p01), a1 = hi_h2(p01), a2 = lo_h2(p23), a3 = hi_h2(p23);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][i], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
        }
      }
    }
    copy_wait<0>();

    // ---- the four warps' parts of the segment
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], w);
    float* mo = reinterpret_cast<float*>(smem);                    // [warp][row][D + 4]
    float2* ml = reinterpret_cast<float2*>(mo + kWarps * L::kRows * (D + 4));  // [warp][row]
    __syncthreads();  // every warp is done with the ring
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = warp * L::kRows + 8 * nt + 2 * t + c;
#pragma unroll
        for (int i = 0; i < MT; ++i)
          *reinterpret_cast<float2*>(mo + r * (D + 4) + (D / 8) * g + 2 * i) = make_float2(o[nt][i][c], o[nt][i][c + 2]);
        if (g == 0) ml[r] = make_float2(M[nt][c], l[nt][c]);
      }
    __syncthreads();
    const bool starts_here = tile0 == 0, ends_here = tile0 + n == tiles;
    float* slot = a.partial + ((int64_t)blockIdx.x * 2 + (starts_here ? 1 : 0)) * a.slot;
    for (int i = tid; i < L::kRows * (D / 4); i += kThreads) {
      const int r = i / (D / 4), d = i % (D / 4) * 4;
      if (r0 + r >= rows) continue;
      float mx = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, ml[w * L::kRows + r].x);
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
      float den = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 v = ml[w * L::kRows + r];
        const float f = v.x == -INFINITY && v.y == 0.f ? 0.f : ex2(v.x - (mx == -INFINITY ? 0.f : mx));
        const float4 ow = *reinterpret_cast<const float4*>(mo + (w * L::kRows + r) * (D + 4) + d);
        sum.x = fmaf(f, ow.x, sum.x), sum.y = fmaf(f, ow.y, sum.y);
        sum.z = fmaf(f, ow.z, sum.z), sum.w = fmaf(f, ow.w, sum.w);
        den = fmaf(f, v.y, den);
      }
      if (starts_here && ends_here) {
        const float inv = den == 0.f ? 0.f : 1.f / den;  // a row that sees no key is zero
        const int64_t at = (int64_t)(s.row0 + (r0 + r) / a.group) * cache.heads * a.group + (int64_t)h * a.group + (r0 + r) % a.group;
        *reinterpret_cast<uint2*>(a.out + at * D + d) = make_uint2(f2h(sum.x * inv, sum.y * inv), f2h(sum.z * inv, sum.w * inv));
      } else {
        *reinterpret_cast<float4*>(slot + r * D + d) = sum;
        if (d == 0) *reinterpret_cast<float2*>(slot + L::kRows * D + 2 * r) = make_float2(mx, den);
      }
    }
    if (starts_here && !ends_here && tid == 0) {
      // the CTA that holds the group's last unit: the last c with first_unit(c) < the group's end
      const int64_t end = u + tiles;
      a.fix[blockIdx.x] = Kv8Fix{1, s.row0, rows, r0, h, (int)((end * ctas + total - 1) / total) - 1, 0, 0};
    }
    u += n;
    __syncthreads();  // the merge buffer is the next segment's ring
  }
}

// Adds the parts of the groups that more than one CTA worked on, in CTA order
// (so the result does not depend on timing). CTA c of this kernel has the
// group that starts in CTA c of the attention kernel: one part in that CTA's
// slot 1, the others in the following CTAs' slots 0. A warp takes a row.
template <int D>
__global__ void __launch_bounds__(256) kv8_fixup_kernel(const AttnArgs a, int heads, int tile_rows) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const Kv8Fix f = a.fix[blockIdx.x];
  if (!f.valid) return;
  const int lane = threadIdx.x & 31, parts = f.last_cta - (int)blockIdx.x + 1;
  constexpr int E = D / 32;  // channels per lane
  auto part = [&](int i) {
    return a.partial + (((int64_t)blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * a.slot;
  };
  for (int r = threadIdx.x >> 5; r < tile_rows && f.tile0 + r < f.rows; r += 8) {
    float mx = -INFINITY;
    for (int i = lane; i < parts; i += 32) mx = fmaxf(mx, part(i)[tile_rows * D + 2 * r]);
#pragma unroll
    for (int w = 16; w; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
    const float m0 = mx == -INFINITY ? 0.f : mx;
    float sum[E] = {}, den = 0.f;
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
      const float* pt = part(i);
      const float2 v = *reinterpret_cast<const float2*>(pt + tile_rows * D + 2 * r);
      const float w = v.x == -INFINITY && v.y == 0.f ? 0.f : ex2(v.x - m0);
      den = fmaf(w, v.y, den);
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 x = *reinterpret_cast<const float2*>(pt + r * D + 64 * (e / 2) + 2 * lane);
        sum[e] = fmaf(w, x.x, sum[e]);
        sum[e + 1] = fmaf(w, x.y, sum[e + 1]);
      }
    }
    const float inv = den == 0.f ? 0.f : 1.f / den;
    const int64_t at = (int64_t)(f.row0 + (f.tile0 + r) / a.group) * heads * a.group + (int64_t)f.head * a.group + (f.tile0 + r) % a.group;
#pragma unroll
    for (int e = 0; e < E; e += 2)
      *reinterpret_cast<uint32_t*>(a.out + at * D + 64 * (e / 2) + 2 * lane) = f2h(sum[e] * inv, sum[e + 1] * inv);
  }
}

template <typename... P, typename... A>
cudaError_t launch_pdl(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

constexpr int kMaxRows = 16;  // query rows of the widest tile
constexpr int kMaxCtasPerSm = 4;

template <int D, int SUB, int NT>
cudaError_t launch_attention(AttnArgs a, const Kv8Cache& cache, const Kv8Batch& bt, uint32_t* status,
                             cudaStream_t stream) {
  using L = Attn<D, SUB, NT>;
  static std::atomic<uint64_t> attr_set{0};  // one bit per device that has the attribute
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return cudaErrorInvalidDevice;
  if (!(attr_set.load(std::memory_order_acquire) >> dev & 1)) {
    cudaError_t e = cudaFuncSetAttribute(kv8_attention_kernel<D, SUB, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
    if (e != cudaSuccess) return e;
    attr_set.fetch_or(uint64_t(1) << dev, std::memory_order_acq_rel);
  }
  a.slot = L::kSlot;
  const int ctas = L::kCtasPerSm * device_info().sm_count;  // all resident: a persistent grid
  cudaError_t e = launch_pdl(kv8_attention_kernel<D, SUB, NT>, dim3((unsigned)ctas), kThreads, L::kSmem, stream, a, cache, bt, status);
  if (e != cudaSuccess) return e;
  return launch_pdl(kv8_fixup_kernel<D>, dim3((unsigned)ctas), 256, 0, stream, a, cache.heads, L::kRows);
}

}  // namespace

size_t kv8_workspace_bytes(int D, int sm_count) {
  const size_t ctas = (size_t)kMaxCtasPerSm * sm_count;
  return kWsHeaderBytes + ctas * sizeof(Kv8Fix) + ctas * 2 * kMaxRows * (D + 2) * sizeof(float);
}

cudaError_t launch_kv8_append(const __half* k, const __half* v, int64_t k_stride, int64_t v_stride,
                              const Kv8Cache& cache, const Kv8Batch& bt, uint32_t* status, cudaStream_t stream) {
  // blocks that get new tokens: at most one per token, and per sequence one
  // per full block of them and two at the ends
  int64_t items = (int64_t)bt.rows / bt.block_tokens + 2 * (int64_t)bt.seqs;
  if (items > bt.rows) items = bt.rows;
  const dim3 grid((unsigned)items, 2 * cache.heads);
  switch (bt.block_tokens * cache.head_dim / 1024) {
    case 1: return launch_pdl(kv8_append_kernel<1>, grid, kThreads, 0, stream, k, v, k_stride, v_stride, cache, bt, status);
    case 2: return launch_pdl(kv8_append_kernel<2>, grid, kThreads, 0, stream, k, v, k_stride, v_stride, cache, bt, status);
    case 4: return launch_pdl(kv8_append_kernel<4>, grid, kThreads, 0, stream, k, v, k_stride, v_stride, cache, bt, status);
    case 8: return launch_pdl(kv8_append_kernel<8>, grid, kThreads, 0, stream, k, v, k_stride, v_stride, cache, bt, status);
    case 16: return launch_pdl(kv8_append_kernel<16>, grid, kThreads, 0, stream, k, v, k_stride, v_stride, cache, bt, status);
    default: return cudaErrorInvalidConfiguration;
  }
}

cudaError_t launch_kv8_attention(const __half* q, int64_t q_stride, int q_heads, float scale, const Kv8Cache& cache,
                                 const Kv8Batch& bt, __half* out, void* workspace, cudaStream_t stream) {
  const size_t ctas = (size_t)kMaxCtasPerSm * device_info().sm_count;
  char* ws = static_cast<char*>(workspace);
  AttnArgs a = {};
  a.q = q;
  a.q_stride = q_stride;
  a.out = out;
  a.group = q_heads / cache.heads;
  a.scale_log2 = scale * kLog2e;
  a.fix = reinterpret_cast<Kv8Fix*>(ws + kWsHeaderBytes);
  a.partial = reinterpret_cast<float*>(ws + kWsHeaderBytes + ctas * sizeof(Kv8Fix));
  uint32_t* status = reinterpret_cast<uint32_t*>(ws);
  // rows that share a kv head, by the mean of new tokens a sequence (lengths are on the device)
  const int64_t rows = ((int64_t)bt.rows + bt.seqs - 1) / bt.seqs * a.group;
  if (cache.head_dim == 128)
    return rows <= 8 ? launch_attention<128, 1, 1>(a, cache, bt, status, stream)
                     : launch_attention<128, 1, 2>(a, cache, bt, status, stream);
  return rows <= 8 ? launch_attention<64, 2, 1>(a, cache, bt, status, stream)
                   : launch_attention<64, 2, 2>(a, cache, bt, status, stream);
}

}  // namespace awq
