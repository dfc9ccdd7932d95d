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
#include <type_traits>

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
  if (!AWQ_CHECK(in_range(b, 1, bt.seqs), status)) return Seq{0, 0, 0};
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
// sequence b. Every thread of the CTA calls this and counts a run of sequences;
// returned is the sum, and whose run item u lies in is told by the counts alone: by
// one thread's, even if the lists change before they are read again.
struct Counted {
  int64_t before, mine;  // items of the threads before this one, and this one's
  __device__ __forceinline__ bool has(int64_t u) const { return u >= before && u < before + mine; }
};
template <typename Items>
__device__ __forceinline__ int64_t total_items(int B, const Items& items, int64_t* scan /* [kWarps] */, Counted& c) {
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
  c = Counted{inc - mine, mine};
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) c.before += scan[w];
    total += scan[w];
  }
  return total;
}

// Codes of the cache's K (or V), for the debug build's checks.
[[maybe_unused]] __device__ __forceinline__ int64_t code_bytes(const Kv8Cache& cache, const Kv8Batch& bt) {
  return cache.blocks * cache.heads * bt.block_tokens * cache.head_dim;
}
// Entry j of sequence b's block table.
__device__ __forceinline__ int table_block(const Kv8Batch& bt, int b, int j, uint32_t* status) {
  const int64_t at = (int64_t)b * bt.table_width + j;
  return AWQ_CHECK(in_range(at, 1, (int64_t)bt.seqs * bt.table_width), status) ? bt.table[at] : -1;
}

struct Place {
  int b;
  int64_t base;
};

// Sequence of item u < total, and the first of its items; `before` is this
// thread's from total_items, whose caller has set *shared to the first sequence.
// If the lists change while a kernel reads them, several threads or none may find
// it: then b is still a sequence's and base at most u.
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
// The codes of two fp16 values times m.
__device__ __forceinline__ uint32_t code2_h(uint32_t w, __half2 m) {
  const __half2 p = __hmul2(*reinterpret_cast<const __half2*>(&w), m);
  return __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(p), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Largest magnitudes of the low and the high fp16 values, as bits; of all
// finite ones.
__device__ __forceinline__ uint32_t max_mag(const uint4& v) {
  constexpr uint32_t k = 0x7FFF7FFFu;
  return __vmaxu2(__vmaxu2(v.x & k, v.y & k), __vmaxu2(v.z & k, v.w & k));
}
__device__ __forceinline__ uint32_t max_finite_mag(const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t m = 0;
  for (int q = 0; q < 8; ++q) {
    const uint32_t a = w[q / 2] >> 16 * (q & 1) & 0x7FFFu;
    if (a < 0x7C00u) m = max(m, a);
  }
  return m;
}

// Smallest e with |v| <= 448 2^e for the fp16 magnitude bits of a finite v:
// v = 1.m 2^x in fp32, 448 = 1.75 * 2^8. Zero needs the least, -32 (what
// 2^-24, the smallest fp16, needs).
__device__ __forceinline__ int needed_exponent(uint32_t mag) {
  if (mag == 0) return -32;
  const uint32_t f = __float_as_uint(__half2float(__ushort_as_half((unsigned short)mag)));
  return (int)(f >> 23) - 127 - 8 + ((f & 0x7FFFFFu) > 0x600000u);
}

// Exponents as both calls use them, whatever a caller's cache holds: with a spread
// of 63 no weight that counts leaves fp32, and 2^e is a number. (The append's own
// are -32 .. 8.)
__device__ __forceinline__ int usable(int e) { return max(min(e, 31), -32); }

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------

// One CTA per (block that gets new tokens, kv head), for K and V. The block's
// new rows stay in registers between the maximum and the conversion, so they
// are read once, and their loads do not wait for the block number.
// Bound by HBM for prompts (2 bytes read, 1 written an element), by the launch
// and four dependent loads for a few hundred single tokens. Heads are the grid's fastest
// dimension: the CTAs that run together read whole rows of k and v.
//
// Every CTA reads the batch's lists to find its block. With many sequences that is
// most of the work and grows with their square, so there (kMany) as many CTAs as
// about fit at once take equal ranges of blocks, find the first and count on from
// it. Single tokens, 8 kv heads 128 wide, blocks of 64: 4096 sequences 2919 us with
// a CTA a block and 202 so, 2048 399 and 89, 1024 67 and 42 (blocks of 16, 32 heads:
// 204 and 98), 1024 prompts of 64 tokens 135 and 87; but 512 prompts of 128 77 and 84,
// 256 single tokens 12.5 and 13.1. Two and eight CTAs an SM: 4096 sequences 270 and
// 245 us.
constexpr int kManySeqs = 1024;
constexpr int kManyCtasPerSm = 4;

template <int kIter, bool kMany>  // kIter: 16-byte pieces of a block's rows per thread, block_tokens * D / 1024
__global__ void __launch_bounds__(kThreads) kv8_append_kernel(const __half* __restrict__ knew,
                                                              const __half* __restrict__ vnew, int64_t k_stride,
                                                              int64_t v_stride, Kv8Cache cache, Kv8Batch bt,
                                                              uint32_t* status) {
  __shared__ int64_t scan[kWarps];
  __shared__ Place place;
  __shared__ uint32_t wmax[2][kWarps];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int bs = bt.block_tokens, shift = __ffs(bs) - 1, D = cache.head_dim;
  // blocks of sequence b that get new tokens
  auto items = [&](int b) -> int64_t {
    const Seq s = load_seq(bt, b, status);
    const int first = max(s.len - s.tokens, 0);
    return first < s.len && s.tokens > 0 ? ((s.len - 1) >> shift) - (first >> shift) + 1 : 0;
  };
  if (threadIdx.x == 0) place = Place{0, 0};
  Counted counted;
  const int64_t total = total_items(bt.seqs, items, scan, counted);
  const int64_t ctas = (int64_t)gridDim.y * gridDim.z, cta = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
  auto first_item = [&](int64_t c) { return !kMany || total <= ctas ? c : total / ctas * c + total % ctas * c / ctas; };
  const int64_t u0 = first_item(cta), u1 = kMany ? min(first_item(cta + 1), total) : u0 + 1;
  if (u0 >= total) return;
  Place p = find_item(bt.seqs, items, counted.before, u0, &place);
  // Every thread takes the same steps, whatever it reads in the lists.
  for (int64_t u = u0; u < u1; ++u) {
    if (kMany && u > u0) {
      __syncthreads();  // the last item's maxima have been read
      if (__shfl_sync(0xffffffffu, u - p.base >= items(p.b), 0)) {  // the next sequence with items, 32 at a time
        p.base = u;
        for (bool found = false; !found && p.b < bt.seqs - 1;) {
          const int b = p.b + 1 + (int)(threadIdx.x & 31);
          const uint32_t m = __ballot_sync(0xffffffffu, b < bt.seqs && items(b) > 0);
          found = m != 0;
          p.b = min(p.b + (found ? __ffs(m) : 32), bt.seqs - 1);
        }
      }
    }
    const Seq s = load_seq(bt, p.b, status);
    const int past = s.len - s.tokens;  // position of the first new row (rows at negative positions have no place)
    // (a grid of a CTA a block has fewer than 2^22 of them)
    const int nth = kMany ? (int)min(u - p.base, (int64_t)bt.table_width) : (int)(u - p.base);
    const int j = min((max(past, 0) >> shift) + nth, bt.table_width - 1);
    const int h = blockIdx.x;
    const int lo = max(max(past, 0) - j * bs, 0), hi = min(s.len - j * bs, bs);  // new rows of the block
    const int pieces = D / 8, rows_per_pass = kThreads / pieces;
    const int r0 = threadIdx.x / pieces, c = threadIdx.x % pieces;
    const int64_t row0 = (int64_t)s.row0 + (int64_t)j * bs - past;  // source row of the block's token 0

    const int blk = table_block(bt, p.b, j, status);
    uint4 x[2][kIter];
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int r = r0 + i * rows_per_pass;
      const int64_t at = (int64_t)h * D + 8 * c;
      x[0][i] = x[1][i] = make_uint4(0, 0, 0, 0);
      if (r >= lo && r < hi && AWQ_CHECK(in_range(row0 + r, 1, bt.rows), status)) {
        x[0][i] = *reinterpret_cast<const uint4*>(knew + (row0 + r) * k_stride + at);
        x[1][i] = *reinterpret_cast<const uint4*>(vnew + (row0 + r) * v_stride + at);
      }
    }
    const bool there = blk >= 0 && blk < cache.blocks;
    if (!there) {
      if (threadIdx.x == 0) record_status(status, AWQ_ERR_BOUNDS);
      if (!kMany) return;
    }
    const int64_t at = there ? (int64_t)blk * cache.heads + h : 0;
    int8_t* const exps[2] = {cache.k_exp + at, cache.v_exp + at};
    int e_there[2];  // not used before the barrier: its load may take that long
    bool odd[2];  // this thread has an infinity or a NaN
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      e_there[part] = lo > 0 && there ? (int)*exps[part] : -128;
      uint32_t m2 = 0;  // two maxima of fp16 magnitudes
#pragma unroll
      for (int i = 0; i < kIter; ++i) m2 = __vmaxu2(m2, max_mag(x[part][i]));
      uint32_t mag = max(m2 & 0xFFFFu, m2 >> 16);
      odd[part] = mag >= 0x7C00u;
      if (odd[part]) {  // infinities and NaN become NaN codes and set no scale: once more, without them
        mag = 0;
        for (int i = 0; i < kIter; ++i) mag = max(mag, max_finite_mag(x[part][i]));
      }
      mag = __reduce_max_sync(0xffffffffu, mag);
      if ((threadIdx.x & 31) == 0) wmax[part][threadIdx.x >> 5] = mag;
    }
    __syncthreads();  // the maxima are there, and every thread has read the old exponents
    if (!there) continue;
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      uint32_t mag = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mag = max(mag, wmax[part][w]);
      const int e_old = lo > 0 ? usable(e_there[part]) : -128;
      const int e = max(needed_exponent(mag), e_old);
      if (threadIdx.x == 0) *exps[part] = (int8_t)e;
      const int64_t dst_at = at * bs * D + 8 * c;
      uint8_t* dst = (part ? cache.v : cache.k) + dst_at;
      const float inv = ldexpf(1.f, -e);
      if (!odd[part] && e >= -15 && e <= 14) {
        // 2^-e is an fp16 number, and a product that fp16 does not hold exactly
        // lies below 2^-14, where every code is zero
        const __half2 inv2 = __float2half2_rn(inv);
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
          const int r = r0 + i * rows_per_pass;
          const uint4& v = x[part][i];
          if (r >= lo && r < hi && AWQ_CHECK(in_range(dst_at + r * D, 8, code_bytes(cache, bt)), status))
            *reinterpret_cast<uint2*>(dst + r * D) = make_uint2(code2_h(v.x, inv2) | (code2_h(v.y, inv2) << 16),
                                                                code2_h(v.z, inv2) | (code2_h(v.w, inv2) << 16));
        }
      } else {
#pragma unroll 1
        for (int r = r0; r < hi; r += rows_per_pass) {
          if (r < lo || !AWQ_CHECK(in_range(row0 + r, 1, bt.rows) &&
                                       in_range(dst_at + r * D, 8, code_bytes(cache, bt)), status))
            continue;
          const __half* s = (part ? vnew + (row0 + r) * v_stride : knew + (row0 + r) * k_stride) + (int64_t)h * D + 8 * c;
          const uint4 v = *reinterpret_cast<const uint4*>(s);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          uint32_t o[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float2 f = h2f(w[q]);
            f.x *= inv, f.y *= inv;                 // exact
            if (!(fabsf(f.x) < INFINITY)) f.x = NAN;  // the conversion would saturate an infinity
            if (!(fabsf(f.y) < INFINITY)) f.y = NAN;
            o[q] = code2(f.x, f.y);
          }
          *reinterpret_cast<uint2*>(dst + r * D) = make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
        }
      }
      if (e > e_old && lo > 0) {  // the codes that were there, under the larger exponent
        const float down = ldexpf(1.f, e_old - e);
        for (int r = r0; r < lo; r += rows_per_pass) {
          if (!AWQ_CHECK(in_range(dst_at + r * D, 8, code_bytes(cache, bt)), status)) continue;
          uint2* old = reinterpret_cast<uint2*>(dst + r * D);
          const uint2 v = *old;
          const float2 a = h2f(lo_h2(v.x)), b = h2f(hi_h2(v.x)), d = h2f(lo_h2(v.y)), f = h2f(hi_h2(v.y));
          *old = make_uint2(code2(a.x * down, a.y * down) | (code2(b.x * down, b.y * down) << 16),
                            code2(d.x * down, d.y * down) | (code2(f.x * down, f.y * down) << 16));
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// attention
// ---------------------------------------------------------------------------

// mma.sync m16n8k16, in two forms. Up to 8 query rows (query heads that share a kv
// head, times new tokens): S^T = K q^T and O^T = V^T P^T, the keys (of S) and the
// head's channels (of O) are the instruction's 16 rows, the query rows its 8
// columns, so few rows waste half as much; the weights are transposed on the way.
// More rows (kWide): S = q K^T and O = P V, 16 query rows are its rows, and the
// weights come out of S as the next operand (drafts of 1 to 5 tokens, 64 wide 25.1
// us against 26.1 as two column tiles of 8). Codes become exact fp16 in registers;
// the products are exact, the sums fp32.
//
// Bound by HBM: every code is read once, 4 flops a code and row. Each warp has
// a ring of its own in shared memory that its lanes fill with 16-byte copies, 512
// contiguous bytes an instruction; warps never wait for one another within a
// segment, and the next segment's first copies start before a segment's parts
// are merged. (Tiled copies by one lane took it 190 cycles a box, a quarter of a
// step: 1 x 131002 tokens 53.1 against 51.9 us, 48 x 64 wide 43.2 against 41.4.)
// The 16-byte pieces are swizzled by token, so that ldmatrix, which takes one
// piece of 8 tokens at a time, has no bank conflicts. As 16-bit elements those
// pieces are pairs of codes: for K, lane (g, t) gets channels 4t .. 4t + 3 of
// token g, the fragment of one k-step (the k order is free as long as q
// follows it); for V, transposed, it gets channels 2g and 2g + 1 of tokens 2t
// and 2t + 1, and one byte permutation makes them fragments.
//
// Softmax in one pass, in powers of two. With x = scale log2(e) q.k and the V
// exponent e of a key's block, the weight kept for a key is p = 2^(x + e - M):
// V's codes then need no scaling, and l = sum p 2^-e is the denominator in the
// same unit. Any M serves that keeps p within fp16. It follows the running
// maximum of x + e, less kPOffset, but only when some exponent has grown past
// kPMost: then p stays at most 2^15 (fp16 ends at 65504), the reduction over
// lanes and the rescaling of O are skipped in most steps, and fp16's
// subnormals begin 2^-26 below the largest weight. p is rounded to fp16 (2^-11
// relative) for the second MMA; l sums the unrounded p.
constexpr float kPOffset = 12.f, kPMost = 15.f;
// A group costs about as much as this many units more: its q, its first copies'
// latency, the merge of the warps' parts. CTAs get equal ranges of units with
// these counted (48 ragged sequences: 78.5 us without, 72.2 with two; with 64-wide
// heads 51.4 and 40.0; three change them by less than 1 %).
constexpr int kGroupCost = 2;
// Where the block table holds no more keys than this, and the groups are not
// many times the CTAs, a CTA takes whole groups and there is no fixup kernel, so a
// launch less. In a graph, 8 kv heads, all of 128 / 256 / 512 tokens: one sequence 5.4 /
// 6.2 / 7.3 us against 7.1 / 7.6 / 7.8 split, 32 sequences 6.7 / 7.9 / 10.5 against 8.2 /
// 10.6 / 13.1 (but four of 512: 9.2 against 8.6, and one of 1024 11.8 against 8.0; 256
// sequences of 20 to 400: 37.5 against 34.9); a call from Python 10.8 us against 13.1.
constexpr int kWholeKeys = 512;
constexpr float kNoM = -1e30f;  // M of a row that has seen no key: finite, far below any x (|x| < 2^96 by the limit of scale)

// The group of units that starts in a CTA's range and ends in a later one's.
struct Kv8Fix {
  int valid, row0, rows, tile0, head, last_cta, past, pad;
};

struct AttnArgs {
  const __half* q;
  int64_t q_stride;
  __half* out;
  int group;          // query heads per kv head
  float scale_log2;   // softmax scale times log2 e
  float* partial;     // [ctas][2][slot], partial_floats in all
  int64_t partial_floats;
  int slot;           // floats of a slot: rows * (D + 2)
  Kv8Fix* fix;        // [ctas]
  bool whole;         // groups are not split between CTAs
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// 16 bytes from global to shared memory; zeros for bytes = 0.
__device__ __forceinline__ void copy16(uint32_t to, const uint8_t* from, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
// Four 8 x 16-byte pieces: lane i gives the address of token i % 8 of piece i / 8.
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}

// A step of a warp is two 16-key subtiles; a unit of work, the same step of the
// four warps, is 128 keys of one group (sequence, kv head, row tile).
constexpr int kSub = 2;
constexpr int kStepKeys = 16 * kSub;
constexpr int kUnitKeys = kWarps * kStepKeys;

// D: head dimension; NT: query rows of a tile, in eights (1 or 2); ST: steps in a warp's ring.
template <int D, int NT, int ST>
struct Attn {
  static constexpr int kRows = 8 * NT;
  static constexpr int kStages = ST;
  static constexpr int kPartBytes = kStepKeys * D;            // a warp's step of K, or of V
  static constexpr int kStageBytes = 2 * kPartBytes;
  static_assert(kStageBytes >= kRows * D * 4, "a warp's part of the output fits a stage");
  static constexpr int kSmem = kWarps * kStages * kStageBytes + 128;  // room to align
  static constexpr int kSlot = kRows * (D + 2);
  static constexpr int kCtasPerSm = kStages * kStageBytes <= 16384 ? 3 : 2;  // by shared memory and registers
};

// The part of a group in a CTA's range.
struct Segment {
  int b, row0, len, past, rows, r0, head, tile0, n;
  int seen;     // keys that some row sees
  bool starts, ends;
  int left;     // units of the group behind it
};

// Where a CTA is in its range.
struct Walk {
  int64_t todo;  // units left
  Seq s;
  int b, head, tile, tiles;  // the sequence, and the group in it: kv head, row tile of `tiles`
  int v0, per;   // the next unit of the group, its units
};

template <int D, int NT, int ST>
__global__ void __launch_bounds__(kThreads, Attn<D, NT, ST>::kCtasPerSm)
    kv8_attention_kernel(const AttnArgs a, const Kv8Cache cache, const Kv8Batch bt, uint32_t* status) {
  using L = Attn<D, NT, ST>;
  constexpr int KS = D / 16;     // k-steps of S
  constexpr int MT = D / 16;     // channel tiles of O
  constexpr bool kWide = NT == 2;
  extern __shared__ char smem_raw[];
  char* const smem = smem_raw + (-ptx::smem_u32(smem_raw) & 127u);  // the pieces' places are computed by XOR
  __shared__ int64_t scan[kWarps];
  __shared__ Walk walk;
  __shared__ float2 ml[kWarps][L::kRows];  // M and l of the warps' rows
  __shared__ const float* parts[kWarps];
  __shared__ Segment ahead[3];
  __shared__ int ahead_valid[3];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int bs = bt.block_tokens, shift = __ffs(bs) - 1;
  // (debug build) whether bytes of shared memory lie in the ring
  [[maybe_unused]] auto in_ring = [&](uint32_t at, int bytes) {
    return AWQ_CHECK(in_range((int64_t)at - ptx::smem_u32(smem), bytes, L::kSmem - 128), status);
  };
  auto row_tiles = [&](const Seq& s) { return (int)(((int64_t)s.tokens * a.group + L::kRows - 1) / L::kRows); };
  // a sequence with no keys still has one (empty) unit per row tile: its rows are zero
  auto key_tiles = [&](const Seq& s) { return max((s.len + kUnitKeys - 1) / kUnitKeys, 1); };
  // what a group of the sequence counts in the split
  auto group_units = [&](const Seq& s) { return a.whole ? 1 : key_tiles(s) + kGroupCost; };
  auto items = [&](int b) -> int64_t {
    const Seq s = load_seq(bt, b, status);
    return (int64_t)row_tiles(s) * group_units(s) * cache.heads;
  };
  if (tid == 0) walk.todo = ahead_valid[0] = 0;
  Counted counted;
  const int64_t total = total_items(bt.seqs, items, scan, counted);
  const int64_t ctas = total < (int64_t)gridDim.x ? total : (int64_t)gridDim.x;
  if (tid == 0) a.fix[blockIdx.x].valid = 0;
  if ((int64_t)blockIdx.x >= ctas) return;
  // a 64-bit division takes as long as a step
  const bool small = total * gridDim.x <= 0x7FFFFFFF;
  auto divide = [&](int64_t x, int64_t y) -> int64_t { return small ? (int64_t)((uint32_t)x / (uint32_t)y) : x / y; };
  auto first_unit = [&](int64_t c) {
    return small ? divide(total * c, ctas) : total / ctas * c + total % ctas * c / ctas;
  };
  const int64_t u = first_unit(blockIdx.x), u1 = first_unit((int64_t)blockIdx.x + 1);

  const uint32_t ring = ptx::smem_u32(smem) + warp * (L::kStages * L::kStageBytes);
  // The lane's row and piece of an ldmatrix: tokens (lane & 15), the first of
  // two neighbouring pieces for lanes below 16; pieces are swizzled by token.
  const uint32_t lrow = lane & 15, swz = D == 128 ? (lane & 7) : (lane >> 1 & 3);
  const uint32_t lane_off = lrow * D + (((lane >> 4) ^ swz) << 4);
  int stage = 0, fill = 0;   // ring positions of the next step to use and to fill
  // The lane's piece of 512 contiguous bytes of codes (512 / D tokens), and its
  // place: pieces are swizzled by token.
  const uint32_t put_row = lane / (D / 16), put_swz = D == 128 ? put_row : (put_row >> 1 & 3);
  const uint32_t put = put_row * D + ((lane % (D / 16) ^ put_swz) << 4);

  // ---- segments: the parts of groups in this CTA's range. One thread walks the
  // batch two segments ahead and hands them out, so that all warps take the same
  // steps even if the lists change under them.
  Segment sg;
  auto hand_out = [&](int slot) {
    Walk w = walk;
    bool found = false;
    while (w.todo > 0) {
      if (w.v0 == w.per) {  // the next group
        w.v0 = 0;
        if (++w.tile >= w.tiles) {
          w.tile = 0;
          if (++w.head >= cache.heads) {
            w.head = 0;
            w.tiles = 0;
            while (w.tiles == 0 && ++w.b < bt.seqs) {
              w.s = load_seq(bt, w.b, status);
              w.tiles = row_tiles(w.s);
            }
            if (w.tiles == 0) break;
            w.per = group_units(w.s);
          }
        }
      }
      const int take = (int)(w.todo < w.per - w.v0 ? w.todo : w.per - w.v0);
      Segment s;
      s.tile0 = max(w.v0 - kGroupCost, 0);
      s.n = a.whole ? key_tiles(w.s) : w.v0 + take - kGroupCost - s.tile0;
      w.v0 += take;
      w.todo -= take;
      if (s.n <= 0) continue;  // only of the units that stand for the group's fixed cost
      s.head = w.head;
      s.r0 = w.tile * L::kRows;
      s.b = w.b;
      s.row0 = w.s.row0;
      s.len = w.s.len;
      s.past = w.s.len - w.s.tokens;
      s.rows = w.s.tokens * a.group;
      s.seen = max(min(s.past + (min(s.r0 + L::kRows, s.rows) - 1) / a.group + 1, s.len), 0);
      s.starts = s.tile0 == 0;
      s.ends = w.v0 == w.per;
      s.left = w.per - w.v0;
      ahead[slot] = s;
      found = true;
      break;
    }
    walk = w;
    ahead_valid[slot] = found;
  };
  if (counted.has(u)) {  // the thread that counted the sequence of the first unit begins
    const int per = (bt.seqs + kThreads - 1) / kThreads;
    int64_t at = counted.before;
    for (int b = tid * per; b < min(bt.seqs, (tid + 1) * per); ++b) {
      const Seq s = load_seq(bt, b, status);
      const int tiles = row_tiles(s), units = group_units(s);
      const int64_t n = (int64_t)tiles * units * cache.heads;
      if (u < at + n) {
        const int64_t group_no = divide(u - at, units);
        Walk w;
        w.todo = u1 - u;
        w.s = s;
        w.b = b;
        w.head = (int)divide(group_no, tiles);
        w.tile = (int)(group_no - (int64_t)w.head * tiles);
        w.tiles = tiles;
        w.v0 = (int)(u - at - group_no * units);
        w.per = units;
        walk = w;
        hand_out(0);
        break;
      }
      at += n;
    }
  }

  // ---- a segment's query rows as fragments, channels in K's order
  uint32_t qf[NT][KS][2];
  auto load_q = [&]() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = sg.r0 + 8 * nt + g;
      const __half* q = a.q + (int64_t)(sg.row0 + r / a.group) * a.q_stride + ((int64_t)sg.head * a.group + r % a.group) * D + 4 * t;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint2 v = make_uint2(0, 0);
        if (r < sg.rows &&
            AWQ_CHECK(in_range(sg.row0 + r / a.group, 1, bt.rows) && in_range(sg.head, 1, cache.heads), status))
          v = *reinterpret_cast<const uint2*>(q + 16 * ks);
        qf[nt][ks][0] = v.x;
        qf[nt][ks][1] = v.y;
      }
    }
  };

  // ---- the warp's steps of a segment
  int key00, steps;  // first key, steps with keys that some row sees
  auto begin_steps = [&]() {
    key00 = sg.tile0 * kUnitKeys + warp * kStepKeys;
    steps = sg.seen > key00 ? min((sg.seen - key00 + kUnitKeys - 1) / kUnitKeys, sg.n) : 0;
  };
  // Which of the lane's two rows element c of an S or O fragment belongs to, their
  // numbers in the tile, the lanes of a row, and the key of an S element in a subtile.
  auto row_of = [](int c) { return kWide ? c >> 1 : c & 1; };
  auto lane_row = [&](int c) { return kWide ? g + 8 * c : 2 * t + c; };
  auto key_of = [&](int nt, int c) { return kWide ? 8 * nt + 2 * t + (c & 1) : g + 8 * (c >> 1); };
  constexpr int kRowLane = kWide ? 1 : 4, kRowLanes = kWide ? 4 : 8;

  // Blocks and exponents of the next 32 subtiles, one per lane.
  int blk = -1;
  int k_exp = 0, v_exp = 0, k_exp_prev = 0, v_exp_prev = 0;
  auto load_info = [&](int sub0) {
    const int sub = sub0 + lane, key = key00 + sub / kSub * kUnitKeys + (sub % kSub) * 16;
    k_exp_prev = k_exp;
    v_exp_prev = v_exp;
    blk = -1;
    k_exp = v_exp = 0;
    if (sub < steps * kSub && key < sg.seen) {
      blk = table_block(bt, sg.b, key >> shift, status);
      if (blk < 0 || blk >= cache.blocks) {
        record_status(status, AWQ_ERR_BOUNDS);
        blk = -1;
      } else {
        const int64_t at = (int64_t)blk * cache.heads + sg.head;
        k_exp = cache.k_exp[at];  // used no sooner than the step's copies have landed
        v_exp = cache.v_exp[at];
      }
    }
  };
  // A step's K and V: 512 contiguous bytes an instruction, 16 tokens of a block
  // after the other. A block that is not there, or that no row sees, is zeros.
  // One group of copies per call, so that a step is the oldest of kStages.
  auto issue = [&](int step) {
    if (step < steps) {
      if ((step * kSub) % 32 == 0) load_info(step * kSub);
      const uint32_t dst = ring + fill * L::kStageBytes + put;
      fill = fill == L::kStages - 1 ? 0 : fill + 1;
      const int key = key00 + step * kUnitKeys;
      __syncwarp();  // every lane has read what the stage held
#pragma unroll
      for (int sb = 0; sb < kSub; ++sb) {
        const int id = __shfl_sync(0xffffffffu, blk, step * kSub + sb);
        const uint32_t bytes = id < 0 ? 0 : 16;
        const int64_t at = ((int64_t)(max(id, 0) * cache.heads + sg.head) * bs + ((key + 16 * sb) & (bs - 1))) * D + 16 * lane;
#pragma unroll
        for (int i = 0; i < 16 * D / 512; ++i) {
          const uint32_t to = (dst + sb * (16 * D) + i * 512) ^ (D == 128 ? (i & 1) << 6 : 0);
          if (!AWQ_CHECK(in_range(at + i * 512, 16, code_bytes(cache, bt)), status) || !in_ring(to, 16) ||
              !in_ring(to + L::kPartBytes, 16))
            continue;
          copy16(to, cache.k + at + i * 512, bytes);
          copy16(to + L::kPartBytes, cache.v + at + i * 512, bytes);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto begin_segment = [&]() {  // its first steps and its q on their way
    begin_steps();
#pragma unroll 1
    for (int i = 0; i < L::kStages - 1; ++i) issue(i);
    load_q();
  };

  __syncthreads();
  bool have = ahead_valid[0];
  sg = ahead[0];
  if (have) begin_segment();
  if (tid == 0) hand_out(1), hand_out(2);
  __syncwarp();
  bool first = true;
  for (int turn = 0, next = 1; have; turn = next, next = next == 2 ? 0 : next + 1) {
    int limit[2];  // keys that the lane's two rows see
#pragma unroll
    for (int c = 0; c < 2; ++c) limit[c] = min(sg.past + (sg.r0 + lane_row(c)) / a.group + 1, sg.len);
    const int least = sg.past + sg.r0 / a.group + 1;  // keys that every row sees

    float o[MT][NT][4], M[2], l[2];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.f;
    M[0] = M[1] = steps > 0 ? 0.f : kNoM;  // 0 until the first step sets it
    l[0] = l[1] = 0.f;

    for (int step = 0; step < steps; ++step) {
      issue(step + L::kStages - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(L::kStages - 1) : "memory");
      __syncwarp();  // the other lanes' copies are there too
      const uint32_t src = ring + stage * L::kStageBytes + lane_off;
      stage = stage == L::kStages - 1 ? 0 : stage + 1;
      const int key0 = key00 + step * kUnitKeys;
      // the issuing side is up to kStages - 1 steps ahead: it may have loaded the next 32 already
      const bool same = (step * kSub) / 32 == min(step + L::kStages - 1, steps - 1) * kSub / 32;
      const float k_of = a.scale_log2 * __int_as_float((usable(same ? k_exp : k_exp_prev) + 127) << 23);
      const float v_of = (float)usable(same ? v_exp : v_exp_prev);

      // The weights' exponents x + e_v - M of the step's keys (masked keys: -inf)
      float x[kSub][NT][4], unit[kSub];  // unit: 2^-e_v
#pragma unroll
      for (int sb = 0; sb < kSub; ++sb)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) x[sb][nt][0] = x[sb][nt][1] = x[sb][nt][2] = x[sb][nt][3] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ks += 2)
#pragma unroll
        for (int sb = 0; sb < kSub; ++sb) {
          uint32_t w[4];  // tokens g and g + 8 of piece ks, then of ks + 1
          const uint32_t from = (src + sb * (16 * D)) ^ (ks << 4);
          ldsm4(in_ring(from, 16) ? from : ring, w);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t k0 = lo_h2(w[2 * i]), k1 = lo_h2(w[2 * i + 1]), k2 = hi_h2(w[2 * i]), k3 = hi_h2(w[2 * i + 1]);
            if constexpr (kWide) {
              const uint32_t(&q0)[2] = qf[0][ks + i], (&q1)[2] = qf[NT - 1][ks + i];
              mma16816(x[sb][0], q0[0], q1[0], q0[1], q1[1], k0, k2);
              mma16816(x[sb][NT - 1], q0[0], q1[0], q0[1], q1[1], k1, k3);
            } else {
              mma16816(x[sb][0], k0, k1, k2, k3, qf[0][ks + i][0], qf[0][ks + i][1]);
            }
          }
        }
#pragma unroll
      for (int sb = 0; sb < kSub; ++sb) {
        const float k_unit = __shfl_sync(0xffffffffu, k_of, step * kSub + sb);
        const float ev = __shfl_sync(0xffffffffu, v_of, step * kSub + sb);
        unit[sb] = ex2(-ev);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) x[sb][nt][c] = fmaf(x[sb][nt][c], k_unit, ev - M[row_of(c)]);
      }
      if (key0 + kStepKeys > least) {  // some row does not see all of the step's keys
#pragma unroll
        for (int sb = 0; sb < kSub; ++sb)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (key0 + 16 * sb + key_of(nt, c) >= limit[row_of(c)]) x[sb][nt][c] = -INFINITY;
      }

      // Where one exceeds kPMost, and in a segment's first step, every row's M
      // follows its running maximum.
      float over = -INFINITY;
#pragma unroll
      for (int sb = 0; sb < kSub; ++sb)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) over = fmaxf(over, x[sb][nt][c]);
      if (__any_sync(0xffffffffu, over > kPMost) || step == 0) {
        float up[2] = {kNoM, kNoM};  // by how much M moves
#pragma unroll
        for (int sb = 0; sb < kSub; ++sb)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) up[row_of(c)] = fmaxf(up[row_of(c)], x[sb][nt][c]);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
          for (int w = kRowLane; w < kRowLane * kRowLanes; w <<= 1) up[r] = fmaxf(up[r], __shfl_xor_sync(0xffffffffu, up[r], w));
          up[r] = step == 0 ? up[r] - kPOffset : fmaxf(up[r] - kPOffset, 0.f);
          M[r] += up[r];
        }
#pragma unroll
        for (int sb = 0; sb < kSub; ++sb)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) x[sb][nt][c] -= up[row_of(c)];
        if (step > 0) {  // in the first step there is nothing to rescale
          const float f[2] = {ex2(-up[0]), ex2(-up[1])};
          l[0] *= f[0], l[1] *= f[1];
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 4; ++c) o[i][nt][c] *= f[row_of(c)];
        }
      }

      uint32_t pf[kSub][2 * NT];
#pragma unroll
      for (int sb = 0; sb < kSub; ++sb) {
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float pr[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) pr[c] = ex2(x[sb][nt][c]);
#pragma unroll
          for (int c = 0; c < 4; ++c) sum[row_of(c)] += pr[c];
          pf[sb][2 * nt] = f2h(pr[0], pr[1]);
          pf[sb][2 * nt + 1] = f2h(pr[2], pr[3]);
          if (!kWide) pf[sb][0] = transpose8x8(pf[sb][0]), pf[sb][1] = transpose8x8(pf[sb][1]);
        }
        l[0] = fmaf(sum[0], unit[sb], l[0]);
        l[1] = fmaf(sum[1], unit[sb], l[1]);
      }
      // O += P V. Where a row does not see all 16 keys of a subtile, a NaN
      // code must reach only the rows that see it: 0 * NaN in the MMA would
      // reach all. Such codes are taken out there, and their channels of the
      // rows that see them set to NaN. (Places behind the end can hold NaN codes
      // too.) The other steps have no branch between their loads.
      auto add_pv = [&](auto careful) {
#pragma unroll
        for (int sb = 0; sb < kSub; ++sb) {
          const int key = key0 + 16 * sb;
#pragma unroll
          for (int i = 0; i < MT; i += 2) {
            uint32_t w[4];  // channels 2g, 2g + 1 of piece i: tokens 2t, 2t + 1, then + 8; the same of piece i + 1
            const uint32_t from = (src + L::kPartBytes + sb * (16 * D)) ^ (i << 4);
            ldsm4_trans(in_ring(from, 16) ? from : ring, w);
            if constexpr (decltype(careful)::value) {
              uint32_t nan[4], any = 0;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                nan[j] = ((w[j] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;  // 0x80 in bytes that are 0x7F or 0xFF
                any |= nan[j];
              }
              if (__any_sync(0xffffffffu, any)) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  w[j] &= ~((nan[j] >> 7) * 0xFFu);
#pragma unroll 1
                  for (int s = 0; s < 4 * NT; ++s) {  // the lanes that share this lane's channels
                    const int gg = kWide ? 2 * t + (s >> 2) : g, tt = s & 3;
                    const uint32_t m = __shfl_sync(0xffffffffu, nan[j], 4 * gg + tt);
                    if (m == 0) continue;
#pragma unroll
                    for (int b = 0; b < 4; ++b)  // byte b: token + (b >> 1), channel + (b & 1)
#pragma unroll
                      for (int r = 0; r < 2; ++r)
                        if ((m >> (8 * b + 7) & 1) && key + 2 * tt + 8 * (j & 1) + (b >> 1) < limit[r]) {
                          float(&to)[NT][4] = o[i + (j >> 1)];
                          if (!kWide) to[0][2 * (b & 1) + r] = NAN;
                          else if (s < 4) to[(b & 1) % NT][2 * r] = NAN;
                          else to[(b & 1) % NT][2 * r + 1] = NAN;
                        }
                  }
                }
              }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t p0 = __byte_perm(w[2 * j], 0, 0x3120), p1 = __byte_perm(w[2 * j + 1], 0, 0x3120);
              const uint32_t v0 = lo_h2(p0), v1 = hi_h2(p0), v2 = lo_h2(p1), v3 = hi_h2(p1);
              if constexpr (kWide) {  // channels of even number, then of odd
                const uint32_t(&p)[2 * NT] = pf[sb];
                mma16816(o[i + j][0], p[0], p[1], p[2 * NT - 2], p[2 * NT - 1], v0, v2);
                mma16816(o[i + j][NT - 1], p[0], p[1], p[2 * NT - 2], p[2 * NT - 1], v1, v3);
              } else {
                mma16816(o[i + j][0], v0, v1, v2, v3, pf[sb][0], pf[sb][1]);
              }
            }
          }
        }
      };
      if (key0 + kStepKeys > least)
        add_pv(std::true_type());
      else
        add_pv(std::false_type());
    }

    // ---- the next segment's copies start before this one's parts are merged
    const Segment& w = ahead[turn];
    if (first) __syncthreads();  // the second segment is there (later ones: the last merge's barrier)
    first = false;
    have = ahead_valid[next];
    sg = ahead[next];
    if (have) begin_segment();
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int x = kRowLane; x < kRowLane * kRowLanes; x <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], x);
    // Each warp leaves its part in the stage of its ring that is still free.
    // Columns are swapped by 16 in every second row (wide), or pair of rows: fewer
    // conflicts.
    float* const mine = reinterpret_cast<float*>(smem + (ring - ptx::smem_u32(smem)) + fill * L::kStageBytes);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int r = lane_row(c);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int col = kWide ? (16 * i + 4 * t) ^ ((r & 1) << 4) : (16 * i + 2 * g) ^ ((t & 1) << 4);
        if (!in_ring(ptx::smem_u32(mine + r * D + col), kWide ? 16 : 8)) continue;
        if constexpr (kWide)
          *reinterpret_cast<float4*>(mine + r * D + col) =
              make_float4(o[i][0][2 * c], o[i][NT - 1][2 * c], o[i][0][2 * c + 1], o[i][NT - 1][2 * c + 1]);
        else
          *reinterpret_cast<float2*>(mine + r * D + col) = make_float2(o[i][0][c], o[i][0][c + 2]);
      }
      if ((kWide ? t : g) == 0) ml[warp][r] = make_float2(M[c], l[c]);
    }
    if (lane == 0) parts[warp] = mine;
    __syncthreads();
    float* slot = a.partial + ((int64_t)blockIdx.x * 2 + (w.starts ? 1 : 0)) * a.slot;
    for (int i = tid; i < L::kRows * (D / 4); i += kThreads) {
      const int r = i / (D / 4), d = i % (D / 4) * 4;
      if (w.r0 + r >= w.rows) continue;
      float mx = kNoM;
#pragma unroll
      for (int j = 0; j < kWarps; ++j) mx = fmaxf(mx, ml[j][r].x);
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
      float den = 0.f;
#pragma unroll
      for (int j = 0; j < kWarps; ++j) {
        const float2 v = ml[j][r];
        const float f = ex2(v.x - mx);
        const float* part = parts[j] + r * D + (d ^ ((kWide ? r & 1 : r >> 1 & 1) << 4));
        if (!in_ring(ptx::smem_u32(part), 16)) continue;
        const float4 ow = *reinterpret_cast<const float4*>(part);
        sum.x = fmaf(f, ow.x, sum.x), sum.y = fmaf(f, ow.y, sum.y);
        sum.z = fmaf(f, ow.z, sum.z), sum.w = fmaf(f, ow.w, sum.w);
        den = fmaf(f, v.y, den);
      }
      if (w.starts && w.ends) {
        const int token = (w.r0 + r) / a.group;
        // a row that sees no key is zero; one whose scores are all -infinity is 0 / 0
        const float inv = min(w.past + token + 1, w.len) > 0 ? 1.f / den : 0.f;
        const int64_t at = (int64_t)(w.row0 + token) * cache.heads * a.group + (int64_t)w.head * a.group + (w.r0 + r) % a.group;
        if (AWQ_CHECK(in_range(at, 1, (int64_t)bt.rows * cache.heads * a.group), status))
          *reinterpret_cast<uint2*>(a.out + at * D + d) = make_uint2(f2h(sum.x * inv, sum.y * inv), f2h(sum.z * inv, sum.w * inv));
      } else if (AWQ_CHECK(in_range(slot - a.partial, a.slot, a.partial_floats) &&
                               in_range(r * D + d, 4, L::kRows * D), status)) {
        *reinterpret_cast<float4*>(slot + r * D + d) = sum;
        if (d == 0) *reinterpret_cast<float2*>(slot + L::kRows * D + 2 * r) = make_float2(mx, den);
      }
    }
    if (w.starts && !w.ends && tid == 0)  // the CTA that holds the group's last unit: the last c with first_unit(c) < its end
      a.fix[blockIdx.x] = Kv8Fix{1, w.row0, w.rows, w.r0, w.head, (int)min(((u1 + w.left) * ctas + total - 1) / total, ctas) - 1, w.past, 0};
    __syncthreads();  // copies will come where the parts were
    if (tid == 0) hand_out(turn);
    __syncwarp();
  }
}

// Adds the parts of the groups that more than one CTA worked on, in a fixed
// order (so the result does not depend on timing). CTA (c, .) has the group
// that starts in CTA c of the attention kernel: one part in that CTA's slot 1,
// the others in the following CTAs' slots 0. Few groups have many parts each
// (long sequences): kSplit gives a CTA one row, its warps every fourth part.
// Many groups have few parts: then a warp takes a row. It does not let the next
// kernel start early: CTAs of a following attention kernel that take the places
// of the first fixup CTAs to end are spread unevenly over the SMs (48 ragged
// sequences with four CTAs per SM: 101 against 76 us).
template <int D, bool kSplit>
__global__ void __launch_bounds__(kThreads) kv8_fixup_kernel(const AttnArgs a, int heads, int rows, int tile_rows,
                                                             uint32_t* status) {
  __shared__ float2 wml[kWarps];
  __shared__ float wsum[kWarps][D];
  ptx::griddep_wait();
  const Kv8Fix f = a.fix[blockIdx.x];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = kSplit ? (int)blockIdx.y : (int)blockIdx.y * kWarps + warp;
  if (!f.valid || f.tile0 + r >= f.rows) return;
  const int parts = f.last_cta - (int)blockIdx.x + 1;
  if (!AWQ_CHECK(in_range(2 * (int64_t)blockIdx.x * a.slot, (2 * (int64_t)parts - 1) * a.slot, a.partial_floats) &&
                     in_range(tile_rows * D + 2 * r, 2, a.slot) && in_range(f.head, 1, heads) &&
                     in_range((f.tile0 + r) / a.group + (int64_t)f.row0, 1, rows), status))
    return;
  constexpr int E = D / 32;  // channels per lane
  auto part = [&](int i) { return a.partial + (((int64_t)blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * a.slot; };
  const int first = kSplit ? warp : 0, by = kSplit ? kWarps : 1;
  float mx = kNoM;
  for (int i = first + by * lane; i < parts; i += 32 * by) mx = fmaxf(mx, part(i)[tile_rows * D + 2 * r]);
#pragma unroll
  for (int w = 16; w; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
  float sum[E] = {}, den = 0.f;
#pragma unroll 8
  for (int i = first; i < parts; i += by) {
    const float* pt = part(i);
    const float2 v = *reinterpret_cast<const float2*>(pt + tile_rows * D + 2 * r);
    const float w = ex2(v.x - mx);
    den = fmaf(w, v.y, den);
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float2 x = *reinterpret_cast<const float2*>(pt + r * D + 32 * e + 2 * lane);
      sum[e] = fmaf(w, x.x, sum[e]);
      sum[e + 1] = fmaf(w, x.y, sum[e + 1]);
    }
  }
  if (kSplit) {
    if (lane == 0) wml[warp] = make_float2(mx, den);
#pragma unroll
    for (int e = 0; e < E; e += 2) *reinterpret_cast<float2*>(&wsum[warp][32 * e + 2 * lane]) = make_float2(sum[e], sum[e + 1]);
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, wml[w].x);
    den = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) sum[e] = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float k = ex2(wml[w].x - mx);
      den = fmaf(k, wml[w].y, den);
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        sum[e] = fmaf(k, wsum[w][32 * e + 2 * lane], sum[e]);
        sum[e + 1] = fmaf(k, wsum[w][32 * e + 2 * lane + 1], sum[e + 1]);
      }
    }
  }
  const int token = (f.tile0 + r) / a.group;
  const float inv = f.past + token + 1 > 0 ? 1.f / den : 0.f;  // as in the attention kernel (such groups have keys)
  const int64_t at = (int64_t)(f.row0 + token) * heads * a.group + (int64_t)f.head * a.group + (f.tile0 + r) % a.group;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t*>(a.out + at * D + 32 * e + 2 * lane) = f2h(sum[e] * inv, sum[e + 1] * inv);
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
constexpr int kMaxCtasPerSm = 3;

template <int D, int NT, int ST>
cudaError_t launch_attention(AttnArgs a, const Kv8Cache& cache, const Kv8Batch& bt, uint32_t* status,
                             cudaStream_t stream) {
  using L = Attn<D, NT, ST>;
  static std::atomic<uint64_t> attr_set{0};  // one bit per device that has the attribute
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return cudaErrorInvalidDevice;
  if (!(attr_set.load(std::memory_order_acquire) >> dev & 1)) {
    cudaError_t e = cudaFuncSetAttribute(kv8_attention_kernel<D, NT, ST>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
    if (e != cudaSuccess) return e;
    attr_set.fetch_or(uint64_t(1) << dev, std::memory_order_acq_rel);
  }
  a.slot = L::kSlot;
  const int ctas = L::kCtasPerSm * device_info().sm_count;  // all resident: a persistent grid
  cudaError_t e = launch_pdl(kv8_attention_kernel<D, NT, ST>, dim3((unsigned)ctas), kThreads, L::kSmem, stream, a, cache, bt, status);
  if (e != cudaSuccess || a.whole) return e;
  // groups of units at most; with eight or more parts each, a CTA per row
  const int64_t groups = (int64_t)cache.heads * (bt.seqs + (int64_t)bt.rows * a.group / L::kRows);
  if (groups * 8 <= ctas)
    return launch_pdl(kv8_fixup_kernel<D, true>, dim3((unsigned)ctas, L::kRows), kThreads, 0, stream, a, cache.heads, bt.rows, L::kRows, status);
  return launch_pdl(kv8_fixup_kernel<D, false>, dim3((unsigned)ctas, L::kRows / kWarps), kThreads, 0, stream, a, cache.heads, bt.rows,
                    L::kRows, status);
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
  const int64_t fit = max(kManyCtasPerSm * device_info().sm_count / cache.heads, 1);
  const bool many = bt.seqs >= kManySeqs && items > fit;
  if (many) items = fit;
  const unsigned gy = items < 65535 ? (unsigned)items : 65535u;
  const dim3 grid(cache.heads, gy, (unsigned)((items + gy - 1) / gy));
  auto launch = [&](auto many) -> cudaError_t {
    auto start = [&](auto kernel) { return launch_pdl(kernel, grid, kThreads, 0, stream, k, v, k_stride, v_stride, cache, bt, status); };
    constexpr bool kMany = decltype(many)::value;
    switch (bt.block_tokens * cache.head_dim / 1024) {
      case 1: return start(kv8_append_kernel<1, kMany>);
      case 2: return start(kv8_append_kernel<2, kMany>);
      case 4: return start(kv8_append_kernel<4, kMany>);
      case 8: return start(kv8_append_kernel<8, kMany>);
      case 16: return start(kv8_append_kernel<16, kMany>);
      default: return cudaErrorInvalidConfiguration;
    }
  };
  return many ? launch(std::true_type()) : launch(std::false_type());
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
  // ("not many": about as many groups as sequences and tokens times kv heads)
  a.whole = (int64_t)bt.table_width * bt.block_tokens <= kWholeKeys &&
            ((int64_t)bt.seqs + bt.rows) * cache.heads <= 8 * device_info().sm_count;
  a.fix = reinterpret_cast<Kv8Fix*>(ws + kWsHeaderBytes);
  a.partial = reinterpret_cast<float*>(ws + kWsHeaderBytes + ctas * sizeof(Kv8Fix));
  a.partial_floats = (int64_t)ctas * 2 * kMaxRows * (cache.head_dim + 2);
  uint32_t* status = reinterpret_cast<uint32_t*>(ws);
  // rows that share a kv head, by the mean of new tokens a sequence (lengths are on the device)
  const int64_t rows = ((int64_t)bt.rows + bt.seqs - 1) / bt.seqs * a.group;
  // Few groups (long sequences) keep one stream per warp: a ring of three steps
  // and two CTAs per SM. Many groups want more of them under way: two steps
  // and three CTAs. One sequence of 131002 tokens: 51.4 against 53.1 us, with four
  // new tokens 53.5 against 58.5; 256 of 20 to 400: 40.5 against 35.2, 48 of 30 to
  // 8000 with two new tokens of 64 query heads 77.7 against 73.6. (64-wide heads do
  // as well with two steps.)
  const int64_t groups = (int64_t)cache.heads * (bt.seqs + (int64_t)bt.rows * a.group / (rows > 8 ? 16 : 8));  // at most
  const bool few = groups * 8 <= 2 * device_info().sm_count;
  if (cache.head_dim == 128) {
    if (rows > 8)
      return few ? launch_attention<128, 2, 3>(a, cache, bt, status, stream)
                 : launch_attention<128, 2, 2>(a, cache, bt, status, stream);
    return few ? launch_attention<128, 1, 3>(a, cache, bt, status, stream)
               : launch_attention<128, 1, 2>(a, cache, bt, status, stream);
  }
  return rows <= 8 ? launch_attention<64, 1, 2>(a, cache, bt, status, stream)
                   : launch_attention<64, 2, 2>(a, cache, bt, status, stream);
}

}  // namespace awq
