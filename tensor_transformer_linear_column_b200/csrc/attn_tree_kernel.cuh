// attn_tree_kernel.cuh -- attention of the T new tokens of one sequence (a
// decoded token, a short chunk, or a tree of drafted tokens) over its
// key-value cache, held in bf16 or in 8 bits.
//
// New token i sees every cached key and the new keys j that bit j of row i of
// `mask` names (no mask: j <= i).  Query head h reads key-value head
// g = h / G, G = nq / nkv; scores are q . k / sqrt(d).  The work is cut where
// the mask begins:
//   attn_tree_kernel        block (chunk c, key-value head g, row group z): the
//                           cached keys of chunk c, which no mask touches,
//                           against kRows of the T G query rows of head g;
//                           writes a partial (maximum, sum, weighted sum of
//                           values).  The blocks also write the new tokens'
//                           keys and values behind the cached ones, where no
//                           block reads in this launch
//   attn_tree_merge_kernel  per (token, query head): the chunks' partials and
//                           the visible new tokens, one by one, in a fixed
//                           order.  A hidden token's score is not used and its
//                           value enters no sum, so a NaN or an infinity in them
//                           reaches no row that does not see it; a row that sees
//                           nothing is zero
// (attn_tree_merge_causal_kernel: the same for many rows without a mask; kJoin: a
// short 8-bit cache, where attn_tree_kernel's blocks do it themselves.)
//
// attn_tree_kernel, per key block b of 128 (16 KB shared-memory stages loaded by
// TMA in the order K_0, K_1, V_0, K_2, V_1, ...):
//   S_b^T[key, n] = K_b Q^T       tcgen05.mma, keys as M (a TMEM lane is a key),
//                                 query rows as N, into one of two TMEM slots
//                                 (8 bits: the parts of an operand lie side by side
//                                 along N and their products in columns of their own,
//                                 so their number costs no instructions: one thread
//                                 issues an MMA every 100 cycles whatever its N)
//   softmax                       one key per thread: its scores against the
//                                 running maximum m_n of each row; weights
//                                 p = 2^(s - m) into one of two shared slots
//   O^T[d, n] += V_b^T P_b^T      tcgen05.mma, d as M, V read as it lies
// The running maximum is raised only when some weight of the block would pass
// 2^16 (8 bits: 2^10): one vote per block in the usual case, and a reduction over
// the block's lanes and a rescale of O in the rare one.  Weights are stored with
// the query rows contiguous (an MN-major B operand), so a thread writes its key's
// weights as 16-byte vectors, without shuffles.
//
// 8-bit cache.  The codes go to the tensor cores as they are (kind::f8f6f4),
// converted nowhere; the operands they meet are split instead:
//   - a bf16 query element has 8 significant bits, E4M3 has 4: the element is
//     scaled by a power of two that brings its row's largest to (224, 448] and
//     becomes hi + lo, both E4M3.  The sum is exact for elements of at least
//     2^-9 of the row's largest and within 2^-17 of the largest below that
//   - a weight p is multiplied by its key's value scale over C, a power of two
//     at or above every value scale of the chunk so far (a running maximum, raised
//     like m), and by 2^5, rounded to fp16, and becomes the sum of three E5M2 terms of
//     3 bits each: within 2^-9 + 2^-11 of itself (a bf16 weight: 2^-9), plus 2^-22 of
//     the largest weight times C, where the terms end.  E5M2 is the upper byte of
//     fp16, so the split is masks and exact subtractions in fp16 pairs
// Keys' scales multiply the scores, one per lane.  Sums of weights are of the
// unrounded ones, in fp32.
//
// Up to 64 query rows per head the cache's bytes bound it (64 / 8 heads, 65536
// cached tokens): 4 tokens over bf16 47 us (5.7 TB/s, 89 % of a plain copy's
// rate).  Over 8 bits a block's chain of latencies for each key block does: 34 us (4.1
// TB/s), and 32 for 1 token with half the softmax work.  About 7 us of a call are not the cache's: the
// launches, the first loads' latency, the last block's end (5 us after the first's
// over a long cache: the SMs do not get the same bandwidth), the merge.
#pragma once

#include "attn_kernel.cuh"
#include "kv_cache_kernel.cuh"
#include "rows_bf16.cuh"

namespace tpb {

constexpr int kTreeMaxTokens = 128;
constexpr int kTreeStageBytes = 16384;  // one TMA item: 128 x 128 codes, or 16 KB of bf16
constexpr int kTreeMaxStages = 8;
// How far a weight may pass 1 before the maximum is raised.  Over a bf16 cache its
// relative error does not depend on its size (at 2^4 instead of 2^16 the raises of
// the first blocks cost a third of the time); over an 8-bit cache the terms of a
// weight end at 2^-17, so the room above 1 is taken from the room below.
constexpr float kLazyLog2 = 16.0f;
constexpr float kLazyLog2Kv8 = 10.0f;
constexpr float kUnsetMax = -1e30f;     // the running maximum before the first key
constexpr int kWeightShift = 5;         // 8 bits: weights are split after times 2^5
// What a preceding kernel may have written is read with plain loads: these kernels
// start before it ends, and the read-only path is for data that stays as it is for a
// kernel's whole life.

struct TreeMergeParams {
  int T, past, nq, nkv, G, rows, chunks, max_len;
  int words;        // mask words per token
  int warps;        // warps per (token, query head): 1, 2, 4 or 8
  float scale;      // 1 / sqrt(d)
  const uint16_t* qkv;
  const uint8_t* cache[2];         // 8 bits: the caches, for the new rows
  const float* cache_scale[2];
  const unsigned long long* mask;  // [T][words], or null: j <= i
  const float* part_o;
  const float* part_ml;
  uint16_t* ctx;    // [T, nq d]
};

struct TreeParams {
  int T, past, nq, nkv, G;
  int R;            // query rows per key-value head: T G
  unsigned g_magic; // ceil(2^32 / G), G > 1: r / G is the upper word of r g_magic, r < 2^16
  int groups;       // row groups of kRows: grid z
  int nblk;         // key blocks of 128 in [0, past)
  int nb, chunks;   // key blocks per chunk, chunks per key-value head: grid x
  int max_len;
  int append;       // this kernel writes the new rows (else the launch before it has)
  int join;         // the chunks of a head are a cluster and leave no partials
  float scale_log2; // log2(e) / sqrt(d)
  const uint16_t* qkv;       // [T, (nq + 2 nkv) d]
  void* cache[2];            // K, V [nkv, max_len, d]: bf16 or E4M3 codes
  float* cache_scale[2];     // [nkv, max_len] (8 bits)
  float* part_o;             // [groups][nkv][chunks][kRows][d]
  float* part_ml;            // [groups][nkv][chunks][kRows][2]
  TreeMergeParams merge;     // where a head's blocks join their partials themselves
};

template <int kRows, bool k8>
struct TreeShape {
  static constexpr int kGroups = kRows / 16;  // softmax warpgroups
  static constexpr int kCols = 16;            // query rows per thread
  static constexpr int kThreads = 64 + 128 * kGroups;           // + TMA warp, MMA warp
  static constexpr int kBlocksPerSm = kRows <= 32 ? 2 : 1;
  static constexpr int kKItems = k8 ? 1 : 2;               // stages per K (and per V) block
  static constexpr int kParts = k8 ? 3 : 1;                // weight operands
  static constexpr int kPartBytes = 128 * kRows * (k8 ? 1 : 2);
  static constexpr int kSlotBytes = kParts * kPartBytes;
  static constexpr int kQBytes = 2 * kRows * 128;          // hi, lo; or the two d halves
  static constexpr int kScoreParts = k8 ? 2 : 1;  // hi | lo along N: summed by the softmax
  static constexpr int kOCol = 2 * kScoreParts * kRows;  // TMEM: two score slots, then O's parts
  static constexpr int kTmemUsed = kOCol + kParts * kRows;
  static constexpr int kTmemCols =
      kTmemUsed <= 64 ? 64 : kTmemUsed <= 128 ? 128 : kTmemUsed <= 256 ? 256 : 512;
  static_assert(kTmemUsed <= 512 && kBlocksPerSm * kTmemCols <= 512, "TMEM of the blocks of an SM");
  static constexpr int kSmallBytes = (4 * kRows + 4 * kRows) * 4 + 64 + 256;
  static constexpr int kSmemTarget = kBlocksPerSm == 2 ? (228 * 1024) / 2 - 1024 : 227 * 1024;
  static constexpr int kFit = (kSmemTarget - 1024 - kSmallBytes - kQBytes - 2 * kSlotBytes) /
                              kTreeStageBytes;
  static constexpr int kStages = kFit > kTreeMaxStages ? kTreeMaxStages : kFit;
  static constexpr int kSmem = 1024 + kStages * kTreeStageBytes + kQBytes + 2 * kSlotBytes +
                               kSmallBytes;
  static_assert(kStages >= 4, "K, K, V and the next K in flight");
};

// Operand layouts in shared memory, as descriptor words:
//   K-major or MN-major with 128-byte swizzling (desc_kmajor_sw128,
//     desc_mnmajor_sw128): lower word desc_lo(address, LBO), upper kDescHiSw128
//   MN-major without swizzling: 16-byte vectors along MN, 8 consecutive K indices 16
//     bytes apart (a 128-byte core matrix), core matrices along K LBO = 128 and along
//     MN SBO = 2048 bytes apart: lower word desc_lo(address, 128), upper kDescHiPlain

// Instruction descriptor, kind::f8f6f4: fp32 D; A and B are E4M3 or E5M2.
__host__ __device__ constexpr uint32_t idesc_f8_f32(int M, int N, bool a_e5m2, bool b_e5m2,
                                                    bool a_mn, bool b_mn) {
  return (1u << 4) | ((a_e5m2 ? 1u : 0u) << 7) | ((b_e5m2 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// The MMAs of these kernels take a descriptor as its two words: the upper one does
// not change, and a step along K adds to the lower one.  The warp that issues them
// runs converged, so the words are uniform, and one elected lane issues.
constexpr uint32_t kDescHiSw128 = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kDescHiPlain = (2048u >> 4) | (1u << 14);  // SBO 2048
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
  return ((saddr >> 4) & 0x3FFFu) | ((lbo >> 4) << 16);  // (a cluster's address holds the rank)
}

// D[tmem] (+)= A[smem] * B[smem]^T, one M x N x 16 (bf16) or x 32 (8 bits) step.
template <bool k8>
__device__ __forceinline__ void umma_words(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi,
                                           uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                           bool accumulate) {
  if constexpr (k8)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc),
        "r"(static_cast<uint32_t>(accumulate))
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc),
        "r"(static_cast<uint32_t>(accumulate))
        : "memory");
}

// The bf16 step with A in tensor memory (umma_bf16_ta's layout).
__device__ __forceinline__ void umma_words_ta(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo,
                                              uint32_t b_hi, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %3};\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Whether `pred` holds in any thread of the `nthreads` at barrier `id`.
__device__ __forceinline__ bool named_barrier_any(uint32_t id, uint32_t nthreads, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(nthreads), "r"(static_cast<uint32_t>(pred))
      : "memory");
  return r != 0;
}

// Smallest e with 2^e >= s, within [-100, 120] (0 and negative s: -100).
__device__ __forceinline__ int scale_exponent(float s) {
  const uint32_t bits = __float_as_uint(s);
  const int e = static_cast<int>((bits >> 23) & 0xFFu) - 127 + ((bits & 0x7FFFFFu) != 0 ? 1 : 0);
  return s > 0.0f ? (e < -100 ? -100 : (e > 120 ? 120 : e)) : -100;
}

__device__ __forceinline__ float pow2i(int e) {  // -126 <= e <= 127
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Two E4M3 codes of an fp16 pair, and back (exact).
__device__ __forceinline__ uint32_t e4m3x2_of(uint32_t h2) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h2));
  return r;
}
__device__ __forceinline__ uint32_t half2_of_e4m3x2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
  return r;
}

// Query rows [row0, row0 + kRows) of head g into shared memory as a K-major
// operand, by kThreads threads (16 lanes a row): bf16 as two 64-wide halves, or
// the 8-bit hi / lo parts with each row's factor in rf_s.  Rows at or past R are
// zero.  The first call starts the copies (16 bytes a thread each; 8 bits: raw,
// into `stage`), the second waits for this thread's and splits them, four rows at a
// time.  The ring's
// loads start after the first call: behind them these few KB would land 6,000
// cycles later.  Rolled loops: a block runs them once, and each instruction line it
// has to fetch costs more than the loop.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(in ? 16 : 0)
               : "memory");
}

template <int kRows, bool k8, int kThreads>
__device__ __forceinline__ void start_queries(const TreeParams& p, int g, int row0, uint8_t* qs,
                                              uint8_t* stage, int st) {
  const int l = st & 15;
#pragma unroll 1
  for (int i = 0; i < kRows * 16 / kThreads; ++i) {
    const int r = (st >> 4) + i * (kThreads >> 4);
    const bool in = row0 + r < p.R;
    const int rr = in ? row0 + r : 0;
    const int tok = p.G == 1 ? rr : static_cast<int>(__umulhi(static_cast<unsigned>(rr), p.g_magic));
    const uint16_t* src =
        p.qkv +
        (static_cast<size_t>(tok) * (p.nq + 2 * p.nkv) + g * p.G + rr - tok * p.G) * kAttnHeadDim +
        8 * l;
    // bf16: half l / 8, 16-byte chunk l % 8 of the 128-byte row, swizzled
    uint8_t* dst = k8 ? stage + r * 256 + l * 16
                      : qs + (l >> 3) * (kRows * 128) + r * 128 + (((l & 7) ^ (r & 7)) << 4);
    cp_async16(smem_u32(dst), src, in);
  }
}

template <int kRows, bool k8, int kThreads>
__device__ __forceinline__ void finish_queries(const TreeParams& p, uint8_t* qs,
                                               const uint8_t* stage, float* rf_s, int st) {
  asm volatile("cp.async.wait_all;" ::: "memory");
  if constexpr (k8) {
    const int l = st & 15;
#pragma unroll 4
    for (int i = 0; i < kRows * 16 / kThreads; ++i) {
      const int r = (st >> 4) + i * (kThreads >> 4);
      float x[8];
      unpack8(*reinterpret_cast<const uint4*>(stage + r * 256 + l * 16), x);
      float amax = abs_max8(x);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      // shift: amax 2^shift in (224, 448]
      const uint32_t bits = __float_as_uint(amax);
      int shift = 8 - (static_cast<int>(bits >> 23) - 127) - ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
      shift = amax > 0.0f ? (shift > 126 ? 126 : shift) : 0;
      const float up = pow2i(shift);  // at least -120
      // in fp16 the scaled elements are exact down to 2^-14, as hi and the rest
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const __half2 v = __floats2half2_rn(x[2 * k] * up, x[2 * k + 1] * up);
        hi[k] = e4m3x2_of(*reinterpret_cast<const uint32_t*>(&v));
        const uint32_t back = half2_of_e4m3x2(hi[k]);
        const __half2 rest = __hsub2(v, *reinterpret_cast<const __half2*>(&back));
        lo[k] = e4m3x2_of(*reinterpret_cast<const uint32_t*>(&rest));
      }
      const int off = r * 128 + (((l >> 1) ^ (r & 7)) << 4) + (l & 1) * 8;
      *reinterpret_cast<uint2*>(qs + off) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
      *reinterpret_cast<uint2*>(qs + kRows * 128 + off) =
          make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
      // a row that holds an infinity scores NaN (its parts are clamped)
      if (l == 0)
        rf_s[r] = amax > 3.3895314e38f ? __int_as_float(0x7fc00000) : p.scale_log2 * pow2i(-shift);
    }
  }
}

// The new tokens' K and V rows of head g behind the cached ones, the rows dealt
// out over the head's blocks (block `part` of `parts`): one pass of the block's TMA
// warp, two rows, from item `base` on.  The warp takes a pass after each key block
// that it has sent for, so the rows cost the softmax warps nothing (in 8 bits their
// divisions held up a call's first scores by 1.5 us).
template <bool k8>
__device__ __forceinline__ void append_pass(const TreeParams& p, int g, int part, int parts,
                                            int base, int lane) {
  const int l = lane & 15;
  const int item = base + (lane >> 4) * parts + part;  // (token, K or V)
  const bool in = item < 2 * p.T;
  uint4 raw = make_uint4(0, 0, 0, 0);
  if (in)
    raw = reinterpret_cast<const uint4*>(
        p.qkv + (static_cast<size_t>(item >> 1) * (p.nq + 2 * p.nkv) + p.nq + (item & 1) * p.nkv +
                 g) * kAttnHeadDim)[l];
  const size_t row = static_cast<size_t>(g) * p.max_len + p.past + (item >> 1);
  void* cache = item & 1 ? p.cache[1] : p.cache[0];
  if constexpr (!k8) {
    if (in) reinterpret_cast<uint4*>(static_cast<uint16_t*>(cache) + row * kAttnHeadDim)[l] = raw;
  } else {
    float x[8];
    unpack8(raw, x);
    float amax = abs_max8(x);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    float scale;
    const uint2 codes = kv8_codes(x, amax, scale);
    if (in) {
      reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + row * kAttnHeadDim)[l] = codes;
      if (l == 0) (item & 1 ? p.cache_scale[1] : p.cache_scale[0])[row] = scale;
    }
  }
}

// 16 weights (already times 2^5 times the value scale over C) as three 16-byte
// vectors of E5M2 terms: a = the leading 3 bits, b = the next of the rest, c =
// the rest of that, rounded.  x - a and x - a - b are exact in fp16.
__device__ __forceinline__ void split_weights(const float2* w, uint4& a4, uint4& b4, uint4& c4) {
  uint32_t a[4], b[4], c[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t av[2], bv[2], cv[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const __half2 x = __float22half2_rn(w[2 * q + h]);
      const uint32_t xb = *reinterpret_cast<const uint32_t*>(&x);
      av[h] = xb & 0xFF00FF00u;
      const __half2 r1 = __hsub2(x, *reinterpret_cast<const __half2*>(&av[h]));
      const uint32_t r1b = *reinterpret_cast<const uint32_t*>(&r1);
      bv[h] = r1b & 0xFF00FF00u;
      const __half2 r2 = __hsub2(r1, *reinterpret_cast<const __half2*>(&bv[h]));
      cv[h] = *reinterpret_cast<const uint32_t*>(&r2) + 0x00800080u;
    }
    a[q] = __byte_perm(av[0], av[1], 0x7531);
    b[q] = __byte_perm(bv[0], bv[1], 0x7531);
    c[q] = __byte_perm(cv[0], cv[1], 0x7531);
  }
  a4 = make_uint4(a[0], a[1], a[2], a[3]);
  b4 = make_uint4(b[0], b[1], b[2], b[3]);
  c4 = make_uint4(c[0], c[1], c[2], c[3]);
}

constexpr int kMergeWarps = 8;
constexpr int kMergeChunks = 4;  // partials a warp has in flight
constexpr int kMergeTokens = 4;  // new tokens a warp has in flight

// One running (maximum, sums, weighted sum) of a warp in base-2 units: lane l
// owns elements 4 l .. 4 l + 3 of the weighted sum; `l` is the chunks' sum, the
// same in every lane, `lt` the new tokens' (lane l: those of slot l / 8).
struct MergeState {
  float m, l, lt;
  float4 o;
};

// Raise the maximum to at least `high`; the reference to take exponents over (0
// while nothing finite has been seen).
__device__ __forceinline__ float merge_raise(MergeState& a, float high) {
  const float mn = fmaxf(a.m, high);
  const float ref = mn == neg_inf() ? 0.0f : mn;
  const float s = exp2_fast(a.m - ref);
  a.o.x *= s;
  a.o.y *= s;
  a.o.z *= s;
  a.o.w *= s;
  a.l *= s;
  a.lt *= s;
  a.m = mn;
  return ref;
}

__device__ __forceinline__ void merge_add(MergeState& a, float w, const float4& v) {
  a.o.x = fmaf(w, v.x, a.o.x);
  a.o.y = fmaf(w, v.y, a.o.y);
  a.o.z = fmaf(w, v.z, a.o.z);
  a.o.w = fmaf(w, v.w, a.o.w);
}

// Four elements of a row.
template <bool k8>
__device__ __forceinline__ float4 cache_values(const uint2& raw) {
  if constexpr (k8) {
    const __half2 a(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(raw.x), __NV_E4M3));
    const __half2 b(
        __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(raw.x >> 16), __NV_E4M3));
    const float2 fa = __half22float2(a), fb = __half22float2(b);
    return make_float4(fa.x, fa.y, fb.x, fb.y);
  } else {
    return make_float4(__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xFFFF0000u),
                       __uint_as_float(raw.y << 16), __uint_as_float(raw.y & 0xFFFF0000u));
  }
}

// The new tokens that token i sees, of those in `mine` (of every 32), for its query
// head h of key-value head g: bf16 from qkv, 8 bits as they were written.
template <bool k8>
__device__ __forceinline__ void merge_tokens(MergeState& st, const TreeMergeParams& p, int i, int h,
                                             int g, uint32_t mine, int lane) {
  const float f = p.scale * 1.4426950408889634f;
  const size_t ld = static_cast<size_t>(p.nq + 2 * p.nkv) * kAttnHeadDim;
  const float4 q = cache_values<false>(
      reinterpret_cast<const uint2*>(p.qkv + i * ld + h * kAttnHeadDim)[lane]);
  const size_t row0 = static_cast<size_t>(g) * p.max_len + p.past;
  for (int j0 = 0; j0 < p.T; j0 += 32) {
    const int left = p.T - j0;  // tokens from this half word on
    uint32_t bits = left >= 32 ? ~0u : (1u << left) - 1u;
    if (p.mask != nullptr) {
      bits &= reinterpret_cast<const uint32_t*>(p.mask + static_cast<size_t>(i) * p.words)[j0 / 32];
    } else {
      const int upto = i - j0 + 1;  // tokens j <= i
      bits &= upto >= 32 ? ~0u : upto > 0 ? (1u << upto) - 1u : 0u;
    }
    bits = __reduce_or_sync(0xffffffffu, bits & mine);  // the same in all lanes, and known to be
    while (bits != 0u) {
      uint2 kr[kMergeTokens], vr[kMergeTokens];
      float s[kMergeTokens], ks = 1.0f, vs = 1.0f;
      const int slot = lane >> 3;  // the token whose score this lane will hold
      int count = 0;
#pragma unroll
      for (int k = 0; k < kMergeTokens; ++k) {
        kr[k] = vr[k] = make_uint2(0, 0);
        if (bits != 0u) {
          const int j = j0 + __ffs(static_cast<int>(bits)) - 1;
          bits &= bits - 1u;
          if constexpr (k8) {
            kr[k].x = __ldcg(reinterpret_cast<const unsigned int*>(
                                 p.cache[0] + (row0 + j) * kAttnHeadDim) + lane);
            vr[k].x = __ldcg(reinterpret_cast<const unsigned int*>(
                                 p.cache[1] + (row0 + j) * kAttnHeadDim) + lane);
          } else {
            const uint16_t* at = p.qkv + j * ld + (p.nq + g) * kAttnHeadDim;
            kr[k] = reinterpret_cast<const uint2*>(at)[lane];
            vr[k] = reinterpret_cast<const uint2*>(at + p.nkv * kAttnHeadDim)[lane];
          }
          if (k8 && slot == k) {
            ks = __ldcg(p.cache_scale[0] + row0 + j);
            vs = __ldcg(p.cache_scale[1] + row0 + j);
          }
          count = k + 1;
        }
      }
#pragma unroll
      for (int k = 0; k < kMergeTokens; ++k) {
        const float4 kv = cache_values<k8>(kr[k]);
        s[k] = fmaf(q.x, kv.x, fmaf(q.y, kv.y, fmaf(q.z, kv.z, q.w * kv.w)));
      }
      const float dot = warp_rows_reduce<kMergeTokens, false>(s, lane);
      // rounded once, for the maximum and for the exponents alike
      const float t = slot < count ? __fmul_rn(dot * ks, f) : neg_inf();
      float high = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
      high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, 16));
      const float ref = merge_raise(st, high);
      const float e = exp2_fast(t - ref);
      st.lt += e;
#pragma unroll
      for (int k = 0; k < kMergeTokens; ++k) {
        const float wk = __shfl_sync(0xffffffffu, e * vs, 8 * k);
        if (k < count) merge_add(st, wk, cache_values<k8>(vr[k]));
      }
    }
  }
}

// The row's sum over the new tokens' slots, and with the chunks'.
__device__ __forceinline__ void merge_sum(MergeState& st) {
  st.lt += __shfl_xor_sync(0xffffffffu, st.lt, 8);
  st.l += st.lt + __shfl_xor_sync(0xffffffffu, st.lt, 16);
}

__device__ __forceinline__ void merge_store(const MergeState& st, const TreeMergeParams& p, int i,
                                            int h, int lane) {
  const float inv = st.l == 0.0f ? 0.0f : 1.0f / st.l;  // a row that sees nothing is zero
  uint2 packed;
  packed.x = pack_bf16x2(st.o.x * inv, st.o.y * inv);
  packed.y = pack_bf16x2(st.o.z * inv, st.o.w * inv);
  *(reinterpret_cast<uint2*>(p.ctx + static_cast<size_t>(i) * p.nq * kAttnHeadDim +
                             static_cast<size_t>(h) * kAttnHeadDim) + lane) = packed;
}

// kMergeChunks partials (maximum, sum, weighted sum) into the state.
__device__ __forceinline__ void merge_chunks(MergeState& st, const float2 (&ml)[kMergeChunks],
                                             const float4 (&o)[kMergeChunks]) {
  float high = ml[0].x;
#pragma unroll
  for (int k = 1; k < kMergeChunks; ++k) high = fmaxf(high, ml[k].x);
  const float ref = merge_raise(st, high);
#pragma unroll
  for (int k = 0; k < kMergeChunks; ++k) {
    const float e = exp2_fast(ml[k].x - ref);
    st.l = fmaf(e, ml[k].y, st.l);
    merge_add(st, e, o[k]);
  }
}

// Shared memory of a block of the cluster.
__device__ __forceinline__ float4 cluster_ld4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ float2 cluster_ld2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

// kJoin: a head's chunks are one cluster, and its blocks join their partials out of
// each other's shared memory instead of leaving them to a second launch (which in
// 8 bits has nothing to do before this one is over: it waits for the new rows' codes).
template <int kRows, bool k8, bool kJoin>
__global__ void __launch_bounds__(TreeShape<kRows, k8>::kThreads, TreeShape<kRows, k8>::kBlocksPerSm)
    attn_tree_kernel(const __grid_constant__ CUtensorMap tmap_k,
                     const __grid_constant__ CUtensorMap tmap_v, const TreeParams p) {
  using Sh = TreeShape<kRows, k8>;
  constexpr int kCols = Sh::kCols;
  constexpr int kStages = Sh::kStages;
  constexpr int kItems = Sh::kKItems;
  constexpr int kSoftmax = 128 * Sh::kGroups;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* ring = smem;
  uint8_t* qs = ring + kStages * kTreeStageBytes;
  uint8_t* ps = qs + Sh::kQBytes;                                   // [2 slots][parts]
  float* nm_s = reinterpret_cast<float*>(ps + 2 * Sh::kSlotBytes);  // minus the running maxima
  float* a_s = nm_s + kRows;      // this raise's factor of O
  float* al_s = a_s + kRows;     // this raise's factor of the sums
  float* rf_s = al_s + kRows;    // 8 bits: score factor of each row
  float* red = rf_s + kRows;     // [4][kRows]
  int* red_c = reinterpret_cast<int*>(red + 4 * kRows);  // [4 warpgroups][4]
  uint64_t* bars = reinterpret_cast<uint64_t*>(red_c + 16);
  uint64_t* full_bar = bars;                      // [kStages]
  uint64_t* empty_bar = full_bar + kTreeMaxStages;
  uint64_t* q_bar = empty_bar + kTreeMaxStages;   // the query operand is written
  uint64_t* q_sent = q_bar + 1;                   // its copies have been started
  uint64_t* s_full = q_sent + 1;                  // [2] scores of a block in their slot
  uint64_t* s_free = s_full + 2;                  // [2] slot read
  uint64_t* p_full = s_free + 2;                  // [2] weights written, O rescaled
  uint64_t* o_done = p_full + 2;                  // [2] the block's value product done
  uint64_t* final_bar = o_done + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(final_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = warp_index();
  const int lane = threadIdx.x & 31;
  const int chunk = blockIdx.x;
  const int g = blockIdx.y;
  const int grp = blockIdx.z;
  const int blk0 = chunk * p.nb;
  const int nbc = p.nblk - blk0 < p.nb ? p.nblk - blk0 : p.nb;  // at least 1
  const int key0 = blk0 * 128;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&full_bar[s]), 1);
      mbar_init(smem_u32(&empty_bar[s]), 1);
    }
    mbar_init(smem_u32(q_bar), kSoftmax / 32);
    mbar_init(smem_u32(q_sent), kSoftmax / 32);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&s_free[i]), kSoftmax / 32);
      mbar_init(smem_u32(&p_full[i]), kSoftmax / 32);
      mbar_init(smem_u32(&o_done[i]), 1);
    }
    mbar_init(smem_u32(final_bar), 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), static_cast<uint32_t>(Sh::kTmemCols));
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  constexpr uint32_t o_col = Sh::kOCol;
  constexpr int kSlotCols = Sh::kScoreParts * kRows;

  if (warp == 0) {
    // ---------------- TMA producer (lane 0), and the new rows
    const int parts = p.chunks * p.groups, part = chunk + p.chunks * grp;
    int append = p.append ? 0 : 2 * p.T;
    if (lane == 0) {
      prefetch_tmap(&tmap_k);
      prefetch_tmap(&tmap_v);
    }
    grid_dependency_wait();  // a preceding kernel may still write the cache, or qkv
    fence_proxy_async_global();
    uint32_t issued = 0u, phases = 0u;
    int s = 0;
    uint32_t ph = 0u;
    bool ok = lane == 0 && wait_parity(smem_u32(q_sent), 0, abort_flag);
    auto load = [&](bool is_v, int b) {
      const int kb = key0 + b * 128;
      for (int it = 0; it < kItems && ok; ++it) {
        if (!wait_parity(smem_u32(&empty_bar[s]), ph ^ 1u, abort_flag)) {
          ok = false;
          break;
        }
        const uint32_t fb = smem_u32(&full_bar[s]);
        const uint32_t dst = smem_u32(ring + s * kTreeStageBytes);
        mbar_arrive_expect_tx(fb, kTreeStageBytes);
        if constexpr (k8) {
          tma_load_3d(dst, is_v ? &tmap_v : &tmap_k, fb, 0, kb, g);
        } else if (!is_v) {  // item: one 64-wide half of d, 128 keys
          tma_load_3d(dst, &tmap_k, fb, it * 64, kb, g);
        } else {             // item: 64 keys, both halves of d
          tma_load_3d(dst, &tmap_v, fb, 0, kb + it * 64, g);
          tma_load_3d(dst + kTreeStageBytes / 2, &tmap_v, fb, 64, kb + it * 64, g);
        }
        issued |= 1u << s;
        phases = (phases & ~(1u << s)) | (ph << s);
        if (++s == kStages) {
          s = 0;
          ph ^= 1u;
        }
      }
    };
    for (int b = 0; b <= nbc; ++b) {
      if (lane == 0) {
        if (b < nbc) load(false, b);
        if (b > 0) load(true, b - 1);
      }
      __syncwarp();
      if (append < 2 * p.T) append_pass<k8>(p, g, part, parts, append, lane);
      append += 2 * parts;
    }
    for (; append < 2 * p.T; append += 2 * parts) append_pass<k8>(p, g, part, parts, append, lane);
    if (lane == 0 && *abort_flag) {
      for (int st = 0; st < kStages; ++st)
        if (issued & (1u << st))
          drain_wait(smem_u32(&full_bar[st]), (phases >> st) & 1u, 50ull * 1000ull * 1000ull);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- MMA issuer, in the producer's order
    const bool elected = elect_one();
    bool ok = __all_sync(0xffffffffu, wait_parity(smem_u32(q_bar), 0, abort_flag));
    tc_fence_after();
    int s = 0;
    uint32_t ph = 0u;
    const uint32_t q_lo = desc_lo(smem_u32(qs), 16);
    // the next stage's tile, once it has landed
    auto next = [&]() -> uint32_t {
      ok = ok && __all_sync(0xffffffffu, wait_parity(smem_u32(&full_bar[s]), ph, abort_flag));
      tc_fence_after();
      return smem_u32(ring) + static_cast<uint32_t>(s * kTreeStageBytes);
    };
    auto release = [&] {
      if (elected) umma_commit(smem_u32(&empty_bar[s]));
      if (++s == kStages) {
        s = 0;
        ph ^= 1u;
      }
    };
    for (int b = 0; b <= nbc && ok; ++b) {
      if (b < nbc) {
        const int slot = b & 1;
        if (b >= 2)
          ok = __all_sync(0xffffffffu, wait_parity(smem_u32(&s_free[slot]), ((b - 2) >> 1) & 1,
                                                   abort_flag));
        const uint32_t d = tmem + static_cast<uint32_t>(slot * kSlotCols);
#pragma unroll
        for (int it = 0; it < kItems; ++it) {
          const uint32_t k_lo = desc_lo(next(), 16);
          if (!ok) break;
          constexpr uint32_t idesc = k8 ? idesc_f8_f32(128, kSlotCols, false, false, false, false)
                                        : idesc_bf16_f32(128, kSlotCols);
          if (elected) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_words<k8>(d, k_lo + kk * 2u, kDescHiSw128, q_lo + it * (kRows * 8u) + kk * 2u,
                             kDescHiSw128, idesc, it + kk > 0);
          }
          release();
        }
        if (!ok) break;
        if (elected) umma_commit(smem_u32(&s_full[slot]));
      }
      if (b > 0) {
        const int v = b - 1, slot = v & 1;
        ok = __all_sync(0xffffffffu,
                        wait_parity(smem_u32(&p_full[slot]), (v >> 1) & 1, abort_flag));
        const uint32_t p_lo =
            desc_lo(smem_u32(ps) + static_cast<uint32_t>(slot * Sh::kSlotBytes), 128);
#pragma unroll
        for (int it = 0; it < kItems; ++it) {
          // bf16: 64 keys an item, its d halves 8 KB apart, 16 keys a step 2048 bytes
          // on; 8 bits: 128 keys, 32 a step 4096 bytes on.  Weights: 2 or 4 core
          // matrices on
          const uint32_t v_lo = desc_lo(next(), k8 ? 0 : kTreeStageBytes / 2);
          if (!ok) break;
          constexpr uint32_t idesc =
              k8 ? idesc_f8_f32(128, Sh::kParts * kRows, false, true, true, true)
                 : idesc_bf16_f32(128, kRows, true, true);
          if (elected) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_words<k8>(tmem + o_col, v_lo + kk * (k8 ? 256u : 128u), kDescHiSw128,
                             p_lo + (it * 4 + kk) * (k8 ? 32u : 16u), kDescHiPlain, idesc,
                             v > 0 || it + kk > 0);
          }
          release();
        }
        if (!ok) break;
        if (elected) umma_commit(smem_u32(&o_done[slot]));
      }
    }
    if (elected) {
      umma_commit(smem_u32(final_bar));
      drain_wait(smem_u32(final_bar), 0, 50ull * 1000ull * 1000ull);
    }
    __syncwarp();
  } else {
    // ---------------- softmax warps.  Thread r of a warpgroup owns TMEM lane r:
    // key r of each block, and element r of O; warpgroup w owns query rows
    // [w kCols, (w + 1) kCols).  Every thread takes the same barriers and
    // arrivals whatever its waits returned.
    grid_dependency_wait();  // qkv; and the partials may still be read
    grid_launch_dependents();
    const int st = threadIdx.x - 64;
    const int wg = (warp - 2) >> 2;
    const int et = st & 127;
    const int q4 = warp & 3;
    const int r = q4 * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(q4 * 32) << 16;
    const uint32_t bar_id = 1u + static_cast<uint32_t>(wg);
    const int row0 = grp * kRows;
    const int c0 = wg * kCols;
    start_queries<kRows, k8, kSoftmax>(p, g, row0, qs, ps, st);
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(q_sent));
    finish_queries<kRows, k8, kSoftmax>(p, qs, ps, rf_s, st);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(q_bar));
    if (et < kCols) nm_s[c0 + et] = -kUnsetMax;
    named_barrier_sync(5, kSoftmax);  // rf_s and nm_s are written

    float2 lsum[kCols / 2];
#pragma unroll
    for (int j = 0; j < kCols / 2; ++j) lsum[j] = make_float2(0.0f, 0.0f);
    int c_exp = -100;  // 8 bits: C = 2^c_exp
    bool ok = true;
    const float* scale_k = nullptr;
    const float* scale_v = nullptr;
    float kscale = p.scale_log2, vscale = 0.0f, k_next = 0.0f, v_next = 0.0f;
    if constexpr (k8) {
      scale_k = p.cache_scale[0] + static_cast<size_t>(g) * p.max_len + key0 + r;
      scale_v = p.cache_scale[1] + static_cast<size_t>(g) * p.max_len + key0 + r;
      if (key0 + r < p.past) {
        k_next = *scale_k;
        v_next = *scale_v;
      }
    }
    for (int b = 0; b < nbc; ++b) {
      const int slot = b & 1;
      const int left = p.past - (key0 + b * 128);  // keys from this block on
      if constexpr (k8) {
        kscale = k_next;
        vscale = v_next;
        k_next = v_next = 0.0f;
        if (b + 1 < nbc && r + 128 < left) {
          k_next = scale_k[(b + 1) * 128];
          v_next = scale_v[(b + 1) * 128];
        }
      }
      ok = __all_sync(0xffffffffu, ok && wait_parity(smem_u32(&s_full[slot]), (b >> 1) & 1,
                                                     abort_flag));
      tc_fence_after();
      const uint32_t s_at = tmem + lane_addr + static_cast<uint32_t>(slot * kSlotCols + c0);
      // e: scores in base-2 units over the running maximum, which stays unless
      // some e passes kLazyLog2.  The product is rounded before the maximum is taken
      // off, as the maximum was: fused, the best key would keep that rounding, up to 8 in
      // its weight's exponent where q . k is 2^30.  (The second rounding costs 0.15 us
      // of 34.6 for 4 tokens over 65536 in 8 bits.)
      float2 e[kCols / 2];
      float over = kUnsetMax;
      auto scores = [&] {
        uint32_t sv[kCols], lo[kCols];
        if (ok) {
          tmem_ld16(s_at, sv);
          if constexpr (k8) tmem_ld16(s_at + kRows, lo);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int j = 0; j < kCols; ++j) sv[j] = lo[j] = 0u;
        }
#pragma unroll
        for (int j = 0; j < kCols / 2; ++j) {
          e[j] = make_float2(__uint_as_float(sv[2 * j]), __uint_as_float(sv[2 * j + 1]));
          if constexpr (k8)
            e[j] = add2(e[j], make_float2(__uint_as_float(lo[2 * j]), __uint_as_float(lo[2 * j + 1])));
        }
      };
      auto factor = [&](int j) {
        float2 f = make_float2(kscale, kscale);
        if constexpr (k8) f = mul2(f, *reinterpret_cast<const float2*>(rf_s + c0 + 2 * j));
        return f;
      };
      auto hide = [&] {  // keys behind the cache's last, in its last block
        if (left < 128 && r >= left) {
#pragma unroll
          for (int j = 0; j < kCols / 2; ++j) e[j] = make_float2(neg_inf(), neg_inf());
        }
      };
      auto excess = [&] {
        scores();
#pragma unroll
        for (int j = 0; j < kCols / 2; ++j)
          e[j] = add2_unfused(mul2(e[j], factor(j)),
                              *reinterpret_cast<const float2*>(nm_s + c0 + 2 * j));
        hide();
      };
      excess();
#pragma unroll
      for (int j = 0; j < kCols / 2; ++j) over = fmaxf(over, fmaxf(e[j].x, e[j].y));
      bool raise = over > (k8 ? kLazyLog2Kv8 : kLazyLog2);
      if constexpr (k8) raise = raise || vscale > pow2i(c_exp);
      if (named_barrier_any(bar_id, 128, raise)) {
        // the block's maximum of every row (and of the value scales), over the
        // lanes of a warp and then the four warps in order
        scores();
#pragma unroll
        for (int j = 0; j < kCols / 2; ++j) e[j] = mul2(e[j], factor(j));
        hide();
        {
          const float m =
              warp_rows_reduce<kCols, true>(*reinterpret_cast<float(*)[kCols]>(e), lane);
          if ((lane & 1) == 0) red[q4 * kRows + c0 + (lane >> 1)] = m;
        }
        int c_new = c_exp;
        if constexpr (k8) {
          const int ce = __reduce_max_sync(0xffffffffu, scale_exponent(vscale));
          if (lane == 0) red_c[wg * 4 + q4] = ce;
        }
        named_barrier_sync(bar_id, 128);
        if constexpr (k8) {
#pragma unroll
          for (int w = 0; w < 4; ++w) c_new = max(c_new, red_c[wg * 4 + w]);
        }
        if (et < kCols) {
          const int n = c0 + et;
          const float mo = -nm_s[n];
          float mn = fmaxf(fmaxf(red[n], red[kRows + n]), fmaxf(red[2 * kRows + n], red[3 * kRows + n]));
          mn = fmaxf(mo, mn);
          const float al = exp2f(mo - mn);
          nm_s[n] = -mn;
          al_s[n] = al;
          a_s[n] = k8 ? al * pow2i(c_exp - c_new < -126 ? -126 : c_exp - c_new) : al;
        }
        c_exp = c_new;
        named_barrier_sync(bar_id, 128);
#pragma unroll
        for (int j = 0; j < kCols / 2; ++j)
          lsum[j] = mul2(lsum[j], *reinterpret_cast<const float2*>(al_s + c0 + 2 * j));
        excess();
        if (b > 0) {
          // O holds the products of blocks 0 .. b - 1: wait for the last
          ok = __all_sync(0xffffffffu, ok && wait_parity(smem_u32(&o_done[slot ^ 1]),
                                                         ((b - 1) >> 1) & 1, abort_flag));
          if (ok) {
            tc_fence_after();
#pragma unroll 1
            for (int part = 0; part < Sh::kParts; ++part) {
              uint32_t o[16];
              const uint32_t at = tmem + lane_addr + o_col + static_cast<uint32_t>(part * kRows + c0);
              tmem_ld16(at, o);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j)
                o[j] = __float_as_uint(__uint_as_float(o[j]) * a_s[c0 + j]);
              tmem_st16(at, o);
            }
            tmem_wait_st();
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s_free[slot]));
      // the slot's weights are free once block b - 2's value product is done
      if (b >= 2)
        ok = __all_sync(0xffffffffu, ok && wait_parity(smem_u32(&o_done[slot]),
                                                       ((b - 2) >> 1) & 1, abort_flag));
      uint8_t* pslot = ps + slot * Sh::kSlotBytes;
      float2 wf = make_float2(1.0f, 1.0f);
      if constexpr (k8) wf.x = wf.y = vscale * pow2i(kWeightShift - c_exp);
#pragma unroll
      for (int c = 0; c < kCols; c += 16) {
        float2 w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          w[j] = make_float2(exp2_fast(e[c / 2 + j].x), exp2_fast(e[c / 2 + j].y));
          lsum[c / 2 + j] = add2(lsum[c / 2 + j], w[j]);
          if constexpr (k8) w[j] = mul2(w[j], wf);
        }
        if constexpr (k8) {
          uint4 a4, b4, c4;
          split_weights(w, a4, b4, c4);
          uint8_t* at = pslot + ((c0 + c) / 16) * 2048 + r * 16;
          *reinterpret_cast<uint4*>(at) = a4;
          *reinterpret_cast<uint4*>(at + Sh::kPartBytes) = b4;
          *reinterpret_cast<uint4*>(at + 2 * Sh::kPartBytes) = c4;
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            *reinterpret_cast<uint4*>(pslot + ((c0 + c) / 8 + h) * 2048 + r * 16) =
                make_uint4(pack_bf16x2(w[4 * h].x, w[4 * h].y),
                           pack_bf16x2(w[4 * h + 1].x, w[4 * h + 1].y),
                           pack_bf16x2(w[4 * h + 2].x, w[4 * h + 2].y),
                           pack_bf16x2(w[4 * h + 3].x, w[4 * h + 3].y));
        }
      }
      fence_proxy_async_smem();  // the weights are read by the MMA through the async proxy
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&p_full[slot]));
    }
    // the rows' sums over the lanes, then the four warps in order
    {
      const float v =
          warp_rows_reduce<kCols, false>(*reinterpret_cast<float(*)[kCols]>(lsum), lane);
      if ((lane & 1) == 0) red[q4 * kRows + c0 + (lane >> 1)] = v;
    }
    named_barrier_sync(bar_id, 128);
    const size_t part = (static_cast<size_t>(grp) * p.nkv + g) * p.chunks + chunk;
    float* part_o = kJoin ? reinterpret_cast<float*>(ring) : p.part_o + part * kRows * kAttnHeadDim;
    float* part_ml = kJoin ? part_o + kRows * kAttnHeadDim : p.part_ml + part * kRows * 2;
    ok = __all_sync(0xffffffffu, ok && wait_parity(smem_u32(&o_done[(nbc - 1) & 1]),
                                                   ((nbc - 1) >> 1) & 1, abort_flag));
    tc_fence_after();
    // (kJoin: the ring is empty by now, every tile has been read)
    if (et < kCols && row0 + c0 + et < p.R) {
      const int n = c0 + et;
      float2 ml = make_float2(-nm_s[n], ((red[n] + red[kRows + n]) + red[2 * kRows + n]) +
                                          red[3 * kRows + n]);
      *reinterpret_cast<float2*>(part_ml + n * 2) = ml;
    }
    const float of = k8 ? pow2i(c_exp - kWeightShift) : 1.0f;
    float* po = part_o + c0 * kAttnHeadDim + r;
    float sum[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) sum[j] = 0.0f;
    if (ok) {
#pragma unroll
      for (int part = 0; part < Sh::kParts; ++part) {
        uint32_t o[16];
        tmem_ld16(tmem + lane_addr + o_col + static_cast<uint32_t>(part * kRows + c0), o);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; ++j) sum[j] += __uint_as_float(o[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (row0 + c0 + j < p.R) po[static_cast<size_t>(j) * kAttnHeadDim] = sum[j] * of;
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, static_cast<uint32_t>(Sh::kTmemCols));
  }
  if constexpr (kJoin) {
    __syncwarp();
    grid_dependency_wait();  // for the warps that have not: qkv, the mask
    cluster_sync_all();  // every block's partial, and in 8 bits the new rows
    // one row a warp: the launch sees to it that there are enough of them
    const int row = warp * p.chunks + chunk;
    if (row < p.R) {
      const int i = row / p.G, h = g * p.G + row - i * p.G;
      MergeState st{neg_inf(), 0.0f, 0.0f, make_float4(0.f, 0.f, 0.f, 0.f)};
      merge_tokens<k8>(st, p.merge, i, h, g, ~0u, lane);
      merge_sum(st);
      float2 ml[kMergeChunks];
      float4 o[kMergeChunks];
      const uint32_t at_o = smem_u32(ring) + static_cast<uint32_t>(row * kAttnHeadDim + lane * 4) * 4u;
      const uint32_t at_ml = smem_u32(ring) + static_cast<uint32_t>(kRows * kAttnHeadDim + row * 2) * 4u;
      for (int c0 = 0; c0 < p.chunks; c0 += kMergeChunks) {
#pragma unroll
        for (int k = 0; k < kMergeChunks; ++k) {
          ml[k] = make_float2(neg_inf(), 0.0f);
          o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (c0 + k < p.chunks) {
            ml[k] = cluster_ld2(dsmem_map(at_ml, static_cast<uint32_t>(c0 + k)));
            o[k] = cluster_ld4(dsmem_map(at_o, static_cast<uint32_t>(c0 + k)));
          }
        }
        merge_chunks(st, ml, o);
      }
      merge_store(st, p.merge, i, h, lane);
    }
    cluster_sync_all();  // a block's shared memory stays until the others have read it
  }
}

// p.warps warps per (token, query head).  Warp w takes the visible new tokens
// j = w, w + warps, ..., four at a time, and then chunks w, w + warps, ..., four
// at a time, in order; the warps' states are then added in order.  Bit-identical
// from run to run.
template <bool k8>
__global__ void __launch_bounds__(kMergeWarps * 32, 4)
    attn_tree_merge_kernel(const TreeMergeParams p) {
  __shared__ float4 red_o[kMergeWarps][32];
  __shared__ float red_l[kMergeWarps], red_m[kMergeWarps];
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int w = warp & (p.warps - 1);
  const int wid = (blockIdx.x * kMergeWarps + warp) / p.warps;
  MergeState st{neg_inf(), 0.0f, 0.0f, make_float4(0.f, 0.f, 0.f, 0.f)};
  const bool in = wid < p.T * p.nq;
  const int i = in ? wid / p.nq : 0;
  const int h = in ? wid - i * p.nq : 0;
  const int g = h / p.G;
  if (in) {
    const int rr = i * p.G + h - g * p.G;
    const int grp = rr / p.rows, n = rr - grp * p.rows;
    const size_t base = (static_cast<size_t>(grp) * p.nkv + g) * p.chunks * p.rows + n;
    // qkv and the mask are complete: the preceding kernel has waited for them
    // before it let this one start
    const uint32_t mine =  // of 32 tokens
        (p.warps == 8 ? 0x01010101u : p.warps == 4 ? 0x11111111u : p.warps == 2 ? 0x55555555u : ~0u)
        << w;
    float2 ml[kMergeChunks];
    float4 o[kMergeChunks];
    auto load_chunks = [&](int c0) {
#pragma unroll
      for (int k = 0; k < kMergeChunks; ++k) {
        const int c = c0 + k * p.warps;
        ml[k] = make_float2(neg_inf(), 0.0f);
        o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c < p.chunks) {
          const size_t at = base + static_cast<size_t>(c) * p.rows;
          ml[k] = __ldcg(reinterpret_cast<const float2*>(p.part_ml + at * 2));
          o[k] = __ldcg(reinterpret_cast<const float4*>(p.part_o + at * kAttnHeadDim) + lane);
        }
      }
    };
    if constexpr (k8) {
      grid_dependency_wait();  // the new rows' codes, and the partials
      grid_launch_dependents();
      load_chunks(w);
    }
    merge_tokens<k8>(st, p, i, h, g, mine, lane);
    if constexpr (!k8) {
      grid_dependency_wait();  // the partials
      grid_launch_dependents();
    }
    for (int c0 = w; c0 < p.chunks; c0 += p.warps * kMergeChunks) {
      if (!k8 || c0 != w) load_chunks(c0);
      merge_chunks(st, ml, o);
    }
    merge_sum(st);
  } else {
    grid_dependency_wait();
  }
  if (p.warps > 1) {
    red_o[warp][lane] = st.o;
    if (lane == 0) {
      red_l[warp] = st.l;
      red_m[warp] = st.m;
    }
    __syncthreads();
    if (w != 0) return;
    float m = st.m;
    for (int k = 1; k < p.warps; ++k) m = fmaxf(m, red_m[warp + k]);
    const float ref = m == neg_inf() ? 0.0f : m;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.0f;
    for (int k = 0; k < p.warps; ++k) {
      const float f = exp2_fast(red_m[warp + k] - ref);
      const float4 v = red_o[warp + k][lane];
      o.x = fmaf(f, v.x, o.x);
      o.y = fmaf(f, v.y, o.y);
      o.z = fmaf(f, v.z, o.z);
      o.w = fmaf(f, v.w, o.w);
      l = fmaf(f, red_l[warp + k], l);
    }
    st.o = o;
    st.l = l;
  }
  if (in) merge_store(st, p, i, h, lane);
}

// The same for many rows that see every new token before them (no mask): there the
// merge's work is the new tokens, 290 instructions for four of them and a row above.
// Here a warp takes kHeads query heads of one token and one key-value head, which
// see the same keys, and a block stages that head's new tokens in shared memory.  A
// lane owns tokens for the scores (no sums across lanes) and elements 4 l .. 4 l + 3
// for the weighted sums; the first partials are loaded meanwhile.  64 tokens of
// 64 / 8 heads over 1000 cached: 33 us a call with the kernel above, 19.8 with this
// (two heads a warp 21.1, one 23.8; partials loaded after the new tokens' work 26.7).
// Bound by latencies: 8 warps an SM, issue slots busy a third of the time.
// Shared memory: K and V [T][256 B] as bf16 or (8 bits) the codes as fp16, 16-byte
// piece c of row j at c ^ (j % 8); per warp its queries in fp32 and the weights
// [64][kHeads] of 64 tokens; 8 bits: the new rows' scales.
constexpr int kManyWarps = 4;
constexpr int kManyFloats = kAttnHeadDim + 64;  // of a head: its query, 64 weights

template <bool k8, int kHeads>
__global__ void __launch_bounds__(kManyWarps * 32)
    attn_tree_merge_causal_kernel(const TreeMergeParams p) {
  extern __shared__ __align__(16) uint8_t many_smem[];
  const int warp = warp_index(), lane = threadIdx.x & 31;
  uint8_t* kt = many_smem;
  uint8_t* vt = kt + p.T * 256;
  float* wq = reinterpret_cast<float*>(vt + p.T * 256) + warp * (kHeads * kManyFloats);
  float* sc = reinterpret_cast<float*>(vt + p.T * 256) + kManyWarps * (kHeads * kManyFloats);
  const int g = blockIdx.y;
  const int parts = (p.G + kHeads - 1) / kHeads;  // of a token's heads
  const int item = blockIdx.x * kManyWarps + warp;
  const bool in = item < p.T * parts;
  const int i = in ? item / parts : 0;
  const int h0 = in ? (item - i * parts) * kHeads : 0;  // first head in the group
  const size_t ld = static_cast<size_t>(p.nq + 2 * p.nkv) * kAttnHeadDim;
  const int seen = in ? i + 1 : 0;  // tokens that the warp's rows see, and the block's
  const int last = (blockIdx.x * kManyWarps + kManyWarps - 1) / parts;
  const int limit = last + 1 < p.T ? last + 1 : p.T;
  grid_dependency_wait();  // the partials, and in 8 bits the new rows
  grid_launch_dependents();
  size_t base[kHeads];
  float2 ml[kHeads][kMergeChunks];
  float4 po[kHeads][kMergeChunks];
#pragma unroll
  for (int k = 0; k < kHeads; ++k) {
    const int rr = i * p.G + (h0 + k < p.G ? h0 + k : p.G - 1);
    const int grp = rr / p.rows;
    base[k] = (static_cast<size_t>(grp) * p.nkv + g) * p.chunks * p.rows + rr - grp * p.rows;
  }
  auto load_chunks = [&](int c0) {
#pragma unroll
    for (int k = 0; k < kHeads; ++k)
#pragma unroll
      for (int x = 0; x < kMergeChunks; ++x) {
        ml[k][x] = make_float2(neg_inf(), 0.0f);
        po[k][x] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c0 + x < p.chunks) {
          const size_t at = base[k] + static_cast<size_t>(c0 + x) * p.rows;
          ml[k][x] = __ldcg(reinterpret_cast<const float2*>(p.part_ml + at * 2));
          po[k][x] = __ldcg(reinterpret_cast<const float4*>(p.part_o + at * kAttnHeadDim) + lane);
        }
      }
  };
  if constexpr (k8) {
    const size_t row0 = static_cast<size_t>(g) * p.max_len + p.past;
    for (int x = threadIdx.x; x < limit * 16; x += kManyWarps * 32) {
      const int j = x >> 4, c = x & 7;
      const uint4 codes = __ldcg(reinterpret_cast<const uint4*>(
                                     (x & 8 ? p.cache[1] : p.cache[0]) + (row0 + j) * kAttnHeadDim) + c);
      uint8_t* at = (x & 8 ? vt : kt) + j * 256;
      *reinterpret_cast<uint4*>(at + (((2 * c) ^ (j & 7)) << 4)) =
          make_uint4(half2_of_e4m3x2(codes.x), half2_of_e4m3x2(codes.x >> 16),
                     half2_of_e4m3x2(codes.y), half2_of_e4m3x2(codes.y >> 16));
      *reinterpret_cast<uint4*>(at + (((2 * c + 1) ^ (j & 7)) << 4)) =
          make_uint4(half2_of_e4m3x2(codes.z), half2_of_e4m3x2(codes.z >> 16),
                     half2_of_e4m3x2(codes.w), half2_of_e4m3x2(codes.w >> 16));
    }
    for (int j = threadIdx.x; j < limit; j += kManyWarps * 32) {
      sc[j] = __ldcg(p.cache_scale[0] + row0 + j);
      sc[kTreeMaxTokens + j] = __ldcg(p.cache_scale[1] + row0 + j);
    }
  } else {
    for (int x = threadIdx.x; x < limit * 32; x += kManyWarps * 32) {
      const int j = x >> 5, c = x & 15, which = (x >> 4) & 1;
      cp_async16(smem_u32((which ? vt : kt) + j * 256 + ((c ^ (j & 7)) << 4)),
                 p.qkv + j * ld + (p.nq + which * p.nkv + g) * kAttnHeadDim + c * 8, true);
    }
  }
#pragma unroll
  for (int k = 0; k < kHeads; ++k) {
    const int h = h0 + k < p.G ? h0 + k : p.G - 1;
    reinterpret_cast<float4*>(wq)[k * 32 + lane] = cache_values<false>(
        reinterpret_cast<const uint2*>(p.qkv + i * ld + (g * p.G + h) * kAttnHeadDim)[lane]);
  }
  load_chunks(0);  // on their way under the new tokens' work
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();

  auto value2 = [](uint32_t w) {  // two elements
    if constexpr (k8)
      return __half22float2(*reinterpret_cast<const __half2*>(&w));
    else
      return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  };
  struct __align__(kHeads * 4) Weights {
    float w[kHeads];
  };
  Weights* weights = reinterpret_cast<Weights*>(wq + kHeads * kAttnHeadDim);
  float m[kHeads], l[kHeads];
  float2 o[kHeads][2];
#pragma unroll
  for (int k = 0; k < kHeads; ++k) {
    m[k] = neg_inf();
    l[k] = 0.0f;
    o[k][0] = o[k][1] = make_float2(0.0f, 0.0f);
  }
  const float f = p.scale * 1.4426950408889634f;
  // 64 tokens at a time
#pragma unroll 1
  for (int j0 = 0; j0 < seen; j0 += 64) {
    // scores of tokens lane and lane + 32
    int j[2];
    float2 acc[2][kHeads];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      j[u] = j0 + u * 32 + lane;
      if (j[u] >= limit) j[u] = limit - 1;
#pragma unroll
      for (int k = 0; k < kHeads; ++k) acc[u][k] = make_float2(0.0f, 0.0f);
    }
#pragma unroll 2
    for (int c = 0; c < 16; ++c) {
      float2 kv[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint4 raw = *reinterpret_cast<const uint4*>(kt + j[u] * 256 + ((c ^ (j[u] & 7)) << 4));
        kv[u][0] = value2(raw.x);
        kv[u][1] = value2(raw.y);
        kv[u][2] = value2(raw.z);
        kv[u][3] = value2(raw.w);
      }
#pragma unroll
      for (int k = 0; k < kHeads; ++k) {
        const float4 qa = reinterpret_cast<const float4*>(wq)[k * 32 + 2 * c];
        const float4 qb = reinterpret_cast<const float4*>(wq)[k * 32 + 2 * c + 1];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          acc[u][k] = fma2(kv[u][0], make_float2(qa.x, qa.y), acc[u][k]);
          acc[u][k] = fma2(kv[u][1], make_float2(qa.z, qa.w), acc[u][k]);
          acc[u][k] = fma2(kv[u][2], make_float2(qb.x, qb.y), acc[u][k]);
          acc[u][k] = fma2(kv[u][3], make_float2(qb.z, qb.w), acc[u][k]);
        }
      }
    }
    // weights
    float by[2] = {f, f}, vs[2] = {1.0f, 1.0f};
    Weights e[2];
    if constexpr (k8) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        by[u] *= sc[j[u]];
        vs[u] = sc[kTreeMaxTokens + j[u]];
      }
    }
    const bool see0 = j0 + lane < seen, see1 = j0 + lane + 32 < seen;
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      // rounded once, for the maximum and for the exponents alike
      const float s0 = see0 ? __fmul_rn(acc[0][k].x + acc[0][k].y, by[0]) : neg_inf();
      const float s1 = see1 ? __fmul_rn(acc[1][k].x + acc[1][k].y, by[1]) : neg_inf();
      float high = fmaxf(s0, s1);
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, x));
      high = fmaxf(high, m[k]);
      const float ref = high == neg_inf() ? 0.0f : high;
      const float a = exp2_fast(m[k] - ref);
      const float e0 = exp2_fast(s0 - ref), e1 = exp2_fast(s1 - ref);
      float sum = e0 + e1;
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      m[k] = high;
      l[k] = fmaf(l[k], a, sum);
      o[k][0] = mul2(o[k][0], make_float2(a, a));
      o[k][1] = mul2(o[k][1], make_float2(a, a));
      e[0].w[k] = e0 * vs[0];
      e[1].w[k] = e1 * vs[1];
    }
    __syncwarp();  // the last 64's have been read
    weights[lane] = e[0];
    weights[lane + 32] = e[1];
    __syncwarp();
    const int n = seen - j0 < 64 ? seen - j0 : 64;
    for (int x0 = 0; x0 < n; x0 += 4) {
      uint2 raw[4];
      Weights w[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int at = x0 + x < n ? x0 + x : n - 1;
        raw[x] = *reinterpret_cast<const uint2*>(vt + (j0 + at) * 256 +
                                                 ((lane * 8) ^ ((at & 7) << 4)));
        w[x] = weights[at];
      }
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (x0 + x < n) {
          const float2 va = value2(raw[x].x), vb = value2(raw[x].y);
#pragma unroll
          for (int k = 0; k < kHeads; ++k) {
            const float2 wk = make_float2(w[x].w[k], w[x].w[k]);
            o[k][0] = fma2(wk, va, o[k][0]);
            o[k][1] = fma2(wk, vb, o[k][1]);
          }
        }
    }
  }
  if (!in) return;
  for (int c0 = 0; c0 < p.chunks; c0 += kMergeChunks) {
    if (c0 != 0) load_chunks(c0);
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      float high = m[k];
#pragma unroll
      for (int x = 0; x < kMergeChunks; ++x) high = fmaxf(high, ml[k][x].x);
      const float ref = high == neg_inf() ? 0.0f : high;
      const float a = exp2_fast(m[k] - ref);
      m[k] = high;
      l[k] *= a;
      o[k][0] = mul2(o[k][0], make_float2(a, a));
      o[k][1] = mul2(o[k][1], make_float2(a, a));
#pragma unroll
      for (int x = 0; x < kMergeChunks; ++x) {
        const float e = exp2_fast(ml[k][x].x - ref);
        l[k] = fmaf(e, ml[k][x].y, l[k]);
        o[k][0] = fma2(make_float2(e, e), make_float2(po[k][x].x, po[k][x].y), o[k][0]);
        o[k][1] = fma2(make_float2(e, e), make_float2(po[k][x].z, po[k][x].w), o[k][1]);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kHeads; ++k) {
    if (h0 + k >= p.G) break;
    const float inv = l[k] == 0.0f ? 0.0f : 1.0f / l[k];  // a row that sees nothing is zero
    uint2 packed;
    packed.x = pack_bf16x2(o[k][0].x * inv, o[k][0].y * inv);
    packed.y = pack_bf16x2(o[k][1].x * inv, o[k][1].y * inv);
    *(reinterpret_cast<uint2*>(p.ctx + static_cast<size_t>(i) * p.nq * kAttnHeadDim +
                               static_cast<size_t>(g * p.G + h0 + k) * kAttnHeadDim) + lane) = packed;
  }
}

}  // namespace tpb
