// kv_cache_kernel.cuh -- new keys and values written into a cache, in bf16 as
// they are or in 8 bits, and an 8-bit cache read back as bf16.
//
// An 8-bit row (one token, one key-value head, K or V) is d E4M3 codes and one
// fp32 scale:
//   scale = max_j |x_j| / 448   (NaN elements are not counted)
//   code_j = E4M3(x_j / scale), to nearest, ties to even, at most 448
// (a row of zeros: scale 0, codes 0 or -0; the attention over a cache bounds its
// weights by the largest value scale, which such a row must not set)
// and stands for scale * code.  Quotients are IEEE divisions, so a row's codes
// do not depend on which kernel wrote them.  448 is the largest E4M3 value.
//
// Bound by HBM: a row is read once and written once (256 bytes in, 132 out at
// d = 128).  A lane holds 8 elements (16 bytes of bf16, 8 codes); a row is a
// group of 2 to 32 lanes.
#pragma once

#include "rows_bf16.cuh"

namespace tpb {

constexpr float kE4m3Max = 448.0f;
constexpr int kCacheThreads = 256;
constexpr int kAppendBatch = 4;  // rows a lane group takes where there are many

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// Codes of 8 of a row's elements, given the largest magnitude of the row.
__device__ __forceinline__ uint2 kv8_codes(const float (&x)[8], float amax, float& scale) {
  scale = __fdiv_rn(amax, kE4m3Max);
  const float by = amax > 0.0f ? scale : 1.0f;
  float q[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) q[k] = __fdiv_rn(x[k], by);
  return make_uint2(e4m3x4(q[0], q[1], q[2], q[3]), e4m3x4(q[4], q[5], q[6], q[7]));
}

__device__ __forceinline__ float abs_max8(const float (&x)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(x[k]));
  return m;
}

struct KvAppendParams {
  const uint16_t* qkv;  // [T, (nq + 2 nkv) d]
  const int* rows;      // [n] rows of qkv, or null: 0 .. n - 1
  void* cache[2];       // K, V: bf16 or codes [nkv, max_len, d]
  float* scale[2];      // [nkv, max_len] (8 bits)
  int T, n, past, max_len, nq, nkv, d;
};

// blockIdx.y = K or V of one head (2 g + which); the block's rows are
// consecutive cache rows, so codes and scales are written in whole lines.
// A row index outside [0, T) leaves its cache row as it was.
// kLanes lanes per row: the power of two >= d / 8; kBatch rows a lane group.
template <bool k8, int kLanes, int kBatch>
__global__ void __launch_bounds__(kCacheThreads) kv_append_rows_kernel(const KvAppendParams p) {
  grid_dependency_wait();  // qkv comes from the preceding kernel
  grid_launch_dependents();
  const int lane_in = threadIdx.x % kLanes;
  const int g = blockIdx.y >> 1, which = blockIdx.y & 1;
  const int e0 = lane_in * 8;
  const bool active = e0 < p.d;
  constexpr int per_block = kCacheThreads / kLanes;
  const int mine = threadIdx.x / kLanes;
  // every load is issued before the first use.  With many rows a lane group takes
  // four: one each took 12.5 us for 4096 tokens of 8 + 8 heads of 128 in 8 bits, now
  // 8.1 (3.1 TB/s).  With few it takes one: 21 tokens took 5.8 us with four, 2.7 with
  // one.  Plain loads: this kernel starts before the one that wrote qkv ends, and the
  // read-only path is for data that stays as it is for a kernel's whole life.
  const int first = blockIdx.x * per_block * kBatch + mine;
  uint4 raw[kBatch];
  bool in[kBatch];
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    const int j = first + b * per_block;
    const int src = j < p.n ? (p.rows != nullptr ? p.rows[j] : j) : -1;
    in[b] = active && src >= 0 && src < p.T;
    raw[b] = make_uint4(0, 0, 0, 0);
    if (in[b])
      raw[b] = *reinterpret_cast<const uint4*>(
          p.qkv + (static_cast<size_t>(src) * (p.nq + 2 * p.nkv) + p.nq + which * p.nkv + g) * p.d +
          e0);
  }
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    const size_t row = static_cast<size_t>(g) * p.max_len + p.past + first + b * per_block;
    void* cache = which ? p.cache[1] : p.cache[0];
    if constexpr (k8) {
      float x[8];
      unpack8(raw[b], x);
      float amax = abs_max8(x);
#pragma unroll
      for (int o = kLanes >> 1; o > 0; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      float scale;
      const uint2 codes = kv8_codes(x, amax, scale);
      if (in[b]) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + row * p.d + e0) = codes;
        if (lane_in == 0) (which ? p.scale[1] : p.scale[0])[row] = scale;
      }
    } else if (in[b]) {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(cache) + row * p.d + e0) = raw[b];
    }
  }
}

struct Kv8ReadParams {
  const uint8_t* codes[2];  // K, V [nkv, max_len, d]
  const float* scale[2];    // [nkv, max_len]
  uint16_t* out[2];         // bf16 [nkv, out_len, d]
  int start, count, max_len, out_len, d;
};

constexpr int kReadBatch = 8;

// Rows [start, start + count) of every head: blockIdx.y = 2 g + which.  A thread
// turns 8 codes into 16 bytes at a time, so a warp's stores are whole lines: 65536
// rows of 8 + 8 heads of 128 in 62 us (6.5 TB/s, as fast as a plain copy of as many
// bytes); with 16 codes into two 16-byte stores each 75.
__global__ void __launch_bounds__(kCacheThreads) kv8_read_kernel(const Kv8ReadParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int g = blockIdx.y >> 1, which = blockIdx.y & 1;
  const int per_row = p.d / 8;
  const long long pieces = static_cast<long long>(p.count) * per_row;
  const size_t in_row = static_cast<size_t>(g) * p.max_len + p.start;
  const size_t out_row = static_cast<size_t>(g) * p.out_len + p.start;
  const uint2* src =
      reinterpret_cast<const uint2*>((which ? p.codes[1] : p.codes[0]) + in_row * p.d);
  const float* sc = (which ? p.scale[1] : p.scale[0]) + in_row;
  uint4* dst = reinterpret_cast<uint4*>((which ? p.out[1] : p.out[0]) + out_row * p.d);
  const long long i0 =
      static_cast<long long>(blockIdx.x) * (kCacheThreads * kReadBatch) + threadIdx.x;
  uint2 raw[kReadBatch];
  float s[kReadBatch];
#pragma unroll
  for (int b = 0; b < kReadBatch; ++b) {
    const long long i = i0 + b * kCacheThreads;
    if (i < pieces) {
      raw[b] = src[i];
      s[b] = sc[i / per_row];
    }
  }
#pragma unroll
  for (int b = 0; b < kReadBatch; ++b) {
    const long long i = i0 + b * kCacheThreads;
    if (i < pieces) {
      uint32_t o[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t w = q < 2 ? raw[b].x : raw[b].y;
        const __half2 h(__nv_cvt_fp8x2_to_halfraw2(
            static_cast<__nv_fp8x2_storage_t>(w >> (16 * (q & 1))), __NV_E4M3));
        const float2 f = __half22float2(h);
        o[q] = pack_bf16x2(f.x * s[b], f.y * s[b]);
      }
      dst[i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

}  // namespace tpb
