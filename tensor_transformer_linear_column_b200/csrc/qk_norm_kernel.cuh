// qk_norm_kernel.cuh -- RMS norms of queries and keys for each head with the
// position rotation in the same pass, between the QKV projection and the
// attention core, and the gradients of both.
//
// Per token i at position t_i and per query or key head x (d wide), with one
// gain per kind of head (gamma_q, gamma_k):
//   r = 1 / sqrt(mean_j x_j^2 + eps),  z = gamma * x * r,  y = R(t_i) z
// R turns pair p of the first rot elements by the angle t_i inv_freq[p]; a pair
// is (p, p + rot / 2) in the half layout and (2 p, 2 p + 1) in the pairs
// layout; elements from rot on pass unturned.  The gradients, with dz = R^T dy:
//   dgamma = sum over tokens and heads of dz * x r
//   dx     = r (gamma dz) - x r^3 / d * sum_j (gamma dz)_j x_j
// (R is orthogonal; r depends on every element of its head).
//
// Both kernels are bound by HBM: qkv is read and written once (the gradient
// reads dout too).  A lane holds 16 bytes (8 elements) of a head, so a head is
// a group of 2 to 32 lanes and its sums are shuffles inside the group; the
// angles depend only on the token and on the lane's place in its head, so a
// lane computes with the same 8 cosines and sines for every head of a token.
// They are evaluated once per token and block: the product t inv_freq and its
// remainder by 2 pi in 64 bits (in 32 bits the angle of a position near 2^20 is
// off by 0.06), then sine and cosine in 32 bits of the remainder in [-pi, pi].
#pragma once

#include "rows_bf16.cuh"

namespace tpb {

constexpr int kQkThreads = 256;
constexpr int kQkMaxDim = 256;
constexpr int kQkBatch = 4;         // head groups whose loads a warp has in flight
constexpr int kQkMaxBlocks = 592;   // blocks of the gradient: four per SM
constexpr int kQkReduceLanes = 16;  // partial sums per element in the gains' last step

struct QkParams {
  const uint16_t* x;       // qkv [T, (nq + 2 nkv) d]
  const uint16_t* dy;      // gradient of the result (backward only)
  const uint16_t* gamma_q; // [d] each, or both null: no norm
  const uint16_t* gamma_k;
  const float* inv_freq;   // [rot / 2]
  const int* positions;    // [T] or null: past + i
  uint16_t* out;           // the result (forward) or dqkv (backward)
  float* partial;          // [blocks][2][d] sums of the gains' gradients (backward)
  int T, past, nq, nkv, d, rot;
  int lanes;               // lanes per head: the power of two >= d / 8
  int heads;               // heads walked: nq + nkv, or nq + 2 nkv where V is copied too
  int slices;              // blocks that share one token's heads (forward)
  int pairs;               // 1: the pairs layout
  float eps;
};

// cos and sin of position * freq, the remainder by 2 pi taken in 64 bits: two
// steps of Cody and Waite's reduction with 2 pi as the sum of two doubles.
__device__ __forceinline__ void far_sincos(int position, float freq, float& s, float& c) {
  const double a = static_cast<double>(position) * static_cast<double>(freq);
  const double n = rint(a * 0.15915494309189535);     // 1 / (2 pi)
  double r = fma(-n, 6.283185307179586, a);           // 2 pi rounded to a double,
  r = fma(-n, 2.4492935982947064e-16, r);             // and what that leaves out
  sincosf(static_cast<float>(r), &s, &c);
}

// cos_s / sin_s [rot / 2] of one token, by the whole block.
__device__ __forceinline__ void token_angles(const QkParams& p, int token, float* cos_s,
                                             float* sin_s) {
  const int position = p.positions != nullptr ? __ldg(p.positions + token) : p.past + token;
  for (int i = threadIdx.x; i < p.rot / 2; i += kQkThreads)
    far_sincos(position, __ldg(p.inv_freq + i), sin_s[i], cos_s[i]);
}

// This lane's factors: element e of the head becomes x_e c_e + partner_e s_e.
// `turn` is +1 for R and -1 for its transpose.
struct LaneTurn {
  float c[8], s[8];
  int partner;   // lane that holds the partner elements (half layout)
  bool on;       // the lane's elements are below rot
};

__device__ __forceinline__ void lane_turn(const QkParams& p, int lane, int e0, float turn,
                                          const float* cos_s, const float* sin_s, LaneTurn& t) {
  t.on = e0 < p.rot;
  t.partner = lane;
  const int half = p.rot / 2;
  if (!t.on) return;
  if (p.pairs) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      t.c[k] = cos_s[e0 / 2 + k / 2];
      t.s[k] = (k & 1 ? turn : -turn) * sin_s[e0 / 2 + k / 2];
    }
  } else {
    const bool second = e0 >= half;  // rot is a multiple of 16: a lane lies in one half
    t.partner = lane + (second ? -half / 8 : half / 8);
    const int i0 = second ? e0 - half : e0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      t.c[k] = cos_s[i0 + k];
      t.s[k] = (second ? turn : -turn) * sin_s[i0 + k];
    }
  }
}

// v <- R v (or R^T v); every lane of the warp takes part.
__device__ __forceinline__ void apply_turn(const LaneTurn& t, bool pairs, float (&v)[8]) {
  float w[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) w[k] = pairs ? v[k ^ 1] : __shfl_sync(0xffffffffu, v[k], t.partner);
  if (t.on) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = fmaf(v[k], t.c[k], w[k] * t.s[k]);
  }
}

__device__ __forceinline__ float group_sum(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The factor that brings a head whose squares leave fp32's range back into it,
// from its sum of squares: 2^-70 above 1e37, 2^70 below 1e-30 where eps does not
// drown it, else 1.  With x' = up x and eps' = up^2 eps, x r = x' r' and r = up r'.
__device__ __forceinline__ float range_factor(float ss, float eps) {
  if (!(ss <= 1e37f)) return 8.470329472543003e-22f;               // NaN takes this way too
  if (ss < 1e-30f && eps < 1e-22f) return 1.1805916207174113e21f;
  return 1.0f;
}

// Forward: block (token, slice of heads).  In place (out == x) the V heads are
// not touched; otherwise they are copied.
__global__ void __launch_bounds__(kQkThreads) qk_norm_rope_kernel(const QkParams p) {
  __shared__ float cos_s[kQkMaxDim / 2], sin_s[kQkMaxDim / 2];
  grid_dependency_wait();  // qkv comes from the preceding kernel
  const int token = blockIdx.x / p.slices;
  const int slice = blockIdx.x % p.slices;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_warp = 32 / p.lanes;              // heads a warp holds at once
  const int e0 = (lane % p.lanes) * 8;            // this lane's elements of its head
  const bool active = e0 < p.d;
  const bool norm = p.gamma_q != nullptr;
  const size_t row = static_cast<size_t>(token) * (p.nq + 2 * p.nkv) * p.d;
  if (p.rot > 0) {
    token_angles(p, token, cos_s, sin_s);
    __syncthreads();
  }
  LaneTurn turn;
  lane_turn(p, lane, e0, 1.0f, cos_s, sin_s, turn);
  uint4 gq = make_uint4(0, 0, 0, 0), gk = gq;
  if (norm && active) {
    gq = __ldg(reinterpret_cast<const uint4*>(p.gamma_q + e0));
    gk = __ldg(reinterpret_cast<const uint4*>(p.gamma_k + e0));
  }
  const int step = (kQkThreads / 32) * per_warp;  // heads a block holds at once
  const int first = warp * per_warp + lane / p.lanes + slice * step;
  const int stride = step * p.slices;
  // every lane of a warp walks the same number of head groups: the shuffles
  // need them all
  for (int h0 = first; h0 - lane / p.lanes < p.heads; h0 += kQkBatch * stride) {
    uint4 raw[kQkBatch];
#pragma unroll
    for (int b = 0; b < kQkBatch; ++b) {
      const int h = h0 + b * stride;
      raw[b] = active && h < p.heads
                   ? *reinterpret_cast<const uint4*>(p.x + row + static_cast<size_t>(h) * p.d + e0)
                   : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int b = 0; b < kQkBatch; ++b) {
      const int h = h0 + b * stride;
      if (h - lane / p.lanes >= p.heads) continue;  // the same for the whole warp
      float v[8];
      unpack8(raw[b], v);
      if (norm) {
        float ss = 0.0f, eps = p.eps;
#pragma unroll
        for (int k = 0; k < 8; ++k) ss = fmaf(v[k], v[k], ss);
        ss = group_sum(ss, p.lanes);
        const float up = range_factor(ss, eps);
        if (__any_sync(0xffffffffu, up != 1.0f)) {
          eps = eps * up * up;
          float s2 = 0.0f;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            v[k] *= up;
            s2 = fmaf(v[k], v[k], s2);
          }
          ss = group_sum(s2, p.lanes);
        }
        const float inv = rsqrtf(ss / static_cast<float>(p.d) + eps);
        float g[8];
        unpack8(h < p.nq ? gq : gk, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = v[k] * inv * g[k];
      }
      if (p.rot > 0) apply_turn(turn, p.pairs != 0, v);
      if (active && h < p.heads)
        *reinterpret_cast<uint4*>(p.out + row + static_cast<size_t>(h) * p.d + e0) =
            h < p.nq + p.nkv ? pack8(v) : raw[b];
    }
  }
  grid_launch_dependents();
}

// Backward: a block walks tokens blockIdx.x, + gridDim.x, ...; each lane keeps
// its share of the gains' gradients (8 elements, queries and keys) in registers
// over all of them.  The block's shares are then added in a fixed order into
// partial[block], and qk_gain_reduce_kernel adds the blocks in a fixed order:
// the gradients are bit-identical from run to run, with no atomics.
__global__ void __launch_bounds__(kQkThreads) qk_norm_rope_backward_kernel(const QkParams p) {
  __shared__ float cos_s[kQkMaxDim / 2], sin_s[kQkMaxDim / 2];
  __shared__ float share[kQkThreads * 8];
  grid_dependency_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_warp = 32 / p.lanes;
  const int e0 = (lane % p.lanes) * 8;
  const bool active = e0 < p.d;
  const bool norm = p.gamma_q != nullptr;
  uint4 gq = make_uint4(0, 0, 0, 0), gk = gq;
  if (norm && active) {
    gq = __ldg(reinterpret_cast<const uint4*>(p.gamma_q + e0));
    gk = __ldg(reinterpret_cast<const uint4*>(p.gamma_k + e0));
  }
  const int stride = (kQkThreads / 32) * per_warp;
  const int first = warp * per_warp + lane / p.lanes;
  float acc_q[8] = {0, 0, 0, 0, 0, 0, 0, 0}, acc_k[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  const float inv_d = 1.0f / static_cast<float>(p.d);
  for (int token = blockIdx.x; token < p.T; token += gridDim.x) {
    const size_t row = static_cast<size_t>(token) * (p.nq + 2 * p.nkv) * p.d;
    if (p.rot > 0) {
      __syncthreads();  // the last token's angles have been read
      token_angles(p, token, cos_s, sin_s);
      __syncthreads();
    }
    LaneTurn turn;
    lane_turn(p, lane, e0, -1.0f, cos_s, sin_s, turn);
    for (int h0 = first; h0 - lane / p.lanes < p.heads; h0 += kQkBatch * stride) {
      uint4 rx[kQkBatch], rd[kQkBatch];
#pragma unroll
      for (int b = 0; b < kQkBatch; ++b) {
        const int h = h0 + b * stride;
        const bool in = active && h < p.heads;
        const size_t at = row + static_cast<size_t>(h) * p.d + e0;
        rd[b] = in ? *reinterpret_cast<const uint4*>(p.dy + at) : make_uint4(0, 0, 0, 0);
        rx[b] = in && norm && h < p.nq + p.nkv ? *reinterpret_cast<const uint4*>(p.x + at)
                                               : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int b = 0; b < kQkBatch; ++b) {
        const int h = h0 + b * stride;
        if (h - lane / p.lanes >= p.heads) continue;
        float dz[8];
        unpack8(rd[b], dz);
        if (p.rot > 0) apply_turn(turn, p.pairs != 0, dz);
        if (norm) {
          float x[8], g[8];
          unpack8(rx[b], x);
          unpack8(h < p.nq ? gq : gk, g);
          float ss = 0.0f, sg = 0.0f;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            ss = fmaf(x[k], x[k], ss);
            sg = fmaf(g[k] * dz[k], x[k], sg);
          }
          ss = group_sum(ss, p.lanes);
          sg = group_sum(sg, p.lanes);
          float eps = p.eps;
          const float up = range_factor(ss, eps);
          if (__any_sync(0xffffffffu, up != 1.0f)) {
            eps = eps * up * up;
            ss = sg = 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              x[k] *= up;
              ss = fmaf(x[k], x[k], ss);
              sg = fmaf(g[k] * dz[k], x[k], sg);
            }
            ss = group_sum(ss, p.lanes);
            sg = group_sum(sg, p.lanes);
          }
          const float inv = rsqrtf(fmaf(ss, inv_d, eps));
          const float mean = sg * inv * inv_d;  // of gamma dz x r over the head
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float n = x[k] * inv;
            if (h < p.nq) acc_q[k] = fmaf(dz[k], n, acc_q[k]);
            else if (h < p.nq + p.nkv) acc_k[k] = fmaf(dz[k], n, acc_k[k]);
            dz[k] = inv * up * fmaf(g[k], dz[k], -n * mean);
          }
        }
        if (active && h < p.heads)
          *reinterpret_cast<uint4*>(p.out + row + static_cast<size_t>(h) * p.d + e0) =
              h < p.nq + p.nkv ? pack8(dz) : rd[b];
      }
    }
  }
  if (norm) {
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 8; ++k) share[threadIdx.x * 8 + k] = kind == 0 ? acc_q[k] : acc_k[k];
      __syncthreads();
      // element e: lane e / 8 of every head group of the block, in order
      for (int e = threadIdx.x; e < p.d; e += kQkThreads) {
        float sum = 0.0f;
        for (int gidx = 0; gidx < kQkThreads / p.lanes; ++gidx)
          sum += share[(gidx * p.lanes + e / 8) * 8 + e % 8];
        p.partial[(static_cast<size_t>(blockIdx.x) * 2 + kind) * p.d + e] = sum;
      }
    }
  }
  grid_launch_dependents();
}

// The gains' gradients: column (kind, element) of partial [blocks][2 d] summed
// over the blocks, kQkReduceLanes interleaved sums per column added in order.
__global__ void __launch_bounds__(16 * kQkReduceLanes)
    qk_gain_reduce_kernel(const float* __restrict__ partial, int blocks, int d,
                          uint16_t* __restrict__ dgamma_q, uint16_t* __restrict__ dgamma_k) {
  __shared__ float sums[kQkReduceLanes][16];
  grid_dependency_wait();
  const int col = blockIdx.x * 16 + (threadIdx.x & 15);  // d is a multiple of 16
  const int part = threadIdx.x >> 4;
  float s = 0.0f;
  for (int b = part; b < blocks; b += kQkReduceLanes)
    s += __ldcg(partial + static_cast<size_t>(b) * 2 * d + col);
  sums[part][threadIdx.x & 15] = s;
  __syncthreads();
  if (threadIdx.x < 16) {
    float total = 0.0f;
#pragma unroll
    for (int k = 0; k < kQkReduceLanes; ++k) total += sums[k][threadIdx.x];
    const __nv_bfloat16 b = __float2bfloat16_rn(total);
    (col < d ? dgamma_q[col] : dgamma_k[col - d]) = *reinterpret_cast<const uint16_t*>(&b);
  }
  grid_launch_dependents();
}

}  // namespace tpb
