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
//   dx     = r (gamma dz - x r mean_j(gamma dz x r))
// (R is orthogonal; r depends on every element of its head).
//
// Both kernels are bound by HBM: qkv is read and written once (the gradient
// reads dout too).  A lane holds 8 elements of a head as two 8-byte vectors, so
// a head is a group of 2 to 32 lanes and its sums are shuffles inside the
// group.  In the half layout the two vectors are the first and second members
// of four pairs, in the pairs layout eight elements in a row: a lane always
// holds whole pairs, and the turn needs no exchange.  The angles depend only on
// the token and on the lane's place in its head, so a lane turns every head of a
// token by the same 4 cosines and sines.  They are evaluated once per segment, by
// warps of their own: the product
// t inv_freq and its remainder by 2 pi in 64 bits (in 32 bits the angle of a
// position near 2^20 is off by 0.06), then sine and cosine in 32 bits of the
// remainder in [-pi, pi].
#pragma once

#include "rows_bf16.cuh"

namespace tpb {

constexpr int kQkWarps = 8;                       // computing warps of a block
constexpr int kQkThreads = 32 * kQkWarps + 64;    // + one for copies, one for angles
constexpr int kQkMaxDim = 256;
constexpr int kQkStages = 4;                      // slots of the ring
constexpr int kQkSlotBytes = 24 * 1024;           // a slot at most: two blocks per SM
constexpr int kQkMaxBlocks = 296;                 // blocks: two per SM
constexpr int kQkMaxHeads = 4096;                 // nq + 2 nkv: at most kQkMaxBlocks segments
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
  int heads;               // heads walked: nq + nkv, or nq + 2 nkv where V is copied too
  int seg;                 // heads per segment of a token: grid y counts them
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

// Where lane `l` of a head's group finds its elements: vectors of four at a0 and
// b0.  `angle`: its four pairs' index, or -1 where they are not turned.
struct QkLane {
  int a0, b0, angle;
  bool active;
};

template <bool kPairs>
__device__ __forceinline__ QkLane qk_lane(int l, int d, int rot) {
  QkLane q;
  q.active = l * 8 < d;
  if (!q.active) l = 0;
  if constexpr (kPairs) {
    q.a0 = 8 * l;
    q.b0 = 8 * l + 4;
    q.angle = 8 * l < rot ? 4 * l : -1;
  } else {
    // the unturned rest is held in the same way, as halves of its own
    const int p0 = 4 * l, half = rot / 2;
    q.a0 = p0 < half ? p0 : half + p0;
    q.b0 = q.a0 + (p0 < half ? half : (d - rot) / 2);
    q.angle = p0 < half ? p0 : -1;
  }
  return q;
}

// A lane's 8 elements: v[0..1] and v[2..3] are the two vectors.
__device__ __forceinline__ void qk_unpack(uint2 a, uint2 b, float2 (&v)[4]) {
  v[0] = make_float2(__uint_as_float(a.x << 16), __uint_as_float(a.x & 0xFFFF0000u));
  v[1] = make_float2(__uint_as_float(a.y << 16), __uint_as_float(a.y & 0xFFFF0000u));
  v[2] = make_float2(__uint_as_float(b.x << 16), __uint_as_float(b.x & 0xFFFF0000u));
  v[3] = make_float2(__uint_as_float(b.y << 16), __uint_as_float(b.y & 0xFFFF0000u));
}

__device__ __forceinline__ uint2 qk_pack(float2 a, float2 b) {
  return make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(b.x, b.y));
}

// This lane's gains.
__device__ __forceinline__ void qk_gain(const float* gain, const QkLane& q, float2 (&g)[4]) {
  const float4 a = *reinterpret_cast<const float4*>(gain + q.a0);
  const float4 b = *reinterpret_cast<const float4*>(gain + q.b0);
  g[0] = make_float2(a.x, a.y);
  g[1] = make_float2(a.z, a.w);
  g[2] = make_float2(b.x, b.y);
  g[3] = make_float2(b.z, b.w);
}

// This lane's cosines and sines (pairs angle .. angle + 3).
__device__ __forceinline__ void qk_load_turn(const float* cos_s, const float* sin_s, int angle,
                                             float4& c, float4& s) {
  if (angle >= 0) {
    c = *reinterpret_cast<const float4*>(cos_s + angle);
    s = *reinterpret_cast<const float4*>(sin_s + angle);
  }
}

// v <- R v; with `s` negated, R^T v.
template <bool kPairs>
__device__ __forceinline__ void qk_turn(float2 (&v)[4], const float4& c, const float4& s) {
  if constexpr (kPairs) {
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float a = v[k].x, b = v[k].y;
      v[k].x = fmaf(a, cc[k], -(b * ss[k]));
      v[k].y = fmaf(b, cc[k], a * ss[k]);
    }
  } else {
    const float2 c2[2] = {make_float2(c.x, c.y), make_float2(c.z, c.w)};
    const float2 s2[2] = {make_float2(s.x, s.y), make_float2(s.z, s.w)};
    const float2 n2[2] = {make_float2(-s.x, -s.y), make_float2(-s.z, -s.w)};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float2 a = v[k], b = v[2 + k];
      v[k] = fma2(a, c2[k], mul2(b, n2[k]));
      v[2 + k] = fma2(b, c2[k], mul2(a, s2[k]));
    }
  }
}

template <int kLanes>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = kLanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A lane's share of a head's dot product (none behind the head's end).
__device__ __forceinline__ float dot8(const QkLane& q, const float2 (&a)[4], const float2 (&b)[4]) {
  float2 s = mul2(a[0], b[0]);
#pragma unroll
  for (int k = 1; k < 4; ++k) s = fma2(a[k], b[k], s);
  return q.active ? s.x + s.y : 0.0f;
}

// Two sums over a group's lanes in one butterfly: at the first step a lane keeps
// one of the two and trades the other away, at the end the halves trade back.
template <int kLanes>
__device__ __forceinline__ void group_sum_two(float& a, float& b) {
  constexpr int kHalf = kLanes / 2;
  const bool upper = (threadIdx.x & kHalf) != 0;
  float mine = (upper ? b : a) + __shfl_xor_sync(0xffffffffu, upper ? a : b, kHalf);
#pragma unroll
  for (int o = kHalf >> 1; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  const float other = __shfl_xor_sync(0xffffffffu, mine, kHalf);
  a = upper ? other : mine;
  b = upper ? mine : other;
}

// The factor that brings a head whose squares leave fp32's range back into it,
// from its sum of squares: 2^-70 above 1e37, 2^70 below 1e-30 where eps does not
// drown it, else 1.  With x' = up x and eps' = up^2 eps, x r = x' r' and r = up r'.
__device__ __forceinline__ float range_factor(float ss, float eps) {
  if (!(ss <= 1e37f)) return 8.470329472543003e-22f;               // NaN takes this way too
  if (ss < 1e-30f && eps < 1e-22f) return 1.1805916207174113e21f;
  return 1.0f;
}

__device__ __forceinline__ uint2 qk_load(const uint16_t* p) {
  return *reinterpret_cast<const uint2*>(p);
}

// ------------------------------------------------------------------ bulk copies
//
// Contiguous global <-> shared copies without a tensor map: addresses and sizes
// are multiples of 16 bytes.

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src),
               "r"(bytes)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// At most one of this thread's stores still reads shared memory / none is open.
__device__ __forceinline__ void bulk_wait_read_but_one() {
  asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait_all() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// One block of eight computing warps and two more takes one segment of p.seg
// heads (blockIdx.y) of tokens blockIdx.x, + gridDim.x, ... .  A ring of
// shared-memory slots is filled by bulk copies ahead of the computing warps, which work on a
// slot in place; a bulk copy writes it out while the next is computed.  One of the
// other warps issues the copies, the other evaluates the tokens' angles ahead.
// The warps meet at mbarriers only, so loads, arithmetic and stores of different
// tokens overlap at any number of registers, and no warp waits for a slower one
// before the ring is used up.  4096 tokens of 64 + 8 + 8 heads of 128, out of
// place: forward 29 us (5.7 TB/s, 89 % of a plain copy's rate), backward 52 us
// (4.8 TB/s; without any arithmetic 42).  With each token's loads waited for by the
// block that computes on it 39 and 67; with a block barrier per token 30 and 59.
// Backward, 10 and 12 computing warps a block took 61 and 65, one block of 16 per
// SM 52, three of five 63.
//   forward: slot = the segment of qkv, turned into the result
//   backward: slot = the segment of dout, turned into dqkv, then that of qkv.
//     Each lane keeps its share of the gains' gradients (8 elements, queries and
//     keys) in registers over all tokens; the block's shares are added in a fixed
//     order into partial[block], and qk_gain_reduce_kernel adds the blocks in a
//     fixed order: bit-identical from run to run, with no atomics.
// In place, the heads behind p.heads (V) are not touched; out of place they are
// copied.
template <int kLanes, bool kPairs, bool kBack>
__global__ void __launch_bounds__(kQkThreads, 2) qk_norm_rope_kernel(const QkParams p) {
  extern __shared__ __align__(128) uint8_t qk_smem[];
  __shared__ __align__(16) float cos_s[kQkStages][kQkMaxDim / 2], sin_s[kQkStages][kQkMaxDim / 2];
  __shared__ __align__(16) float gain_s[2][kQkMaxDim];  // of queries, of keys
  __shared__ __align__(8) uint64_t full_bar[kQkStages];   // the slot's copies have landed
  __shared__ __align__(8) uint64_t angle_bar[kQkStages];  // the token's angles are written
  __shared__ __align__(8) uint64_t done_bar[kQkStages];   // the computing warps are done with both
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;
  const int warp = warp_index(), lane = threadIdx.x & 31;
  constexpr int kPerWarp = 32 / kLanes;         // heads a warp holds at once
  constexpr int kStep = kQkWarps * kPerWarp;    // heads a block holds at once
  const QkLane q = qk_lane<kPairs>(lane % kLanes, p.d, p.rot);
  const int sub = lane / kLanes;
  const bool norm = p.gamma_q != nullptr;
  const int turned = p.nq + p.nkv;
  const size_t row = static_cast<size_t>(p.nq + 2 * p.nkv) * p.d;
  const int seg_elems = p.seg * p.d;
  const int slot_bytes = seg_elems * (kBack ? 4 : 2);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kQkStages; ++i) {
      mbar_init(smem_u32(&full_bar[i]), 1);
      mbar_init(smem_u32(&angle_bar[i]), 1);
      mbar_init(smem_u32(&done_bar[i]), kQkWarps);
    }
    abort_word = 0;
    fence_barrier_init();
  }
  __syncthreads();
  grid_dependency_wait();  // qkv comes from the preceding kernel
  grid_launch_dependents();

  const int h0 = blockIdx.y * p.seg;  // this block's heads
  const int n = p.heads - h0 < p.seg ? p.heads - h0 : p.seg;
  const int last = turned - h0 < n ? turned - h0 : n;  // of them, queries and keys
  const uint32_t bytes = static_cast<uint32_t>(n * p.d * 2);
  const uint32_t bytes_x = kBack && norm && last > 0 ? static_cast<uint32_t>(last * p.d * 2) : 0u;
  const int tokens = (p.T - static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) - 1) /
                     static_cast<int>(gridDim.x);
  auto offset = [&](int k) -> size_t {  // of the block's k-th token's segment
    return (blockIdx.x + static_cast<size_t>(k) * gridDim.x) * row + static_cast<size_t>(h0) * p.d;
  };
  auto fill = [&](int k) {
    if (k >= tokens) return;
    const uint32_t dst = smem_u32(qk_smem) + static_cast<uint32_t>((k % kQkStages) * slot_bytes);
    const uint32_t bar = smem_u32(&full_bar[k % kQkStages]);
    mbar_arrive_expect_tx(bar, bytes + bytes_x);
    bulk_load(dst, (kBack ? p.dy : p.x) + offset(k), bytes, bar);
    if (bytes_x > 0)
      bulk_load(dst + static_cast<uint32_t>(seg_elems * 2), p.x + offset(k), bytes_x, bar);
  };
  if (norm)
    for (int e = threadIdx.x; e < p.d; e += kQkThreads) {
      gain_s[0][e] = bf16_to_f32(p.gamma_q[e]);
      gain_s[1][e] = bf16_to_f32(p.gamma_k[e]);
    }
  float2 acc_q[4], acc_k[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) acc_q[k] = acc_k[k] = make_float2(0.0f, 0.0f);
  const float inv_d = 1.0f / static_cast<float>(p.d);
  __syncthreads();

  if (warp < kQkWarps) {
    // ---------------- computing warps
    bool ok = true;
    for (int k = 0; k < tokens; ++k) {
      const int st = k % kQkStages;
      const uint32_t phase = (k / kQkStages) & 1;
      uint16_t* slot = reinterpret_cast<uint16_t*>(qk_smem + st * slot_bytes);
      ok = ok && wait_parity(smem_u32(&full_bar[st]), phase, abort_flag);
      if (p.rot > 0) ok = ok && wait_parity(smem_u32(&angle_bar[st]), phase, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      float4 c = make_float4(0.f, 0.f, 0.f, 0.f), s = c;
      qk_load_turn(cos_s[st], sin_s[st], q.angle, c, s);
      if (kBack) s = make_float4(-s.x, -s.y, -s.z, -s.w);  // the transpose
      // a warp's lanes walk the same head groups: the shuffles need all of them
      // and start one place further for each token, so that a last group of heads
      // that does not fill all warps falls to each of them in turn
      for (int w0 = ((warp + k) % kQkWarps) * kPerWarp; w0 < last && ok; w0 += kStep) {
        // lanes behind the last head or element compute on others' and store nothing
        const int hl = w0 + sub < last ? w0 + sub : last - 1, h = h0 + hl;
        const bool in = q.active && w0 + sub < last;
        uint16_t* at = slot + hl * p.d;
        float2 v[4];
        qk_unpack(qk_load(at + q.a0), qk_load(at + q.b0), v);
        if constexpr (!kBack) {
          if (norm) {
            float ss = group_sum<kLanes>(dot8(q, v, v)), eps = p.eps;
            const float up = range_factor(ss, eps);
            if (__any_sync(0xffffffffu, up != 1.0f)) {
              eps = eps * up * up;
#pragma unroll
              for (int j = 0; j < 4; ++j) v[j] = mul2(v[j], make_float2(up, up));
              ss = group_sum<kLanes>(dot8(q, v, v));
            }
            const float inv = rsqrtf(fmaf(ss, inv_d, eps));
            float2 g[4];
            qk_gain(gain_s[h < p.nq ? 0 : 1], q, g);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = mul2(mul2(v[j], make_float2(inv, inv)), g[j]);
          }
          if (q.angle >= 0) qk_turn<kPairs>(v, c, s);
        } else {
          if (q.angle >= 0) qk_turn<kPairs>(v, c, s);
          if (norm) {
            float2 x[4], g[4];
            qk_unpack(qk_load(at + seg_elems + q.a0), qk_load(at + seg_elems + q.b0), x);
            qk_gain(gain_s[h < p.nq ? 0 : 1], q, g);
#pragma unroll
            for (int j = 0; j < 4; ++j) g[j] = mul2(g[j], v[j]);
            float ss = dot8(q, x, x), sg = dot8(q, g, x);
            group_sum_two<kLanes>(ss, sg);
            float eps = p.eps;
            const float up = range_factor(ss, eps);
            if (__any_sync(0xffffffffu, up != 1.0f)) {
              eps = eps * up * up;
#pragma unroll
              for (int j = 0; j < 4; ++j) x[j] = mul2(x[j], make_float2(up, up));
              ss = dot8(q, x, x);
              sg = dot8(q, g, x);
              group_sum_two<kLanes>(ss, sg);
            }
            const float inv = rsqrtf(fmaf(ss, inv_d, eps));
            const float mean = sg * inv * inv_d;  // of gamma dz x r over the head
            const float scale = inv * up;
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = mul2(x[j], make_float2(inv, inv));
            // the whole warp; lanes behind the head's end keep sums that nobody reads
            if (h0 + w0 + kPerWarp <= p.nq && w0 + kPerWarp <= last) {
#pragma unroll
              for (int j = 0; j < 4; ++j) acc_q[j] = fma2(v[j], x[j], acc_q[j]);
            } else {
              const bool of_q = in && h < p.nq, of_k = in && h >= p.nq;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float2 t = mul2(v[j], x[j]);
                if (of_q) acc_q[j] = add2(acc_q[j], t);
                if (of_k) acc_k[j] = add2(acc_k[j], t);
              }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
              v[j] = mul2(make_float2(scale, scale), fma2(x[j], make_float2(-mean, -mean), g[j]));
          }
        }
        if (in) {
          *reinterpret_cast<uint2*>(at + q.a0) = qk_pack(v[0], v[1]);
          *reinterpret_cast<uint2*>(at + q.b0) = qk_pack(v[2], v[3]);
        }
      }
      fence_proxy_async_smem();  // the slot is read by the bulk store
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&done_bar[st]));
    }
  } else if (warp == kQkWarps) {
    // ---------------- copies
    if (lane == 0) {
      fence_proxy_async_global();  // qkv was written by plain stores
      int filled = 0;
      for (; filled < kQkStages - 1; ++filled) fill(filled);
      for (int k = 0; k < tokens; ++k) {
        const int st = k % kQkStages;
        if (!wait_parity(smem_u32(&done_bar[st]), (k / kQkStages) & 1, abort_flag)) break;
        bulk_store(p.out + offset(k), smem_u32(qk_smem) + static_cast<uint32_t>(st * slot_bytes),
                   bytes);
        // the slot before this one is free once its store has read it
        bulk_wait_read_but_one();
        fill(k + kQkStages - 1);
        ++filled;
      }
      bulk_wait_all();
      if (*abort_flag)  // a wait gave up: copies may still be on their way into the ring
        for (int k = filled > kQkStages ? filled - kQkStages : 0; k < filled && k < tokens; ++k)
          drain_wait(smem_u32(&full_bar[k % kQkStages]), (k / kQkStages) & 1,
                     50ull * 1000ull * 1000ull);
    }
    __syncwarp();
  } else if (p.rot > 0) {
    // ---------------- angles, up to kQkStages tokens ahead.  Plain loads: the kernel
    // before this one may have written the frequencies and the positions
    const int half = p.rot / 2;
    float freq[kQkMaxDim / 64];
#pragma unroll
    for (int j = 0; j < kQkMaxDim / 64; ++j)
      freq[j] = lane + 32 * j < half ? p.inv_freq[lane + 32 * j] : 0.0f;
    for (int k = 0; k < tokens; ++k) {
      const int st = k % kQkStages;
      const int token = static_cast<int>(blockIdx.x) + k * static_cast<int>(gridDim.x);
      const int position = p.positions != nullptr ? p.positions[token] : p.past + token;
      if (k >= kQkStages &&
          !__all_sync(0xffffffffu, wait_parity(smem_u32(&done_bar[st]),
                                               ((k - kQkStages) / kQkStages) & 1, abort_flag)))
        break;
#pragma unroll
      for (int j = 0; j < kQkMaxDim / 64; ++j)
        if (32 * j < half) {
          float sn, cs;
          far_sincos(position, freq[j], sn, cs);
          if (lane + 32 * j < half) {
            sin_s[st][lane + 32 * j] = sn;
            cos_s[st][lane + 32 * j] = cs;
          }
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&angle_bar[st]));
    }
  }
  if constexpr (kBack) {
    if (norm) {
      float* share = reinterpret_cast<float*>(qk_smem);
#pragma unroll
      for (int kind = 0; kind < 2; ++kind) {
        __syncthreads();  // the stores have read the ring
        if (warp < kQkWarps) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<float2*>(share + threadIdx.x * 8 + 2 * j) =
                kind == 0 ? acc_q[j] : acc_k[j];
        }
        __syncthreads();
        // lane l of every head group of the block, in order, for its 8 elements
        for (int e = threadIdx.x; e < p.d; e += kQkThreads) {
          const int l = e >> 3, j = e & 7;
          float sum = 0.0f;
          for (int gidx = 0; gidx < kQkWarps * kPerWarp; ++gidx)
            sum += share[(gidx * kLanes + l) * 8 + j];
          const QkLane where = qk_lane<kPairs>(l, p.d, p.rot);
          const int at = j < 4 ? where.a0 + j : where.b0 + j - 4;
          p.partial[((static_cast<size_t>(blockIdx.y) * gridDim.x + blockIdx.x) * 2 + kind) * p.d +
                    at] = sum;
        }
      }
    }
  }
  __syncthreads();
}

// The gains' gradients: column (kind, element) of partial [blocks][2 d] summed
// over the blocks, kQkReduceLanes interleaved sums per column added in order.
__global__ void __launch_bounds__(16 * kQkReduceLanes)
    qk_gain_reduce_kernel(const float* __restrict__ partial, int blocks, int d,
                          uint16_t* __restrict__ dgamma_q, uint16_t* __restrict__ dgamma_k) {
  __shared__ float sums[kQkReduceLanes][16];
  grid_dependency_wait();
  grid_launch_dependents();
  const int col = blockIdx.x * 16 + (threadIdx.x & 15);  // d is a multiple of 16
  const int part = threadIdx.x >> 4;
  float s = 0.0f;
#pragma unroll 8
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
}

}  // namespace tpb
