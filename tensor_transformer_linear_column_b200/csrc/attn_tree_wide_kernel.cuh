// attn_tree_wide_kernel.cuh -- attn_tree_kernel's part of the work (the cached keys
// against the T G query rows of a key-value head) for more than 64 rows, where
// the tensor cores and the exponentials bound it and no longer the cache.
//
// Query rows as M, keys as N: a thread owns a query row (a TMEM lane), so the
// row's maximum and sum are a register each and nothing is exchanged between
// threads.  Two warpgroups of softmax threads each work on a tile of their own,
// with its own scores S_t, accumulator O_t (TMEM) and weights P_t (shared
// memory), so that one's exponentials overlap the other's products:
//   bf16, more than 128 rows ("shared"): 256 rows a block, tile t = rows
//     [128 t, 128 t + 128); both tiles read every key block, so a key block
//     crosses from L2 once for 256 rows
//   else ("split"): 128 rows a block, tile t = key blocks t, t + 2, ...; each
//     writes a partial of its own
// Unit i of the block's work belongs to tile i % 2 and to key block i / 2
// (shared) or i (split):
//   S_t = Q_t K_b^T             tcgen05.mma, after unit i - 2's value product: a
//                               tile's scores are ready only when its weights are
//                               free again, so one wait covers both
//   softmax                     p = 2^(t - m) straight from the scores with the
//                               running m, 64 keys at a time; only if their sum
//                               passes 2^20 (8 bits: a product with a value scale
//                               leaves fp16) is m raised and the half done again
//   O_t += P_t V_b              tcgen05.mma, V read MN-major as it lies
// A tile waits for its own two products, and the other tile's exponentials fill
// that time.  64 tokens of 64 / 8 heads over 65536 cached tokens (512 rows per head):
// 139 us, 990 TFLOP/s, in a burst, and 164 (840) after some hundred calls in a row,
// when the power cap holds the clock down; 4,100 cycles for 256 rows of a key block,
// of which the softmax of a tile takes 2,300 and its products 1,600.  On the way: keys
// as M and weights through shared memory 312 us; rows as M 180; bf16 weights over the
// scores in tensor memory instead of in shared memory, the ring twice as deep 177; the
// issuing warp converged 158; weights handed over by halves 139.
// 8-bit caches: scores as in attn_tree_kernel (queries in two E4M3 parts against
// the codes); here two more warps turn each block's value codes into fp16 once for
// all rows, and a row's weights times the value scales are fp16 against those
// (within 2^-11, plus 2^-26 of the largest product; splitting them into three E5M2
// terms, as for few rows, costs three of eight instructions an element: 266 us instead
// of 186 for 64 tokens over 65536 rows).  A row's m bounds the products p * scale
// themselves, so a key of a large value scale and a small weight costs the others
// nothing.
#pragma once

#include <type_traits>

#include "attn_tree_kernel.cuh"

namespace tpb {

// TMA warp, MMA warp, (8 bits) two converting warps, two softmax warpgroups
__host__ __device__ constexpr int wide_first(bool k8) { return k8 ? 4 : 2; }
__host__ __device__ constexpr int wide_threads(bool k8) { return 32 * wide_first(k8) + 256; }
constexpr int kWideMaxStages = 10;
constexpr float kWideSumMax = 1048576.0f;       // bf16: 64 keys' sum of weights up to 2^20
constexpr float kWideProductMax = 60000.0f;     // 8 bits: products are fp16
constexpr float kWideProductLog2 = 2.0f;        // a raise leaves products up to 2^2 and
constexpr float kWideWeightLog2 = 94.0f;        // weights up to 2^94: with that, products of
constexpr float kWideSumMaxKv8 = 1.2676506e30f; // value scales from 2^-92 on stay there, and
                                                // 64 weights' sum within 2^100
// Above this a row's scores (in base-2 units) are far: a score is rounded before m is
// taken off, as m was.  In one fused step the best key would keep that rounding, up to
// 8 in its weight's exponent from 2^27 on.  And over 8 bits the range of the products
// is an offset c beside m, which m + c would lose.  Two operations instead of one for
// every score cost 0.4 us of 22.3 (26 tokens of 64 / 8 heads over 8191).
constexpr float kWideFarScore = 1048576.0f;     // 2^20: m is held to 2^-4

template <bool k8, bool kShared>
struct WideShape {
  static constexpr int kKItems = k8 ? 1 : 2;            // stages per K (and per V) block
  static constexpr int kTileRows = kShared ? 256 : 128; // rows of a block
  static constexpr int kQBytes = (kShared ? 2 : 1) * 32768;
  static constexpr int kValueBytes = k8 ? 2 * 32768 : 0;  // two blocks' values as fp16
  static constexpr int kScaleBytes = k8 ? (2 * 2 * 3 + 2) * 128 * 4 : 0;  // [tile][slot][3][128], c
  static constexpr int kSmallBytes = kScaleBytes + 256 * 4 + 384;
  static constexpr int kFit =
      (227 * 1024 - 1024 - kSmallBytes - kQBytes - kValueBytes) / kTreeStageBytes;
  static constexpr int kStages = kFit > kWideMaxStages ? kWideMaxStages : kFit;
  static constexpr int kSmem = 1024 + kStages * kTreeStageBytes + kQBytes + kValueBytes + kSmallBytes;
  static_assert(kStages >= 4 && kStages >= 2 * kKItems + 1, "K and V of a block and the next K in flight");
};

template <bool k8, bool kShared>
__global__ void __launch_bounds__(wide_threads(k8), 1)
    attn_tree_wide_kernel(const __grid_constant__ CUtensorMap tmap_k,
                          const __grid_constant__ CUtensorMap tmap_v, const TreeParams p) {
  using Sh = WideShape<k8, kShared>;
  constexpr int kStages = Sh::kStages;
  constexpr int kItems = Sh::kKItems;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* ring = smem;
  uint8_t* qs = ring + kStages * kTreeStageBytes;
  uint8_t* vs = qs + Sh::kQBytes;                                // 8 bits: [2][2 x 64 keys]
  float* rf_s = reinterpret_cast<float*>(vs + Sh::kValueBytes);  // [256] score factors
  float* sc_s = rf_s + 256;                                       // 8 bits: [tile][slot][3][128]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sc_s + Sh::kScaleBytes / 4);
  uint64_t* full_bar = bars;                       // [kWideMaxStages]
  uint64_t* empty_bar = full_bar + kWideMaxStages; // [kWideMaxStages]
  uint64_t* q_bar = empty_bar + kWideMaxStages;
  uint64_t* q_sent = q_bar + 1;    // the queries' copies have been started
  uint64_t* s_full = q_sent + 1;   // [tile] scores of a unit, P_t free, O_t up to date
  uint64_t* p_full = s_full + 2;   // [tile][half] weights written, O rescaled
  uint64_t* h_done = p_full + 4;   // [tile] the first half's value product done
  uint64_t* o_done = h_done + 2;   // [tile] the last unit's value product done
  uint64_t* v_full = o_done + 2;   // [2] 8 bits: a block's values are fp16
  uint64_t* v_free = v_full + 2;   // [2] and have been read
  uint64_t* final_bar = v_free + 2;
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
  const int units = kShared ? 2 * nbc : nbc;
  // The ring's order: the first blocks' keys (`pre` of them), then the values of
  // block x and the keys of block x + pre in turn (shared: the other way round,
  // for tile 0 reads the next keys before tile 1 reads the values).
  const int pre = kShared || nbc < 2 ? 1 : 2;
  auto k_pos = [&](int x) { return x < pre ? x : 2 * x - pre + (kShared ? 0 : 1); };
  auto v_pos = [&](int x) {
    return kShared ? pre + (x + 1 < nbc - pre ? x + 1 : nbc - pre) + x
                   : pre + (x < nbc - pre ? x : nbc - pre) + x;
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&full_bar[s]), 1);
      mbar_init(smem_u32(&empty_bar[s]), 1);
    }
    mbar_init(smem_u32(q_bar), 8);
    mbar_init(smem_u32(q_sent), 8);
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&s_full[t]), 1);
      mbar_init(smem_u32(&p_full[2 * t]), 4);
      mbar_init(smem_u32(&p_full[2 * t + 1]), 4);
      mbar_init(smem_u32(&h_done[t]), 1);
      mbar_init(smem_u32(&v_full[t]), 1);
      mbar_init(smem_u32(&v_free[t]), 1);
      mbar_init(smem_u32(&o_done[t]), 1);
    }
    mbar_init(smem_u32(final_bar), 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;  // S_0, S_1 at columns 0 and 128, O_0, O_1 at 256, 384

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
    if (lane == 0)
      for (int x = 0; x < pre; ++x) load(false, x);
    for (int x = 0; x < nbc; ++x) {
      if (lane == 0) {
        if (kShared && x + pre < nbc) load(false, x + pre);
        load(true, x);
        if (!kShared && x + pre < nbc) load(false, x + pre);
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
    // ---------------- MMA issuer: units 0 and 1's scores, then unit i's values and
    // unit i + 2's scores.  One issuer for both tiles keeps them half a period apart;
    // with one each they fell into step, and 64 tokens over 65536 rows took 205 us
    // instead of 158.
    const bool elected = elect_one();
    bool ok = __all_sync(0xffffffffu, wait_parity(smem_u32(q_bar), 0, abort_flag));
    tc_fence_after();
    const uint32_t q_lo = desc_lo(smem_u32(qs), 16);
    // the tile at position `pos` (item it) of the ring's order, once it has landed
    auto landed = [&](int pos, int it, int& s) -> uint32_t {
      const int n = pos * kItems + it;
      s = n % kStages;
      ok = ok && __all_sync(0xffffffffu, wait_parity(smem_u32(&full_bar[s]),
                                                     static_cast<uint32_t>(n / kStages) & 1u,
                                                     abort_flag));
      tc_fence_after();
      return smem_u32(ring) + static_cast<uint32_t>(s * kTreeStageBytes);
    };
    auto scores = [&](int i) {
      const int t = i & 1, b = kShared ? i >> 1 : i;
      const uint32_t d = tmem + static_cast<uint32_t>(t * 128);
      const uint32_t a_lo = q_lo + (kShared ? t * 2048u : 0u);
#pragma unroll
      for (int it = 0; it < kItems; ++it) {
        int s;
        const uint32_t k_lo = desc_lo(landed(k_pos(b), it, s), 16);
        if (!ok) return;
        constexpr uint32_t idesc = k8 ? idesc_f8_f32(128, 128, false, false, false, false)
                                      : idesc_bf16_f32(128, 128);
        if (elected) {
#pragma unroll
          for (int part = 0; part < (k8 ? 2 : 1); ++part)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_words<k8>(d, a_lo + (it + part) * 1024u + kk * 2u, kDescHiSw128, k_lo + kk * 2u,
                             kDescHiSw128, idesc, it + part + kk > 0);
          if (!kShared || t == 1) umma_commit(smem_u32(&empty_bar[s]));
        }
      }
      if (elected) umma_commit(smem_u32(&s_full[t]));
    };
    auto values = [&](int i) {
      const int t = i & 1, b = kShared ? i >> 1 : i;
      const uint32_t d = tmem + 256u + static_cast<uint32_t>(t * 128);
      const uint32_t a_tmem = tmem + static_cast<uint32_t>(t * 128);
#pragma unroll
      for (int half = 0; half < 2; ++half) {  // 64 keys, d halves 8 KB apart
        ok = ok && __all_sync(0xffffffffu, wait_parity(smem_u32(&p_full[2 * t + half]),
                                                       (i >> 1) & 1, abort_flag));
        int s = 0;
        uint32_t tile;
        if constexpr (k8) {
          if (half == 0)
            ok = ok && __all_sync(0xffffffffu, wait_parity(smem_u32(&v_full[b & 1]), (b >> 1) & 1,
                                                           abort_flag));
          tc_fence_after();
          tile = smem_u32(vs) + static_cast<uint32_t>((b & 1) * 32768 + half * 16384);
        } else {
          tile = landed(v_pos(b), half, s);
        }
        const uint32_t v_lo = desc_lo(tile, kTreeStageBytes / 2);
        if (!ok) return;
        // A in tensor memory, B MN-major: both fp16, or both bf16
        constexpr uint32_t idesc =
            idesc_bf16_f32(128, 128, false, true) & ~(k8 ? (1u << 7) | (1u << 10) : 0u);
        if (elected) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_words_ta(d, a_tmem + static_cast<uint32_t>(half * 32 + kk * 8), v_lo + kk * 128u,
                          kDescHiSw128, idesc, i >= 2 || half + kk > 0);
          if (half == 0) umma_commit(smem_u32(&h_done[t]));
          if (!kShared || t == 1) {
            if constexpr (!k8)
              umma_commit(smem_u32(&empty_bar[s]));
            else if (half == 1)
              umma_commit(smem_u32(&v_free[b & 1]));
          }
        }
      }
      if (elected && i + 2 >= units) umma_commit(smem_u32(&o_done[t]));
    };
    if (ok) scores(0);
    if (ok && units > 1) scores(1);
    for (int i = 0; i < units && ok; ++i) {
      values(i);
      if (ok && i + 2 < units) scores(i + 2);
    }
    if (elected) {
      umma_commit(smem_u32(final_bar));
      drain_wait(smem_u32(final_bar), 0, 50ull * 1000ull * 1000ull);
    }
    __syncwarp();
  } else if (k8 && warp < 4) {
    // ---------------- value codes to fp16: [key][d] codes (16-byte chunk c of a row at
    // c ^ (key % 8)) to the bf16 cache's tiles: per 64 keys two d halves of 128-byte rows
    // (chunk j at j ^ (key % 8)).  A quarter warp takes chunks 0 .. 3 of a half of keys
    // k and k ^ 5: these differ in the bits that keep its loads and its stores apart
    // in the banks.
    const int c4 = lane & 3, k8th = (lane >> 3) ^ ((lane & 4) ? 5 : 0);
    bool ok = wait_parity(smem_u32(q_bar), 0, abort_flag);  // the queries were split in `vs`
    for (int b = 0; b < nbc; ++b) {  // all of them: both warps take every barrier
      const int n = v_pos(b);
      const int s = n % kStages;
      ok = ok && wait_parity(smem_u32(&full_bar[s]), static_cast<uint32_t>(n / kStages) & 1u,
                             abort_flag);
      if (b >= 2)
        ok = ok && wait_parity(smem_u32(&v_free[b & 1]), ((b - 2) >> 1) & 1, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      const uint8_t* src = ring + s * kTreeStageBytes;
      uint8_t* dst = vs + (b & 1) * 32768;
#pragma unroll 4
      for (int i = warp - 2; i < 32 && ok; i += 2) {
        const int key = (i >> 1) * 8 + k8th, dh = i & 1;
        const uint4 codes =
            *reinterpret_cast<const uint4*>(src + key * 128 + (((dh * 4 + c4) ^ (key & 7)) << 4));
        uint8_t* at = dst + (key >> 6) * 16384 + dh * 8192 + (key & 63) * 128;
        *reinterpret_cast<uint4*>(at + (((2 * c4) ^ (key & 7)) << 4)) =
            make_uint4(half2_of_e4m3x2(codes.x), half2_of_e4m3x2(codes.x >> 16),
                       half2_of_e4m3x2(codes.y), half2_of_e4m3x2(codes.y >> 16));
        *reinterpret_cast<uint4*>(at + (((2 * c4 + 1) ^ (key & 7)) << 4)) =
            make_uint4(half2_of_e4m3x2(codes.z), half2_of_e4m3x2(codes.z >> 16),
                       half2_of_e4m3x2(codes.w), half2_of_e4m3x2(codes.w >> 16));
      }
      fence_proxy_async_smem();  // read by the MMA through the async proxy
      named_barrier_sync(4, 64);
      if (ok && threadIdx.x == 64) {
        mbar_arrive(smem_u32(&v_full[b & 1]));
        mbar_arrive(smem_u32(&empty_bar[s]));
      }
    }
  } else {
    // ---------------- softmax: thread r of tile t owns its query row r.  Every
    // thread takes the same barriers and arrivals whatever its waits returned.
    grid_dependency_wait();  // qkv; and the partials may still be read
    grid_launch_dependents();
    const int st = threadIdx.x - 32 * wide_first(k8);
    const int t = (warp - wide_first(k8)) >> 2;
    const int q4 = warp & 3;
    const int r = q4 * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(q4 * 32) << 16;
    const int row0 = grp * Sh::kTileRows + (kShared ? t * 128 : 0);
    constexpr int kQThreads = kShared ? 128 : 256;  // a tile's own rows, or both the same
    const int qt = kShared ? st & 127 : st;
    uint8_t* qd = qs + (kShared ? t * 32768 : 0);
    uint8_t* stage = vs + (kShared ? t * 32768 : 0);  // 8 bits: no values there yet
    start_queries<128, k8, kQThreads>(p, g, row0, qd, stage, qt);
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(q_sent));
    finish_queries<128, k8, kQThreads>(p, qd, stage, rf_s + (kShared ? t * 128 : 0), qt);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(q_bar));
    named_barrier_sync(3, 256);  // rf_s is written
    const float rf = k8 ? rf_s[(kShared ? t * 128 : 0) + r] : p.scale_log2;
    const int mine = kShared ? nbc : (nbc - t + 1) / 2;  // this tile's units
    auto key_of = [&](int k) { return key0 + (kShared ? k : 2 * k + t) * 128; };

    // weights are 2^(score - m - c).  c is 0 but over 8 bits and for far scores, and not
    // worth a register: held in one, some of the others spilled (188 us instead of 186
    // for 64 tokens over 65536)
    float m = kUnsetMax, l = 0.0f;
    float* const c_at = sc_s + 2 * 2 * 3 * 128 + t * 128 + r;
    if constexpr (k8) *c_at = 0.0f;
    bool far = false;  // any of the warp's rows
    bool ok = true;
    float k_next = 0.0f, v_next = 0.0f;
    const size_t sc_row = static_cast<size_t>(g) * p.max_len + r;
    if constexpr (k8) {
      if (mine > 0 && key_of(0) + r < p.past) {
        k_next = p.cache_scale[0][sc_row + key_of(0)];
        v_next = p.cache_scale[1][sc_row + key_of(0)];
      }
    }
    const uint32_t s_at = tmem + lane_addr + static_cast<uint32_t>(t * 128);
    const uint32_t o_at = tmem + lane_addr + 256u + static_cast<uint32_t>(t * 128);
    for (int k = 0; k < mine; ++k) {
      const int left = p.past - key_of(k);  // keys from this block on
      const float* ks = nullptr;            // this block's key scales, value scales, log2 of them
      if constexpr (k8) {
        float* slot = sc_s + (t * 2 + (k & 1)) * 3 * 128;
        slot[r] = k_next;
        slot[128 + r] = v_next;
        slot[256 + r] = __log2f(v_next);
        ks = slot;
        k_next = v_next = 0.0f;
        if (k + 1 < mine && key_of(k + 1) + r < p.past) {
          k_next = p.cache_scale[0][sc_row + key_of(k + 1)];
          v_next = p.cache_scale[1][sc_row + key_of(k + 1)];
        }
        named_barrier_sync(1u + static_cast<uint32_t>(t), 128);
      }
      ok = __all_sync(0xffffffffu, ok && wait_parity(smem_u32(&s_full[t]), k & 1, abort_flag));
      tc_fence_after();
      // 32 raw scores from column `col` on
      auto fetch = [&](int col, uint32_t (&sv)[32]) {
        if (ok) {
          tmem_ld32(s_at + static_cast<uint32_t>(col), sv);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) sv[j] = 0u;
        }
      };
      // ... in base-2 units
      auto factor = [&](int col) {
        const float2 f = make_float2(rf, rf);
        return k8 ? mul2(f, *reinterpret_cast<const float2*>(ks + col)) : f;
      };
      auto products = [&](const uint32_t (&sv)[32], int col, float2 (&e)[16]) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          e[j] = mul2(make_float2(__uint_as_float(sv[2 * j]), __uint_as_float(sv[2 * j + 1])),
                      factor(col + 2 * j));
      };
      // behind the cache's last key: -inf
      auto hide = [&](int col, float2 (&e)[16]) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          if (col + 2 * j >= left) e[j].x = neg_inf();
          if (col + 2 * j + 1 >= left) e[j].y = neg_inf();
        }
      };
      // The block's halves of 64 keys in turn: weights with the running m, their sum
      // and (8 bits) the largest product with a value scale.  If the sum (the product)
      // has left its range, m is raised and the half done again; its scores are still
      // there, for the weights wait in registers until they are known to be good.
      // The first half's value product runs under the second half's exponentials.
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        const int base = half * 64;
        float2 acc;
        float top;
        uint32_t pk[32];
        auto weights32 = [&](const uint32_t (&sv)[32], int col, auto careful) {  // keys base + col ...
          float2 e[16];
          const float2 nm = make_float2(-m, -m);
          if constexpr (careful) {  // far scores, or the cache's end
            const float c = k8 ? *c_at : 0.0f;
            products(sv, base + col, e);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              e[j] = add2_unfused(e[j], nm);
              if constexpr (k8) e[j] = add2(e[j], make_float2(-c, -c));
            }
            hide(base + col, e);
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              e[j] = fma2(make_float2(__uint_as_float(sv[2 * j]), __uint_as_float(sv[2 * j + 1])),
                          factor(base + col + 2 * j), nm);
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            e[j] = make_float2(exp2_fast(e[j].x), exp2_fast(e[j].y));
            acc = add2(acc, e[j]);
            if constexpr (k8) {
              e[j] = mul2(e[j], *reinterpret_cast<const float2*>(ks + 128 + base + col + 2 * j));
              top = fmaxf(top, fmaxf(e[j].x, e[j].y));
              const __half2 h = __float22half2_rn(e[j]);
              pk[col / 2 + j] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
              pk[col / 2 + j] = pack_bf16x2(e[j].x, e[j].y);
            }
          }
        };
        auto weights = [&](auto careful) {
          uint32_t sa[32], sb[32];
          acc = make_float2(0.0f, 0.0f);
          top = 0.0f;
          fetch(base, sa);
          tmem_wait_ld();
          fetch(base + 32, sb);  // on their way meanwhile
          weights32(sa, 0, careful);
          tmem_wait_ld();
          weights32(sb, 32, careful);
        };
        bool need = k + half == 0, raised = false;
        for (;;) {
          if (__any_sync(0xffffffffu, need)) {
            raised = true;
            // the scores' maximum, and (8 bits) that of the products; where scores are
            // far once more, over that maximum
            float high = kUnsetMax, product = kUnsetMax, anchor = 0.0f;
            bool is_far = false;
#pragma unroll 1
            for (int pass = 0; pass < 2; ++pass) {
              float top_score = kUnsetMax;
              product = kUnsetMax;
#pragma unroll 1
              for (int col = base; col < base + 64; col += 32) {
                uint32_t sv[32];
                float2 e[16];
                fetch(col, sv);
                tmem_wait_ld();
                products(sv, col, e);
                if (k8 && pass > 0) {
#pragma unroll
                  for (int j = 0; j < 16; ++j) e[j] = add2_unfused(e[j], make_float2(-anchor, -anchor));
                }
                if (left < 128) hide(col, e);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                  top_score = fmaxf(top_score, fmaxf(e[j].x, e[j].y));
                  if constexpr (k8) {
                    const float2 lv = *reinterpret_cast<const float2*>(ks + 256 + col + 2 * j);
                    product = fmaxf(product, fmaxf(e[j].x + lv.x, e[j].y + lv.y));
                  }
                }
              }
              if (pass > 0) break;
              high = top_score;
              is_far = fabsf(high) > kWideFarScore && high != kUnsetMax;
              if (!k8 || !__any_sync(0xffffffffu, is_far)) break;
              anchor = is_far ? high : 0.0f;
            }
            float mn = high, cn = 0.0f;
            if constexpr (k8) {
              const float by = fmaxf(product - kWideProductLog2,
                                     (is_far ? 0.0f : high) - kWideWeightLog2);
              if (is_far)
                cn = rintf(fminf(by, 126.0f));  // a power of two, for the partial
              else
                mn = by;
            }
            const float c = k8 ? *c_at : 0.0f;
            const float rise = (mn - m) + (cn - c);
            const bool up = need && rise > 0.0f;
            // in two steps: an 8-bit row's reference may rise by more than fp32's exponents
            const float part = up ? exp2f(-0.5f * rise) : 1.0f;
            l = l * part * part;
            m = up ? mn : m;
            if (k8 && up) *c_at = cn;
            far = __any_sync(0xffffffffu, fabsf(m) > kWideFarScore && m != kUnsetMax);
            // O holds the products of the tile's earlier units and of this one's
            // first half: wait for that one
            if (half == 1)
              ok = __all_sync(0xffffffffu, ok && wait_parity(smem_u32(&h_done[t]), k & 1, abort_flag));
            if (k + half > 0 && ok) {
              tc_fence_after();
#pragma unroll 1
              for (int col = 0; col < 128; col += 16) {
                uint32_t o[16];
                tmem_ld16(o_at + static_cast<uint32_t>(col), o);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j)
                  o[j] = __float_as_uint(__uint_as_float(o[j]) * part * part);
                tmem_st16(o_at + static_cast<uint32_t>(col), o);
              }
              tmem_wait_st();
            }
          }
          if (left < 128 || far)
            weights(std::true_type{});
          else
            weights(std::false_type{});
          // (NaN raises once, for nothing)
          const float sum = acc.x + acc.y;
          need = k8 ? !(top <= kWideProductMax) || !(sum <= kWideSumMaxKv8) : !(sum <= kWideSumMax);
          if (raised || !__any_sync(0xffffffffu, need)) break;
        }
        l += acc.x + acc.y;
        // two keys a column, over scores that have been read
#pragma unroll
        for (int j = 0; j < 32; j += 16)
          tmem_st16(s_at + static_cast<uint32_t>(half * 32 + j),
                    *reinterpret_cast<const uint32_t(*)[16]>(pk + j));
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&p_full[2 * t + half]));
      }
    }
    // both tiles': the ring is used again below
    for (int x = 0; x < 2 && x < units; ++x)
      ok = __all_sync(0xffffffffu, ok && wait_parity(smem_u32(&o_done[x]), 0, abort_flag));
    tc_fence_after();
    // the partial, with the sum brought to [1, 2): m then stands for the row's
    // mass whatever the value scales were.  A far row's m cannot take that in: its sum
    // is left (its best weight was 1 at the last raise), but for c
    const bool far_row = fabsf(m) > kWideFarScore;
    const int le = static_cast<int>((__float_as_uint(l) >> 23) & 0xFFu) - 127;
    int shift = l > 0.0f && le > -127 && le < 128 ? (le < -126 ? -126 : le > 126 ? 126 : le) : 0;
    if (far_row) shift = k8 ? -static_cast<int>(*c_at) : 0;
    const float down = pow2i(-shift);
    const size_t part = (static_cast<size_t>(grp) * p.nkv + g) * p.chunks * (kShared ? 1 : 2) +
                        (kShared ? chunk : 2 * chunk + t);
    const size_t out_row = part * Sh::kTileRows + (kShared ? t * 128 : 0) + r;
    const bool in = row0 + r < p.R;
    if (in)
      *reinterpret_cast<float2*>(p.part_ml + out_row * 2) =
          make_float2(far_row ? m : m + static_cast<float>(shift), l * down);
    // O row by row: a warp turns 64 columns of its 32 rows at a time through 8 KB
    // of the ring, which is empty by now (16-byte piece c of row r at c ^ (r % 16)),
    // so that 16 lanes write 256 contiguous bytes
    uint8_t* turn = ring + t * 32768 + q4 * 8192;
    float4* po = reinterpret_cast<float4*>(p.part_o + (out_row - lane) * kAttnHeadDim);
    const bool have = ok && mine > 0;  // unwritten TMEM may hold anything
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      uint32_t o[64];
      if (have) {
        tmem_ld32(o_at + static_cast<uint32_t>(half * 64), *reinterpret_cast<uint32_t(*)[32]>(o));
        tmem_ld32(o_at + static_cast<uint32_t>(half * 64 + 32),
                  *reinterpret_cast<uint32_t(*)[32]>(o + 32));
        tmem_wait_ld();
      }
#pragma unroll
      for (int j = 0; j < 16; ++j)
        *reinterpret_cast<float4*>(turn + lane * 256 + ((j ^ (lane & 15)) << 4)) =
            have ? make_float4(__uint_as_float(o[4 * j]) * down, __uint_as_float(o[4 * j + 1]) * down,
                               __uint_as_float(o[4 * j + 2]) * down,
                               __uint_as_float(o[4 * j + 3]) * down)
                 : make_float4(0.f, 0.f, 0.f, 0.f);
      __syncwarp();
#pragma unroll 8
      for (int i = 0; i < 32; i += 2) {
        const int rl = i + (lane >> 4), piece = lane & 15;
        const float4 v = *reinterpret_cast<const float4*>(turn + rl * 256 + ((piece ^ (rl & 15)) << 4));
        if (row0 + q4 * 32 + rl < p.R) po[rl * (kAttnHeadDim / 4) + half * 16 + piece] = v;
      }
      __syncwarp();
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace tpb
