// Attention over packed whole prompts on sm_100a: sequences of different lengths end to end, grouped heads,
// causal or not.
//     o_i = sum_j p_ij v_j,   p_ij = softmax_j(scale q_i . k_j),   j over i's own sequence (j <= i if causal)
// The Hq / Hk = g query heads that share a key head are computed together: a work item is 128 query rows,
// floor(128 / g) consecutive tokens of one sequence times those g heads (row = token * g + head), so K and V
// are read once for all of them and the causal diagonal of an item stays narrow.  It walks its keys 128 at a
// time:
//     S [128 rows x 128 keys] = Q (K-major) * K_blk^T          fp32 in TMEM
//     O [128 rows x D]       += P (bf16, TMEM) * V_blk          fp32 in TMEM
// S and P have two buffers each in TMEM beside O.  An S buffer is free again as soon as its scores are in the
// softmax threads' registers, so the scores of the next two blocks are ahead of the softmax, across the ends of
// items too, and neither the softmax nor the tensor core waits for the other's latency.  (With P in the columns
// of its S, every S waits for a P.V product: 1,520 cycles a block with three buffers, and 1,640 to 1,930 with two
// query tiles that share K and V.)  Products cover only the keys an item can see, rounded up to 16.
//
// Two softmax warpgroups take alternate blocks, one thread per query row of 128 scores, so that one group's waits
// and votes pass during the other's exponentials (2^x on the special function unit alone: a part of them as
// polynomials on the FMA pipe cost more issue slots than it freed, 640 -> 673 us on one prompt of 8192).  The
// running maximum m of a row is kept lazily: a block is exponentiated against the current m, which is raised
// (O and the sums rescaled) only when a logit exceeds it by more than kPackedRescale (log2 units): any m
// without overflow gives the same softmax.  m goes from block to block, so from one group to the other,
// through shared memory: a group hands it on as soon as it has its block's maximum.  Sums are binary32 over
// the unrounded weights, one partial sum per group; P is rounded to bf16, the tensor core's operand type
// (relative 2^-8 on every weight, averaged over the row).
//
// The items of each CTA are listed by the plan, longest first, balanced over the SMs on the host: no work
// counter, so nothing is shared between calls but the status word that a failed wait sets.
//
// A key block may end inside another sequence or past the tensor.  Keys there are masked in S; values there
// meet zero weights, but 0 * NaN is NaN, so the warp that issues P.V overwrites the up to 15 value rows
// between a sequence's end and the next multiple of 16 with zeros before the product may read them.
//
// What bounds it: the softmax chain of a block, about 1,500 cycles where its two products take 1,024 at D = 128
// (tensor and special function pipes both 63% busy), then the power limit on long prompts.  One thread loads 128 scores,
// takes their maximum and waits for the other group's before its first exponential.  Calls in a row, with the sampled SM
// clock (in brackets: bursts of nine calls, before the power limit lowers it):
//   40 heads on 8, D = 128, causal, one sequence of 8192                 675 us at 1,515 MHz, 1,018 TFLOP/s (575 to 590)
//   56 heads, D = 96, four sequences of 700 to 2048, not causal          244 us at 1,582 MHz, 739 TFLOP/s (206 to 211)
//   64 heads on 8, D = 64, ragged, causal (9.7e8 exponentials: 214 us)   390 us at 1,950 MHz, 634 TFLOP/s (381)
//   40 heads on 8, D = 128, causal, 24 prompts of 1 to 1000 tokens       78 us at 1,770 MHz (69.6)
// An item's first block is a chain of load, product, softmax, product and store that little overlaps (one O buffer; each
// thread stores its own row): the time from 4 to 8 one-block items a CTA grows by 8,600 cycles an item of 128 tokens at
// D = 128, 6,300 at D = 96, 4,600 at D = 64; 6,000 for 25 tokens of five heads, 3,400 for single tokens.  A call on one token
// takes 5.2 us: the launch, the set-up (TMEM, barriers, tensor maps) and that item.
//
// Roles (352 threads): warps 0..3 and 4..7 softmax of even and odd blocks, and the epilogue (half of O's columns
// each); 8 TMA loads; 9 issues S and owns TMEM, 10 issues P.V.  Every mbarrier wait is bounded.
#pragma once
#include <cuda.h>
#include <cstdint>

#include "attn_sm100.cuh"

namespace vsa {

struct PackedItem {
  int32_t row0;  // the sequence's first token among the packed rows
  int32_t len;   // its tokens
  int32_t t0;    // the item's first token inside it
  int32_t kvh;   // key head
};

struct PackedArgs {
  const PackedItem* items;
  const int32_t* first;  // [grid + 1]: the items of CTA c are [first[c], first[c + 1])
  uint16_t* out;
  int64_t out_ld, out_hd;  // elements between tokens, between heads
  int* status;
  int group;        // g
  int tile_tokens;  // floor(128 / g)
  int causal;
  float scale_log2;  // softmax scale * log2(e)
};

constexpr int kPackedThreads = 352;
constexpr int kAllKeys = 0x40000000;
// Weights stay below 2^24, sums of fewer than 2^31 of them below 2^55; at 8 (a raise for every row whose logits
// have a spread of 6 nats) the raises cost a third of the time on keys of uneven length.
constexpr float kPackedRescale = 24.0f;
// TMEM columns: two S buffers, two P buffers (two bf16 to a column), O
constexpr uint32_t kPackedP = 256, kPackedO = 384;

template <int D>
struct PackedLayout {
  static constexpr int kHalves = (D + 63) / 64;          // 64-column halves of a row (D = 96: two)
  static constexpr int kTileBytes = kHalves * 128 * 128;  // 128 rows of one operand
  static constexpr int kKStages = D == 64 ? 4 : 2, kVStages = kKStages;
  static constexpr int oQ = 0;  // two items' queries
  static constexpr int oK = oQ + 2 * kTileBytes;
  static constexpr int oV = oK + kKStages * kTileBytes;
  static constexpr int oBar = oV + kVStages * kTileBytes;
  static constexpr int bQFull = 0, bQEmpty = bQFull + 2;
  static constexpr int bKFull = bQEmpty + 2, bKEmpty = bKFull + kKStages;
  static constexpr int bVFull = bKEmpty + kKStages, bVEmpty = bVFull + kVStages;
  static constexpr int bSFull = bVEmpty + kVStages, bPEmpty = bSFull + 2;
  static constexpr int bSEmpty = bPEmpty + 2, bPFull = bSEmpty + 2;  // 128 arrivals each
  static constexpr int bMax = bPFull + 2;                            // 128 arrivals: the row maxima after a block
  static constexpr int bSum = bMax + 2, bOEmpty = bSum + 1;  // 256 arrivals
  static constexpr int bOFull = bOEmpty + 1, bDone = bOFull + 1;
  static constexpr int kNumBars = bDone + 2;
  static constexpr int oMisc = oBar + kNumBars * 8;  // TMEM base, abort flag
  static constexpr int oMax = oMisc + 8;             // float [2 blocks][128 rows]
  static constexpr int oSum = oMax + 1024;           // float2 [2 items][2 groups][128 rows]: sum, the maximum it is relative to
  static constexpr int oEnd = oSum + 4096;
  static size_t bytes() { return 1024 /*alignment slack*/ + oEnd; }
};

__device__ __forceinline__ void tma_load_3d(void* dst, const void* tmap, uint64_t* bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(tmap), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// Largest of three; a NaN wins.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// mbar_wait and mbar_wait_drain without a call (the softmax's registers would be saved around it): the abort flag at the
// first look that fails and at every eighth, the time at every 1024th.  With kIdle, for the loader and the two issuers, kIdleNs
// of sleep between looks (their waits lie on the chain of an item's first block too).
constexpr unsigned kIdleNs = 100;
template <bool kIdle = false>
__device__ __forceinline__ bool packed_wait(uint64_t* bar, uint32_t parity, const WaitCtl& ctl, int site,
                                            bool drain = false) {
  uint64_t t0 = 0;
  for (uint32_t it = 0; !mbar_try_wait(bar, parity); ++it) {
    if (kIdle) __nanosleep(kIdleNs);
    if ((it & 7u) != 0) continue;
    if (!drain && *ctl.abort_flag) return false;
    if ((it & 1016u) != 1016u) continue;
    const uint64_t now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > ctl.timeout_ns) {
      *ctl.abort_flag = 1;
      if (atomicCAS(ctl.status, 0, kStatusTimeout) == 0) atomicExch(ctl.status + 1, site);
      return false;
    }
  }
  return true;
}

// Self-test of packed_wait, both forms, on a barrier that nothing arrives on: site 240 + warp if the wait ran out (or saw
// the other warp's abort) and every later wait returned at once, 242 + warp if those took longer than one limit.
__global__ void packed_wait_selftest_kernel(int* status, uint64_t timeout_ns) {
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    abort_flag = 0;
    mbar_init(&bar, 1);
    fence_mbar_init();
  }
  __syncthreads();
  const WaitCtl ctl{&abort_flag, status, timeout_ns};
  const auto wait = [&]() {
    return warp == 0 ? packed_wait(&bar, 0, ctl, 240) : packed_wait<true>(&bar, 0, ctl, 241);  // phase 0 never completes
  };
  bool done = wait();
  const uint64_t t0 = globaltimer_ns();
  for (int i = 0; i < 1000; ++i) done = wait() || done;
  if (done || globaltimer_ns() - t0 > timeout_ns) atomicExch(status + 1, 242 + warp);
}

// One thread of a converged warp, the same at every call.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(p));
  return p != 0;
}

// Shared-memory descriptor in two words (as umma_desc_sw128): the low one moves with the address, the high one
// is a constant; 1 KB between 8-row groups, `lbo` bytes between the 64-column halves of a K-major step's
// operand (unused) or of an MN-major operand.
__device__ __forceinline__ uint32_t umma_desc_lo(uint32_t saddr) { return (saddr & 0x3FFFFu) >> 4; }
__device__ __forceinline__ uint64_t umma_desc(uint32_t lo, uint32_t lbo) {
  const uint32_t hi = (1024u >> 4) | (1u << 14) | (2u << 29);
  return (static_cast<uint64_t>(hi) << 32) | lo | ((lbo >> 4) << 16);
}

// An item as every lane of a warp has it, the keys it can see and the blocks they make.
struct PackedWork {
  int row0, len, t0, kvh, keys, blocks;
};
__device__ __forceinline__ PackedWork packed_work(const PackedArgs& a, int i) {
  const int4 v = __ldg(reinterpret_cast<const int4*>(a.items) + i);
  PackedWork w;
  w.row0 = __shfl_sync(0xffffffffu, v.x, 0);
  w.len = __shfl_sync(0xffffffffu, v.y, 0);
  w.t0 = __shfl_sync(0xffffffffu, v.z, 0);
  w.kvh = __shfl_sync(0xffffffffu, v.w, 0);
  w.keys = a.causal ? min(w.len, w.t0 + a.tile_tokens) : w.len;
  w.blocks = (w.keys + 127) >> 7;
  return w;
}

template <int D>
__global__ void __launch_bounds__(kPackedThreads, 1)
    packed_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const PackedArgs a) {
  using Ly = PackedLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Ly::oBar);
  uint32_t* tmem_base_s = reinterpret_cast<uint32_t*>(sm + Ly::oMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + Ly::oMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtl ctl{abort_flag, a.status, kWaitTimeoutNs};
  const int i0 = __shfl_sync(0xffffffffu, __ldg(a.first + blockIdx.x), 0);
  const int i1 = __shfl_sync(0xffffffffu, __ldg(a.first + blockIdx.x + 1), 0);
  // a wait of a whole warp, with one answer for all of it
  auto warp_wait = [&](int bar, uint32_t parity, int site) {
    return __shfl_sync(0xffffffffu, static_cast<int>(packed_wait<true>(&bars[bar], parity, ctl, site)), 0) != 0;
  };

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < Ly::kNumBars; ++i) {
      const bool one_group = i >= Ly::bSEmpty && i < Ly::bMax + 2, both = i == Ly::bSum || i == Ly::bOEmpty;
      mbar_init(&bars[i], one_group ? 128 : both ? 256 : 1);
    }
    fence_mbar_init();
  }
  if (warp == 8 && lane == 0) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  if (warp == 9) {
    tmem_alloc(tmem_base_s, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_base_s, 0);

  if (warp == 8) {
    // ============================================================ TMA producer
    // one lane per 64-column half (a thread alone reaches 28 B/clk); K runs two blocks ahead of V, as S does of P.V
    const uint32_t q_bytes = static_cast<uint32_t>(Ly::kHalves * 128 * a.group * a.tile_tokens);
    constexpr int kAhead = 2;
    bool ok = true;
    int n = 0;
    auto load = [&](int b_full, int b_empty, uint32_t stages, int base, const void* map, const PackedWork& w, int j,
                    uint32_t g) {
      const uint32_t st = g % stages;
      ok = ok && warp_wait(b_empty + st, ((g / stages) & 1) ^ 1, 202);
      if (!ok) return;
      if (lane == 0) mbar_arrive_expect_tx(&bars[b_full + st], Ly::kTileBytes);
      __syncwarp();
      if (lane < Ly::kHalves)
        tma_load_3d(sm + base + st * Ly::kTileBytes + lane * 16384, map, &bars[b_full + st], lane * 64, w.kvh,
                    w.row0 + 128 * j);
      __syncwarp();
    };
    // two walks over the items' blocks, of K and of V
    PackedWork wk{}, wv{};
    int ik = i0, iv = i0, jk = 0, jv = 0;
    uint32_t gk = 0, gv = 0;
    auto next_k = [&]() {
      if (ik >= i1) return;
      if (jk == 0) {
        wk = packed_work(a, ik);
        const int b = n & 1;
        ok = ok && warp_wait(Ly::bQEmpty + b, ((n >> 1) & 1) ^ 1, 201);
        if (!ok) return;
        if (lane == 0) mbar_arrive_expect_tx(&bars[Ly::bQFull + b], q_bytes);
        __syncwarp();
        if (lane < Ly::kHalves)
          tma_load_3d(sm + Ly::oQ + b * Ly::kTileBytes + lane * 16384, &tm_q, &bars[Ly::bQFull + b], lane * 64,
                      wk.kvh * a.group, wk.row0 + wk.t0);
        __syncwarp();
        ++n;
      }
      load(Ly::bKFull, Ly::bKEmpty, Ly::kKStages, Ly::oK, &tm_k, wk, jk, gk);
      if (!ok) return;
      ++gk;
      if (++jk == wk.blocks) {
        jk = 0;
        ++ik;
      }
    };
    for (int e = 0; e < kAhead && ok; ++e) next_k();
    while (iv < i1 && ok) {
      next_k();
      if (!ok) break;
      if (jv == 0) wv = packed_work(a, iv);
      load(Ly::bVFull, Ly::bVEmpty, Ly::kVStages, Ly::oV, &tm_v, wv, jv, gv);
      if (!ok) break;
      ++gv;
      if (++jv == wv.blocks) {
        jv = 0;
        ++iv;
      }
    }
    // every load of this warp lands before the CTA exits (some are left only after a failed wait)
    if (lane == 0) {
      for (uint32_t s = 0; s < Ly::kKStages && s < gk; ++s)
        packed_wait(&bars[Ly::bKFull + (gk - 1 - s) % Ly::kKStages], ((gk - 1 - s) / Ly::kKStages) & 1, ctl, 203, true);
      for (uint32_t s = 0; s < Ly::kVStages && s < gv; ++s)
        packed_wait(&bars[Ly::bVFull + (gv - 1 - s) % Ly::kVStages], ((gv - 1 - s) / Ly::kVStages) & 1, ctl, 204, true);
      for (int s = 0; s < 2 && s < n; ++s)
        packed_wait(&bars[Ly::bQFull + ((n - 1 - s) & 1)], ((n - 1 - s) >> 1) & 1, ctl, 205, true);
    }
    __syncwarp();
  } else if (warp == 9) {
    // ============================================================ S issuer (one elected thread)
    // A thread takes about 80 cycles to issue a product whatever its N, and one of 128 x 128 x 16 runs for 64, so
    // S and P.V have an issuer each.  The whole warp walks the items with values made uniform by a shuffle, and
    // only the products and commits are the elected thread's: their descriptors then live in uniform registers
    // (with the walk itself inside `lane == 0` a product took about 130 cycles).
    const uint32_t q_desc = __shfl_sync(0xffffffffu, umma_desc_lo(smem_u32(sm + Ly::oQ)), 0);
    const uint32_t k_desc = __shfl_sync(0xffffffffu, umma_desc_lo(smem_u32(sm + Ly::oK)), 0);
    uint32_t g = 0;
    int n = 0;
    bool ok = true;
    for (int i = i0; i < i1 && ok; ++i, ++n) {
      const PackedWork w = packed_work(a, i);
      ok = warp_wait(Ly::bQFull + (n & 1), (n >> 1) & 1, 211);
      const uint32_t ad = q_desc + (n & 1) * (Ly::kTileBytes >> 4);
      for (int j = 0; j < w.blocks && ok; ++j, ++g) {
        const uint32_t st = g % Ly::kKStages, sb = g & 1;
        ok = warp_wait(Ly::bKFull + st, (g / Ly::kKStages) & 1, 212);
        ok = ok && warp_wait(Ly::bSEmpty + sb, ((g >> 1) & 1) ^ 1, 213);
        if (!ok) break;
        tc_fence_after();
        const uint32_t idesc = umma_idesc_bf16(128, min(128, (w.keys - 128 * j + 15) & ~15), 0, 0);
        const uint32_t bd = k_desc + st * (Ly::kTileBytes >> 4);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
            umma_ss(tmem + sb * 128, umma_desc(ad + off, 16), umma_desc(bd + off, 16), idesc, kk > 0 ? 1u : 0u);
          }
          umma_commit(&bars[Ly::bSFull + sb]);
          umma_commit(&bars[Ly::bKEmpty + st]);
          if (j == w.blocks - 1) umma_commit(&bars[Ly::bQEmpty + (n & 1)]);
        }
        __syncwarp();
      }
    }
    if (elect_one()) {
      umma_commit(&bars[Ly::bDone]);
      packed_wait(&bars[Ly::bDone], 0, ctl, 214, true);
    }
    __syncwarp();
  } else if (warp == 10) {
    // ============================================================ P.V issuer (one elected thread)
    constexpr uint32_t kIdesc = umma_idesc_bf16(128, D, 0, 1);
    const uint32_t v_desc = __shfl_sync(0xffffffffu, umma_desc_lo(smem_u32(sm + Ly::oV)), 0);
    uint32_t g = 0;
    int n = 0;
    bool ok = true;
    for (int i = i0; i < i1 && ok; ++i, ++n) {
      const PackedWork w = packed_work(a, i);
      for (int j = 0; j < w.blocks && ok; ++j, ++g) {
        const uint32_t st = g % Ly::kVStages, sb = g & 1;
        ok = warp_wait(Ly::bVFull + st, (g / Ly::kVStages) & 1, 221);
        const int left = w.len - 128 * j;  // rows of the block inside the sequence
        if (ok && left < 128 && (left & 15) != 0) {
          uint8_t* v = sm + Ly::oV + st * Ly::kTileBytes + left * 128;
          const int chunks = (((left + 15) & ~15) - left) * 8;
          for (int e = lane; e < Ly::kHalves * chunks; e += 32) {
            const int hh = e / chunks;
            *reinterpret_cast<uint4*>(v + hh * 16384 + (e - hh * chunks) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (j == 0) ok = ok && warp_wait(Ly::bOEmpty, (n & 1) ^ 1, 222);
        ok = ok && warp_wait(Ly::bPFull + sb, (g >> 1) & 1, 223);
        if (!ok) break;
        tc_fence_after();
        const int steps = min(8, (w.keys - 128 * j + 15) >> 4);
        const uint32_t bd = v_desc + st * (Ly::kTileBytes >> 4);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            if (kk >= steps) break;
            umma_ts(tmem + kPackedO, tmem + kPackedP + sb * 64 + kk * 8, umma_desc(bd + kk * 128, 16384), kIdesc,
                    (j > 0 || kk > 0) ? 1u : 0u);
          }
          umma_commit(&bars[Ly::bPEmpty + sb]);
          umma_commit(&bars[Ly::bVEmpty + st]);
          if (j == w.blocks - 1) umma_commit(&bars[Ly::bOFull]);
        }
        __syncwarp();
      }
    }
    if (elect_one()) {
      umma_commit(&bars[Ly::bDone + 1]);
      packed_wait(&bars[Ly::bDone + 1], 0, ctl, 224, true);
    }
    __syncwarp();
  } else {
    // ============================================================ softmax and epilogue: one thread per row
    const int x = warp >> 2, r = threadIdx.x & 127;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_col = t_lane + x * 128, p_col = t_lane + kPackedP + x * 64, o_col = t_lane + kPackedO;
    const float cl = a.scale_log2;
    float* max_s = reinterpret_cast<float*>(sm + Ly::oMax);
    float2* sum_s = reinterpret_cast<float2*>(sm + Ly::oSum);
    uint32_t g = 0;  // blocks so far, of both groups

    // Once a wait of the CTA has given up, nothing that follows is worth storing: both groups look at the abort flag
    // before they store or rescale and at the end of an item, and leave.  Until then every wait that is not ready
    // returns at its first look, a few microseconds a block.  (A look in every block: 378 -> 386 us on the ragged D = 64
    // batch; these 381.)
    const auto gave_up = [&]() { return __any_sync(0xffffffffu, *abort_flag != 0) != 0; };
    // (what little lives through the block loop is recomputed or packed: a row of scores leaves 40 registers)
    // item n - 1 is complete: this group's half of its O columns, over both groups' sums
    int pending = 0;  // 0: stored; 1 + parity of its last block
    auto epilogue = [&](int n) {
      const bool odd = pending == 2;
      pending = 0;
      const PackedWork last = packed_work(a, i0 + n - 1);
      const int tl = r / a.group, hl = r - tl * a.group;  // token and head of the row inside the item
      const int tok = last.t0 + tl;
      const bool live = tl < a.tile_tokens && tok < last.len;
      packed_wait(&bars[Ly::bSum], (n - 1) & 1, ctl, 232);
      const float2* sums = sum_s + ((n - 1) & 1) * 256;
      const float2 s0 = sums[r], s1 = sums[128 + r];
      packed_wait(&bars[Ly::bOFull], (n - 1) & 1, ctl, 233);
      if (gave_up()) return;
      tc_fence_after();
      // O is relative to the maximum after the last block; a group without blocks has sum 0
      const float m = odd ? s1.y : s0.y;
      const float sum = (s0.x == 0.0f ? 0.0f : s0.x * ex2_approx(s0.y - m)) + (s1.x == 0.0f ? 0.0f : s1.x * ex2_approx(s1.y - m));
      const float rl = 1.0f / sum;
      uint16_t* dst = a.out + (static_cast<int64_t>(last.row0) + tok) * a.out_ld +
                      static_cast<int64_t>(last.kvh * a.group + hl) * a.out_hd + x * (D / 2);
#pragma unroll
      for (int c0 = 0; c0 < D / 2; c0 += 16) {
        float o[16];
        tmem_ld16(o_col + x * (D / 2) + c0, o);
        tmem_wait_ld();
        if (live) {
#pragma unroll
          for (int e = 0; e < 16; e += 8) {
            U128 v;
            v.x = pack_bf16x2(o[e] * rl, o[e + 1] * rl);
            v.y = pack_bf16x2(o[e + 2] * rl, o[e + 3] * rl);
            v.z = pack_bf16x2(o[e + 4] * rl, o[e + 5] * rl);
            v.w = pack_bf16x2(o[e + 6] * rl, o[e + 7] * rl);
            *reinterpret_cast<U128*>(dst + c0 + e) = v;
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&bars[Ly::bOEmpty]);  // also: the sums are read
    };

    for (int i = i0; i < i1; ++i) {
      const PackedWork w = packed_work(a, i);
      const int tl = r / a.group, tok = w.t0 + tl;
      // the row sees keys [0, seen); rows that are not stored see all and never vote
      const int seen = !(tl < a.tile_tokens && tok < w.len) ? kAllKeys : a.causal ? tok + 1 : w.len;
      float l[4], lm = 0.0f;  // this group's partial sums, relative to lm
#pragma unroll
      for (int q = 0; q < 4; ++q) l[q] = 0.0f;
      for (int j = 0; j < w.blocks; ++j, ++g) {
        if ((g & 1) != static_cast<uint32_t>(x)) continue;
        const uint32_t use = (g >> 1) & 1;  // parity of this use of the group's S and P buffers
        const int cols = min(128, w.keys - 128 * j), lim = seen - 128 * j;
        const bool masked = (a.causal ? w.t0 + 1 : w.len) - 128 * j < 128;  // some row does not see all of them
        packed_wait(&bars[Ly::bSFull + x], use, ctl, 234);
        tc_fence_after();
        // the whole row of S in registers; columns past `cols` hold older scores and are masked
        float s[128];
        auto load_row = [&]() {
#pragma unroll
          for (int c0 = 0; c0 < 128; c0 += 32) tmem_ld32(s_col + c0, s + c0);
          tmem_wait_ld();
          if (masked) {
#pragma unroll
            for (int e = 0; e < 128; ++e)
              if (e >= lim) s[e] = -INFINITY;
          }
        };
        load_row();
        // the row's largest logit, NaN where it holds a NaN (max.f32 would drop it)
        float mx[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) mx[q] = max3_nan(s[3 * q], s[3 * q + 1], s[3 * q + 2]);
#pragma unroll
        for (int e = 12; e < 124; e += 8) {
#pragma unroll
          for (int q = 0; q < 4; ++q) mx[q] = max3_nan(mx[q], s[e + 2 * q], s[e + 2 * q + 1]);
        }
        mx[0] = max3_nan(mx[0], s[124], s[125]);
        mx[1] = max3_nan(mx[1], s[126], s[127]);
        const float t = max3_nan(max3_nan(mx[0], mx[1], mx[2]), mx[3], mx[3]) * cl;
        // the maximum the block before left; raised where this block exceeds it (each row by its own scores only)
        if (g > 0) packed_wait(&bars[Ly::bMax + ((g - 1) & 1)], ((g - 1) >> 1) & 1, ctl, 235);
        const float before = max_s[((g - 1) & 1) * 128 + r];
        const bool raise = j > 0 && before == before && !(t <= before + kPackedRescale);
        const float m = (j == 0 || raise) ? t : before;
        max_s[(g & 1) * 128 + r] = m;
        mbar_arrive(&bars[Ly::bMax + (g & 1)]);
        if (__any_sync(0xffffffffu, seen != kAllKeys && raise)) {
          // O must hold every block before this one, which may be waiting for this group's part of the last epilogue
          if (pending) epilogue(i - i0);
          packed_wait(&bars[Ly::bPEmpty + x], use ^ 1, ctl, 238);  // two blocks back, so that the next parity is the last block's
          packed_wait(&bars[Ly::bPEmpty + ((g - 1) & 1)], ((g - 1) >> 1) & 1, ctl, 236);
          if (gave_up()) break;
          tc_fence_after();
          const float f = raise ? ex2_approx(before - m) : 1.0f;
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 16) {
            float o[16];
            tmem_ld16(o_col + c0, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] *= f;
            tmem_st16(o_col + c0, o);
          }
          load_row();  // once more: the registers were needed here
        }
        tc_fence_before();
        mbar_arrive(&bars[Ly::bSEmpty + x]);  // the buffer is free for the group's next block
        if (j >= 2 && lm != m) {  // raised here, or by the other group since
          const float f = ex2_approx(lm - m);
#pragma unroll
          for (int q = 0; q < 4; ++q) l[q] *= f;
        }
        lm = m;
        // weights of 32 keys, their sum, and P, once the product two blocks back has read this buffer
        const float nm = m == -INFINITY ? 0.0f : -m;  // every score so far -inf: all weights zero
        auto keys32 = [&](int c0) {
#pragma unroll
          for (int e = c0; e < c0 + 32; e += 2) {
            fma2(s[e], s[e + 1], s[e], s[e + 1], cl, cl, nm, nm);
            s[e] = ex2_approx(s[e]);
            s[e + 1] = ex2_approx(s[e + 1]);
          }
#pragma unroll
          for (int e = c0; e < c0 + 32; e += 2)
            add2(l[e & 3], l[(e & 3) + 1], l[e & 3], l[(e & 3) + 1], s[e], s[e + 1]);
          uint32_t p[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) p[e] = pack_bf16x2(s[c0 + 2 * e], s[c0 + 2 * e + 1]);
          if (c0 == 0) {
            packed_wait(&bars[Ly::bPEmpty + x], use ^ 1, ctl, 237);
            tc_fence_after();
          }
          tmem_st16(p_col + c0 / 2, reinterpret_cast<const float*>(p));
        };
        keys32(0);
        if (cols > 32) keys32(32);
        if (cols > 64) keys32(64);
        if (cols > 96) keys32(96);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bars[Ly::bPFull + x]);
        if (pending) epilogue(i - i0);  // the item before: its last product has run meanwhile, and this item's wait for it
      }
      if (gave_up()) break;
      if (pending) epilogue(i - i0);  // no block of this item was this group's
      sum_s[((i - i0) & 1) * 256 + x * 128 + r] =
          make_float2((l[0] + l[1]) + (l[2] + l[3]), lm);
      mbar_arrive(&bars[Ly::bSum]);
      pending = 1 + ((g - 1) & 1);
    }
    if (pending) epilogue(i1 - i0);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace vsa
