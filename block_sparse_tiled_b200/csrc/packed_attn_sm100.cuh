// Attention over packed whole prompts on sm_100a: sequences of different lengths end to end, grouped heads,
// causal or not.
//     o_i = sum_j p_ij v_j,   p_ij = softmax_j(scale q_i . k_j),   j over i's own sequence (j <= i if causal)
// The Hq / Hk = g query heads that share a key head are computed together: a tile of 128 query rows is
// floor(128 / g) tokens times those g heads (row = token * g + head), so K and V are read once for all of
// them and the causal diagonal of a tile stays narrow.  A work item is two such tiles, A and B, of one key
// head: consecutive tokens of one sequence, walking its keys 128 at a time:
//     S_X [128 rows x 128 keys] = Q_X (K-major) * K_blk^T          fp32 in TMEM
//     O_X [128 rows x D]       += P_X (bf16, TMEM) * V_blk          fp32 in TMEM
// P_X overwrites the columns of S_X, so the two tiles' S and O fill TMEM's 512 columns exactly, and while
// one tile's softmax runs the tensor core works for the other.  One thread issues every product, in order:
// P_X.V_j, then S_X of block j + 1 into the columns that product has just read.  Products cover only the
// keys a tile can see, rounded up to 16 (the last block's K-steps and columns are cut), and blocks past
// the causal limit of a tile are not visited.
//
// The softmax of tile X runs in one warpgroup, one thread per query row.  The running maximum is kept
// lazily: a block is exponentiated against the current maximum m, which is raised (O and the sum rescaled)
// only when a logit exceeds it by more than kPackedRescale (log2 units): any m without overflow gives the
// same softmax.  The sum is binary32 over the unrounded probabilities; P is rounded to bf16, the tensor
// core's operand type (relative 2^-8 on every weight, averaged over the row).
//
// The items of each CTA are listed by the plan, longest first, balanced over the SMs on the host: no work
// counter, so nothing is shared between calls but the status word that a failed wait sets.
//
// A key block may end inside another sequence or past the tensor.  Keys there are masked in S; values there
// meet zero weights, but 0 * NaN is NaN, so a helper warp overwrites the up to 15 value rows between a
// sequence's end and the next multiple of 16 with zeros before the product may read them.
//
// Roles (384 threads): warps 0..3 softmax and epilogue of tile A, 4..7 of tile B, 8 TMA producer, 9 issuer
// and TMEM owner, 10 value rows past a sequence's end, 11 idle.  Every mbarrier wait is bounded (ptx.cuh).
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

constexpr int kPackedThreads = 384;
constexpr float kPackedRescale = 8.0f;
constexpr uint32_t kPackedS = 0, kPackedO = 256;  // TMEM columns: S_A, S_B, O_A, O_B, 128 each

template <int D>
struct PackedLayout {
  static constexpr int kHalves = (D + 63) / 64;          // 64-column halves of a row (D = 96: two)
  static constexpr int kTileBytes = kHalves * 128 * 128;  // 128 rows of one operand
  static constexpr int kStages = D == 64 ? 8 : 5;         // ring of K and V blocks, in order of use
  static constexpr int oQ = 0;
  static constexpr int oKV = oQ + 2 * kTileBytes;
  static constexpr int oBar = oKV + kStages * kTileBytes;
  static constexpr int bQFull = 0, bQEmpty = 2, bSFull = 4, bPFull = 6, bOFull = 8, bDone = 10;
  static constexpr int bFull = 11, bEmpty = bFull + kStages, bRaw = bEmpty + kStages;
  static constexpr int kNumBars = bRaw + kStages;
  static constexpr int oMisc = oBar + kNumBars * 8;  // TMEM base, abort flag
  static constexpr int oEnd = oMisc + 8;
  static size_t bytes() { return 1024 /*alignment slack*/ + oEnd; }
};

__device__ __forceinline__ void tma_load_3d(void* dst, const void* tmap, uint64_t* bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(tmap), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// What every role derives from an item: the keys each tile can see (0: the tile has no tokens) and blocks.
struct PackedSpan {
  int keys[2], blocks[2], n;
};
__device__ __forceinline__ PackedSpan packed_span(const PackedItem& it, const PackedArgs& a) {
  PackedSpan s;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int t = it.t0 + x * a.tile_tokens;
    s.keys[x] = t >= it.len ? 0 : a.causal ? min(it.len, t + a.tile_tokens) : it.len;
    s.blocks[x] = (s.keys[x] + 127) >> 7;
  }
  s.n = max(s.blocks[0], s.blocks[1]);
  return s;
}
// The last value block of an item holds rows past the sequence's end that a product would read.
__device__ __forceinline__ bool packed_ragged(const PackedItem& it, int n) {
  return 128 * n > it.len && (it.len & 15) != 0;
}

template <int D>
__global__ void __launch_bounds__(kPackedThreads, 1)
    packed_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const PackedArgs a) {
  using Ly = PackedLayout<D>;
  constexpr int kStages = Ly::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Ly::oBar);
  uint32_t* tmem_base_s = reinterpret_cast<uint32_t*>(sm + Ly::oMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + Ly::oMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtl ctl{abort_flag, a.status, kWaitTimeoutNs};
  const int i0 = __ldg(a.first + blockIdx.x), i1 = __ldg(a.first + blockIdx.x + 1);
  auto item_at = [&](int i) -> PackedItem {
    const int4 v = __ldg(reinterpret_cast<const int4*>(a.items) + i);
    return PackedItem{v.x, v.y, v.z, v.w};
  };

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < Ly::kNumBars; ++i) {
      const bool p = i == Ly::bPFull || i == Ly::bPFull + 1;
      mbar_init(&bars[i], p ? 128 : 1);
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
  const uint32_t tmem = *tmem_base_s;

  if (warp == 8) {
    // ============================================================ TMA producer (one thread)
    if (lane == 0) {
      const uint32_t q_bytes = static_cast<uint32_t>(Ly::kHalves * 128 * a.group * a.tile_tokens);
      uint32_t c = 0, qn[2] = {0, 0}, raw_parity = 0, last_raw = 0;
      bool ok = true;
      auto load_q = [&](const PackedItem& it, int x) {
        ok = ok && mbar_wait(&bars[Ly::bQEmpty + x], (qn[x] & 1) ^ 1, ctl, 201);
        if (!ok) return;
        mbar_arrive_expect_tx(&bars[Ly::bQFull + x], q_bytes);
        for (int hh = 0; hh < Ly::kHalves; ++hh)
          tma_load_3d(sm + Ly::oQ + x * Ly::kTileBytes + hh * 16384, &tm_q, &bars[Ly::bQFull + x], hh * 64,
                      it.kvh * a.group, it.row0 + it.t0 + x * a.tile_tokens);
        ++qn[x];
      };
      auto load_kv = [&](const PackedItem& it, const void* map, int j, bool raw) {
        const int st = c % kStages;
        ok = ok && mbar_wait(&bars[Ly::bEmpty + st], ((c / kStages) & 1) ^ 1, ctl, 202);
        if (!ok) return;
        uint64_t* bar = &bars[(raw ? Ly::bRaw : Ly::bFull) + st];
        mbar_arrive_expect_tx(bar, Ly::kTileBytes);
        for (int hh = 0; hh < Ly::kHalves; ++hh)
          tma_load_3d(sm + Ly::oKV + st * Ly::kTileBytes + hh * 16384, map, bar, hh * 64, it.kvh, it.row0 + 128 * j);
        last_raw = (last_raw & ~(1u << st)) | (raw ? 1u << st : 0u);
        if (raw) raw_parity ^= 1u << st;
        ++c;
      };
      for (int i = i0; i < i1 && ok; ++i) {
        const PackedItem it = item_at(i);
        const PackedSpan sp = packed_span(it, a);
        const bool ragged = packed_ragged(it, sp.n);
        load_q(it, 0);
        load_kv(it, &tm_k, 0, false);
        if (sp.blocks[1] > 0) load_q(it, 1);
        for (int j = 0; j < sp.n && ok; ++j) {
          load_kv(it, &tm_v, j, ragged && j == sp.n - 1);
          if (j + 1 < sp.n) load_kv(it, &tm_k, j + 1, false);
        }
      }
      // every load this thread issued lands before the CTA exits (only after a failed wait are some left)
      for (uint32_t s = 0; s < kStages && s < c; ++s) {
        const uint32_t u = c - 1 - s, st = u % kStages;
        if ((last_raw >> st) & 1u)
          mbar_wait_drain(&bars[Ly::bRaw + st], ((raw_parity >> st) & 1u) ^ 1u, ctl, 203);
        else
          mbar_wait_drain(&bars[Ly::bFull + st], (u / kStages) & 1, ctl, 203);
      }
      for (int x = 0; x < 2; ++x)
        if (qn[x] > 0) mbar_wait_drain(&bars[Ly::bQFull + x], (qn[x] - 1) & 1, ctl, 204);
    }
    __syncwarp();
  } else if (warp == 9) {
    // ============================================================ issuer (one thread)
    if (lane == 0) {
      uint32_t c = 0, qn[2] = {0, 0}, pn[2] = {0, 0};
      bool ok = true;
      auto issue_s = [&](int x, int j, int blocks, int keys, uint32_t kst) {
        const int cols = min(128, (keys - 128 * j + 15) & ~15);
        const uint32_t idesc = umma_idesc_bf16(128, cols, 0, 0);
        const uint64_t ad = umma_desc_sw128(smem_u32(sm + Ly::oQ + x * Ly::kTileBytes), 16, 1024);
        const uint64_t bd = umma_desc_sw128(smem_u32(sm + Ly::oKV + kst * Ly::kTileBytes), 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t off = static_cast<uint64_t>(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4);
          umma_ss(tmem + kPackedS + x * 128, ad + off, bd + off, idesc, kk > 0 ? 1u : 0u);
        }
        umma_commit(&bars[Ly::bSFull + x]);
        if (j == blocks - 1) umma_commit(&bars[Ly::bQEmpty + x]);
      };
      auto issue_o = [&](int x, int j, int keys, uint32_t vst) {
        constexpr uint32_t kIdesc = umma_idesc_bf16(128, D, 0, 1);
        const int steps = min(8, (keys - 128 * j + 15) >> 4);
        const uint64_t bd = umma_desc_sw128(smem_u32(sm + Ly::oKV + vst * Ly::kTileBytes), 16384, 1024);
        for (int kk = 0; kk < steps; ++kk)
          umma_ts(tmem + kPackedO + x * 128, tmem + kPackedS + x * 128 + kk * 8, bd + static_cast<uint64_t>(kk * 128),
                  kIdesc, (j > 0 || kk > 0) ? 1u : 0u);
      };
      for (int i = i0; i < i1 && ok; ++i) {
        const PackedItem it = item_at(i);
        const PackedSpan sp = packed_span(it, a);
        uint32_t st = c % kStages;
        ok = mbar_wait(&bars[Ly::bFull + st], (c / kStages) & 1, ctl, 211);
        for (int x = 0; x < 2 && ok; ++x) {
          if (sp.blocks[x] == 0) continue;
          ok = mbar_wait(&bars[Ly::bQFull + x], qn[x] & 1, ctl, 212);
          ++qn[x];
          if (!ok) break;
          tc_fence_after();
          issue_s(x, 0, sp.blocks[x], sp.keys[x], st);
        }
        if (!ok) break;
        umma_commit(&bars[Ly::bEmpty + st]);
        ++c;
        for (int j = 0; j < sp.n && ok; ++j) {
          const uint32_t vst = c % kStages, kst = (c + 1) % kStages;
          const bool more = j + 1 < sp.n;
          ok = mbar_wait(&bars[Ly::bFull + vst], (c / kStages) & 1, ctl, 213);
          bool k_here = false;
          for (int x = 0; x < 2 && ok; ++x) {
            if (j >= sp.blocks[x]) continue;
            ok = mbar_wait(&bars[Ly::bPFull + x], pn[x] & 1, ctl, 214);
            ++pn[x];
            if (!ok) break;
            tc_fence_after();
            issue_o(x, j, sp.keys[x], vst);
            if (j == sp.blocks[x] - 1) umma_commit(&bars[Ly::bOFull + x]);
            if (x == 1 || j >= sp.blocks[1]) umma_commit(&bars[Ly::bEmpty + vst]);
            if (j + 1 < sp.blocks[x]) {
              if (!k_here) ok = mbar_wait(&bars[Ly::bFull + kst], ((c + 1) / kStages) & 1, ctl, 215);
              k_here = true;
              if (!ok) break;
              tc_fence_after();
              issue_s(x, j + 1, sp.blocks[x], sp.keys[x], kst);
            }
          }
          if (!ok) break;
          if (more) umma_commit(&bars[Ly::bEmpty + kst]);
          c += more ? 2 : 1;
        }
      }
      umma_commit(&bars[Ly::bDone]);
      mbar_wait_drain(&bars[Ly::bDone], 0, ctl, 216);
    }
    __syncwarp();
  } else if (warp == 10) {
    // ============================================================ zero the value rows past a sequence's end
    uint32_t c = 0, parity = 0;
    for (int i = i0; i < i1; ++i) {
      const PackedItem it = item_at(i);
      const PackedSpan sp = packed_span(it, a);
      c += 2 * sp.n;
      if (!packed_ragged(it, sp.n)) continue;
      const uint32_t st = (c - 1) % kStages;  // the item's last value block
      const bool ok = mbar_wait(&bars[Ly::bRaw + st], (parity >> st) & 1u, ctl, 221);
      parity ^= 1u << st;
      const int from = it.len - 128 * (sp.n - 1), rows = ((from + 15) & ~15) - from;
      uint8_t* v = sm + Ly::oKV + st * Ly::kTileBytes + from * 128;
      for (int e = lane; e < Ly::kHalves * rows * 8 && ok; e += 32) {
        const int hh = e / (rows * 8), o = e - hh * rows * 8;
        *reinterpret_cast<uint4*>(v + hh * 16384 + o * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[Ly::bFull + st]);
    }
  } else if (warp < 8) {
    // ============================================================ softmax and epilogue: one thread per row
    const int x = warp >> 2, r = threadIdx.x & 127;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_col = t_lane + kPackedS + x * 128, o_col = t_lane + kPackedO + x * 128;
    const int tl = r / a.group, hl = r - tl * a.group;  // token and head of the row inside a tile
    const float cl = a.scale_log2;
    uint32_t sn = 0, on = 0;
    for (int i = i0; i < i1; ++i) {
      const PackedItem it = item_at(i);
      const PackedSpan sp = packed_span(it, a);
      const int blocks = sp.blocks[x], keys = sp.keys[x];
      if (blocks == 0) continue;
      const int tok = it.t0 + x * a.tile_tokens + tl;
      const bool live = tl < a.tile_tokens && tok < it.len;
      // the row sees keys [0, seen); rows that are not stored see all and never vote
      const int seen = !live ? 0x40000000 : a.causal ? tok + 1 : it.len;
      float m = 0.0f, l0 = 0.0f, l1 = 0.0f;
      for (int j = 0; j < blocks; ++j, ++sn) {
        const int cols = min(128, keys - 128 * j), lim = seen - 128 * j;
        const bool masked = __any_sync(0xffffffffu, lim < ((cols + 31) & ~31));
        mbar_wait(&bars[Ly::bSFull + x], sn & 1, ctl, 231);
        tc_fence_after();
        float top = -INFINITY;
#pragma unroll
        for (int c0 = 0; c0 < 128; c0 += 32) {
          if (c0 >= cols) break;
          float s[32];
          tmem_ld32(s_col + c0, s);
          tmem_wait_ld();
          if (masked) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (c0 + e >= lim) s[e] = -INFINITY;
          }
#pragma unroll
          for (int e = 0; e < 32; e += 2) top = max3(top, s[e], s[e + 1]);
        }
        const float t = top * cl;
        if (j == 0) {
          m = t;
        } else if (__any_sync(0xffffffffu, live && t > m + kPackedRescale)) {
          // S of this block was committed after the product of the previous one, so O is complete
          const float up = fmaxf(m, t), f = up == m ? 1.0f : ex2_approx(m - up);
          m = up;
          l0 *= f;
          l1 *= f;
#pragma unroll
          for (int c0 = 0; c0 < D; c0 += 16) {
            float o[16];
            tmem_ld16(o_col + c0, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] *= f;
            tmem_st16(o_col + c0, o);
          }
        }
        const float nm = m == -INFINITY ? 0.0f : -m;  // every score so far -inf: all weights zero
#pragma unroll
        for (int c0 = 0; c0 < 128; c0 += 32) {
          if (c0 >= cols) break;
          float s[32];
          tmem_ld32(s_col + c0, s);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; e += 2) fma2(s[e], s[e + 1], s[e], s[e + 1], cl, cl, nm, nm);
          if (masked) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (c0 + e >= lim) s[e] = -INFINITY;
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) s[e] = ex2_approx(s[e]);
#pragma unroll
          for (int e = 0; e < 32; e += 2) add2(l0, l1, l0, l1, s[e], s[e + 1]);
          uint32_t p[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) p[e] = pack_bf16x2(s[2 * e], s[2 * e + 1]);
          // P of these keys goes where S of keys at or before them was
          tmem_st16(s_col + c0 / 2, reinterpret_cast<const float*>(p));
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bars[Ly::bPFull + x]);
      }
      mbar_wait(&bars[Ly::bOFull + x], on & 1, ctl, 232);
      ++on;
      tc_fence_after();
      const float rl = 1.0f / (l0 + l1);
      uint16_t* dst = a.out + (static_cast<int64_t>(it.row0) + tok) * a.out_ld +
                      static_cast<int64_t>(it.kvh * a.group + hl) * a.out_hd;
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += 32) {
        float o[32];
        tmem_ld32(o_col + c0, o);
        tmem_wait_ld();
        if (live) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            U128 v;
            v.x = pack_bf16x2(o[e] * rl, o[e + 1] * rl);
            v.y = pack_bf16x2(o[e + 2] * rl, o[e + 3] * rl);
            v.z = pack_bf16x2(o[e + 4] * rl, o[e + 5] * rl);
            v.w = pack_bf16x2(o[e + 6] * rl, o[e + 7] * rl);
            *reinterpret_cast<U128*>(dst + c0 + e) = v;
          }
        }
      }
      tc_fence_before();  // O read: ordered before the next item's first P by that P's arrival
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace vsa
