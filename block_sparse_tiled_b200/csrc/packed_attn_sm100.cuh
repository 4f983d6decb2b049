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
constexpr int kPolyPairs = 1;  // of every four pairs of exponentials, those on the FMA pipe
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

// 2^x of two values with the FMA pipe: 2^floor(x) times a degree-4 polynomial in the remaining fraction
// (least largest relative error on [0, 1] with p(0) = 1, by linear programming: 3.0e-6 evaluated in binary32).
// x <= -127 gives exactly 0, so a weight that has vanished stays exactly nothing; x must stay below 127.
__device__ __forceinline__ void ex2_poly2(float& x0, float& x1) {
  constexpr float kFloor = 12582912.0f;  // 1.5 * 2^23: adding it, rounded down, leaves floor(x) in the low bits
  const float a0 = fmaxf(x0, -127.0f), a1 = fmaxf(x1, -127.0f);
  float t0, t1, f0, f1, p0, p1;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %4};\n\t"
      "add.rm.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(t0), "=f"(t1)
      : "f"(a0), "f"(a1), "f"(kFloor));
  add2(f0, f1, t0, t1, -kFloor, -kFloor);
  fma2(f0, f1, f0, f1, -1.0f, -1.0f, a0, a1);
  fma2(p0, p1, f0, f1, 0.013427376f, 0.013427376f, 0.052241072f, 0.052241072f);
  fma2(p0, p1, p0, p1, f0, f1, 0.24128109f, 0.24128109f);
  fma2(p0, p1, p0, p1, f0, f1, 0.69304466f, 0.69304466f);
  fma2(p0, p1, p0, p1, f0, f1, 1.0f, 1.0f);
  x0 = __uint_as_float(__float_as_uint(p0) + (__float_as_uint(t0) << 23));
  x1 = __uint_as_float(__float_as_uint(p1) + (__float_as_uint(t1) << 23));
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

__device__ __forceinline__ PackedItem uniform_item(const PackedItem& it) {
  return PackedItem{__shfl_sync(0xffffffffu, it.row0, 0), __shfl_sync(0xffffffffu, it.len, 0),
                    __shfl_sync(0xffffffffu, it.t0, 0), __shfl_sync(0xffffffffu, it.kvh, 0)};
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
  const int i0 = __shfl_sync(0xffffffffu, __ldg(a.first + blockIdx.x), 0);
  const int i1 = __shfl_sync(0xffffffffu, __ldg(a.first + blockIdx.x + 1), 0);
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
    // ============================================================ issuer (one elected thread)
    // The whole warp walks the items with values made uniform by a shuffle, and only the products and commits
    // are the elected thread's: their descriptors then live in uniform registers.  With the walk itself inside
    // `lane == 0` every product took about 130 cycles to issue, twice what it takes to run.
    {
      uint32_t c = 0, qn[2] = {0, 0}, pn[2] = {0, 0};
      bool ok = true;
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t q_desc = __shfl_sync(0xffffffffu, umma_desc_lo(smem_u32(sm + Ly::oQ)), 0);
      const uint32_t kv_desc = __shfl_sync(0xffffffffu, umma_desc_lo(smem_u32(sm + Ly::oKV)), 0);
      auto wait = [&](int bar, uint32_t parity, int site) {
        return __shfl_sync(0xffffffffu, static_cast<int>(mbar_wait(&bars[bar], parity, ctl, site)), 0) != 0;
      };
      auto issue_s = [&](int x, int j, int blocks, int keys, uint32_t kst) {
        const int cols = min(128, (keys - 128 * j + 15) & ~15);
        const uint32_t idesc = umma_idesc_bf16(128, cols, 0, 0);
        const uint32_t ad = q_desc + x * (Ly::kTileBytes >> 4), bd = kv_desc + kst * (Ly::kTileBytes >> 4);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
            umma_ss(tm + kPackedS + x * 128, umma_desc(ad + off, 16), umma_desc(bd + off, 16), idesc, kk > 0 ? 1u : 0u);
          }
          umma_commit(&bars[Ly::bSFull + x]);
          if (j == blocks - 1) umma_commit(&bars[Ly::bQEmpty + x]);
        }
        __syncwarp();
      };
      auto issue_o = [&](int x, int j, int blocks, int keys, uint32_t vst, bool last_use) {
        constexpr uint32_t kIdesc = umma_idesc_bf16(128, D, 0, 1);
        const int steps = min(8, (keys - 128 * j + 15) >> 4);
        const uint32_t bd = kv_desc + vst * (Ly::kTileBytes >> 4);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            if (kk >= steps) break;
            umma_ts(tm + kPackedO + x * 128, tm + kPackedS + x * 128 + kk * 8, umma_desc(bd + kk * 128, 16384), kIdesc,
                    (j > 0 || kk > 0) ? 1u : 0u);
          }
          if (j == blocks - 1) umma_commit(&bars[Ly::bOFull + x]);
          if (last_use) umma_commit(&bars[Ly::bEmpty + vst]);
        }
        __syncwarp();
      };
      for (int i = i0; i < i1 && ok; ++i) {
        const PackedItem it = uniform_item(item_at(i));
        const PackedSpan sp = packed_span(it, a);
        const uint32_t st = c % kStages;
        ok = wait(Ly::bFull + st, (c / kStages) & 1, 211);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (!ok || sp.blocks[x] == 0) continue;
          ok = wait(Ly::bQFull + x, qn[x] & 1, 212);
          ++qn[x];
          if (!ok) continue;
          tc_fence_after();
          issue_s(x, 0, sp.blocks[x], sp.keys[x], st);
        }
        if (!ok) break;
        if (elect_one()) umma_commit(&bars[Ly::bEmpty + st]);
        __syncwarp();
        ++c;
        for (int j = 0; j < sp.n && ok; ++j) {
          const uint32_t vst = c % kStages, kst = (c + 1) % kStages;
          const bool more = j + 1 < sp.n;
          ok = wait(Ly::bFull + vst, (c / kStages) & 1, 213);
          bool k_here = false;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (!ok || j >= sp.blocks[x]) continue;
            ok = wait(Ly::bPFull + x, pn[x] & 1, 214);
            ++pn[x];
            if (!ok) continue;
            tc_fence_after();
            issue_o(x, j, sp.blocks[x], sp.keys[x], vst, x == 1 || j >= sp.blocks[1]);
            if (j + 1 < sp.blocks[x]) {
              if (!k_here) ok = wait(Ly::bFull + kst, ((c + 1) / kStages) & 1, 215);
              k_here = true;
              if (!ok) continue;
              tc_fence_after();
              issue_s(x, j + 1, sp.blocks[x], sp.keys[x], kst);
            }
          }
          if (!ok) break;
          if (more) {
            if (elect_one()) umma_commit(&bars[Ly::bEmpty + kst]);
            __syncwarp();
          }
          c += more ? 2 : 1;
        }
      }
      if (elect_one()) {
        umma_commit(&bars[Ly::bDone]);
        mbar_wait_drain(&bars[Ly::bDone], 0, ctl, 216);
      }
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
      float m = 0.0f, l[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) l[q] = 0.0f;
      for (int j = 0; j < blocks; ++j, ++sn) {
        const int cols = min(128, keys - 128 * j), lim = seen - 128 * j;
        const bool masked = __any_sync(0xffffffffu, lim < 128);
        mbar_wait(&bars[Ly::bSFull + x], sn & 1, ctl, 231);
        tc_fence_after();
        // the whole row of S in registers; columns past `cols` hold older scores, masked below
        float s[128];
#pragma unroll
        for (int c0 = 0; c0 < 128; c0 += 32) tmem_ld32(s_col + c0, s + c0);
        tmem_wait_ld();
        if (masked) {
#pragma unroll
          for (int e = 0; e < 128; ++e)
            if (e >= lim) s[e] = -INFINITY;
        }
        float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int e = 4; e < 128; e += 8) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (e + 2 * q + 1 < 128) mx[q] = max3(mx[q], s[e + 2 * q], s[e + 2 * q + 1]);
        }
        const float t = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * cl;
        if (j == 0) {
          m = t;
        } else if (__any_sync(0xffffffffu, live && t > m + kPackedRescale)) {
          // S of this block was committed after the product of the previous one, so O is complete
          const float up = fmaxf(m, t), f = up == m ? 1.0f : ex2_approx(m - up);
          m = up;
#pragma unroll
          for (int q = 0; q < 8; ++q) l[q] *= f;
#pragma unroll 1
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
#pragma unroll
          for (int e = c0; e < c0 + 32; e += 2) {
            fma2(s[e], s[e + 1], s[e], s[e + 1], cl, cl, nm, nm);
            if ((e & 7) >= 8 - 2 * kPolyPairs) {
              ex2_poly2(s[e], s[e + 1]);
            } else {
              s[e] = ex2_approx(s[e]);
              s[e + 1] = ex2_approx(s[e + 1]);
            }
          }
#pragma unroll
          for (int e = c0; e < c0 + 32; e += 2) add2(l[e & 7], l[(e & 7) + 1], l[e & 7], l[(e & 7) + 1], s[e], s[e + 1]);
          uint32_t p[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) p[e] = pack_bf16x2(s[c0 + 2 * e], s[c0 + 2 * e + 1]);
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
      const float rl = 1.0f / (((l[0] + l[1]) + (l[2] + l[3])) + ((l[4] + l[5]) + (l[6] + l[7])));
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
