// Row operators of a block around the attention, in sequence order: the root-mean-square norm with the
// residual's addition (vsa_rms_norm), and the head norm and rotary positions of Q and K (vsa_qk_rope).
// Each reads its inputs once and writes its outputs once.  HBM bounds the norm and the rotary positions of long wide
// sequences; instruction issue bounds the rotary positions at D = 96.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <new>
#include <type_traits>

#include "rows.h"
#include "status.h"
#include "vsa.h"

namespace {

using vsa::set_error;

__device__ __forceinline__ void unpack8(const uint4& u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = __uint_as_float(w[j] << 16);
    f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
}

// Two elements per instruction, each rounded as by the scalar operation (the 8-bit norm of wide rows is bound by issue).
__device__ __forceinline__ void fma2(float* d, float a0, float a1, float b0, float b1, float c0, float c1) {
  asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(d[0]), "=f"(d[1])
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void mul2(float* d, float a0, float a1, float b0, float b1) {
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(d[0]), "=f"(d[1])
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void add2(float* d, float a0, float a1, float b0, float b1) {
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(d[0]), "=f"(d[1])
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
// Largest of three; a NaN wins.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

// ---------------------------------------------------------------------------------------------
// vsa_rms_norm.  With t = x + r (binary32):
//   r' = t rounded to the residual's type,   y = t * rsqrt(mean(t^2) + eps) * w,
//   out = y rounded to bf16, or s = max|y| / 448 and out = E4M3(y / s).
// The row stays in registers between the sums and the output, so it is read once.
// max|y| = rsqrt(..) max|t w|, so one reduction gives both the sum of squares and the scale, and the
// codes are E4M3(t w (448 / max|t w|)): the row factor cancels.
//
// A row is kC chunks of eight elements for each of its threads: one warp's 32 threads for rows of up to 1024
// elements, else a CTA's (a barrier instead of shuffles alone).  The grid is as large as fits the GPU and
// walks the rows, so that the weights are read once into registers and the next row's loads are in flight
// while this one is summed and written.  Bound by HBM where there are rows enough: 75,008 rows of 5376, bf16 residual,
// 8-bit output 433 us = 6.52 TB/s; 14,208 rows without a residual 51 us = 6.0 TB/s; 1537 rows of 5120, binary32
// residual 16.3 us = 5.3 TB/s; one row 2.6 us, the launch.
// ---------------------------------------------------------------------------------------------
struct NormArgs {
  const uint16_t* x;
  const void* residual;
  const void* weight;
  void* out;
  void* residual_out;
  float* scale;
  int64_t x_ld, res_ld, out_ld, res_out_ld;
  int rows, width;
  float eps;
};

enum : int { kNoRes = 0, kResBf16 = 1, kResF32 = 2 };

// Threads of a row at most, by its chunks per thread, and the CTAs per SM to compile for (more of them hold more loads
// in flight, until the registers for them run out: 14,208 rows of 5376 without a residual at 3 chunks 58 us at two
// CTAs, 51 at three, 55 at four; 30,000 bf16-residual rows of 4096 at 2 chunks 155 us at four, 137 at three; 75,008 rows
// of 5376 with a residual at 3 chunks 433 us at two, 509 at three).  Four chunks, the widths above 6144, take one CTA of up
// to 512 threads; a binary32 residual then spills 16 to 32 bytes.  At 1.6e8 elements and widths of 6152 to 16384: without
// a residual 5.4 to 6.2 TB/s (8-bit 4.2 to 5.2), bf16 residual 5.8 to 6.6, binary32 residual 5.5 to 6.3.
template <int kC>
constexpr int kNormThreads = kC == 4 ? 512 : 256;
template <int kC, bool kRes>
constexpr int kNormCtas = kC == 4 ? 1 : kC == 3 ? (kRes ? 2 : 3) : (kRes ? 3 : 4);

template <int kRes, bool kF8, bool kWF32, int kC, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 256 : kNormThreads<kC>, kWarp ? 1 : kNormCtas<kC, kRes != kNoRes>) rms_norm_kernel(const NormArgs a) {
  constexpr int kResWords = kRes == kResF32 ? 2 : 1;  // 16-byte words of a residual chunk
  const int chunks = a.width >> 3;
  const int lanes = kWarp ? 32 : blockDim.x, lane = kWarp ? threadIdx.x & 31 : threadIdx.x;
  const int step = kWarp ? gridDim.x * (blockDim.x >> 5) : gridDim.x;
  int row = kWarp ? blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;

  uint4 xr[kC], rr[kRes ? kC * kResWords : 1];
  const auto load = [&](int64_t row) {
    const uint4* x = reinterpret_cast<const uint4*>(a.x + row * a.x_ld);
    const uint4* r = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.residual) + row * a.res_ld * (2 * kResWords));
#pragma unroll
    for (int u = 0; u < kC; ++u) {
      const int c = lane + u * lanes;
      xr[u] = make_uint4(0u, 0u, 0u, 0u);  // chunks past the row add nothing to its sums
      if (c < chunks) xr[u] = x[c];
      if constexpr (kRes != kNoRes) {
#pragma unroll
        for (int k = 0; k < kResWords; ++k) {
          rr[u * kResWords + k] = make_uint4(0u, 0u, 0u, 0u);
          if (c < chunks) rr[u * kResWords + k] = r[c * kResWords + k];
        }
      }
    }
  };
  if (row < a.rows) load(row);
  // the weights as they are stored: packed bf16 is half the registers, and more CTAs hold more loads in flight
  constexpr int kWWords = kWF32 ? 2 : 1;
  uint4 wr[kC * kWWords];
#pragma unroll
  for (int u = 0; u < kC; ++u) {
    const int c = lane + u * lanes;
#pragma unroll
    for (int k = 0; k < kWWords; ++k) {
      const uint32_t one = kWF32 ? 0x3f800000u : 0x3f803f80u;
      wr[u * kWWords + k] = make_uint4(one, one, one, one);
      if (a.weight != nullptr && c < chunks) wr[u * kWWords + k] = static_cast<const uint4*>(a.weight)[c * kWWords + k];
    }
  }
  const auto weights = [&](int u, float* w) {
    if constexpr (kWF32) {
      const uint4 p = wr[2 * u], q = wr[2 * u + 1];
      const uint32_t v[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = __uint_as_float(v[e]);
    } else {
      unpack8(wr[u], w);
    }
  };
  constexpr int kWarps = kNormThreads<kC> / 32;  // of a row, at most
  __shared__ float2 part[2][kWarps];
  int slot = 0;
  const auto most_of = [](float v) {  // over the warp, of values >= 0 (their bits are in their order, a NaN's above all)
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
  };
  const auto reduce = [&](float* sum, float* most) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) *sum += __shfl_xor_sync(0xffffffffu, *sum, off);
    if constexpr (kF8) *most = most_of(*most);
    if constexpr (!kWarp) {
      // two slots in turn: a slot is written again only behind the barrier that follows its last reads
      if ((threadIdx.x & 31) == 0) part[slot][threadIdx.x >> 5] = make_float2(*sum, *most);
      __syncthreads();
      // every warp adds up the warps' partial sums: lane i reads the (i mod kWarps)-th, if there is one
      const int i = threadIdx.x & (kWarps - 1);
      const float2 v = i < (blockDim.x >> 5) ? part[slot][i] : make_float2(0.0f, 0.0f);
      *sum = v.x;
#pragma unroll
      for (int off = kWarps / 2; off > 0; off >>= 1) *sum += __shfl_xor_sync(0xffffffffu, *sum, off);
      if constexpr (kF8) *most = most_of(v.y);
      slot ^= 1;
    }
  };
  const float n = static_cast<float>(a.width);
  for (; row < a.rows; row = a.rows - row > step ? row + step : a.rows) {  // (rows may be up to 2^31 - 1)
    float t[kC][8];
    float ss = 0.0f, top = 0.0f;
#pragma unroll
    for (int u = 0; u < kC; ++u) {
      unpack8(xr[u], t[u]);
      if constexpr (kRes == kResBf16) {
        float r[8];
        unpack8(rr[u], r);
#pragma unroll
        for (int e = 0; e < 8; e += 2) add2(t[u] + e, t[u][e], t[u][e + 1], r[e], r[e + 1]);
      } else if constexpr (kRes == kResF32) {
        const uint4 p = rr[2 * u], q = rr[2 * u + 1];
        const uint32_t r[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
        for (int e = 0; e < 8; e += 2)
          add2(t[u] + e, t[u][e], t[u][e + 1], __uint_as_float(r[e]), __uint_as_float(r[e + 1]));
      }
    }
    if (a.rows - row > step) load(row + step);
    if constexpr (kRes != kNoRes) {
      if (a.residual_out != nullptr) {
        uint4* ro = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.residual_out) +
                                             static_cast<int64_t>(row) * a.res_out_ld * (2 * kResWords));
#pragma unroll
        for (int u = 0; u < kC; ++u) {
          const int c = lane + u * lanes;
          if (c >= chunks) continue;
          if constexpr (kRes == kResF32) {
            const float* f = t[u];
            ro[2 * c] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
            ro[2 * c + 1] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
          } else {
            ro[c] = pack8(t[u]);
          }
        }
      }
    }
    const auto sums = [&]() {
      float s[2] = {0.0f, 0.0f};
#pragma unroll
      for (int u = 0; u < kC; ++u) {
        float w[8];
        if constexpr (kF8) weights(u, w);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          fma2(s, t[u][e], t[u][e + 1], t[u][e], t[u][e + 1], s[0], s[1]);
          if constexpr (kF8) {
            float p[2];
            mul2(p, t[u][e], t[u][e + 1], w[e], w[e + 1]);
            top = max3(top, fabsf(p[0]), fabsf(p[1]));
          }
        }
      }
      ss = s[0] + s[1];
      reduce(&ss, &top);
    };
    sums();
    float mean = ss / n + a.eps;
    // The squares left binary32's range: once more, of the row times 2^-80 (squares of 16384 values below 2^48 fit) or 2^70.
    if (isinf(ss) || mean < 1e-30f) {
      const float unit = isinf(ss) ? 0x1p-80f : 0x1p70f;
      top = 0.0f;
#pragma unroll
      for (int u = 0; u < kC; ++u) {
#pragma unroll
        for (int e = 0; e < 8; ++e) t[u][e] *= unit;
      }
      sums();
      mean = ss / n + a.eps * unit * unit;
    }
    const float rstd = rsqrtf(mean);  // of the row as t holds it (within 2 ulp)
    if constexpr (kF8) {
      // (an infinite element makes top infinite, or NaN where its weight is 0, and rstd 0: the scale is NaN like max|y|)
      if (lane == 0) a.scale[row] = top == 0.0f ? 0.0f : top * rstd / 448.0f;
      if (top < 1e-30f) {  // 448 / top may overflow: the row is raised by 2^64 (exactly)
        top *= 0x1p64f;
#pragma unroll
        for (int u = 0; u < kC; ++u) {
#pragma unroll
          for (int e = 0; e < 8; ++e) t[u][e] *= 0x1p64f;
        }
      }
      // 448 / top = f + rest
      const float f = top > 0.0f ? 448.0f / top : 0.0f;
      const float rest = f > 0.0f ? fmaf(-f, top, 448.0f) / top : 0.0f;
      uint2* out = reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + row * a.out_ld);
#pragma unroll
      for (int u = 0; u < kC; ++u) {
        const int c = lane + u * lanes;
        uint32_t code[2] = {0u, 0u};
        float w[8];
        weights(u, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // t w (f + rest) with the product's remainder, rounded once: a code is off only where that rounding crosses a
          // tie (1 or 2 codes of 7.9e6; 2 to 8 without the remainders)
          const int i = 2 * j;
          float p[2], q[2];
          mul2(p, t[u][i], t[u][i + 1], w[i], w[i + 1]);
          mul2(q, p[0], p[1], rest, rest);
          fma2(q, fmaf(t[u][i], w[i], -p[0]), fmaf(t[u][i + 1], w[i + 1], -p[1]), f, f, q[0], q[1]);
          fma2(q, p[0], p[1], f, f, q[0], q[1]);
          const uint32_t two = __nv_cvt_float2_to_fp8x2(make_float2(q[0], q[1]), __NV_SATFINITE, __NV_E4M3);
          code[j >> 1] |= two << (16 * (j & 1));
        }
        if (c < chunks) out[c] = make_uint2(code[0], code[1]);
      }
    } else {
      uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + row * a.out_ld);
#pragma unroll
      for (int u = 0; u < kC; ++u) {
        const int c = lane + u * lanes;
        float w[8];
        weights(u, w);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          mul2(t[u] + e, t[u][e], t[u][e + 1], rstd, rstd);
          mul2(t[u] + e, t[u][e], t[u][e + 1], w[e], w[e + 1]);
        }
        if (c < chunks) out[c] = pack8(t[u]);
      }
    }
  }
}

// ---------------------------------------------------------------------------------------------
// vsa_qk_rope.  Per head row x of Q or K: with a weight w first y = x * rsqrt(mean(x^2) + eps) * w; then
// pair p, (a, b) = (y[p], y[p + D/2]) or, interleaved, (y[2p], y[2p + 1]), becomes
//   (a cos - b sin, a sin + b cos),   angle = position[token][axis_p] * f_p.
// The angle is reduced in turns in binary64 (position times f / 2 pi, less the nearest whole number), so
// far positions lose nothing; its sine and cosine are taken once per token and pair, and every head of
// the token uses them from shared memory.
// ---------------------------------------------------------------------------------------------
constexpr int kMaxPairs = 64;
constexpr int kMaxAxes = 4;

struct RopeTable {
  double turns[kMaxPairs];  // f_p / (2 pi)
  uint8_t axis[kMaxPairs];
};

struct RopeArgs {
  const uint16_t *q, *k;
  uint16_t *q_out, *k_out;
  int64_t q_ld, q_hd, k_ld, k_hd, qo_ld, qo_hd, ko_ld, ko_hd;  // token and head strides, elements
  const uint16_t *q_weight, *k_weight;
  const void* positions;
  uint32_t tokens, pos_rows;
  int heads, kv_heads, n_axes;
  int groups;      // lane groups per token (each takes every groups-th head)
  int tokens_cta;  // tokens at a time
  int span;        // how often, per CTA
  float eps;
};

constexpr int kRopeThreads = 256;
// Tokens a CTA takes one after another, their sines computed together (it waits for positions once), and CTAs per SM
// to compile for.  On 56 + 56 heads with the head norm, 75,008 tokens, D = 128, neighbouring pairs / 14,208 tokens,
// D = 96, halves: 705 us (6.1 TB/s) / 117 us (5.2 TB/s).  Issue bounds it (78% of the slots at D = 96), HBM the long
// wide case: with token numbers of 64 bits 729 / 122, with one element per instruction as well 737 / 139.  Measured at
// 729 / 122: two tokens 743 / 127, eight 733 / 124; 80 registers and three CTAs 717 / 129.
constexpr int kRopeSpan = 4, kRopeCtas = 4;

// Lanes per head row, 16 elements each, and head rows side by side in a warp (D = 96: six lanes, five rows).
template <int D>
struct RopeShape {
  static constexpr int kLanes = D / 16, kRows = 32 / kLanes;
};

template <int D, bool kInter, bool kPosF32>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) qk_rope_kernel(const RopeArgs a, const __grid_constant__ RopeTable tab) {
  constexpr int kPairs = D / 2, kLanes = RopeShape<D>::kLanes, kRows = RopeShape<D>::kRows;
  extern __shared__ float2 cs[];  // [span * tokens_cta][kPairs] (cos, sin)
  const int tokens = a.span * a.tokens_cta;  // of this CTA, tokens_cta at a time
  const uint32_t token0 = blockIdx.x * static_cast<uint32_t>(tokens);  // tokens stay below 2^31
  const int wl = threadIdx.x & 31, lane = wl % kLanes;
  const int group = (threadIdx.x >> 5) * kRows + wl / kLanes;
  const int tl = group / a.groups, g = group - tl * a.groups;
  const bool mine = wl < kRows * kLanes && tl < a.tokens_cta;
  const uint32_t all = a.heads + a.kv_heads, heads = a.heads;
  const auto row_at = [](uint32_t token, int64_t ld, uint32_t head, int64_t hd) {
    return static_cast<uint64_t>(token) * static_cast<uint64_t>(ld) + static_cast<uint64_t>(head) * static_cast<uint64_t>(hd);
  };
  uint4 lo, hi;  // this group's next head row, in flight
  const auto load = [&](uint32_t token, uint32_t h) {
    lo = hi = make_uint4(0u, 0u, 0u, 0u);
    if (!mine || h >= all || token >= a.tokens) return;
    const uint16_t* src = h >= heads ? a.k + row_at(token, a.k_ld, h - heads, a.k_hd) : a.q + row_at(token, a.q_ld, h, a.q_hd);
    lo = reinterpret_cast<const uint4*>(src)[lane];
    hi = reinterpret_cast<const uint4*>(src + D / 2)[lane];
  };
  load(token0 + tl, g);
  // while it comes, the sines and cosines of all the CTA's tokens
  for (int i = threadIdx.x; i < tokens * kPairs; i += blockDim.x) {
    const int t = i / kPairs, p = i - t * kPairs;
    if (token0 + t >= a.tokens) break;
    const int64_t row = a.pos_rows == a.tokens ? token0 + t : (token0 + t) % a.pos_rows;
    const int64_t at = row * a.n_axes + tab.axis[p];
    const double pos = kPosF32 ? static_cast<double>(static_cast<const float*>(a.positions)[at])
                               : static_cast<double>(static_cast<const int32_t*>(a.positions)[at]);
    const double turn = pos * tab.turns[p];
    float s, c;
    sincospif(2.0f * static_cast<float>(turn - rint(turn)), &s, &c);
    cs[i] = make_float2(c, s);
  }
  __syncthreads();
  // the sum over the lanes of a head row
  const auto row_sum = [&](float v) {
    if constexpr (kLanes == 6) {
      const int first = wl - lane;
      v += __shfl_sync(0xffffffffu, v, first + (lane + 3) % 6);
      const float u = __shfl_sync(0xffffffffu, v, first + (lane + 1) % 6);
      return (v + u) + __shfl_sync(0xffffffffu, v, first + (lane + 2) % 6);
    } else {
#pragma unroll
      for (int off = kLanes / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
      return v;
    }
  };
  const int rounds = (all + a.groups - 1) / a.groups;
  float co[8], si[8];
  for (int i = 0, s = 0, round = 0; i < a.span * rounds; ++i) {
    const uint32_t token = token0 + s * a.tokens_cta + tl;
    const uint32_t h = round * a.groups + g;
    const bool on = mine && token < a.tokens && h < all, is_k = h >= heads;
    if (round == 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int p = kInter ? (e < 4 ? 4 * lane + e : kPairs / 2 + 4 * lane + e - 4) : 8 * lane + e;
        const float2 v = on ? cs[(s * a.tokens_cta + tl) * kPairs + p] : make_float2(1.0f, 0.0f);
        co[e] = v.x;
        si[e] = v.y;
      }
    }
    uint32_t raw[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    if (++round == rounds) {
      round = 0;
      ++s;
    }
    if (i + 1 < a.span * rounds) load(token0 + s * a.tokens_cta + tl, round * a.groups + g);
    // the row's factors: y = x rstd w (packed weights, unpacked where they are used: 64 registers a thread)
    float rstd = 1.0f;
    uint32_t wt[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) wt[j] = 0x3f803f80u;
    if (a.q_weight != nullptr || a.k_weight != nullptr) {
      const uint16_t* weight = is_k ? a.k_weight : a.q_weight;
      const auto mean_square = [&]() {
        float ss[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < 8; ++j) fma2(ss, low(raw[j]), high(raw[j]), low(raw[j]), high(raw[j]), ss[0], ss[1]);
        return row_sum(ss[0] + ss[1]) * (1.0f / static_cast<float>(D));
      };
      float mean = mean_square(), eps = a.eps;
      const bool far = weight != nullptr && (isinf(mean) || mean + eps < 1e-30f);
      if (__any_sync(0xffffffffu, far)) {  // squares outside binary32's range: once more, of the row times 2^-70 or 2^70
        // (for all lanes of a row alike: six lanes add in different orders, and at the border their sums may disagree)
        const uint32_t row = ((1u << kLanes) - 1) << (wl - lane);
        const bool over = (__ballot_sync(0xffffffffu, isinf(mean)) & row) != 0;
        const float unit = (__ballot_sync(0xffffffffu, far) & row) == 0 ? 1.0f : over ? 0x1p-70f : 0x1p70f;
#pragma unroll
        for (int j = 0; j < 8; ++j) raw[j] = pack2(low(raw[j]) * unit, high(raw[j]) * unit);
        eps = eps * unit * unit;  // (unit squared leaves the range)
        mean = mean_square();
      }
      if (weight != nullptr && on) {
        rstd = rsqrtf(mean + eps);
        const uint4 w0 = reinterpret_cast<const uint4*>(weight)[lane], w1 = reinterpret_cast<const uint4*>(weight + D / 2)[lane];
        wt[0] = w0.x; wt[1] = w0.y; wt[2] = w0.z; wt[3] = w0.w;
        wt[4] = w1.x; wt[5] = w1.y; wt[6] = w1.z; wt[7] = w1.w;
      }
    }
    if (on) {
      uint32_t out[8];
      // two pairs (x, y) at a time: x c - y s and x s + y c
      const auto turn = [&](float* x, float* y, int p) {
        float u[2], v[2];
        mul2(u, y[0], y[1], si[p], si[p + 1]);
        mul2(v, y[0], y[1], co[p], co[p + 1]);
        fma2(y, x[0], x[1], si[p], si[p + 1], v[0], v[1]);
        x[0] = fmaf(x[0], co[p], -u[0]);
        x[1] = fmaf(x[1], co[p + 1], -u[1]);
      };
      const auto norm2 = [&](float* x, float w0, float w1) {
        mul2(x, x[0], x[1], rstd, rstd);
        mul2(x, x[0], x[1], w0, w1);
      };
      if constexpr (kInter) {  // a word holds a pair
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float x[2] = {low(raw[j]), high(raw[j])};
          norm2(x, low(wt[j]), high(wt[j]));
          out[j] = pack2(x[0] * co[j] - x[1] * si[j], x[0] * si[j] + x[1] * co[j]);
        }
      } else {  // word j of the first half and of the second hold two
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float x[2] = {low(raw[j]), high(raw[j])}, y[2] = {low(raw[j + 4]), high(raw[j + 4])};
          norm2(x, low(wt[j]), high(wt[j]));
          norm2(y, low(wt[j + 4]), high(wt[j + 4]));
          turn(x, y, 2 * j);
          out[j] = pack2(x[0], x[1]);
          out[j + 4] = pack2(y[0], y[1]);
        }
      }
      uint16_t* dst =
          is_k ? a.k_out + row_at(token, a.ko_ld, h - heads, a.ko_hd) : a.q_out + row_at(token, a.qo_ld, h, a.qo_hd);
      reinterpret_cast<uint4*>(dst)[lane] = make_uint4(out[0], out[1], out[2], out[3]);
      reinterpret_cast<uint4*>(dst + D / 2)[lane] = make_uint4(out[4], out[5], out[6], out[7]);
    }
  }
}

template <typename K, typename... Args>
vsa_status launch(const char* what, K kernel, unsigned grid, unsigned block, size_t smem, void* stream,
                  const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e != cudaSuccess) return set_error(VSA_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
  return VSA_OK;
}

// As many CTAs as the GPU holds at once.  75,008 rows of 5376, bf16 residual, 8-bit: 432 us; at half of them 572, at 7/8
// 458, at 1.5 times 506, at twice 434 (14,208 rows without a residual: 51; 65, 53, 55, 52).
template <int kRes, bool kF8, bool kWF32, bool kWarp>
vsa_status launch_norm(const NormArgs& a, int per, int threads, int64_t groups, int sms, void* stream) {
  static std::atomic<int> held[4][33];  // CTAs per SM, by chunks per thread and warps; 0: not asked yet
  const auto kernel = kWarp && per == 1 ? rms_norm_kernel<kRes, kF8, kWF32, 1, true>
                      : per == 2 ? rms_norm_kernel<kRes, kF8, kWF32, 2, kWarp>
                      : per == 3 ? rms_norm_kernel<kRes, kF8, kWF32, 3, kWarp>
                                 : rms_norm_kernel<kRes, kF8, kWF32, 4, kWarp>;
  std::atomic<int>& h = held[per - 1][threads / 32];
  int n = h.load(std::memory_order_relaxed);
  if (n == 0) {
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0);
    if (e != cudaSuccess) return set_error(VSA_ERR_CUDA, "rms_norm: %s", cudaGetErrorString(e));
    n = std::max(1, n);
    h.store(n, std::memory_order_relaxed);
  }
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(groups, static_cast<int64_t>(sms) * n));
  return launch("rms_norm", kernel, grid, static_cast<unsigned>(threads), 0, stream, a);
}

// A row stride in elements: a multiple of 8; an output's rows must not overlap.
vsa_status check_stride(const char* what, int64_t rows, int64_t ld, int64_t width, bool output) {
  if (ld < 0 || (ld & 7) != 0)
    return set_error(VSA_ERR_INVALID_ARG, "%s: strides must be non-negative multiples of 8 elements, got %lld", what,
                     static_cast<long long>(ld));
  if (output && rows > 1 && ld < width)
    return set_error(VSA_ERR_SHAPE, "%s: its rows overlap (stride %lld, width %lld)", what, static_cast<long long>(ld),
                     static_cast<long long>(width));
  return VSA_OK;
}

#define VSA_TRY(expr)                 \
  do {                                \
    const vsa_status s_ = (expr);     \
    if (s_ != VSA_OK) return s_;      \
  } while (0)

vsa_status check_ptr(const char* what, const void* p, unsigned align = 16) {
  if (p == nullptr) return set_error(VSA_ERR_INVALID_ARG, "%s is NULL", what);
  if ((reinterpret_cast<uintptr_t>(p) & (align - 1)) != 0)
    return set_error(VSA_ERR_INVALID_ARG, "%s must be %u-byte aligned", what, align);
  return VSA_OK;
}

// An output may lie over an operand only where it replaces an input row for row.
struct Operand {
  const char* name;
  vsa::Rows rows;  // base NULL: not given
};
vsa_status check_overlap(const Operand& out, const Operand& other, bool may_replace) {
  if (out.rows.base == nullptr || other.rows.base == nullptr || (may_replace && vsa::same_rows(out.rows, other.rows)) ||
      !vsa::rows_meet(out.rows, other.rows))
    return VSA_OK;
  return set_error(VSA_ERR_INVALID_ARG, "%s lies over %s%s", out.name, other.name,
                   may_replace ? " but does not replace it row for row (same address, type and strides)" : "");
}

}  // namespace

struct vsa_rope_s {
  int D, interleaved, n_axes;
  double freq[kMaxPairs];
  int32_t axis[kMaxPairs];
  RopeTable table;
};

extern "C" {

vsa_status vsa_rms_norm(const vsa_rms_norm_args* p, void* stream) {
  if (p == nullptr) return set_error(VSA_ERR_INVALID_ARG, "args is NULL");
  if (p->rows < 0 || p->rows > 0x7fffffff)
    return set_error(VSA_ERR_INVALID_ARG, "rows must lie in [0, 2^31), got %lld", static_cast<long long>(p->rows));
  if (p->width < 8 || p->width > 16384 || (p->width & 7) != 0)
    return set_error(VSA_ERR_UNSUPPORTED, "width must be a multiple of 8 in [8, 16384], got %d", p->width);
  for (const int32_t f : {p->residual_f32, p->weight_f32, p->out_e4m3})
    if (f != 0 && f != 1) return set_error(VSA_ERR_INVALID_ARG, "type flags must be 0 or 1");
  if (!(p->eps >= 0.0f) || !std::isfinite(p->eps)) return set_error(VSA_ERR_INVALID_ARG, "eps must be finite and >= 0");
  const bool res = p->residual != nullptr;
  if (!res && p->residual_out != nullptr)
    return set_error(VSA_ERR_INVALID_ARG, "residual_out needs a residual");
  if (p->rows == 0) return VSA_OK;
  VSA_TRY(check_ptr("x", p->x));
  VSA_TRY(check_ptr("out", p->out));
  VSA_TRY(check_stride("x", p->rows, p->x_stride, p->width, false));
  VSA_TRY(check_stride("out", p->rows, p->out_stride, p->width, true));
  if (p->weight != nullptr) VSA_TRY(check_ptr("weight", p->weight));
  if (p->out_e4m3) VSA_TRY(check_ptr("scale", p->scale, 4));
  if (res) {
    VSA_TRY(check_ptr("residual", p->residual));
    VSA_TRY(check_stride("residual", p->rows, p->residual_stride, p->width, false));
  }
  if (p->residual_out != nullptr) {
    VSA_TRY(check_ptr("residual_out", p->residual_out));
    VSA_TRY(check_stride("residual_out", p->rows, p->residual_out_stride, p->width, true));
  }
  const auto rows_of = [&](const char* name, const void* base, int64_t ld, int size) {
    return Operand{name, {base, p->rows, ld * size, 1, 0, static_cast<int64_t>(p->width) * size}};
  };
  const auto flat = [](const char* name, const void* base, int64_t bytes) { return Operand{name, {base, 1, 0, 1, 0, bytes}}; };
  const int res_size = p->residual_f32 ? 4 : 2;
  const Operand x = rows_of("x", p->x, p->x_stride, 2), residual = rows_of("residual", p->residual, p->residual_stride, res_size);
  const Operand weight = flat("weight", p->weight, static_cast<int64_t>(p->width) * (p->weight_f32 ? 4 : 2));
  const Operand out = rows_of("out", p->out, p->out_stride, p->out_e4m3 ? 1 : 2);
  const Operand res_out = rows_of("residual_out", p->residual_out, p->residual_out_stride, res_size);
  const Operand scale = flat("scale", p->out_e4m3 ? p->scale : nullptr, 4 * p->rows);
  for (const Operand* o : {&out, &res_out}) {
    VSA_TRY(check_overlap(*o, x, true));
    VSA_TRY(check_overlap(*o, residual, true));
    VSA_TRY(check_overlap(*o, weight, false));
  }
  VSA_TRY(check_overlap(out, res_out, false));
  for (const Operand* o : {&x, &residual, &weight, &out, &res_out}) VSA_TRY(check_overlap(scale, *o, false));
  NormArgs a = {};
  a.x = p->x;
  a.residual = p->residual;
  a.weight = p->weight;
  a.out = p->out;
  a.residual_out = p->residual_out;
  a.scale = p->scale;
  a.x_ld = p->x_stride;
  a.res_ld = p->residual_stride;
  a.out_ld = p->out_stride;
  a.res_out_ld = p->residual_out_stride;
  a.rows = static_cast<int>(p->rows);
  a.width = p->width;
  a.eps = p->eps;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return set_error(VSA_ERR_CUDA, "rms_norm: %s", cudaGetErrorString(e));
  // Chunks per thread and threads per row: a warp up to 1024 elements; beyond, two to four chunks, for about 256 threads
  // (5376 elements without a residual: 51 us at 3 chunks, 58 at 2, 96 at one; 40,000 rows of 2048: 52.5 us at two
  // chunks, 61.6 at one).  A binary32 residual of 385 to 512 chunks takes three: 30,000 rows of 3080, 3584 and 4096 in
  // 196, 237 and 244 us, at two 201, 232 and 261 (8-bit output 174, 213 and 212; 177, 209 and 242).  Without one, and with
  // a bf16 residual and 8-bit output, two are as good or better at 4096 (77 us, 78 at three; 136, 147).
  const int chunks = p->width / 8;
  const bool warp = chunks <= 128;
  const int wide = res && p->residual_f32 && chunks <= 512 ? 192 : 256;
  const int per = warp ? (chunks + 31) / 32 : std::min(4, std::max(2, (chunks + wide - 1) / wide));
  const int threads = warp ? 256 : ((chunks + per - 1) / per + 31) / 32 * 32;
  const int64_t groups = warp ? (p->rows + 7) / 8 : p->rows;
  const auto go = [&](auto res_c) {
    constexpr int R = decltype(res_c)::value;
    const auto by_weight = [&](auto f8_c, auto wf_c) {
      constexpr bool F = decltype(f8_c)::value, W = decltype(wf_c)::value;
      return warp ? launch_norm<R, F, W, true>(a, per, threads, groups, sms, stream)
                  : launch_norm<R, F, W, false>(a, per, threads, groups, sms, stream);
    };
    const std::true_type yes{};
    const std::false_type no{};
    if (p->out_e4m3) return p->weight_f32 ? by_weight(yes, yes) : by_weight(yes, no);
    return p->weight_f32 ? by_weight(no, yes) : by_weight(no, no);
  };
  if (!res) return go(std::integral_constant<int, kNoRes>{});
  return p->residual_f32 ? go(std::integral_constant<int, kResF32>{}) : go(std::integral_constant<int, kResBf16>{});
}

vsa_status vsa_rope_create(const vsa_rope_desc* d, vsa_rope* out) {
  if (out == nullptr) return set_error(VSA_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (d == nullptr) return set_error(VSA_ERR_INVALID_ARG, "desc is NULL");
  if (d->head_dim != 64 && d->head_dim != 96 && d->head_dim != 128)
    return set_error(VSA_ERR_UNSUPPORTED, "head_dim must be 64, 96 or 128, got %d", d->head_dim);
  if (d->n_axes < 1 || d->n_axes > kMaxAxes)
    return set_error(VSA_ERR_INVALID_ARG, "n_axes must lie in [1, %d], got %d", kMaxAxes, d->n_axes);
  if ((d->interleaved != 0 && d->interleaved != 1) || (d->shared_ladder != 0 && d->shared_ladder != 1))
    return set_error(VSA_ERR_INVALID_ARG, "interleaved and shared_ladder must be 0 or 1");
  if ((d->inv_freq == nullptr) != (d->axis == nullptr))
    return set_error(VSA_ERR_INVALID_ARG, "inv_freq and axis must be both NULL or both set");
  const int pairs = d->head_dim / 2;
  vsa_rope_s r = {};
  r.D = d->head_dim;
  r.interleaved = d->interleaved;
  r.n_axes = d->n_axes;
  if (d->inv_freq != nullptr) {
    for (int i = 0; i < pairs; ++i) {
      if (!std::isfinite(d->inv_freq[i])) return set_error(VSA_ERR_INVALID_ARG, "inv_freq[%d] is not finite", i);
      if (d->axis[i] < 0 || d->axis[i] >= d->n_axes)
        return set_error(VSA_ERR_INVALID_ARG, "axis[%d] = %d is outside [0, %d)", i, d->axis[i], d->n_axes);
      r.freq[i] = d->inv_freq[i];
      r.axis[i] = d->axis[i];
    }
  } else {
    if (d->sections == nullptr) return set_error(VSA_ERR_INVALID_ARG, "sections is NULL");
    if (!(d->theta > 0.0) || !std::isfinite(d->theta)) return set_error(VSA_ERR_INVALID_ARG, "theta must be > 0");
    int at = 0;
    for (int x = 0; x < d->n_axes; ++x) {
      const int n = d->sections[x];
      if (n < 0 || n > pairs - at)
        return set_error(VSA_ERR_SHAPE, "the sections must be non-negative and sum to at most head_dim / 2 = %d", pairs);
      for (int i = 0; i < n; ++i, ++at) {
        const double share = d->shared_ladder ? static_cast<double>(at) / pairs : static_cast<double>(i) / n;
        r.freq[at] = std::pow(d->theta, -share);
        r.axis[at] = x;
      }
    }
  }
  for (int i = 0; i < pairs; ++i) {
    r.table.turns[i] = r.freq[i] / 6.283185307179586476925286766559;
    r.table.axis[i] = static_cast<uint8_t>(r.axis[i]);
  }
  vsa_rope_s* p = new (std::nothrow) vsa_rope_s(r);
  if (p == nullptr) return set_error(VSA_ERR_INVALID_ARG, "out of host memory");
  *out = p;
  return VSA_OK;
}

vsa_status vsa_rope_table(vsa_rope r, double* inv_freq, int32_t* axis) {
  if (r == nullptr) return set_error(VSA_ERR_INVALID_ARG, "rope is NULL");
  for (int i = 0; i < r->D / 2; ++i) {
    if (inv_freq != nullptr) inv_freq[i] = r->freq[i];
    if (axis != nullptr) axis[i] = r->axis[i];
  }
  return VSA_OK;
}

vsa_status vsa_rope_destroy(vsa_rope r) {
  delete r;
  return VSA_OK;
}

vsa_status vsa_qk_rope(vsa_rope r, const vsa_qk_rope_args* p, void* stream) {
  if (r == nullptr) return set_error(VSA_ERR_INVALID_ARG, "rope is NULL");
  if (p == nullptr) return set_error(VSA_ERR_INVALID_ARG, "args is NULL");
  const int D = r->D;
  if (p->tokens < 0 || p->tokens > 0x7fffffff)
    return set_error(VSA_ERR_INVALID_ARG, "tokens must lie in [0, 2^31), got %lld", static_cast<long long>(p->tokens));
  if (p->heads < 1 || p->kv_heads < 0 || p->heads > 65535 || p->kv_heads > 65535)
    return set_error(VSA_ERR_INVALID_ARG, "heads must lie in [1, 65535] and kv_heads in [0, 65535]");
  if (p->positions_f32 != 0 && p->positions_f32 != 1)
    return set_error(VSA_ERR_INVALID_ARG, "positions_f32 must be 0 or 1");
  if (!(p->eps >= 0.0f) || !std::isfinite(p->eps)) return set_error(VSA_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (p->tokens == 0) return VSA_OK;
  if (p->pos_rows < 1 || p->tokens % p->pos_rows != 0)
    return set_error(VSA_ERR_SHAPE, "pos_rows must divide the %lld tokens, got %lld", static_cast<long long>(p->tokens),
                     static_cast<long long>(p->pos_rows));
  VSA_TRY(check_ptr("positions", p->positions, 4));
  const auto rows_of = [&](const char* name, const void* base, int heads, int64_t ld, int64_t hd) {
    return Operand{name, {base, p->tokens, ld * 2, heads, hd * 2, D * 2}};
  };
  const auto check = [&](const char* what, int heads, const void* in, int64_t ld, int64_t hd, const void* out,
                         int64_t old, int64_t ohd, const void* w) -> vsa_status {
    VSA_TRY(check_ptr(what, in));
    VSA_TRY(check_ptr(what, out));
    if (w != nullptr) VSA_TRY(check_ptr(what, w));
    VSA_TRY(check_stride(what, p->tokens, ld, D, false));
    VSA_TRY(check_stride(what, heads, hd, D, false));
    VSA_TRY(check_stride(what, p->tokens, old, D, true));
    VSA_TRY(check_stride(what, heads, ohd, D, true));
    if (!vsa::rows_disjoint(rows_of(what, out, heads, old, ohd).rows))
      return set_error(VSA_ERR_SHAPE, "%s: the output's rows overlap", what);
    return VSA_OK;
  };
  VSA_TRY(check("q", p->heads, p->q, p->q_stride, p->q_head_stride, p->q_out, p->q_out_stride, p->q_out_head_stride,
                p->q_weight));
  if (p->kv_heads > 0)
    VSA_TRY(check("k", p->kv_heads, p->k, p->k_stride, p->k_head_stride, p->k_out, p->k_out_stride,
                  p->k_out_head_stride, p->k_weight));
  {
    const bool with_k = p->kv_heads > 0;
    const auto flat = [](const char* name, const void* base, int64_t bytes) { return Operand{name, {base, 1, 0, 1, 0, bytes}}; };
    const Operand q = rows_of("q", p->q, p->heads, p->q_stride, p->q_head_stride);
    const Operand q_out = rows_of("q_out", p->q_out, p->heads, p->q_out_stride, p->q_out_head_stride);
    const Operand k = rows_of("k", with_k ? p->k : nullptr, p->kv_heads, p->k_stride, p->k_head_stride);
    const Operand k_out = rows_of("k_out", with_k ? p->k_out : nullptr, p->kv_heads, p->k_out_stride, p->k_out_head_stride);
    const Operand shared[] = {flat("q_weight", p->q_weight, 2 * D), flat("k_weight", with_k ? p->k_weight : nullptr, 2 * D),
                              flat("positions", p->positions, p->pos_rows * r->n_axes * 4)};
    VSA_TRY(check_overlap(q_out, q, true));
    VSA_TRY(check_overlap(k_out, k, true));
    VSA_TRY(check_overlap(q_out, k, false));
    VSA_TRY(check_overlap(k_out, q, false));
    VSA_TRY(check_overlap(q_out, k_out, false));
    for (const Operand& o : shared) {
      VSA_TRY(check_overlap(q_out, o, false));
      VSA_TRY(check_overlap(k_out, o, false));
    }
  }
  RopeArgs a = {};
  a.q = p->q;
  a.k = p->k;
  a.q_out = p->q_out;
  a.k_out = p->k_out;
  a.q_ld = p->q_stride;
  a.q_hd = p->q_head_stride;
  a.k_ld = p->k_stride;
  a.k_hd = p->k_head_stride;
  a.qo_ld = p->q_out_stride;
  a.qo_hd = p->q_out_head_stride;
  a.ko_ld = p->k_out_stride;
  a.ko_hd = p->k_out_head_stride;
  a.q_weight = p->q_weight;
  a.k_weight = p->k_weight;
  a.positions = p->positions;
  a.tokens = p->tokens;
  a.pos_rows = p->pos_rows;
  a.heads = p->heads;
  a.kv_heads = p->kv_heads;
  a.n_axes = r->n_axes;
  a.eps = p->eps;
  // the heads of a token go over as many lane groups as share them evenly in the fewest rounds, several tokens to
  // a CTA where one has few heads
  const int rows = D == 64 ? RopeShape<64>::kRows : D == 96 ? RopeShape<96>::kRows : RopeShape<128>::kRows;
  const int per_cta = kRopeThreads / 32 * rows, all = p->heads + p->kv_heads;
  const int rounds = (all + per_cta - 1) / per_cta;
  a.groups = (all + rounds - 1) / rounds;
  a.tokens_cta = std::max(1, per_cta / a.groups);
  const int threads = (a.groups * a.tokens_cta + rows - 1) / rows * 32;
  // a CTA computes the sines of several tokens at once, since it waits for their positions; few tokens: one at a time
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return set_error(VSA_ERR_CUDA, "qk_rope: %s", cudaGetErrorString(e));
  const int64_t turns = (p->tokens + a.tokens_cta - 1) / a.tokens_cta;
  const int64_t sines = static_cast<int64_t>(a.tokens_cta) * (D / 2) * sizeof(float2);  // at most 16 KB
  a.span = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({kRopeSpan, turns / (8 * sms), (48 << 10) / sines})));
  const int64_t grid = (turns + a.span - 1) / a.span;
  const size_t smem = static_cast<size_t>(a.span * sines);
  const auto go = [&](auto kernel) {
    return launch("qk_rope", kernel, static_cast<unsigned>(grid), static_cast<unsigned>(threads), smem, stream, a, r->table);
  };
  const auto by_kind = [&](auto half_i, auto half_f, auto next_i, auto next_f) {
    if (r->interleaved) return p->positions_f32 ? go(next_f) : go(next_i);
    return p->positions_f32 ? go(half_f) : go(half_i);
  };
  if (D == 64)
    return by_kind(qk_rope_kernel<64, false, false>, qk_rope_kernel<64, false, true>, qk_rope_kernel<64, true, false>,
                   qk_rope_kernel<64, true, true>);
  if (D == 96)
    return by_kind(qk_rope_kernel<96, false, false>, qk_rope_kernel<96, false, true>, qk_rope_kernel<96, true, false>,
                   qk_rope_kernel<96, true, true>);
  return by_kind(qk_rope_kernel<128, false, false>, qk_rope_kernel<128, false, true>, qk_rope_kernel<128, true, false>,
                 qk_rope_kernel<128, true, true>);
}

}  // extern "C"
