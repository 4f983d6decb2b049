// Row operators of a block around the attention, in sequence order: the root-mean-square norm with the
// residual's addition (vsa_rms_norm), and the head norm and rotary positions of Q and K (vsa_qk_rope).
// Both are bound by HBM traffic: each reads its inputs once and writes its outputs once.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>

#include "status.h"
#include "vsa.h"

namespace {

using vsa::set_error;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

__device__ __forceinline__ void unpack8(const uint4& u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = __uint_as_float(w[j] << 16);
    f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

// Eight values of a bf16 or binary32 row, starting at element 8 * chunk (16-byte aligned).
template <bool kF32>
__device__ __forceinline__ void load8(const void* row, int chunk, float* f) {
  if constexpr (kF32) {
    const float4* p = reinterpret_cast<const float4*>(row) + 2 * chunk;
    const float4 a = p[0], b = p[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else {
    unpack8(reinterpret_cast<const uint4*>(row)[chunk], f);
  }
}

// ---------------------------------------------------------------------------------------------
// vsa_rms_norm.  With t = x + r (binary32):
//   r' = t rounded to the residual's type,   y = t * rsqrt(mean(t^2) + eps) * w,
//   out = y rounded to bf16, or s = max|y| / 448 and out = E4M3(y / s).
// The row stays in registers between the sums and the output, so it is read once.
// max|y| = rsqrt(..) max|t w|, so one reduction gives both the sum of squares and the scale, and the
// codes are E4M3(t w (448 / max|t w|)): the row factor cancels.
// ---------------------------------------------------------------------------------------------
struct NormArgs {
  const uint16_t* x;
  const void* residual;
  const void* weight;
  void* out;
  void* residual_out;
  float* scale;
  int64_t x_ld, res_ld, out_ld, res_out_ld;
  int width;
  float eps;
};

constexpr int kNormThreads = 256;
constexpr int kNormChunks = 8;  // 16384 / 8 / 256: eight-element chunks of a row each thread may hold

template <bool kRes, bool kResF32, bool kWF32, bool kF8>
__global__ void __launch_bounds__(kNormThreads) rms_norm_kernel(const NormArgs a) {
  const int64_t row = blockIdx.x;
  const int chunks = a.width >> 3;
  const uint16_t* x = a.x + row * a.x_ld;
  const uint8_t* res = static_cast<const uint8_t*>(a.residual) + row * a.res_ld * (kResF32 ? 4 : 2);
  uint8_t* res_out = a.residual_out == nullptr
                         ? nullptr
                         : static_cast<uint8_t*>(a.residual_out) + row * a.res_out_ld * (kResF32 ? 4 : 2);
  const auto weight = [&](int c, float* w) {
    if (a.weight != nullptr) {
      load8<kWF32>(a.weight, c, w);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = 1.0f;
    }
  };
  float t[kNormChunks][8];
  float ss = 0.0f, top = 0.0f;
#pragma unroll
  for (int u = 0; u < kNormChunks; ++u) {
    const int c = threadIdx.x + u * kNormThreads;
    if (c >= chunks) break;
    load8<false>(x, c, t[u]);
    if constexpr (kRes) {
      float r[8];
      load8<kResF32>(res, c, r);
#pragma unroll
      for (int e = 0; e < 8; ++e) t[u][e] += r[e];
      if (res_out != nullptr) {
        if constexpr (kResF32) {
          float4* p = reinterpret_cast<float4*>(res_out) + 2 * c;
          p[0] = make_float4(t[u][0], t[u][1], t[u][2], t[u][3]);
          p[1] = make_float4(t[u][4], t[u][5], t[u][6], t[u][7]);
        } else {
          reinterpret_cast<uint4*>(res_out)[c] = pack8(t[u]);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(t[u][e], t[u][e], ss);
    if constexpr (kF8) {
      float w[8];
      weight(c, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(t[u][e] * w[e]));
    }
  }
  __shared__ float2 part[2][kNormThreads / 32];
  const auto reduce = [&](float2* slot, float* sum, float* most) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      *sum += __shfl_xor_sync(0xffffffffu, *sum, off);
      *most = fmaxf(*most, __shfl_xor_sync(0xffffffffu, *most, off));
    }
    if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = make_float2(*sum, *most);
    __syncthreads();
    *sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kNormThreads / 32; ++i) {
      *sum += slot[i].x;
      *most = fmaxf(*most, slot[i].y);
    }
  };
  reduce(part[0], &ss, &top);
  const float n = static_cast<float>(a.width);
  float mean = ss / n + a.eps, unit = 1.0f;
  if (isinf(ss) || mean < 1e-30f) {  // the squares left binary32's range: once more, of the row times 2^-70 or 2^70
    unit = isinf(ss) ? 0x1p-70f : 0x1p70f;
    ss = top = 0.0f;
#pragma unroll
    for (int u = 0; u < kNormChunks; ++u) {
      const int c = threadIdx.x + u * kNormThreads;
      if (c >= chunks) break;
      float w[8];
      weight(c, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        t[u][e] *= unit;
        ss = fmaf(t[u][e], t[u][e], ss);
        top = fmaxf(top, fabsf(t[u][e] * w[e]));
      }
    }
    reduce(part[1], &ss, &top);
    mean = ss / n + a.eps * unit * unit;
  }
  const float rstd = 1.0f / sqrtf(mean);  // of the row as t holds it
  if constexpr (kF8) {
    // rows whose 448 / max would overflow are raised by 2^64 first (exactly)
    const float up = top < 1e-30f ? 0x1p64f : 1.0f;
    const float f = top > 0.0f ? 448.0f / (top * up) : 0.0f;
    if (threadIdx.x == 0) a.scale[row] = top > 0.0f ? top * rstd / 448.0f : isnan(ss) ? ss : 0.0f;
    uint8_t* out = static_cast<uint8_t*>(a.out) + row * a.out_ld;
#pragma unroll
    for (int u = 0; u < kNormChunks; ++u) {
      const int c = threadIdx.x + u * kNormThreads;
      if (c >= chunks) break;
      uint32_t code[2] = {0u, 0u};
      float w[8];
      weight(c, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) t[u][e] = t[u][e] * w[e] * up * f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t two =
            __nv_cvt_float2_to_fp8x2(make_float2(t[u][2 * j], t[u][2 * j + 1]), __NV_SATFINITE, __NV_E4M3);
        code[j >> 1] |= two << (16 * (j & 1));
      }
      reinterpret_cast<uint2*>(out)[c] = make_uint2(code[0], code[1]);
    }
  } else {
    uint16_t* out = static_cast<uint16_t*>(a.out) + row * a.out_ld;
#pragma unroll
    for (int u = 0; u < kNormChunks; ++u) {
      const int c = threadIdx.x + u * kNormThreads;
      if (c >= chunks) break;
      float w[8];
      weight(c, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) t[u][e] = t[u][e] * rstd * w[e];
      reinterpret_cast<uint4*>(out)[c] = pack8(t[u]);
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
  int64_t tokens, pos_rows;
  int heads, kv_heads, n_axes;
  int groups;      // lane groups per token (each takes every groups-th head)
  int tokens_cta;  // tokens per CTA
  float eps;
};

constexpr int kRopeThreads = 256;

template <int D, bool kInter, bool kPosF32>
__global__ void __launch_bounds__(kRopeThreads) qk_rope_kernel(const RopeArgs a, const __grid_constant__ RopeTable tab) {
  constexpr int kPairs = D / 2;
  constexpr int kLanes = D == 64 ? 4 : 8;  // lanes per head row: 16 elements each (D = 96: six of eight)
  extern __shared__ float2 cs[];  // [tokens_cta][kPairs] (cos, sin)
  const int64_t token0 = static_cast<int64_t>(blockIdx.x) * a.tokens_cta;
  for (int i = threadIdx.x; i < a.tokens_cta * kPairs; i += kRopeThreads) {
    const int tl = i / kPairs, p = i - tl * kPairs;
    const int64_t token = token0 + tl;
    if (token >= a.tokens) break;
    const int64_t at = (token % a.pos_rows) * a.n_axes + tab.axis[p];
    const double pos = kPosF32 ? static_cast<double>(static_cast<const float*>(a.positions)[at])
                               : static_cast<double>(static_cast<const int32_t*>(a.positions)[at]);
    const double turn = pos * tab.turns[p];
    float s, c;
    sincospif(2.0f * static_cast<float>(turn - rint(turn)), &s, &c);
    cs[i] = make_float2(c, s);
  }
  __syncthreads();
  const int group = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const int tl = group / a.groups, g = group - tl * a.groups;
  const int64_t token = token0 + tl;
  const bool live = tl < a.tokens_cta && token < a.tokens && lane < D / 16;
  float co[8], si[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int p = kInter ? (e < 4 ? 4 * lane + e : kPairs / 2 + 4 * lane + e - 4) : 8 * lane + e;
    const float2 v = live ? cs[tl * kPairs + p] : make_float2(1.0f, 0.0f);
    co[e] = v.x;
    si[e] = v.y;
  }
  const int all = a.heads + a.kv_heads;
  for (int h0 = 0; h0 < all; h0 += a.groups) {
    const int h = h0 + g;
    const bool on = live && h < all;
    const bool is_k = h >= a.heads;
    const uint16_t* src = is_k ? a.k + token * a.k_ld + (h - a.heads) * a.k_hd : a.q + token * a.q_ld + h * a.q_hd;
    const uint16_t* wt = is_k ? a.k_weight : a.q_weight;
    float x[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = 0.0f;
    if (on) {
      load8<false>(src, lane, x);
      load8<false>(src + D / 2, lane, x + 8);
    }
    float ss = 0.0f;
#pragma unroll
    for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    if (on) {
      if (wt != nullptr) {
        const float rstd = 1.0f / sqrtf(ss / static_cast<float>(D) + a.eps);
        float w[16];
        load8<false>(wt, lane, w);
        load8<false>(wt + D / 2, lane, w + 8);
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] *= rstd * w[e];
      }
      float y[16];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int ia = kInter ? (e < 4 ? 2 * e : 8 + 2 * (e - 4)) : e;
        const int ib = kInter ? ia + 1 : e + 8;
        y[ia] = x[ia] * co[e] - x[ib] * si[e];
        y[ib] = x[ia] * si[e] + x[ib] * co[e];
      }
      uint16_t* dst =
          is_k ? a.k_out + token * a.ko_ld + (h - a.heads) * a.ko_hd : a.q_out + token * a.qo_ld + h * a.qo_hd;
      reinterpret_cast<uint4*>(dst)[lane] = pack8(y);
      reinterpret_cast<uint4*>(dst + D / 2)[lane] = pack8(y + 8);
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

vsa_status check_ptr(const char* what, const void* p) {
  if (p == nullptr) return set_error(VSA_ERR_INVALID_ARG, "%s is NULL", what);
  if (!aligned16(p)) return set_error(VSA_ERR_INVALID_ARG, "%s must be 16-byte aligned", what);
  return VSA_OK;
}

// In place means the same rows: an output that starts where an input starts has its strides.
vsa_status check_alias(const char* what, const void* in, int64_t in_ld, const void* out, int64_t out_ld, int64_t rows,
                       bool same_type) {
  if (in != out || in == nullptr || rows <= 1) return VSA_OK;
  if (!same_type || in_ld != out_ld)
    return set_error(VSA_ERR_INVALID_ARG, "%s: an output in place of an input needs its type and stride", what);
  return VSA_OK;
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
  if (p->out_e4m3) VSA_TRY(check_ptr("scale", p->scale));
  if (res) {
    VSA_TRY(check_ptr("residual", p->residual));
    VSA_TRY(check_stride("residual", p->rows, p->residual_stride, p->width, false));
  }
  if (p->residual_out != nullptr) {
    VSA_TRY(check_ptr("residual_out", p->residual_out));
    VSA_TRY(check_stride("residual_out", p->rows, p->residual_out_stride, p->width, true));
    if (p->residual_out == p->out) return set_error(VSA_ERR_INVALID_ARG, "out and residual_out are the same buffer");
  }
  VSA_TRY(check_alias("out", p->x, p->x_stride, p->out, p->out_stride, p->rows, !p->out_e4m3));
  VSA_TRY(check_alias("out", p->residual, p->residual_stride, p->out, p->out_stride, p->rows,
                      !p->out_e4m3 && !p->residual_f32));
  VSA_TRY(check_alias("residual_out", p->x, p->x_stride, p->residual_out, p->residual_out_stride, p->rows,
                      !p->residual_f32));
  VSA_TRY(check_alias("residual_out", p->residual, p->residual_stride, p->residual_out, p->residual_out_stride, p->rows,
                      true));
  NormArgs a = {p->x,        p->residual,        p->weight,     p->out,
                p->residual_out, p->scale,       p->x_stride,   p->residual_stride,
                p->out_stride,   p->residual_out_stride, p->width, p->eps};
  const auto go = [&](auto kernel) {
    return launch("rms_norm", kernel, static_cast<unsigned>(p->rows), kNormThreads, 0, stream, a);
  };
  const bool wf = p->weight_f32 != 0, f8 = p->out_e4m3 != 0;
  if (!res) {
    if (f8) return wf ? go(rms_norm_kernel<false, false, true, true>) : go(rms_norm_kernel<false, false, false, true>);
    return wf ? go(rms_norm_kernel<false, false, true, false>) : go(rms_norm_kernel<false, false, false, false>);
  }
  if (p->residual_f32) {
    if (f8) return wf ? go(rms_norm_kernel<true, true, true, true>) : go(rms_norm_kernel<true, true, false, true>);
    return wf ? go(rms_norm_kernel<true, true, true, false>) : go(rms_norm_kernel<true, true, false, false>);
  }
  if (f8) return wf ? go(rms_norm_kernel<true, false, true, true>) : go(rms_norm_kernel<true, false, false, true>);
  return wf ? go(rms_norm_kernel<true, false, true, false>) : go(rms_norm_kernel<true, false, false, false>);
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
  VSA_TRY(check_ptr("positions", p->positions));
  const auto check = [&](const char* what, int heads, const void* in, int64_t ld, int64_t hd, const void* out,
                         int64_t old, int64_t ohd, const void* w) -> vsa_status {
    VSA_TRY(check_ptr(what, in));
    VSA_TRY(check_ptr(what, out));
    if (w != nullptr) VSA_TRY(check_ptr(what, w));
    VSA_TRY(check_stride(what, p->tokens, ld, D, false));
    VSA_TRY(check_stride(what, heads, hd, D, false));
    VSA_TRY(check_stride(what, p->tokens, old, D, true));
    VSA_TRY(check_stride(what, heads, ohd, D, true));
    // rows of the output must be disjoint: heads inside a token's stride, or tokens inside a head's
    if (p->tokens > 1 && heads > 1 && old < (heads - 1) * ohd + D && ohd < (p->tokens - 1) * old + D)
      return set_error(VSA_ERR_SHAPE, "%s: the output's rows overlap", what);
    if (in == out && ((p->tokens > 1 && ld != old) || (heads > 1 && hd != ohd)))
      return set_error(VSA_ERR_INVALID_ARG, "%s: an output in place of the input needs its strides", what);
    return VSA_OK;
  };
  VSA_TRY(check("q", p->heads, p->q, p->q_stride, p->q_head_stride, p->q_out, p->q_out_stride, p->q_out_head_stride,
                p->q_weight));
  if (p->kv_heads > 0)
    VSA_TRY(check("k", p->kv_heads, p->k, p->k_stride, p->k_head_stride, p->k_out, p->k_out_stride,
                  p->k_out_head_stride, p->k_weight));
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
  const int lanes = D == 64 ? 4 : 8, per_cta = kRopeThreads / lanes, all = p->heads + p->kv_heads;
  const int rounds = (all + per_cta - 1) / per_cta;
  a.groups = (all + rounds - 1) / rounds;
  a.tokens_cta = std::max(1, per_cta / a.groups);
  const int64_t grid = (p->tokens + a.tokens_cta - 1) / a.tokens_cta;
  const size_t smem = static_cast<size_t>(a.tokens_cta) * (D / 2) * sizeof(float2);
  const auto go = [&](auto kernel) {
    return launch("qk_rope", kernel, static_cast<unsigned>(grid), kRopeThreads, smem, stream, a, r->table);
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
