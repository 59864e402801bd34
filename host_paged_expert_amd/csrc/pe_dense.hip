// HIP kernels of the dense operators around a paged MoE layer (gfx950):
// residual + RMS norm with a bf16 or e4m3 output, top-k routing, and the
// matrix products of the projections, the gated feed-forward block and its
// gradients.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "../../include/pe.h"
#include "pe_dense.h"

namespace pe {

namespace {

__device__ __forceinline__ float bf16_to_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

// fp32 -> bf16 bits, round to nearest even; NaN stays NaN.
__device__ __forceinline__ uint16_t f32_to_bf16(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

__device__ __forceinline__ float e4m3_to_f32(uint8_t c) { return __builtin_amdgcn_cvt_f32_fp8((int)c, 0); }

// fp32 -> OCP e4m3 code, nearest even; callers keep |v| <= 448 (NaN gives the NaN code).
__device__ __forceinline__ uint8_t f32_to_e4m3(float v) {
  return (uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(v, 0.f, 0, false) & 0xFF);
}

constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 1.17549435e-38f;   // 2^-126

// Scale of a group of values whose largest magnitude is `amax`: at least the
// smallest normal number, so that a zero group divides by it.  NaN and
// infinite groups scale by infinity: their values stay NaN.
__device__ __forceinline__ float group_scale(float amax) { return fmaxf(amax / kE4m3Max, kMinScale); }

__device__ __forceinline__ float act_f(float v, int act) {
  if (act == PE_ACT_SILU) return v / (1.f + __expf(-v));
  if (act == PE_ACT_GELU) return 0.5f * v * (1.f + erff(v * 0.70710678f));
  return v;
}

// act'(v)
__device__ __forceinline__ float act_grad_f(float v, int act) {
  if (act == PE_ACT_SILU) {
    const float p = 1.f / (1.f + __expf(-v));
    return p * (1.f + v * (1.f - p));
  }
  return 0.5f * (1.f + erff(v * 0.70710678f)) + v * __expf(-0.5f * v * v) * 0.39894228f;
}

template <int W>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int m = W / 2; m; m >>= 1) v = fmaxf(v, __shfl_xor(v, m));
  return v;
}

}  // namespace

// ------------------------------------------------------------------ RMS norm

// One workgroup per row: v = x + residual, y = v * rsqrt(mean(v^2) + eps) * weight.
__global__ __launch_bounds__(128) void rmsnorm_kernel(NormArgs a) {
  __shared__ float part[2];
  const int64_t t = blockIdx.x;
  const uint16_t* x = a.x + t * a.ldx;
  const uint16_t* r = a.residual ? a.residual + t * a.ldr : nullptr;
  float ss = 0.f;
  for (int i = threadIdx.x; i < a.H; i += 128) {
    const float v = bf16_to_f32(x[i]) + (r ? bf16_to_f32(r[i]) : 0.f);
    ss += v * v;
  }
#pragma unroll
  for (int m = 32; m; m >>= 1) ss += __shfl_xor(ss, m);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = ss;
  __syncthreads();
  const float inv = 1.f / sqrtf((part[0] + part[1]) / (float)a.H + a.eps);
  for (int i0 = 0; i0 < a.H; i0 += 128) {
    const int i = i0 + threadIdx.x;
    const bool in = i < a.H;
    const float v = in ? bf16_to_f32(x[i]) + (r ? bf16_to_f32(r[i]) : 0.f) : 0.f;
    const float y = in ? v * inv * bf16_to_f32(a.weight[i]) : 0.f;
    if (a.sum && in) a.sum[t * a.lds + i] = f32_to_bf16(v);
    if (!a.yscale) {
      if (in) static_cast<uint16_t*>(a.y)[t * a.ldy + i] = f32_to_bf16(y);
      continue;
    }
    __syncthreads();
    const float m = group_max<64>(fabsf(y));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
    const float s = group_scale(fmaxf(part[0], part[1]));
    static_cast<uint8_t*>(a.y)[t * a.ldy + i] = f32_to_e4m3(y / s);
    if (threadIdx.x == 0) a.yscale[t * (a.H / 128) + i0 / 128] = s;
  }
}

void launch_rmsnorm(const NormArgs& a, hipStream_t s) {
  rmsnorm_kernel<<<dim3(a.T), 128, 0, s>>>(a);
}

// ------------------------------------------------------------------ routing

// One wavefront per token, lane l holding experts l, l + 64, ...: k rounds of
// the largest remaining logit (ties to the lowest index).  Logits that are
// -infinity or NaN are never chosen and weigh nothing.
constexpr int kRoutePer = 16;    // 1024 experts / 64 lanes

__global__ __launch_bounds__(64) void route_kernel(RouteArgs a) {
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x;
  const float kNone = -__builtin_inff();
  float v[kRoutePer];
  float mx = kNone;
#pragma unroll
  for (int j = 0; j < kRoutePer; ++j) {
    const int e = lane + 64 * j;
    const float l = e < a.E ? a.logits[t * a.ldl + e] : kNone;
    v[j] = l == l ? l : kNone;
    mx = fmaxf(mx, v[j]);
  }
  mx = group_max<64>(mx);
  // softmax numerator of a logit (1 at the maximum, also where that is +infinity), or its sigmoid
  auto num = [&](float l) {
    if (l == kNone) return 0.f;
    if (a.sigmoid) return 1.f / (1.f + expf(-l));
    return l == mx ? 1.f : expf(l - mx);
  };
  float den = 0.f;
  if (!a.sigmoid) {
#pragma unroll
    for (int j = 0; j < kRoutePer; ++j) den += num(v[j]);
#pragma unroll
    for (int m = 32; m; m >>= 1) den += __shfl_xor(den, m);
  }
  float chosen = 0.f;
  for (int r = 0; r < a.k; ++r) {
    float best = kNone;
    int at = 1 << 30;
#pragma unroll
    for (int j = 0; j < kRoutePer; ++j)
      if (v[j] > best) { best = v[j]; at = lane + 64 * j; }
#pragma unroll
    for (int m = 32; m; m >>= 1) {
      const float ob = __shfl_xor(best, m);
      const int oa = __shfl_xor(at, m);
      if (ob > best || (ob == best && oa < at)) { best = ob; at = oa; }
    }
    const bool found = best > kNone;
    const float p = !found ? 0.f : a.sigmoid ? num(best) : num(best) / den;
    chosen += p;
    if (lane == 0) {
      a.ids[t * a.k + r] = found ? at : -1;
      a.w[t * a.k + r] = p * a.scale;
    }
#pragma unroll
    for (int j = 0; j < kRoutePer; ++j)
      if (at == lane + 64 * j) v[j] = kNone;
  }
  if (a.renorm && chosen > 0.f && lane == 0)
    for (int r = 0; r < a.k; ++r) a.w[t * a.k + r] = a.w[t * a.k + r] / chosen;
}

void launch_route(const RouteArgs& a, hipStream_t s) {
  route_kernel<<<dim3(a.T), 64, 0, s>>>(a);
}

// ------------------------------------------------------------------ matrix products

// A 32 x 128 tile of the output per workgroup, fp32 arithmetic on operands
// staged in LDS 16 values of k at a time; each thread has 4 x 4 outputs.
template <DenseOp OP, bool FP8, bool AK, bool BK>
__global__ __launch_bounds__(256) void dense_kernel(DenseArgs a) {
  constexpr int MT = 32, MN = 128, KB = 16, NB = OP == DENSE_GLU ? 2 : 1;
  __shared__ float sa[KB][MT + 1];
  __shared__ float sb[NB][KB][MN + 1];
  const int t0 = blockIdx.y * MT, n0 = blockIdx.x * MN;
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int64_t nk = a.K / 128;
  auto left = [&](int t, int k) {
    if (t >= a.T || k >= a.K) return 0.f;
    if constexpr (FP8)
      return e4m3_to_f32(static_cast<const uint8_t*>(a.a)[t * a.lda + k]) * a.as[t * nk + k / 128];
    else
      return bf16_to_f32(static_cast<const uint16_t*>(a.a)[AK ? t * a.lda + k : k * a.lda + t]);
  };
  auto right = [&](int n, int k, int part) {
    if (n >= a.N || k >= a.K) return 0.f;
    const int64_t row = (int64_t)part * a.N + n;
    if constexpr (FP8)
      return e4m3_to_f32(static_cast<const uint8_t*>(a.b)[row * a.ldb + k]) * a.bs[(row / 128) * nk + k / 128];
    else
      return bf16_to_f32(static_cast<const uint16_t*>(a.b)[BK ? row * a.ldb + k : k * a.ldb + n]);
  };
  float acc[NB][4][4] = {};
  for (int k0 = 0; k0 < a.K; k0 += KB) {
    for (int i = threadIdx.x; i < KB * MT; i += 256) {
      const int k = AK ? i % KB : i / MT, t = AK ? i / KB : i % MT;
      sa[k][t] = left(t0 + t, k0 + k);
    }
    for (int p = 0; p < NB; ++p)
      for (int i = threadIdx.x; i < KB * MN; i += 256) {
        const int k = BK ? i % KB : i / MN, n = BK ? i / KB : i % MN;
        sb[p][k][n] = right(n0 + n, k0 + k, p);
      }
    __syncthreads();
    for (int k = 0; k < KB; ++k)
#pragma unroll
      for (int p = 0; p < NB; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[p][i][j] = __builtin_fmaf(sa[k][ty * 4 + i], sb[p][k][tx * 4 + j], acc[p][i][j]);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t t = t0 + ty * 4 + i;
    const bool in_t = t < a.T;
    if constexpr (OP == DENSE_LINEAR) {
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + tx * 4 + j;
        if (!in_t || n >= a.N) continue;
        float v = act_f(acc[0][i][j] + (a.bias ? bf16_to_f32(a.bias[n]) : 0.f), a.act);
        if (a.residual) v += bf16_to_f32(a.residual[t * a.ldr + n]);
        if (a.y_f32) static_cast<float*>(a.y)[t * a.ldy + n] = v;
        else static_cast<uint16_t*>(a.y)[t * a.ldy + n] = f32_to_bf16(v);
      }
    } else if constexpr (OP == DENSE_GLU) {
      float h[4], m = 0.f;
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + tx * 4 + j;
        const float g = acc[0][i][j], u = acc[NB - 1][i][j];
        h[j] = act_f(g, a.act) * u;
        m = fmaxf(m, fabsf(h[j]));
        if (a.gu && in_t && n < a.N) {
          a.gu[t * 2 * a.N + n] = f32_to_bf16(g);
          a.gu[t * 2 * a.N + a.N + n] = f32_to_bf16(u);
        }
      }
      // the 32 threads of a row hold one group of 128 columns
      const float s = group_scale(group_max<32>(m));
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + tx * 4 + j;
        if (!in_t || n >= a.N) continue;
        if (a.hs) static_cast<uint8_t*>(a.y)[t * a.ldy + n] = f32_to_e4m3(h[j] / s);
        else static_cast<uint16_t*>(a.y)[t * a.ldy + n] = f32_to_bf16(h[j]);
      }
      if (a.hs && in_t && tx == 0) a.hs[t * (a.N / 128) + n0 / 128] = s;
    } else {
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + tx * 4 + j;
        if (!in_t || n >= a.N) continue;
        const float g = bf16_to_f32(a.gu[t * 2 * a.N + n]), u = bf16_to_f32(a.gu[t * 2 * a.N + a.N + n]);
        const float dh = acc[0][i][j], ag = act_f(g, a.act);
        a.dgu[t * 2 * a.N + n] = f32_to_bf16(dh * u * act_grad_f(g, a.act));
        a.dgu[t * 2 * a.N + a.N + n] = f32_to_bf16(dh * ag);
        if (a.y) static_cast<uint16_t*>(a.y)[t * a.ldy + n] = f32_to_bf16(ag * u);
      }
    }
  }
}

void launch_dense(DenseOp op, bool fp8, bool ak, bool bk, const DenseArgs& a, hipStream_t s) {
  const dim3 grid((a.N + 127) / 128, (a.T + 31) / 32);
  if (op == DENSE_GLU && fp8) dense_kernel<DENSE_GLU, true, true, true><<<grid, 256, 0, s>>>(a);
  else if (op == DENSE_GLU) dense_kernel<DENSE_GLU, false, true, true><<<grid, 256, 0, s>>>(a);
  else if (op == DENSE_DGLU) dense_kernel<DENSE_DGLU, false, true, false><<<grid, 256, 0, s>>>(a);
  else if (fp8) dense_kernel<DENSE_LINEAR, true, true, true><<<grid, 256, 0, s>>>(a);
  else if (ak && bk) dense_kernel<DENSE_LINEAR, false, true, true><<<grid, 256, 0, s>>>(a);
  else if (ak) dense_kernel<DENSE_LINEAR, false, true, false><<<grid, 256, 0, s>>>(a);
  else dense_kernel<DENSE_LINEAR, false, false, false><<<grid, 256, 0, s>>>(a);
}

}  // namespace pe
