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

constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 1.17549435e-38f;   // 2^-126

// Scale of a group of values whose largest magnitude is `amax`: at least the
// smallest normal number, so that a zero group divides by it.  An infinity makes
// it infinite, and every value of the group NaN.  A NaN is not in `amax` (the
// maxima drop it) and keeps only its own code NaN.
__device__ __forceinline__ float group_scale(float amax) { return fmaxf(amax / kE4m3Max, kMinScale); }

// The standard normal distribution's cdf, good to (v^2 + 18) 2^-24 of itself at either end: (1 + erf(v / sqrt(2))) / 2
// would leave a multiple of 2^-24, and so nothing of the tail below -5.  With a = |v| / sqrt(2) and t = 1 / (1 + 0.3 a)
// the tail is erfc(a) / 2 = e t P(t), e = exp(-v^2 / 2): P is a polynomial fitted to erfc(a) exp(a^2) / (2 t) on
// 0 <= a <= 10 for the least largest relative error, 2e-8.  (erfcf is as good and takes longer: 4096 x 4096 x 512 with
// GELU 46.3 us, this 34.1, erff 34.4.)
__device__ __forceinline__ float normal_cdf(float v, float e) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.21213203f, fabsf(v), 1.f));
  const float c[9] = {-0.06476136f, 0.24278118f, -0.25613818f, 0.27385902f, -0.04732468f,
                      0.10746274f,  0.07416966f, 0.08535761f,  0.08459400f};
  float p = c[0];
#pragma unroll
  for (int i = 1; i < 9; ++i) p = __builtin_fmaf(p, t, c[i]);
  const float tail = e * t * p;
  return v < 0.f ? tail : 1.f - tail;
}
__device__ __forceinline__ float half_square_exp(float v) { return __expf(-0.5f * v * v); }

__device__ __forceinline__ float act_f(float v, int act) {
  if (act == PE_ACT_SILU) return v / (1.f + __expf(-v));
  if (act == PE_ACT_GELU) return v * normal_cdf(v, half_square_exp(v));
  return v;
}

// act'(v)
__device__ __forceinline__ float act_grad_f(float v, int act) {
  if (act == PE_ACT_SILU) {
    const float p = 1.f / (1.f + __expf(-v));
    return p * (1.f + v * (1.f - p));
  }
  const float e = half_square_exp(v);
  return normal_cdf(v, e) + v * e * 0.39894228f;
}

// The value of another lane of the same 16: DPP controls of the butterfly below.
template <int CTRL, class V>
__device__ __forceinline__ V dpp(V v) {
  return __builtin_bit_cast(
      V, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}

// Combine the values of W consecutive lanes in all of them.  Up to 16 lanes by
// DPP (pairs, pairs of pairs, mirrored halves of 8 and 16: after each stage every
// lane of the smaller group already has the same value), wider by shuffles.
template <int W, class V, class Op>
__device__ __forceinline__ V group_reduce(V v, Op op) {
  if constexpr (W >= 2) v = op(v, dpp<0xB1>(v));
  if constexpr (W >= 4) v = op(v, dpp<0x4E>(v));
  if constexpr (W >= 8) v = op(v, dpp<0x141>(v));
  if constexpr (W >= 16) v = op(v, dpp<0x140>(v));
  if constexpr (W >= 32) v = op(v, __shfl_xor(v, 16));
  if constexpr (W >= 64) v = op(v, __shfl_xor(v, 32));
  return v;
}
template <int W>
__device__ __forceinline__ float group_max(float v) {
  return group_reduce<W>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int W>
__device__ __forceinline__ float group_sum(float v) {
  return group_reduce<W>(v, [](float a, float b) { return a + b; });
}

// Four e4m3 codes of v / s, the first in the low byte.
__device__ __forceinline__ uint32_t quant4(const float* v, float s) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] / s, v[1] / s, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2] / s, v[3] / s, lo, true);
}

// 8 bf16 values of a 16-byte chunk.
__device__ __forceinline__ void widen8(const uint4& w, float (&v)[8]) {
  const uint32_t d[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(d[i] << 16);
    v[2 * i + 1] = __uint_as_float(d[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 narrow8(const float (&v)[8]) {
  uint32_t d[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) d[i] = f32_to_bf16(v[2 * i]) | (uint32_t)f32_to_bf16(v[2 * i + 1]) << 16;
  return make_uint4(d[0], d[1], d[2], d[3]);
}

}  // namespace

// ------------------------------------------------------------------ RMS norm
//
// v = x + residual, y = v * rsqrt(mean(v^2) + eps) * weight: one pass, the row
// in registers between the sum of squares and the output.  WPR wavefronts share
// a row, each lane holding CH chunks of 8 columns; a scale group of 128 columns
// is 16 neighbouring lanes.  Bound by its bytes: x, residual, sum and y once
// each.  Rows of up to 1024 columns take one wavefront (no barrier), longer ones
// the whole workgroup, which leaves a lane at most 8 chunks and gives a decode
// step's few rows four wavefronts each (8192 rows of 512: 7.3 us with one wavefront,
// 11.5 with four; of 1024 12.0 and 14.0; of 2048 22.4 and 22.0; 4 rows of 2048 4.2 and 3.5).
template <int WPR, int CH>
__global__ __launch_bounds__(256) void rmsnorm_kernel(NormArgs a) {
  __shared__ float part[4];
  constexpr int kLanes = WPR * 64;
  const int64_t t = (int64_t)blockIdx.x * (4 / WPR) + threadIdx.x / kLanes;
  const int l = threadIdx.x % kLanes;
  const bool row = t < a.T;
  const int n_ch = row ? a.H / 8 : 0;
  const uint4* x = reinterpret_cast<const uint4*>(a.x + t * a.ldx);
  const uint4* r = reinterpret_cast<const uint4*>(a.residual + t * a.ldr);
  const uint4* w = reinterpret_cast<const uint4*>(a.weight);
  uint4 xc[CH], rc[CH], wc[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = l + i * kLanes;
    xc[i] = rc[i] = wc[i] = make_uint4(0, 0, 0, 0);
    if (c < n_ch) {
      xc[i] = x[c];
      if (a.residual) rc[i] = r[c];
      wc[i] = w[c];
    }
  }
  float v[CH][8], ss = 0.f;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    float rv[8];
    widen8(xc[i], v[i]);
    widen8(rc[i], rv);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (a.residual) v[i][e] += rv[e];
      ss = __builtin_fmaf(v[i][e], v[i][e], ss);
    }
  }
  auto over_row = [&](float s) {
    s = group_sum<64>(s);
    if constexpr (WPR == 4) {
      __syncthreads();
      if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
      __syncthreads();
      s = (part[0] + part[1]) + (part[2] + part[3]);
    }
    return s;
  };
  ss = over_row(ss);
  float pre = 1.f, eps = a.eps;
  const bool large = ss == __builtin_inff() || a.eps > 0x1p100f, small = ss < 0x1p-80f && a.eps < 0x1p-60f;
  if (large || small) {                  // (the same in all of a row's lanes)
    // Squares that pass fp32's range, or might with eps: sum those of 2^-75 v (at most 2^106 each, 2^120 in 16384
    // columns); or, where so small an eps lets squares below the range count, those of 2^80 v.  eps is scaled alike.
    pre = large ? 0x1p-75f : 0x1p80f;
    eps = eps * pre * pre;
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(v[i][e] * pre, v[i][e] * pre, ss);
    ss = over_row(ss);
  }
  const float inv = 1.f / sqrtf(ss / (float)a.H + eps);
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = l + i * kLanes;
    float wv[8], y[8];
    widen8(wc[i], wv);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = v[i][e] * pre * inv * wv[e];
    if (a.sum && c < n_ch) reinterpret_cast<uint4*>(a.sum + t * a.lds)[c] = narrow8(v[i]);
    if (!a.yscale) {
      if (c < n_ch) reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.y) + t * a.ldy)[c] = narrow8(y);
      continue;
    }
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(y[e]));
    const float s = group_scale(group_max<16>(m));      // H is a multiple of 128: groups are whole
    if (c < n_ch) {
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.y) + t * a.ldy + c * 8) = make_uint2(quant4(y, s), quant4(y + 4, s));
      if (c % 16 == 0) a.yscale[t * (a.H / 128) + c / 16] = s;
    }
  }
}

void launch_rmsnorm(const NormArgs& a, hipStream_t s) {
  const dim3 one((a.T + 3) / 4), four(a.T);
  if (a.H <= 512) rmsnorm_kernel<1, 1><<<one, 256, 0, s>>>(a);
  else if (a.H <= 1024) rmsnorm_kernel<1, 2><<<one, 256, 0, s>>>(a);
  else if (a.H <= 2048) rmsnorm_kernel<4, 1><<<four, 256, 0, s>>>(a);
  else if (a.H <= 4096) rmsnorm_kernel<4, 2><<<four, 256, 0, s>>>(a);
  else if (a.H <= 8192) rmsnorm_kernel<4, 4><<<four, 256, 0, s>>>(a);
  else rmsnorm_kernel<4, 8><<<four, 256, 0, s>>>(a);
}

// ------------------------------------------------------------------ routing
//
// LPT lanes per token, lane l holding experts l, l + LPT, ... (PER of them): k
// rounds of the largest remaining logit, ties to the lowest id, so the choice
// compares logits as they are, never rounded scores.  Logits that are -infinity
// or NaN are never chosen and weigh nothing.  The fewest lanes that hold a
// token's experts, 8 each, keep the butterflies short (all DPP up to 128
// experts) and put several tokens on a wavefront (128 experts, 16 lanes: 5.6 us for
// 4 tokens and 6.9 for 8192; 8 lanes 7.6 and 8.0, 32 lanes 5.5 and 8.0, 64 lanes 5.8 and 11.8).
template <int LPT, int PER>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a) {
  const int64_t t = (int64_t)blockIdx.x * (256 / LPT) + threadIdx.x / LPT;
  const int l = threadIdx.x % LPT;
  if (t >= a.T) return;                                  // whole groups of LPT lanes leave
  const float kNone = -__builtin_inff();
  float v[PER];
  float mx = kNone;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = l + LPT * j;
    const float x = e < a.E ? a.logits[t * a.ldl + e] : kNone;
    v[j] = x == x ? x : kNone;
    mx = fmaxf(mx, v[j]);
  }
  mx = group_max<LPT>(mx);
  // softmax numerator of a logit (1 at the maximum, also where that is +infinity), or its sigmoid, of e^-|x| so that
  // small ones keep what fp32 can hold of them.  Where only the sigmoids' ratios are asked for and all are small, those
  // are the softmax's numerators' too (e^x / (1 + e^x) without its last term, 2^-28), as long as the largest is not 0
  // in fp32.
  const bool sigmoid = a.sigmoid && !(a.renorm && mx < -20.f && mx > -103.5f);
  auto num = [&](float x) {
    if (x == kNone) return 0.f;
    if (sigmoid) {
      const float e = expf(-fabsf(x));
      return (x < 0.f ? e : 1.f) / (1.f + e);
    }
    return x == mx ? 1.f : expf(x - mx);
  };
  float den = 1.f;
  if (!a.sigmoid) {
    den = 0.f;
#pragma unroll
    for (int j = 0; j < PER; ++j) den += num(v[j]);
    den = group_sum<LPT>(den);
  }
  // Round r's choice is kept by lane r % LPT: in registers for r < LPT, beyond that in the output.
  int my_id = -1;
  float my_p = 0.f, chosen = 0.f;
  for (int r = 0; r < a.k; ++r) {
    float best = kNone;
#pragma unroll
    for (int j = 0; j < PER; ++j) best = fmaxf(best, v[j]);
    best = group_max<LPT>(best);
    int at = 1 << 30;
    if (best > kNone) {
#pragma unroll
      for (int j = PER - 1; j >= 0; --j)
        if (v[j] == best) at = l + LPT * j;
    }
    at = group_reduce<LPT>(at, [](int p, int q) { return min(p, q); });
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (at == l + LPT * j) v[j] = kNone;
    const float p = best > kNone ? num(best) / den : 0.f;
    chosen += p;
    if (l == r % LPT) {
      const int id = best > kNone ? at : -1;
      if (r < LPT) {
        my_id = id;
        my_p = p;
      } else {
        a.ids[t * a.k + r] = id;
        a.w[t * a.k + r] = p;
      }
    }
  }
  const float by = a.renorm && chosen > 0.f ? chosen : 1.f;
  if (l < a.k) {
    a.ids[t * a.k + l] = my_id;
    a.w[t * a.k + l] = my_p / by * a.scale;
  }
  for (int r = l + LPT; r < a.k; r += LPT) a.w[t * a.k + r] = a.w[t * a.k + r] / by * a.scale;
}

template <int LPT, int PER>
static void launch_route_n(const RouteArgs& a, hipStream_t s) {
  const int per = 256 / LPT;
  route_kernel<LPT, PER><<<dim3((a.T + per - 1) / per), 256, 0, s>>>(a);
}

void launch_route(const RouteArgs& a, hipStream_t s) {
  if (a.E <= 64) launch_route_n<8, 8>(a, s);
  else if (a.E <= 128) launch_route_n<16, 8>(a, s);
  else if (a.E <= 256) launch_route_n<32, 8>(a, s);
  else if (a.E <= 512) launch_route_n<64, 8>(a, s);
  else launch_route_n<64, 16>(a, s);
}

// ------------------------------------------------------------------ matrix products, tiled
//
// out[t, n] = sum_k A[t, k] B[n, k] on the matrix cores, a BT x BN tile per
// workgroup.  Both operands come through LDS in steps of 128 bytes of k (64
// bf16, 128 e4m3 values: one scale group), NST stages deep: each wavefront
// copies its share of a later step straight from global memory into LDS (no
// registers), while the step that has arrived feeds the MFMAs.  One barrier per
// step: it follows each wavefront's wait for its own copies, so the step is
// whole, and every wavefront is then done reading the buffer the next copies
// overwrite.
//
// A K-major operand's tile is [rows][128 bytes]; a k-slow operand (a gradient's
// transposed factor) is [64 k][rows], and the transposing LDS read gives each
// lane four consecutive k of its row.  LDS-direct copies write lane after lane,
// so bank conflicts are avoided by permuting which global chunk a lane fetches:
// K-major rows keep their 16-byte chunk c at position c ^ (row / 2 % 8) (the 16
// rows one read touches fall on all 16 chunk slots of two rows), k-slow rows
// their 32-byte unit u at u ^ f(k), with f different for the rows of one read.
//
// The MFMA takes B's rows as its first operand, so a lane's four accumulators
// are four consecutive n of one t: 8-byte stores, vector loads of the residual.
// FP8 operands with bf16 outputs take v_mfma_f32_16x16x128_f8f6f4; the step's
// partial products are multiplied by the row's and the block's fp32 scale when
// they are added up in fp32.  Inside, the instruction lines up the eight products
// of eight consecutive k to the largest of their exponents and drops what lies
// more than 13 bits below it (measured product by product); the sums of eight are
// added in fp32.  Each product is so off by less than 2^-13 of the largest of its
// eight.  In a sum that does not cancel that is below the output's own rounding;
// one that does, within itself or with the bias or residual added later, may be
// left with it.  That is taken for twice the matrix rate, and a caller has the
// choice: where an output is kept in fp32 (y, or the scales of an e4m3 h) the
// codes are widened to bf16 in registers instead, for full-width sums.
//
// Rows past the end are read as the last row (their results are not stored); k
// past the end is read from a page of zeros.

namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;
typedef __attribute__((ext_vector_type(4))) float f32x4_t;
typedef __attribute__((ext_vector_type(4))) short s16x4_t;
typedef __attribute__((ext_vector_type(8))) int i32x8_t;

__device__ __attribute__((aligned(16))) const uint32_t g_zeros[4] = {0, 0, 0, 0};

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)(const char*)p;
}

// Copy 16 bytes per lane from base + off (64 lanes) to the 1024 bytes of LDS at
// `lds` (wavefront-uniform).  The compiler orders LDS-direct loads against
// every LDS read it sees with a full wait, which would end the pipelining; as
// inline assembly without outputs they are ordered by wait_stage alone.
__device__ __forceinline__ void copy_to_lds(uint32_t lds, const char* base, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base));
}
// Same from an address of each lane.
__device__ __forceinline__ void copy_to_lds(uint32_t lds, const char* p) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(p));
}
// Same for 4 bytes per lane to 256 bytes of LDS.
__device__ __forceinline__ void copy_to_lds4(uint32_t lds, const char* p) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(p));
}

// A pointer that is the same in all lanes, which the compiler does not always see.
__device__ __forceinline__ const char* uniform(const char* p) {
  const uint64_t b = (uint64_t)p;
  return (const char*)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(b >> 32)) << 32 |
                       (uint32_t)__builtin_amdgcn_readfirstlane((int)b));
}

// This wavefront's copies are done but for the newest N, its LDS reads are
// done, and so are every other wavefront's.
template <int N>
__device__ __forceinline__ void wait_stage() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// Eight e4m3 codes as bf16 (exactly).
__device__ __forceinline__ bf16x8_t widen_e4m3(uint32_t lo, uint32_t hi) {
  typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;
  const bf16x2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const bf16x2_t p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const bf16x2_t p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const bf16x2_t p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return bf16x8_t{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// One operand's tile of ROWS rows: what this wavefront copies per step, and
// where its lanes read fragments.
template <int ROWS, int NW, bool KMAJOR>
struct Operand {
  static constexpr int kInstr = ROWS / 8;               // 1024-byte copies per step
  static constexpr int kPer = (kInstr + NW - 1) / NW;   // of which per wavefront, at most
  static constexpr int kMin = kInstr / NW;              // and at least
  static_assert((kInstr % NW == 0 || kPer == 1) && NW % 2 == 0, "copies divide evenly, or go one each to the first");

  uint32_t off[kPer];     // K-major: byte offset of the lane's chunk from the tile's first row; k-slow: from row k0
  int kc[kPer];           // K-major: the chunk's byte within the 128; k-slow: its k row

  // `row(r)`: the matrix row (clamped) of tile row r, relative to the tile's base; ld in bytes
  template <class RowOf>
  __device__ __forceinline__ void init(int wave, int lane, int64_t ld, RowOf row, int c0, int n_cols) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int j = wave + i * NW;
      if constexpr (KMAJOR) {
        const int r = 8 * j + (lane >> 3);
        const int c = (lane & 7) ^ ((r >> 1) & 7);
        kc[i] = c * 16;
        off[i] = (uint32_t)(row(r) * ld) + c * 16;
      } else {
        constexpr int CPR = ROWS / 8;                   // 16-byte chunks per k row
        const int idx = 64 * j + lane, k = idx / CPR, pos = idx % CPR;
        const int c = (((pos >> 1) ^ swz(k)) << 1) | (pos & 1);
        kc[i] = k;
        // columns past the end are read as the last chunk of the row
        off[i] = (uint32_t)(k * ld) + 2 * min(c0 + 8 * c, n_cols - 8);
      }
    }
  }

  // f(k): as many bits as the number of units is a multiple of, so that u ^ f(k) stays in the row, and
  // different for the k whose rows start on the same banks
  static __device__ __forceinline__ int swz(int k) {
    if constexpr (ROWS % 128 == 0) return (k & 3) | ((k >> 1) & 4);
    if constexpr (ROWS % 64 == 0) return ((k >> 1) & 1) | ((k >> 2) & 2);
    return (k >> 3) & 1;
  }

  // Copy the step whose first chunk (or k row) is at `base`.
  __device__ __forceinline__ void copy(uint32_t lds, int wave, const char* base) const {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (kMin == kPer || wave < kInstr) copy_to_lds(lds + (wave + i * NW) * 1024, base, off[i]);
  }
  // The same where only the first `valid` bytes (k rows) of the step exist: the other lanes copy zeros.
  __device__ __forceinline__ void copy_tail(uint32_t lds, int wave, const char* base, int valid) const {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (kMin == kPer || wave < kInstr)
        copy_to_lds(lds + (wave + i * NW) * 1024,
                    kc[i] < valid ? base + off[i] : reinterpret_cast<const char*>(g_zeros));
  }
};

// Fragment reads of rows w0 .. w0 + 16 F - 1 of an operand's tile.
template <int ROWS, bool KMAJOR, int F>
struct Frags {
  uint32_t at[KMAJOR ? 2 : F];

  __device__ __forceinline__ void init(int w0, int lane) {
    const int q = lane >> 4, j = lane & 15;
    if constexpr (KMAJOR) {
      const uint32_t row = (w0 + j) * 128;
      at[0] = row + ((q ^ (j >> 1)) << 4);
      at[1] = at[0] ^ 64;
    } else {
      const int k = 8 * q + (j >> 2);
      const int g = Operand<ROWS, 2, false>::swz(k);
#pragma unroll
      for (int f = 0; f < F; ++f) at[f] = k * ROWS * 2 + (((w0 / 16 + f) ^ g) << 5) + (j & 3) * 8;
    }
  }

  // Fragment f of k values 32 s .. 32 s + 31 of the step staged at `stage`.
  __device__ __forceinline__ bf16x8_t bf16(const char* stage, int f, int s) const {
    if constexpr (KMAJOR) {
      return *reinterpret_cast<const bf16x8_t*>(stage + at[s] + f * 2048);
    } else {
      typedef __attribute__((address_space(3))) s16x4_t* tr_p;
      const char* p = stage + at[f] + s * 32 * ROWS * 2;
      const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((tr_p)(uintptr_t)lds_addr(p));
      const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((tr_p)(uintptr_t)lds_addr(p + 4 * ROWS * 2));
      return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
  // Fragment f of the whole step in e4m3: both operands take the two chunks in
  // this order, so the pairing of k values is right whatever order the MFMA has.
  __device__ __forceinline__ i32x8_t fp8(const char* stage, int f) const {
    const uint4 lo = *reinterpret_cast<const uint4*>(stage + at[0] + f * 2048);
    const uint4 hi = *reinterpret_cast<const uint4*>(stage + at[1] + f * 2048);
    return i32x8_t{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
  }
};

// C (4 or 8) consecutive bf16 values: as one vector, or the first n of them.
template <int C>
__device__ __forceinline__ void load_bf16(const uint16_t* p, bool vec, int n, float (&v)[C]) {
  if (vec) {
    uint32_t w[C / 2];
    if constexpr (C == 8) *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(p);
    else *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(p);
#pragma unroll
    for (int i = 0; i < C / 2; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = i < n ? bf16_to_f32(p[i]) : 0.f;
  }
}
template <int C>
__device__ __forceinline__ void store_bf16(uint16_t* p, bool vec, int n, const float (&v)[C]) {
  if (vec) {
    uint32_t w[C / 2];
#pragma unroll
    for (int i = 0; i < C / 2; ++i) w[i] = f32_to_bf16(v[2 * i]) | (uint32_t)f32_to_bf16(v[2 * i + 1]) << 16;
    if constexpr (C == 8) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(w);
    else *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(w);
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (i < n) p[i] = f32_to_bf16(v[i]);
  }
}

// y[t, n .. n + C - 1] = act(v + bias) + residual.
template <int C>
__device__ __forceinline__ void finish_linear(const DenseArgs& a, int64_t t, int n, float (&v)[C]) {
  const int left = a.N - n;
  const bool vec = a.vec && left >= C;
  float w[C];
  if (a.bias) {
    load_bf16(a.bias + n, vec, left, w);
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] += w[i];
  }
  if (a.act != PE_ACT_NONE) {
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = act_f(v[i], a.act);
  }
  if (a.residual) {
    load_bf16(a.residual + t * a.ldr + n, vec, left, w);
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] += w[i];
  }
  if (!a.y_f32) {
    store_bf16(static_cast<uint16_t*>(a.y) + t * a.ldy + n, vec, left, v);
  } else {
    float* y = static_cast<float*>(a.y) + t * a.ldy + n;
    if (vec) {
#pragma unroll
      for (int i = 0; i < C; i += 4) *reinterpret_cast<float4*>(y + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i)
        if (i < left) y[i] = v[i];
    }
  }
}

// h[t, n .. n + C - 1] = act(g) * u, and g and u themselves if they are kept.
// With e4m3 output the 128 / C lanes of a scale group hold its columns in order
// (all of them come here, `in` saying whether the row exists).
template <int C>
__device__ __forceinline__ void finish_glu(const DenseArgs& a, int64_t t, int n, bool in, const float (&g)[C],
                                           const float (&u)[C]) {
  float h[C];
#pragma unroll
  for (int i = 0; i < C; ++i) h[i] = act_f(g[i], a.act) * u[i];
  if (a.gu && in) {                                     // 16-byte aligned rows, N a multiple of 8
    store_bf16(a.gu + t * 2 * a.N + n, true, C, g);
    store_bf16(a.gu + t * 2 * a.N + a.N + n, true, C, u);
  }
  if (!a.hs) {
    if (in) store_bf16(static_cast<uint16_t*>(a.y) + t * a.ldy + n, a.vec, C, h);
    return;
  }
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < C; ++i) m = fmaxf(m, fabsf(h[i]));
  const float s = group_scale(group_max<128 / C>(m));
  if (!in) return;
  if (n % 128 == 0) a.hs[t * (a.N / 128) + n / 128] = s;
  uint8_t* y = static_cast<uint8_t*>(a.y) + t * a.ldy + n;
#pragma unroll
  for (int i = 0; i < C; i += 4) {
    const uint32_t c = quant4(h + i, s);
    if (a.vec) {
      *reinterpret_cast<uint32_t*>(y + i) = c;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) y[i + e] = (uint8_t)(c >> (8 * e));
    }
  }
}

// From dh[t, n .. n + C - 1] and the kept g and u: their gradients, and h.  dh stays in fp32; what the products after
// it read is rounded to bf16, as their matrix operands are (in fp32 they would take three bf16 products each).
template <int C>
__device__ __forceinline__ void finish_dglu(const DenseArgs& a, int64_t t, int n, const float (&dh)[C]) {
  float g[C], u[C], dg[C], du[C], h[C];
  load_bf16(a.gu + t * 2 * a.N + n, true, C, g);
  load_bf16(a.gu + t * 2 * a.N + a.N + n, true, C, u);
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const float ag = act_f(g[i], a.act);
    dg[i] = dh[i] * u[i] * act_grad_f(g[i], a.act);
    du[i] = dh[i] * ag;
    h[i] = ag * u[i];
  }
  store_bf16(a.dgu + t * 2 * a.N + n, true, C, dg);
  store_bf16(a.dgu + t * 2 * a.N + a.N + n, true, C, du);
  if (a.y) store_bf16(static_cast<uint16_t*>(a.y) + t * a.ldy + n, true, C, h);
}

// Columns n .. n + 7 of row t, whose accumulators are columns c .. c + 7 of the
// fp32 row at `row` (a GLU's gate and up blocks of 16 alternate there).  KS partial
// sums of a split k lie `apart` floats from each other and are added in order.
template <DenseOp OP, int KS = 1>
__device__ __forceinline__ void finish_chunk(const DenseArgs& a, int64_t t, int n, const float* row, int c, int apart = 0) {
  const bool in = t < a.T && n < a.N;
  const float* p = row + (OP == DENSE_GLU ? (c >> 4) * 32 + (c & 15) : c);
  auto sum8 = [&](const float* at, float (&v)[8]) {
#pragma unroll
    for (int g = 0; g < KS; ++g, at += apart) {
      const float4 lo = reinterpret_cast<const float4*>(at)[0], hi = reinterpret_cast<const float4*>(at)[1];
      const float w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = g ? v[e] + w[e] : w[e];
    }
  };
  float v[8];
  sum8(p, v);
  if constexpr (OP == DENSE_GLU) {
    float u[8];
    sum8(p + 16, u);
    finish_glu(a, t, n, in, v, u);
  } else if constexpr (OP == DENSE_DGLU) {
    if (in) finish_dglu(a, t, n, v);
  } else {
    if (in) finish_linear(a, t, n, v);
  }
}

// Workgroups go round-robin over the 8 XCDs, each with its own L2.  Every XCD
// takes a contiguous run of tiles, in bands of kBand tiles of t, column by
// column, so that the tiles in flight together share rows of both operands.
__device__ __forceinline__ void tile_of(int b, int nt, int nn, int& tt, int& tn) {
  constexpr int kXcds = 8, kBand = 8;
  const int total = nt * nn;
  const int xcd = b % kXcds, per = total / kXcds, rem = total % kXcds;
  const int q = xcd * per + min(xcd, rem) + b / kXcds;
  const int band = q / (kBand * nn), rows = min(kBand, nt - band * kBand), r = q - band * kBand * nn;
  tt = band * kBand + r % rows;
  tn = r / rows;
}

}  // namespace

// LDS of a tile kernel: the stages of both operands and, after them, the fp32 tile.
constexpr int tile_lds(int bt, int bn, int nst, int fp8, int ks = 1) {
  const int stages = nst * ((bt + bn) * 128 + (fp8 ? bt * 4 : 0)), tile = bt * (bn + 4) * 4;
  return ks * (stages > tile ? stages : tile);
}

// FP8: 0 bf16 operands, 1 e4m3 through the FP8 MFMA, 2 e4m3 widened to bf16.
// A WT x WN grid of wavefronts, each with FT x FN blocks of 16 x 16 outputs, KS times: where there are few tiles and
// their k is long, KS such grids take every KS-th step each and their sums meet at the end.
// A GLU tile's B rows alternate 16 gate rows and the 16 up rows of the same
// columns, so that a wavefront holds both products of its columns.
template <DenseOp OP, int FP8, bool AK, bool BK, int WT, int WN, int FT, int FN, int NST, int KS>
__device__ __forceinline__ void dense_tile(const DenseArgs& a, int block) {
  constexpr int NW = WT * WN, BT = WT * FT * 16, BN = WN * FN * 16;
  constexpr int NO = OP == DENSE_GLU ? BN / 2 : BN;       // output columns per tile
  constexpr int ES = FP8 ? 1 : 2;
  constexpr int kA = BT * 128, kB = BN * 128, kStage = kA + kB + (FP8 ? BT * 4 : 0);
  extern __shared__ __align__(16) char lds[];
  const int lane = threadIdx.x & 63, wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave = wave_all % NW, share = wave_all / NW;  // wavefront of its share of k
  const int wt = wave / WN, wn = wave % WN;
  const int q4 = (lane >> 4) * 4, ln = lane & 15;
  int tt, tn;
  tile_of(block, (a.T + BT - 1) / BT, (a.N + NO - 1) / NO, tt, tn);
  const int t0 = tt * BT, n0 = tn * NO;
  const int64_t lda = a.lda * ES, ldb = a.ldb * ES;

  Operand<BT, NW, AK> oa;
  Operand<BN, NW, BK> ob;
  const char* pa = static_cast<const char*>(a.a) + (AK ? t0 * lda : 0);
  const char* pb = static_cast<const char*>(a.b) + (BK ? n0 * ldb : 0);
  oa.init(wave, lane, lda, [&](int r) { return (int64_t)min(r, a.T - 1 - t0); }, t0, a.T);
  // the up half's rows can be further than 32-bit offsets reach: OP == GLU adds them to the base of its copies
  ob.init(wave, lane, ldb, [&](int r) {
    if constexpr (OP == DENSE_GLU) return (int64_t)min((r >> 5) * 16 + (r & 15), a.N - 1 - n0);
    return (int64_t)min(r, a.N - 1 - n0);
  }, n0, a.N);
  Frags<BT, AK, FT> fa;
  Frags<BN, BK, FN> fb;
  fa.init(wt * FT * 16, lane);
  fb.init(wn * FN * 16, lane);

  const int64_t sa = AK ? 128 : 64 * lda, sb = BK ? 128 : 64 * ldb;    // bytes per step
  constexpr int kstep = 128 / ES;
  const int nk = (a.K + kstep - 1) / kstep;
  const int tail = a.K - (nk - 1) * kstep;                              // k of the last step
  const int64_t up = OP == DENSE_GLU ? (int64_t)a.N * ldb : 0;
  const uint32_t lds0 = lds_addr(lds);
  // this wavefront copies 8-row pieces wave, wave + NW, ...: with a GLU's 16-row alternation and NW a
  // multiple of 4, they all lie in one half
  static_assert(OP != DENSE_GLU || NW % 4 == 0, "a wavefront's copies stay in one half");
  if (OP == DENSE_GLU && (wave & 2)) pb += up;
  const int scales_k = FP8 ? a.K / 128 : 0;
  const char* ps = nullptr;
  if constexpr (FP8)
    ps = reinterpret_cast<const char*>(a.as + (int64_t)min(t0 + wave * 64 + lane, a.T - 1) * scales_k);

  auto fetch = [&](int it) {     // this share's copies of turn `it`: step it * KS + share
    const int k = it * KS + share;
    if (KS > 1 && k >= nk) return;
    const uint32_t st = lds0 + (it % NST * KS + share) * kStage;
    if (FP8 || k < nk - 1 || tail == kstep) {
      oa.copy(st, wave, pa + k * sa);
      ob.copy(st + kA, wave, pb + k * sb);
    } else {
      oa.copy_tail(st, wave, pa + k * sa, AK ? tail * ES : tail);
      ob.copy_tail(st + kA, wave, pb + k * sb, BK ? tail * ES : tail);
    }
    if constexpr (FP8)
      if (wave * 64 < BT && (BT % 64 == 0 || lane < BT)) copy_to_lds4(st + kA + kB + wave * 256, ps + k * 4);
  };
  // Copies per step of the wavefront with the fewest (waiting for that many more is waiting for enough).
  constexpr int kCopies = decltype(oa)::kMin + decltype(ob)::kMin;

  f32x4_t acc[FT][FN];
#pragma unroll
  for (int i = 0; i < FT; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  // FP8: the scale of this wavefront's weight rows (they lie in one 128-row block; a GLU's two halves in one each)
  const int brow = n0 + (OP == DENSE_GLU ? wn * FN * 8 : wn * FN * 16);
  const float* sw0 = nullptr;
  const float* sw1 = nullptr;
  if constexpr (FP8) {
    static_assert(FN * 16 <= 128, "a wavefront's columns lie in one scale block");
    sw0 = a.bs + (int64_t)(min(brow, a.N - 1) / 128) * scales_k;
    sw1 = OP == DENSE_GLU ? a.bs + (int64_t)((a.N + min(brow, a.N - 1)) / 128) * scales_k : sw0;
  }

  const int turns = (nk + KS - 1) / KS;
#pragma unroll
  for (int it = 0; it < NST - 1; ++it)
    if (it < turns) fetch(it);
  for (int it = 0; it < turns; ++it) {
    if (NST > 2 && (it + NST - 1) * KS <= nk) wait_stage<(NST - 2) * kCopies>();
    else wait_stage<0>();
    const char* st = lds + (it % NST * KS + share) * kStage;
    if (it + NST - 1 < turns) fetch(it + NST - 1);
    const int k = it * KS + share;
    if (KS > 1 && k >= nk) continue;
    if constexpr (FP8) {
      const float* sc = reinterpret_cast<const float*>(st + kA + kB) + wt * FT * 16 + ln;
      const float w0 = sw0[k], w1 = sw1[k];
      i32x8_t bf[FP8 == 1 ? FN : 1];
      bf16x8_t bw[FP8 == 2 ? FN : 1][4];
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        if constexpr (FP8 == 1) {
          bf[j] = fb.fp8(st + kA, j);
        } else {
          const i32x8_t v = fb.fp8(st + kA, j);
#pragma unroll
          for (int s = 0; s < 4; ++s) bw[j][s] = widen_e4m3(v[2 * s], v[2 * s + 1]);
        }
      }
#pragma unroll
      for (int i = 0; i < FT; ++i) {
        const i32x8_t af = fa.fp8(st, i);
        const float s0 = sc[16 * i] * w0, s1 = sc[16 * i] * w1;
        bf16x8_t aw[4];
        if constexpr (FP8 == 2) {
#pragma unroll
          for (int s = 0; s < 4; ++s) aw[s] = widen_e4m3(af[2 * s], af[2 * s + 1]);
        }
        f32x4_t p[FN];
        if constexpr (FP8 == 2) {
#pragma unroll
          for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int j = 0; j < FN; ++j)
              p[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bw[j][s], aw[s],
                                                             s ? p[j] : f32x4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
        } else {
#pragma unroll
          for (int j = 0; j < FN; ++j)
            p[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bf[j], af, f32x4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0,
                                                                    0);   // no block scales
        }
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc[i][j][e] = __builtin_fmaf(p[j][e], OP == DENSE_GLU && (j & 1) ? s1 : s0, acc[i][j][e]);
      }
    } else {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        bf16x8_t af[FT], bf[FN];
#pragma unroll
        for (int j = 0; j < FN; ++j) bf[j] = fb.bf16(st + kA, j, s);
#pragma unroll
        for (int i = 0; i < FT; ++i) af[i] = fa.bf16(st, i, s);
#pragma unroll
        for (int i = 0; i < FT; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[j], af[i], acc[i][j], 0, 0, 0);
      }
    }
  }

  // The accumulators go through LDS as fp32 rows of the tile (padded by 16 bytes
  // against bank conflicts), so that each thread finishes 8 consecutive columns
  // with 16-byte loads and stores.
  constexpr int LR = BN + 4;
  static_assert(KS * BT * LR * 4 <= tile_lds(BT, BN, NST, FP8, KS), "the tiles fit the stages' LDS");
  float* tile = reinterpret_cast<float*>(lds);
  wait_stage<0>();                                       // the stages have been read
#pragma unroll
  for (int i = 0; i < FT; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
      *reinterpret_cast<f32x4_t*>(tile + (share * BT + (wt * FT + i) * 16 + ln) * LR + (wn * FN + j) * 16 + q4) = acc[i][j];
  __syncthreads();
  constexpr int kChunks = NO / 8;
  static_assert(BT * kChunks % 64 == 0, "whole wavefronts finish chunks: scale groups stay together");
#pragma unroll 1
  for (int idx = threadIdx.x; idx < BT * kChunks; idx += KS * NW * 64) {
    const int r = idx / kChunks, c = (idx % kChunks) * 8;
    finish_chunk<OP, KS>(a, t0 + r, n0 + c, tile + r * LR, c, BT * LR);
  }
}

template <DenseOp OP, int FP8, bool AK, bool BK, int WT, int WN, int FT, int FN, int NST, int KS>
__global__ __launch_bounds__(KS * WT * WN * 64) void dense_tile_kernel(DenseArgs a) {
  dense_tile<OP, FP8, AK, BK, WT, WN, FT, FN, NST, KS>(a, blockIdx.x);
}

// The three products of the feed-forward gradients in one launch of 64 x 64 tiles, the
// longest sums first: `weights_first` where there are more tokens than dx's 2 * inter terms.
template <int KS>
__global__ __launch_bounds__(KS * 256) void dense_grads_kernel(DenseArgs dx, DenseArgs dw13, DenseArgs dw2, int n_dx,
                                                               int n_dw13, int n_dw2, int weights_first) {
  int b = blockIdx.x;
  if (weights_first) b = b < n_dw13 + n_dw2 ? b + n_dx : b - n_dw13 - n_dw2;
  if (b < n_dx) {
    dense_tile<DENSE_LINEAR, 0, true, false, 2, 2, 2, 2, 2, KS>(dx, b);
  } else {
    const bool first = b < n_dx + n_dw13;
    dense_tile<DENSE_LINEAR, 0, false, false, 2, 2, 2, 2, 2, KS>(first ? dw13 : dw2, b - n_dx - (first ? 0 : n_dw13));
  }
}

// The large bf16 tile: 256 rows of A by 32 FN (128, 192 or 256) of B, eight wavefronts as
// 4 x 2.  What bounds the 128 x 128 tile is the LDS port (fragment reads at 128 bytes a
// clock plus the copies' writes at 60): 1058 clocks a step for 515 of MFMA.  A larger
// tile moves fewer bytes per MFMA, but one workgroup then fills the unit and nothing
// runs while its wavefronts read.  So they work in two groups of four (one wavefront
// per SIMD each) half a step apart: while one group reads its fragments of 32 k and
// issues copies, the other one's MFMAs run, and a barrier ends each phase.  A's step
// is copied two steps ahead (three slots), B's one step ahead (two).
template <DenseOp OP, bool AK, bool BK, int FN>
__global__ __launch_bounds__(512) void dense_pair_kernel(DenseArgs a) {
  constexpr int FT = 4, WN = 2, NW = 8, BT = 256, BN = WN * FN * 16;
  constexpr int NO = OP == DENSE_GLU ? BN / 2 : BN;
  constexpr int kA = BT * 128, kB = BN * 128;
  extern __shared__ __align__(16) char lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wt = wave / WN, wn = wave % WN, group = wave / 4;
  const int q4 = (lane >> 4) * 4, ln = lane & 15;
  int tt, tn;
  tile_of(blockIdx.x, (a.T + BT - 1) / BT, (a.N + NO - 1) / NO, tt, tn);
  const int t0 = tt * BT, n0 = tn * NO;
  const int64_t lda = a.lda * 2, ldb = a.ldb * 2;

  Operand<BT, NW, AK> oa;
  Operand<BN, NW, BK> ob;
  const char* pa = static_cast<const char*>(a.a) + (AK ? t0 * lda : 0);
  const char* pb = static_cast<const char*>(a.b) + (BK ? n0 * ldb : 0);
  oa.init(wave, lane, lda, [&](int r) { return (int64_t)min(r, a.T - 1 - t0); }, t0, a.T);
  ob.init(wave, lane, ldb, [&](int r) {
    if constexpr (OP == DENSE_GLU) return (int64_t)min((r >> 5) * 16 + (r & 15), a.N - 1 - n0);
    return (int64_t)min(r, a.N - 1 - n0);
  }, n0, a.N);
  if (OP == DENSE_GLU && (wave & 2)) pb += (int64_t)a.N * ldb;
  pa = uniform(pa);
  pb = uniform(pb);
  Frags<BT, AK, FT> fa;
  Frags<BN, BK, FN> fb;
  fa.init(wt * FT * 16, lane);
  fb.init(wn * FN * 16, lane);
  const int64_t sa = AK ? 128 : 64 * lda, sb = BK ? 128 : 64 * ldb;
  const int nk = (a.K + 63) / 64;
  const int tail = a.K - (nk - 1) * 64;
  const uint32_t lds0 = lds_addr(lds);
  auto copy_a = [&](int k) {
    const uint32_t st = lds0 + k % 3 * kA;
    if (k < nk - 1 || tail == 64) oa.copy(st, wave, pa + k * sa);
    else oa.copy_tail(st, wave, pa + k * sa, AK ? tail * 2 : tail);
  };
  auto copy_b = [&](int k) {
    const uint32_t st = lds0 + 3 * kA + k % 2 * kB;
    if (k < nk - 1 || tail == 64) ob.copy(st, wave, pb + k * sb);
    else ob.copy_tail(st, wave, pb + k * sb, BK ? tail * 2 : tail);
  };
  f32x4_t acc[FT][FN];
#pragma unroll
  for (int i = 0; i < FT; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  bf16x8_t af[FT], bf[FN];
  auto read = [&](int k, int s) {
    const char* la = lds + k % 3 * kA;
    const char* lb = lds + 3 * kA + k % 2 * kB;
#pragma unroll
    for (int j = 0; j < FN; ++j) bf[j] = fb.bf16(lb, j, s);
#pragma unroll
    for (int i = 0; i < FT; ++i) af[i] = fa.bf16(la, i, s);
  };
  auto multiply = [&] {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int i = 0; i < FT; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[j], af[i], acc[i][j], 0, 0, 0);
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_barrier" ::: "memory");
  };
  // everything has arrived but, with `newer`, the copies of A issued last
  auto wait_all_but_a = [&](bool newer) {
    if (newer) wait_stage<decltype(oa)::kPer>();
    else wait_stage<0>();
  };
  if (nk > 0) {
    copy_b(0);
    copy_a(0);
  }
  if (nk > 1) copy_a(1);
  wait_all_but_a(nk > 1);
  if (group == 1) asm volatile("s_barrier" ::: "memory");
  for (int k = 0; k < nk; ++k) {
    read(k, 0);
    if (k + 1 < nk) copy_b(k + 1);          // into the slot of step k - 1, which both groups have read
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    multiply();
    read(k, 1);
    if (k + 2 < nk) copy_a(k + 2);          // likewise
    wait_all_but_a(k + 2 < nk);             // step k + 1 is there before the first group reads it, two phases on
    multiply();
  }
  if (group == 0) asm volatile("s_barrier" ::: "memory");

  // As in the smaller tile, half of each wavefront's blocks of rows at a time.
  constexpr int LR = BN + 4, kChunks = NO / 8;
  float* tile = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
        *reinterpret_cast<f32x4_t*>(tile + (wt * 32 + i * 16 + ln) * LR + (wn * FN + j) * 16 + q4) = acc[2 * half + i][j];
    __syncthreads();
    static_assert(128 * kChunks % 64 == 0, "whole wavefronts finish chunks: scale groups stay together");
#pragma unroll 1
    for (int idx = threadIdx.x; idx < 128 * kChunks; idx += 512) {
      const int r = idx / kChunks, c = (idx % kChunks) * 8;
      finish_chunk<OP>(a, t0 + (r >> 5) * 64 + half * 32 + (r & 31), n0 + c, tile + r * LR, c);
    }
  }
}

// ------------------------------------------------------------------ matrix products of few rows
//
// A few rows of A (a decode step's tokens): the weights' bytes bound the
// product, so they stream straight from memory into MFMA operands, read once (by
// each block of 16 rows of A).  A wavefront takes 16 of the workgroup's weight
// rows (fragment rw of RW) and every KW-th 128-byte step of k, U steps in
// flight; the KW partial sums meet in LDS in a fixed order.  With at most 8 rows of
// A most columns of the MFMA's 16 x 16 block would be idle: P parts of k share it
// instead (16 / P weight rows and 16 / P rows of A each, part p in rows and columns
// p * 16 / P ...; of the block only the P diagonal squares are used).  One compute
// unit cannot draw more than some 55 GB/s from memory, so what counts is that the
// smaller workgroups are P times as many: gate/up 2 x 6144 x 2048 in bf16 for one
// row, 10.7 us (4.7 TB/s) with P = 2 or 4 against 13.5 us with P = 1.  A GLU's fragments
// alternate gate rows and the up rows of the same columns.
template <DenseOp OP, int FP8, int RW, int KW, int P, int U>
__global__ __launch_bounds__(RW * KW * 64) void dense_few_kernel(DenseArgs a) {
  constexpr int NR = 16 / P;                              // weight rows per fragment, rows of A per workgroup
  constexpr int NO = NR * RW / (OP == DENSE_GLU ? 2 : 1); // output columns of the workgroup
  constexpr int ES = FP8 ? 1 : 2;
  __shared__ f32x4_t red[RW][KW][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rw = wave / KW, kw = wave % KW, q = lane >> 4, ln = lane & 15;
  const int part = ln / NR, lr = ln % NR;
  const int n0 = blockIdx.x * NO, t0 = blockIdx.y * NR;
  const int wn = min(n0 + (OP == DENSE_GLU ? rw / 2 * NR : rw * NR) + lr, a.N - 1);
  const int64_t wrow = wn + (OP == DENSE_GLU && (rw & 1) ? (int64_t)a.N : 0);
  const int64_t xrow = min(t0 + lr, a.T - 1);
  const char* pw = static_cast<const char*>(a.b) + wrow * a.ldb * ES + 16 * q;
  const char* px = static_cast<const char*>(a.a) + xrow * a.lda * ES + 16 * q;
  const int kb = a.K * ES;                                // bytes of a row
  const int nk = (kb + 127) / 128;
  const int scales_k = FP8 ? a.K / 128 : 0;
  const float* sw = FP8 ? a.bs + wrow / 128 * scales_k : nullptr;
  const float* sx = FP8 ? a.as + xrow * scales_k : nullptr;
  f32x4_t acc = f32x4_t{0.f, 0.f, 0.f, 0.f};

  auto chunk = [&](const char* p, int at) {               // 16 bytes of this lane's row, zeros past its end
    return at + 16 * q < kb ? *reinterpret_cast<const uint4*>(p + at) : make_uint4(0, 0, 0, 0);
  };
  for (int k0 = kw * P; k0 < nk; k0 += KW * P * U) {
    uint4 w[U][2], x[U][2];
    float s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * KW * P + part, at = k * 128;
      w[u][0] = chunk(pw, at);
      w[u][1] = chunk(pw, at + 64);
      x[u][0] = chunk(px, at);
      x[u][1] = chunk(px, at + 64);
      // a lane's products belong to the k part of its column, and so does its scale; every weight row of
      // the fragment lies in one scale block
      if constexpr (FP8) s[u] = k < nk ? sx[k] * sw[k] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t wd[8] = {w[u][0].x, w[u][0].y, w[u][0].z, w[u][0].w, w[u][1].x, w[u][1].y, w[u][1].z, w[u][1].w};
      const uint32_t xd[8] = {x[u][0].x, x[u][0].y, x[u][0].z, x[u][0].w, x[u][1].x, x[u][1].y, x[u][1].z, x[u][1].w};
      if constexpr (FP8) {
        f32x4_t p = f32x4_t{0.f, 0.f, 0.f, 0.f};
        if constexpr (FP8 == 1) {
          i32x8_t wv, xv;
#pragma unroll
          for (int e = 0; e < 8; ++e) { wv[e] = (int)wd[e]; xv[e] = (int)xd[e]; }
          p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv, xv, p, 0, 0, 0, 0, 0, 0);   // no block scales
        } else {
#pragma unroll
          for (int e = 0; e < 8; e += 2)
            p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_e4m3(wd[e], wd[e + 1]), widen_e4m3(xd[e], xd[e + 1]), p,
                                                        0, 0, 0);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(p[e], s[u], acc[e]);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w[u][h]),
                                                        __builtin_bit_cast(bf16x8_t, x[u][h]), acc, 0, 0, 0);
      }
    }
  }
  red[rw][kw][lane] = acc;
  __syncthreads();

  // Four consecutive columns of one row per thread: their P parts of the KW sums.
  constexpr int kChunks = NO / 4;
  if (threadIdx.x >= NR * kChunks) return;
  const int tr = threadIdx.x / kChunks, c4 = (threadIdx.x % kChunks) * 4;
  auto total = [&](int frag, int r4, float (&v)[4]) {     // rows r4 .. r4 + 3 of fragment `frag`
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = 0.f;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        const f32x4_t m = red[frag][w][(p * NR + r4) / 4 * 16 + p * NR + tr];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += m[e];
      }
  };
  const int64_t t = t0 + tr;
  const int n = n0 + c4;
  if (t >= a.T || n >= a.N) return;
  float v[4];
  if constexpr (OP == DENSE_GLU) {
    float u[4];
    total(c4 / NR * 2, c4 % NR, v);
    total(c4 / NR * 2 + 1, c4 % NR, u);
    finish_glu(a, t, n, true, v, u);
  } else {
    total(c4 / NR, c4 % NR, v);
    finish_linear(a, t, n, v);
  }
}

namespace {

template <DenseOp OP, int FP8, bool AK, bool BK, int WT, int WN, int FT, int FN, int NST, int KS = 1>
void launch_tile(const DenseArgs& a, hipStream_t s) {
  constexpr int BT = WT * FT * 16, BN = WN * FN * 16, NO = OP == DENSE_GLU ? BN / 2 : BN;
  constexpr size_t kLds = tile_lds(BT, BN, NST, FP8, KS);
  static_assert(kLds <= 160 * 1024, "LDS of one workgroup");
  const int64_t tiles = (int64_t)((a.T + BT - 1) / BT) * ((a.N + NO - 1) / NO);
  auto k = dense_tile_kernel<OP, FP8, AK, BK, WT, WN, FT, FN, NST, KS>;
  k<<<dim3((unsigned)tiles), KS * WT * WN * 64, kLds, s>>>(a);
}

}  // namespace

template <DenseOp OP, bool AK, bool BK, int FN>
static void launch_pair(const DenseArgs& a, hipStream_t s) {
  constexpr int BN = 32 * FN, NO = OP == DENSE_GLU ? BN / 2 : BN;
  constexpr size_t kLds = 3 * 256 * 128 + 2 * BN * 128;
  static_assert(kLds <= 160 * 1024 && 128 * (BN + 4) * 4 <= kLds, "LDS of one workgroup");
  const int64_t tiles = (int64_t)((a.T + 255) / 256) * ((a.N + NO - 1) / NO);
  dense_pair_kernel<OP, AK, BK, FN><<<dim3((unsigned)tiles), 512, kLds, s>>>(a);
}

template <DenseOp OP, int FP8, int RW, int KW, int P, int U>
static void launch_few_n(const DenseArgs& a, hipStream_t s) {
  constexpr int NR = 16 / P, NO = NR * RW / (OP == DENSE_GLU ? 2 : 1);
  dense_few_kernel<OP, FP8, RW, KW, P, U><<<dim3((a.N + NO - 1) / NO, (a.T + NR - 1) / NR), RW * KW * 64, 0, s>>>(a);
}

// GLU with an e4m3 output: 128 output columns in one tile, a scale group.  The fewest rows that fill the units once
// (2 x 1536 x 2048 in FP8, by 16, 32, 64 and 128 rows: 256 rows 14.0, 17.1, 23.7, 34.3 us; 1024 rows 43.0, 32.7, 24.9,
// 35.0; 2048 rows 81.5, 48.3, 46.3, 36.0).
template <int FP8>
static void launch_glu_groups(const DenseArgs& a, hipStream_t s) {
  auto tiles = [&](int rows) { return (int64_t)((a.T + rows - 1) / rows) * (a.N / 128); };
  if (tiles(16) <= 256) launch_tile<DENSE_GLU, FP8, true, true, 1, 8, 1, 2, 4>(a, s);
  else if (tiles(32) <= 256) launch_tile<DENSE_GLU, FP8, true, true, 1, 8, 2, 2, 4>(a, s);
  else if (tiles(64) <= 256) launch_tile<DENSE_GLU, FP8, true, true, 1, 8, 4, 2, 3>(a, s);
  else launch_tile<DENSE_GLU, FP8, true, true, 2, 4, 4, 4, 3>(a, s);
}

template <DenseOp OP, int FP8, bool AK, bool BK>
static void launch_sized(const DenseArgs& a, hipStream_t s) {
  auto tiles = [&](int bt, int bn) {
    return (int64_t)((a.T + bt - 1) / bt) * (((OP == DENSE_GLU ? 2 : 1) * (int64_t)a.N + bn - 1) / bn);
  };
  // Few rows: blocks of 16, 8 or 4 weight rows, for 16, 8 or 4 rows of x.  Fewer weight rows a block spread a small
  // weight over the units (8 x 2048 x 6144 in bf16: 16 rows 11.8, 8 rows 8.5 us; 1 x 512 x 6144: 9.3, 6.3 and, with
  // 4, 5.1), more of them use the matrix instructions better (4 x 4096 x 6144: 12.3, 12.6, 14.7; 8 x 3080 x 6144: 12.3,
  // 14.3).  From 3 rows on the tiles below win where the blocks are more than the units (8 x 6144 x 6144: 21.0 against
  // 14.4 us) until their own are too (8 x 12288 x 2048: 11.7 against 12.6), and not where their start and end are
  // most of the time (6 x 4828 x 440: 4.9 against 5.6).
  if constexpr (OP == DENSE_LINEAR && AK && BK) {
    if (a.T <= 4 && a.N < 2048) {
      launch_few_n<OP, FP8, 1, 8, 4, 4>(a, s);
      return;
    }
    if (a.T <= 8 && a.N < 2560) {
      launch_few_n<OP, FP8, 1, 8, 2, 4>(a, s);
      return;
    }
    if ((int64_t)((a.T + 15) / 16) * ((a.N + 15) / 16) <= 256 || a.T <= 2 || (a.T <= 8 && (a.N > 8192 || a.K < 1024))) {
      launch_few_n<OP, FP8, 1, 8, 1, 4>(a, s);
      return;
    }
  }
  // A GLU reads two weight rows per column, so it needs half the columns (T x I x H = 1 x 1024 x 2048: 4 rows 4.5, 8 rows
  // 5.3 us; 1 x 2048 x 2048: 5.7, 5.4), and tiles win earlier (8 x 4096 x 2048: 10.5 against 9.2 us; 1 x 6144 x 2048: 10.7
  // against 11.0) but for short sums (9 x 608 x 984: 4.6 against 6.6; 16 x 4096 x 1024: 6.8 and 6.8; x 2048: 10.6
  // against 9.1).
  if constexpr (OP == DENSE_GLU) {
    if (a.T <= 4 && a.N < 1280) {
      launch_few_n<OP, FP8, 2, 2, 4, 4>(a, s);
      return;
    }
    if (a.T <= 2 || (a.T <= 8 && a.N < 2560)) {
      launch_few_n<OP, FP8, 2, 4, 2, 4>(a, s);
      return;
    }
    if (a.K <= 1280 && (int64_t)((a.T + 15) / 16) * ((a.N + 15) / 16) <= 256) {
      launch_few_n<OP, FP8, 2, 4, 1, 4>(a, s);
      return;
    }
  }
  if (tiles(128, 128) >= 256) {
    // The fewest rounds of tiles over the 256 units, each in the time of a 256 x 256 tile's (us for one round of
    // 4096 k: 99 with K-major operands, 98 with both k-slow): 256 x 192 takes 0.75 (0.86), 256 x 128 0.62 (0.72: never
    // the least), and two 128 x 128 a unit 0.68 (0.62).  Of K-major operands also two 128 x 96 a unit, 0.53 (2048 x
    // 2880 x 2880: 36.0 us, as 256 x 128 40.9), and two 64 x 128, three stages deep, if they are all of it, 0.42 (2048 x
    // 2048 x 6144: 60.9 us, as 256 x 128 74.3).  The fractions are measured at these sizes; elsewhere they are a model.
    // Not for the gradient of h: there the epilogue's bytes weigh as much, and the smaller tiles of two workgroups a
    // unit overlap them (4096 x 6144 x 2048: 144 against 164 us).
    if constexpr (FP8 == 0 && OP != DENSE_DGLU) {
      auto rounds = [](int64_t n, int64_t per) { return (float)((n + per - 1) / per); };
      constexpr bool slow = !AK && !BK;
      const float c256 = rounds(tiles(256, 256), 256), c192 = (slow ? 0.86f : 0.75f) * rounds(tiles(256, 192), 256);
      const float c128 = 0.62f * rounds(tiles(256, 128), 256);
      const float small = (slow ? 0.62f : 0.68f) * rounds(tiles(128, 128), 512);
      const float best = std::min(std::min(c256, c192), slow ? small : std::min(c128, small));
      if constexpr (AK && BK) {
        const float c96 = 0.53f * rounds(tiles(128, 96), 512);
        if (tiles(64, 128) <= 512) {   // (none of the others takes less)
          launch_tile<OP, FP8, AK, BK, 2, 2, 2, 4, 3>(a, s);
          return;
        }
        if (c96 < best) {
          launch_tile<OP, FP8, AK, BK, 2, 2, 4, 3, 2>(a, s);
          return;
        }
      }
      if (best == c256) {
        launch_pair<OP, AK, BK, 8>(a, s);
        return;
      }
      if (best == c192) {
        launch_pair<OP, AK, BK, 6>(a, s);
        return;
      }
      if constexpr (!slow) {
        if (best == c128) {
          launch_pair<OP, AK, BK, 4>(a, s);
          return;
        }
      }
      launch_tile<OP, FP8, AK, BK, 2, 2, 4, 4, 2>(a, s);
      return;
    }
    if constexpr (FP8 != 0) {
      // one 128 x 128 tile a unit, or little more, leaves units waiting for their copies: two of 64 x 128 (N = 2048: T =
      // 2048, 256 tiles, k = 6144 57 -> 50 us; 2176, 272 tiles, k = 2048 21.6 -> 20.7 and k = 6144 57.7 -> 51.2; with
      // more neither is always better: 2560, 320 tiles, k = 2048 20.9 -> 21.1, k = 6144 55.5 -> 54.1; GLU of 640 x
      // 3840 x 2048, 300 tiles, 21.0 -> 22.8; 4096, 512 tiles, k = 2048 23.0 -> 33.2)
      if (tiles(128, 128) <= 288) launch_tile<OP, FP8, AK, BK, 2, 2, 2, 4, 2>(a, s);
      else launch_tile<OP, FP8, AK, BK, 4, 2, 2, 4, 2>(a, s);
    } else {
      launch_tile<OP, FP8, AK, BK, 2, 4, 4, 2, 2>(a, s);
    }
  } else if (tiles(64, 64) > 256) {
    // less than one 128 x 128 tile a unit: 64 x 64 (512 x 3000 x 2048: 14.7 against 20.9 us).  Of K-major bf16 operands,
    // where those are more than two a unit, two of 64 x 96 (1023 x 2880 x 2880: 28.5 -> 26.0 us, 1300 x 2048 x 5000: 67.4 ->
    // 57.9), and where they are not, four stages for long sums, which leave the caches (400 x 2880 x 2880: 24.7 -> 18.8 us,
    // 1024 x 2048 x 6144: 49.4 -> 40.0; of 2048 k 15.3 -> 15.7).
    if constexpr (FP8 == 0 && AK && BK) {
      if (tiles(64, 64) <= 512 && a.K > 2560) {
        launch_tile<OP, FP8, AK, BK, 2, 2, 2, 2, 4>(a, s);
        return;
      }
      if (tiles(64, 64) > 512 && tiles(64, 96) <= 512) {
        launch_tile<OP, FP8, AK, BK, 2, 2, 2, 3, 4>(a, s);
        return;
      }
    }
    launch_tile<OP, FP8, AK, BK, 2, 2, 2, 2, 2>(a, s);
  } else if (tiles(64, 64) <= 128 || tiles(32, OP == DENSE_GLU ? 64 : 32) <= 256 ||
             (FP8 != 0 && OP == DENSE_LINEAR && (a.T <= 32 || a.K >= 6144))) {
    // few of those too, or few rows: smaller ones, their k in four shares (100 x 2048 x 6144: 30.1 -> 15.0 us, GLU of
    // 8 x 6144 x 2048: 12.7 -> 11.4).  In FP8 also up to 256, where its long sums wait for single tiles' copies (320 x
    // 2048 x 8192: 43.8 -> 30.6 us, x 7168 38.2 -> 27.3, x 6144 24.6 -> 24.3; 600 x 1536 x 6144 34.1 -> 27.3; 320 x
    // 2048 x 4096 is 17.3 against 18.9).
    if (OP == DENSE_GLU || tiles(32, 32) <= 256)
      launch_tile<OP, FP8, AK, BK, 2, 2, 1, OP == DENSE_GLU ? 2 : 1, 3, 4>(a, s);
    else                             // two a unit: two stages each (500 x 1024 x 4096: 20.5 -> 17.0 us)
      launch_tile<OP, FP8, AK, BK, 2, 2, 1, OP == DENSE_GLU ? 2 : 1, 2, 4>(a, s);
  } else {
    // one a unit: four stages (320 x 2048 x 4096: 32.5 -> 21.8 us; of 2048 k 11.5 -> 12.5)
    launch_tile<OP, FP8, AK, BK, 2, 2, 2, 2, 4>(a, s);
  }
}

void launch_dense(DenseOp op, bool fp8, bool ak, bool bk, const DenseArgs& a, hipStream_t s) {
  // e4m3 operands are widened to bf16 where the output or its scales are kept in fp32
  if (op == DENSE_GLU && a.hs && fp8) launch_glu_groups<2>(a, s);
  else if (op == DENSE_GLU && a.hs) launch_glu_groups<0>(a, s);
  else if (op == DENSE_GLU && fp8) launch_sized<DENSE_GLU, 1, true, true>(a, s);
  else if (op == DENSE_GLU) launch_sized<DENSE_GLU, 0, true, true>(a, s);
  else if (op == DENSE_DGLU) launch_sized<DENSE_DGLU, 0, true, false>(a, s);
  else if (fp8 && a.y_f32) launch_sized<DENSE_LINEAR, 2, true, true>(a, s);
  else if (fp8) launch_sized<DENSE_LINEAR, 1, true, true>(a, s);
  else if (ak && bk) launch_sized<DENSE_LINEAR, 0, true, true>(a, s);
  else if (ak) launch_sized<DENSE_LINEAR, 0, true, false>(a, s);
  else launch_sized<DENSE_LINEAR, 0, false, false>(a, s);
}

void launch_dense_grads(const DenseArgs* dx, const DenseArgs* dw13, const DenseArgs* dw2, hipStream_t s) {
  auto tiles = [](const DenseArgs& a, int side) {
    return (int64_t)((a.T + side - 1) / side) * ((a.N + side - 1) / side);
  };
  // Where none fills the units with larger tiles, one launch (257 x 2048 x 768: 16 us for what took 22 in three);
  // larger ones go by themselves, each with the tile it is best with.  So does dx if its tiles are few and its
  // sums long (29 x 216 x 2512: 38 -> 24 us): by itself its k is split.
  if (dw13 && dw2 && (!dx || tiles(*dx, 128) < 256) && tiles(*dw13, 128) < 256 && tiles(*dw2, 128) < 256) {
    if (dx && tiles(*dx, 64) <= 128 && dx->K >= 1024) {
      launch_dense(DENSE_LINEAR, false, true, false, *dx, s);
      dx = nullptr;
    }
    const int n0 = dx ? (int)tiles(*dx, 64) : 0, n1 = (int)tiles(*dw13, 64), n2 = (int)tiles(*dw2, 64);
    const DenseArgs x = dx ? *dx : *dw13;
    const int weights_first = dw13->K > x.K;
    // at most a tile a unit: their k in four shares (132 x 1184 x 1456: 35 -> 28 us; at 304 and 464 tiles 45 -> 37, 36 -> 38)
    if (n0 + n1 + n2 <= 256)
      dense_grads_kernel<4><<<dim3(n0 + n1 + n2), 1024, tile_lds(64, 64, 2, 0, 4), s>>>(x, *dw13, *dw2, n0, n1, n2,
                                                                                     weights_first);
    else
      dense_grads_kernel<1><<<dim3(n0 + n1 + n2), 256, tile_lds(64, 64, 2, 0), s>>>(x, *dw13, *dw2, n0, n1, n2,
                                                                                  weights_first);
    return;
  }
  if (dx) launch_dense(DENSE_LINEAR, false, true, false, *dx, s);
  if (dw13) launch_dense(DENSE_LINEAR, false, false, false, *dw13, s);
  if (dw2) launch_dense(DENSE_LINEAR, false, false, false, *dw2, s);
}

}  // namespace pe
