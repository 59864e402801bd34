// Device code that the tiled and the streaming matrix products share (pe_dense.hip,
// pe_grouped.hip): number formats, activations, reductions over lanes, copies into
// LDS, operand tiles and their fragments, and what is done with the accumulators.
#pragma once
#include <hip/hip_runtime.h>

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

}  // namespace pe
