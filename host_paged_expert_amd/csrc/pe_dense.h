// Launchers of the dense operators around a paged MoE layer (defined in
// pe_dense.hip): residual addition + RMS norm, top-k routing, and the matrix
// products of the projections, the gated feed-forward block and its gradients.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace pe {

struct NormArgs {
  const uint16_t* x;          // bf16 [T, H], rows ldx apart
  int64_t ldx;
  const uint16_t* residual;   // bf16 [T, H] or nullptr
  int64_t ldr;
  const uint16_t* weight;     // bf16 [H]
  float eps;
  int T, H;
  uint16_t* sum;              // bf16 [T, H] or nullptr
  int64_t lds;
  void* y;                    // bf16 [T, H], or e4m3 codes if yscale
  int64_t ldy;
  float* yscale;              // fp32 [T, H / 128] or nullptr
};

struct RouteArgs {
  const float* logits;        // fp32 [T, E], rows ldl apart
  int64_t ldl;
  int T, E, k;
  int sigmoid, renorm;
  float scale;
  int32_t* ids;               // [T, k]
  float* w;                   // [T, k]
};

// What a product does with its accumulators.  t is a row of the left operand,
// n a row of the right one.
enum DenseOp {
  DENSE_LINEAR,     // y[t, n] = act(acc + bias[n]) + residual[t, n]
  DENSE_GLU,        // gate and up accumulators of column n: h[t, n] = act(g) * u
  DENSE_DGLU,       // acc = dh[t, n]: dgu[t, n], dgu[t, N + n] and h[t, n]
};

// out[t, n] = sum_k A[t, k] B[n, k].  A K-major operand has rows of k (ld
// elements apart); a k-slow one is stored transposed, row k holding every t
// (or n).
struct DenseArgs {
  const void* a;              // left operand
  int64_t lda;
  const float* as;            // FP8: [T, K / 128] scales
  const void* b;              // right operand
  int64_t ldb;
  const float* bs;            // FP8: [ceil(N / 128), K / 128] scales (GLU: gate rows, then up rows)
  int T, N, K;
  int act;
  const uint16_t* bias;       // LINEAR: bf16 [N] or nullptr
  const uint16_t* residual;   // LINEAR: bf16 [T, N] or nullptr
  int64_t ldr;
  void* y;                    // LINEAR: bf16 or fp32; GLU: h, bf16 or e4m3 (if hs); DGLU: h bf16 or nullptr
  int64_t ldy;
  int y_f32;
  float* hs;                  // GLU: [T, N / 128] scales of an e4m3 h, or nullptr
  uint16_t* gu;               // GLU: bf16 [T, 2N] to keep, or nullptr; DGLU: the kept one
  uint16_t* dgu;              // DGLU: bf16 [T, 2N]
  int vec;                    // outputs, residual and bias may be accessed 8 columns at a time
};

void launch_rmsnorm(const NormArgs& a, hipStream_t s);
void launch_route(const RouteArgs& a, hipStream_t s);
// fp8: both operands are e4m3 with scales; ak / bk: the operand is K-major.
void launch_dense(DenseOp op, bool fp8, bool ak, bool bk, const DenseArgs& a, hipStream_t s);
// The products dx (A K-major, B k-slow), dw13 and dw2 (both k-slow); any may be null.
void launch_dense_grads(const DenseArgs* dx, const DenseArgs* dw13, const DenseArgs* dw2, hipStream_t s);

}  // namespace pe
