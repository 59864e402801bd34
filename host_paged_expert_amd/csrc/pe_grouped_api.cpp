// C entry points of the products grouped by expert, of the 4-bit products and of
// what stands around them (include/pe.h): argument checks, the device of the
// call, and the launches.  They hold no state and allocate nothing.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "../../include/pe.h"
#include "pe_check.h"
#include "pe_error.h"
#include "pe_grouped.h"
#include "pe_layout.h"

namespace {

// A launch has fewer than 2^32 threads, so fewer than 2^23 workgroups of 512.  The products' smallest tiles are 16 x 64,
// the weight gradients' 128 x 128 for each matrix.
int check_tiles(int64_t tiles) {
  if (tiles >= (1 << 23)) return fail(PE_ERR_INVALID_ARG, "the matrices are too large for one call");
  return PE_OK;
}
int64_t row_tiles(int64_t rows, int64_t matrices, int64_t cols) { return (rows / 16 + matrices + 1) * ((cols + 63) / 64); }
int64_t weight_tiles(int64_t matrices, int64_t rows, int64_t cols) {
  return matrices * (((rows + 127) / 128 * ((cols + 127) / 128) + 7) / 8 * 8);
}

int check_experts(int num_experts) {
  if (num_experts < 1 || num_experts > pe::kMaxExperts)
    return fail(PE_ERR_INVALID_ARG, "num_experts=%d outside [1, %d]", num_experts, pe::kMaxExperts);
  return PE_OK;
}

// Weights of `rows` rows and `k` columns for each of E matrices, and their scales.
struct Weights {
  Mat w, s;
};
int check_weights(const char* name, const char* scale_name, int wtype, const void* w, const void* scales, int64_t E,
                  int64_t rows, int K, bool bf16_ok, Weights* out) {
  const bool q = wtype == PE_W_INT4_G128 || wtype == PE_W_MXFP4_B32;
  if (!q && !(bf16_ok && wtype == PE_W_BF16))
    return fail(PE_ERR_UNSUPPORTED, "weights must be %sPE_W_INT4_G128 or PE_W_MXFP4_B32", bf16_ok ? "PE_W_BF16, " : "");
  const int step = !q ? 8 : wtype == PE_W_INT4_G128 ? 128 : 32;
  if (K % step) return fail(PE_ERR_INVALID_ARG, "the summed dimension must be a multiple of %d for these weights", step);
  const int64_t cols = q ? K / 2 : K;
  out->w = Mat{name, w, E * rows, cols, cols, q ? 1 : 2, 16};
  out->s = Mat{scale_name, scales, E * rows, K / step, K / step, wtype == PE_W_INT4_G128 ? 2 : 1, 16};
  if (q) out->s.align = 1;   // rows of any length; the address is checked below
  PE_TRY(check_mat(out->w, false));
  if (!q) {
    if (scales) return fail(PE_ERR_INVALID_ARG, "bf16 weights take no scales");
    return PE_OK;
  }
  PE_TRY(check_mat(out->s, false));
  if ((uintptr_t)scales % 16) return fail(PE_ERR_INVALID_ARG, "%s: address must be a multiple of 16 bytes", scale_name);
  return PE_OK;
}

// A product's arguments in common.
pe::GroupedArgs product(const void* x, int64_t ldx, int x_rows, const int32_t* rows, const int32_t* offsets, int E, int R,
                        const void* w, const void* scales, int N, int K, int act) {
  pe::GroupedArgs g{};
  g.d.a = x; g.d.lda = ldx;
  g.d.b = w; g.d.ldb = K;
  g.d.T = R; g.d.N = N; g.d.K = K; g.d.act = act;
  g.offsets = offsets; g.rows = rows;
  g.E = E; g.R = R; g.x_rows = x_rows;
  g.ws = scales;
  return g;
}

}  // namespace

extern "C" {

int pe_linear_w4(int device, int wtype, const void* x, int64_t ldx, const void* w, const void* wscale, const void* bias,
                 int act, const void* residual, int64_t ldr, int T, int N, int K, void* y, int64_t ldy, int ytype,
                 void* stream) {
  PE_TRY(check_dims(device, T, {N, K}));
  PE_TRY(check_act(act, true));
  if (ytype != PE_Y_BF16 && ytype != PE_Y_FP32) return fail(PE_ERR_INVALID_ARG, "unknown output type %d", ytype);
  const int ys = ytype == PE_Y_FP32 ? 4 : 2;
  const Mat mx{"x", x, T, K, ldx, 2, 16}, mb{"bias", bias, 1, N, N, 2, 2}, mr{"residual", residual, T, N, ldr, 2, 2};
  const Mat my{"y", y, T, N, ldy, ys, ys};
  Weights mw;
  if (T == 0) return PE_OK;
  PE_TRY(check_weights("w", "wscale", wtype, w, wscale, 1, N, K, false, &mw));
  PE_TRY(check_mat(mx, false));
  PE_TRY(check_mat(mb, true));
  PE_TRY(check_mat(mr, true));
  PE_TRY(check_mat(my, false));
  PE_TRY(check_tiles(row_tiles(T, 1, N)));
  PE_TRY(check_apart({{&my, {&mr}}}, {&mx, &mw.w, &mw.s, &mb, &mr}));
  DeviceScope dev(device);
  PE_HIP(dev.err);
  pe::GroupedArgs g = product(x, ldx, T, nullptr, nullptr, 1, T, w, wscale, N, K, act);
  g.d.bias = static_cast<const uint16_t*>(bias);
  g.d.residual = static_cast<const uint16_t*>(residual); g.d.ldr = ldr;
  g.d.y = y; g.d.ldy = ldy; g.d.y_f32 = ytype == PE_Y_FP32;
  g.d.vec = vec8(my) && vec8(mr) && (uintptr_t)bias % 16 == 0;
  pe::launch_grouped(pe::DENSE_LINEAR, wtype, g, static_cast<hipStream_t>(stream));
  PE_HIP(hipGetLastError());
  return PE_OK;
}

int pe_glu_w4(int device, int wtype, int act, const void* x, int64_t ldx, const void* w13, const void* s13, int T,
              int hidden, int inter, void* h, int64_t ldh, void* stream) {
  const int H = hidden, I = inter;
  PE_TRY(check_dims(device, T, {H, I}));
  PE_TRY(check_act(act, false));
  if (I % 8) return fail(PE_ERR_INVALID_ARG, "inter must be a multiple of 8");
  const Mat mx{"x", x, T, H, ldx, 2, 16}, mh{"h", h, T, I, ldh, 2, 2};
  Weights mw;
  if (T == 0) return PE_OK;
  PE_TRY(check_weights("w13", "s13", wtype, w13, s13, 1, 2 * (int64_t)I, H, false, &mw));
  PE_TRY(check_mat(mx, false));
  PE_TRY(check_mat(mh, false));
  PE_TRY(check_tiles(row_tiles(T, 1, I)));
  PE_TRY(check_apart({{&mh, {}}}, {&mx, &mw.w, &mw.s}));
  DeviceScope dev(device);
  PE_HIP(dev.err);
  pe::GroupedArgs g = product(x, ldx, T, nullptr, nullptr, 1, T, w13, s13, I, H, act);
  g.d.y = h; g.d.ldy = ldh;
  g.d.vec = vec8(mh);
  pe::launch_grouped(pe::DENSE_GLU, wtype, g, static_cast<hipStream_t>(stream));
  PE_HIP(hipGetLastError());
  return PE_OK;
}

int pe_group_rows(int device, const int32_t* topk_ids, int T, int top_k, int num_experts, int32_t* offsets, int32_t* rows,
                  int32_t* places, void* stream) {
  const int E = num_experts, k = top_k;
  PE_TRY(check_dims(device, T, {k}));
  PE_TRY(check_experts(E));
  if ((int64_t)T * k >= kMaxRows) return fail(PE_ERR_INVALID_ARG, "T * top_k=%lld is not below 2^24", (long long)T * k);
  const int n = T * k;
  const Mat mi{"topk_ids", topk_ids, T, k, k, 4, 4}, mo{"offsets", offsets, 1, E + 1, E + 1, 4, 4};
  const Mat mr{"rows", rows, 1, n, n, 4, 4}, mp{"places", places, T, k, k, 4, 4};
  PE_TRY(check_mat(mo, false));
  if (n) {
    if (!topk_ids || !rows || !places) return fail(PE_ERR_INVALID_ARG, "topk_ids, rows or places is NULL");
    if (((uintptr_t)topk_ids | (uintptr_t)rows | (uintptr_t)places) % 4)
      return fail(PE_ERR_INVALID_ARG, "topk_ids, rows and places must be multiples of 4 bytes");
    PE_TRY(check_apart({{&mo, {}}, {&mr, {}}, {&mp, {}}}, {&mi}));
  }
  DeviceScope dev(device);
  PE_HIP(dev.err);
  pe::GroupRowsArgs a{topk_ids, n, k, E, offsets, rows, places};
  pe::launch_group_rows(a, static_cast<hipStream_t>(stream));
  PE_HIP(hipGetLastError());
  return PE_OK;
}

int pe_grouped_linear(int device, int wtype, const void* x, int64_t ldx, int x_rows, const int32_t* rows,
                      const int32_t* offsets, const void* w, const void* wscale, const void* bias, int act, int R,
                      int num_experts, int N, int K, void* y, int64_t ldy, int ytype, void* stream) {
  const int E = num_experts;
  PE_TRY(check_dims(device, R, {N, K}));
  PE_TRY(check_experts(E));
  PE_TRY(check_act(act, true));
  if (ytype != PE_Y_BF16 && ytype != PE_Y_FP32) return fail(PE_ERR_INVALID_ARG, "unknown output type %d", ytype);
  if (R == 0) return PE_OK;
  const int xr = rows ? x_rows : R, ys = ytype == PE_Y_FP32 ? 4 : 2;
  if (xr < 1 || xr >= kMaxRows) return fail(PE_ERR_INVALID_ARG, "x_rows=%d outside [1, 2^24)", xr);
  const Mat mx{"x", x, xr, K, ldx, 2, 16}, mrow{"rows", rows, 1, R, R, 4, 4}, mo{"offsets", offsets, 1, E + 1, E + 1, 4, 4};
  const Mat mb{"bias", bias, E, N, N, 2, 2}, my{"y", y, R, N, ldy, ys, ys};
  Weights mw;
  PE_TRY(check_weights("w", "wscale", wtype, w, wscale, E, N, K, true, &mw));
  PE_TRY(check_mat(mx, false));
  if ((uintptr_t)rows % 4) return fail(PE_ERR_INVALID_ARG, "rows must be a multiple of 4 bytes");
  PE_TRY(check_mat(mo, false));
  PE_TRY(check_mat(mb, true));
  PE_TRY(check_mat(my, false));
  PE_TRY(check_tiles(row_tiles(R, E, N)));
  PE_TRY(check_apart({{&my, {}}}, {&mx, &mrow, &mo, &mw.w, &mw.s, &mb}));
  DeviceScope dev(device);
  PE_HIP(dev.err);
  pe::GroupedArgs g = product(x, ldx, xr, rows, offsets, E, R, w, wscale, N, K, act);
  g.d.bias = static_cast<const uint16_t*>(bias);
  g.d.y = y; g.d.ldy = ldy; g.d.y_f32 = ytype == PE_Y_FP32;
  g.d.vec = vec8(my) && (!bias || ((uintptr_t)bias % 16 == 0 && N % 8 == 0));
  pe::launch_grouped(pe::DENSE_LINEAR, wtype, g, static_cast<hipStream_t>(stream));
  PE_HIP(hipGetLastError());
  return PE_OK;
}

int pe_grouped_glu(int device, int wtype, int act, const void* x, int64_t ldx, int x_rows, const int32_t* rows,
                   const int32_t* offsets, const void* w13, const void* s13, int R, int num_experts, int hidden, int inter,
                   void* h, int64_t ldh, void* gu, void* stream) {
  const int E = num_experts, H = hidden, I = inter;
  PE_TRY(check_dims(device, R, {H, I}));
  PE_TRY(check_experts(E));
  PE_TRY(check_act(act, false));
  if (I % 8) return fail(PE_ERR_INVALID_ARG, "inter must be a multiple of 8");
  if (R == 0) return PE_OK;
  const int xr = rows ? x_rows : R;
  if (xr < 1 || xr >= kMaxRows) return fail(PE_ERR_INVALID_ARG, "x_rows=%d outside [1, 2^24)", xr);
  const Mat mx{"x", x, xr, H, ldx, 2, 16}, mrow{"rows", rows, 1, R, R, 4, 4}, mo{"offsets", offsets, 1, E + 1, E + 1, 4, 4};
  const Mat mh{"h", h, R, I, ldh, 2, 2}, mg{"gu", gu, R, 2 * (int64_t)I, 2 * (int64_t)I, 2, 16};
  Weights mw;
  PE_TRY(check_weights("w13", "s13", wtype, w13, s13, E, 2 * (int64_t)I, H, true, &mw));
  PE_TRY(check_mat(mx, false));
  if ((uintptr_t)rows % 4) return fail(PE_ERR_INVALID_ARG, "rows must be a multiple of 4 bytes");
  PE_TRY(check_mat(mo, false));
  PE_TRY(check_mat(mh, false));
  PE_TRY(check_mat(mg, true));
  PE_TRY(check_tiles(row_tiles(R, E, I)));
  PE_TRY(check_apart({{&mh, {}}, {&mg, {}}}, {&mx, &mrow, &mo, &mw.w, &mw.s}));
  DeviceScope dev(device);
  PE_HIP(dev.err);
  pe::GroupedArgs g = product(x, ldx, xr, rows, offsets, E, R, w13, s13, I, H, act);
  g.d.y = h; g.d.ldy = ldh;
  g.d.gu = static_cast<uint16_t*>(gu);
  g.d.vec = vec8(mh);
  pe::launch_grouped(pe::DENSE_GLU, wtype, g, static_cast<hipStream_t>(stream));
  PE_HIP(hipGetLastError());
  return PE_OK;
}

int pe_combine(int device, const void* y, int64_t ldy, int R, const int32_t* places, const float* topk_w,
               const void* residual, int64_t ldr, int T, int top_k, int H, void* out, int64_t ldo, void* stream) {
  const int k = top_k;
  PE_TRY(check_dims(device, T, {k, H}));
  if (R < 0 || R >= kMaxRows) return fail(PE_ERR_INVALID_ARG, "R=%d outside [0, 2^24)", R);
  if ((int64_t)T * k >= (1ll << 31)) return fail(PE_ERR_INVALID_ARG, "T * top_k=%lld is not below 2^31", (long long)T * k);
  if (H % 8) return fail(PE_ERR_INVALID_ARG, "H must be a multiple of 8");
  if (T == 0) return PE_OK;
  const Mat my{"y", y, R, H, ldy, 2, 16}, mp{"places", places, 1, (int64_t)T * k, (int64_t)T * k, 4, 4};
  const Mat mw{"topk_w", topk_w, 1, (int64_t)T * k, (int64_t)T * k, 4, 4};
  const Mat mr{"residual", residual, T, H, ldr, 2, 16}, mo{"out", out, T, H, ldo, 2, 16};
  PE_TRY(check_mat(my, R == 0));
  if (!places || ((uintptr_t)places | (uintptr_t)topk_w) % 4)
    return fail(PE_ERR_INVALID_ARG, "places is NULL, or places or topk_w is no multiple of 4 bytes");
  PE_TRY(check_mat(mr, true));
  PE_TRY(check_mat(mo, false));
  PE_TRY(check_apart({{&mo, {&mr}}}, {&my, &mp, &mw, &mr}));
  DeviceScope dev(device);
  PE_HIP(dev.err);
  pe::CombineArgs a{static_cast<const uint16_t*>(y), ldy, places, topk_w, static_cast<const uint16_t*>(residual), ldr, T, k,
                    H, y ? R : 0, static_cast<uint16_t*>(out), ldo};
  pe::launch_combine(a, static_cast<hipStream_t>(stream));
  PE_HIP(hipGetLastError());
  return PE_OK;
}

int pe_combine_backward(int device, const void* dout, int64_t lddo, const int32_t* places, const float* topk_w,
                        const void* y, int64_t ldy, int R, int T, int top_k, int H, void* dy, int64_t lddy, float* dtopk_w,
                        void* stream) {
  const int k = top_k;
  PE_TRY(check_dims(device, T, {k, H}));
  if (R < 0 || R >= kMaxRows) return fail(PE_ERR_INVALID_ARG, "R=%d outside [0, 2^24)", R);
  // a wavefront for each entry
  if ((int64_t)T * k >= (1 << 25)) return fail(PE_ERR_INVALID_ARG, "T * top_k=%lld is not below 2^25", (long long)T * k);
  if (H % 8) return fail(PE_ERR_INVALID_ARG, "H must be a multiple of 8");
  if (T == 0 || (R == 0 && !dtopk_w)) return PE_OK;   // (an empty dy has no address)
  if (!dy && !dtopk_w) return fail(PE_ERR_INVALID_ARG, "no gradient is asked for");
  const Mat mdo{"dout", dout, T, H, lddo, 2, 16}, mp{"places", places, 1, (int64_t)T * k, (int64_t)T * k, 4, 4};
  const Mat mw{"topk_w", topk_w, 1, (int64_t)T * k, (int64_t)T * k, 4, 4}, my{"y", y, R, H, ldy, 2, 16};
  const Mat mdy{"dy", dy, R, H, lddy, 2, 16}, mdw{"dtopk_w", dtopk_w, 1, (int64_t)T * k, (int64_t)T * k, 4, 4};
  PE_TRY(check_mat(mdo, false));
  if (!places || ((uintptr_t)places | (uintptr_t)topk_w | (uintptr_t)dtopk_w) % 4)
    return fail(PE_ERR_INVALID_ARG, "places is NULL, or places, topk_w or dtopk_w is no multiple of 4 bytes");
  PE_TRY(check_mat(my, R == 0 || !dtopk_w));
  PE_TRY(check_mat(mdy, true));
  PE_TRY(check_apart({{&mdy, {}}, {&mdw, {}}}, {&mdo, &mp, &mw, &my}));
  DeviceScope dev(device);
  PE_HIP(dev.err);
  pe::CombineBackArgs a{static_cast<const uint16_t*>(dout), lddo, places, topk_w, static_cast<const uint16_t*>(y), ldy, T, k,
                        H, R, static_cast<uint16_t*>(dy), lddy, dtopk_w};
  pe::launch_combine_back(a, static_cast<hipStream_t>(stream));
  PE_HIP(hipGetLastError());
  return PE_OK;
}

int pe_grouped_ffn_backward(int device, int act, const void* dy, int64_t lddy, const void* x, int64_t ldx, int x_rows,
                            const int32_t* rows, const int32_t* offsets, const void* gu, const void* w13, const void* w2,
                            int R, int num_experts, int hidden, int inter, void* dgu, void* h, void* dx, int64_t lddx,
                            void* dw13, void* dw2, void* stream) {
  const int E = num_experts, H = hidden, I = inter;
  PE_TRY(check_dims(device, R, {H, I}));
  PE_TRY(check_experts(E));
  PE_TRY(check_act(act, false));
  if (H % 8 || I % 8) return fail(PE_ERR_INVALID_ARG, "hidden and inter must be multiples of 8");
  if (H >= kMaxStride || I >= kMaxStride / 2)
    return fail(PE_ERR_INVALID_ARG, "hidden=%d or 2 * inter=2 * %d is not below 2^22", H, I);
  if (R > 0 && !dx && !dw13 && !dw2) return fail(PE_ERR_INVALID_ARG, "no gradient is asked for");   // (an empty dx has no address)
  const int64_t I2 = 2 * (int64_t)I;
  const int xr = rows ? x_rows : R;
  const Mat mdy{"dy", dy, R, H, lddy, 2, 16}, mx{"x", x, xr, H, ldx, 2, 16}, mgu{"gu", gu, R, I2, I2, 2, 16};
  const Mat mrow{"rows", rows, 1, R, R, 4, 4}, mo{"offsets", offsets, 1, E + 1, E + 1, 4, 4};
  const Mat mw13{"w13", w13, E * I2, H, H, 2, 16}, mw2{"w2", w2, (int64_t)E * H, I, I, 2, 16};
  const Mat mdgu{"dgu", dgu, R, I2, I2, 2, 16}, mh{"h", h, R, I, I, 2, 16}, mdx{"dx", dx, R, H, lddx, 2, 16};
  const Mat mdw13{"dw13", dw13, E * I2, H, H, 2, 16}, mdw2{"dw2", dw2, (int64_t)E * H, I, I, 2, 16};
  PE_TRY(check_mat(mo, false));
  PE_TRY(check_mat(mdw13, true));
  PE_TRY(check_mat(mdw2, true));
  if (R > 0) {
    PE_TRY(check_mat(mdy, false));
    PE_TRY(check_mat(mgu, false));
    PE_TRY(check_mat(mw13, !dx));
    PE_TRY(check_mat(mw2, false));
    PE_TRY(check_mat(mdgu, false));
    PE_TRY(check_mat(mh, !dw2));
    PE_TRY(check_mat(mdx, true));
    if (dw13) {
      if (xr < 1 || xr >= kMaxRows) return fail(PE_ERR_INVALID_ARG, "x_rows=%d outside [1, 2^24)", xr);
      PE_TRY(check_mat(mx, false));
    }
    if ((uintptr_t)rows % 4) return fail(PE_ERR_INVALID_ARG, "rows must be a multiple of 4 bytes");
    PE_TRY(check_tiles(row_tiles(R, E, std::max(H, I))));
  }
  PE_TRY(check_tiles(weight_tiles(E, I2, H)));
  PE_TRY(check_tiles(weight_tiles(E, H, I)));
  PE_TRY(check_apart({{&mdgu, {}}, {&mh, {}}, {&mdx, {}}, {&mdw13, {}}, {&mdw2, {}}},
                     {&mdy, &mx, &mgu, &mrow, &mo, &mw13, &mw2}));
  DeviceScope dev(device);
  PE_HIP(dev.err);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (R > 0) {
    // dh = dy W2, and from it and the kept gate and up values their gradients and h
    pe::GroupedArgs g = product(dy, lddy, R, nullptr, offsets, E, R, w2, nullptr, I, H, act);
    g.d.ldb = I;
    g.d.vec = 1;
    g.d.gu = static_cast<uint16_t*>(const_cast<void*>(gu));
    g.d.dgu = static_cast<uint16_t*>(dgu);
    g.d.y = dw2 ? h : nullptr; g.d.ldy = I;
    pe::launch_grouped_back(pe::DENSE_DGLU, g, s);
    PE_HIP(hipGetLastError());
    if (dx) {
      pe::GroupedArgs p = product(dgu, I2, R, nullptr, offsets, E, R, w13, nullptr, H, 2 * I, PE_ACT_NONE);
      p.d.ldb = H;
      p.d.vec = 1;
      p.d.y = dx; p.d.ldy = lddx;
      pe::launch_grouped_back(pe::DENSE_LINEAR, p, s);
      PE_HIP(hipGetLastError());
    }
  }
  // sums over the rows of each expert; zeros where there are none
  auto weights = [&](const void* left, int64_t ld_l, const void* right, int64_t ld_r, const int32_t* list, int m, int n,
                     void* out) {
    pe::GroupedArgs g = product(left, ld_l, list ? x_rows : R, list, offsets, E, R, right, nullptr, n, 0, PE_ACT_NONE);
    g.d.ldb = ld_r;
    g.d.T = m;
    g.d.vec = 1;
    g.d.y = out; g.d.ldy = n;
    pe::launch_grouped_weights(g, s);
  };
  if (dw13) {
    weights(dgu, I2, x, ldx, rows, 2 * I, H, dw13);
    PE_HIP(hipGetLastError());
  }
  if (dw2) {
    weights(dy, lddy, h, I, nullptr, H, I, dw2);
    PE_HIP(hipGetLastError());
  }
  return PE_OK;
}

}  // extern "C"
