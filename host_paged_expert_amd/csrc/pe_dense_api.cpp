// C entry points of the dense operators around a paged MoE layer (include/pe.h):
// argument checks, the device of the call, and the launches.  They hold no
// state and allocate nothing.
#include <hip/hip_runtime.h>

#include <initializer_list>

#include "../../include/pe.h"
#include "pe_dense.h"
#include "pe_error.h"
#include "pe_layout.h"

namespace {

using pe::fail;

// A matrix argument: `rows` rows of `cols` elements of `es` bytes, `ld` elements apart.
struct Mat {
  const char* name;
  const void* p;
  int64_t rows, cols, ld;
  int es;
  int align;            // bytes the address and the row stride must be multiples of
  double end() const {  // one past the last byte; a double holds any sum of these without overflow
    return (double)(uintptr_t)p + (rows > 0 ? ((double)(rows - 1) * ld + cols) * es : 0.0);
  }
};

// The products address the rows of one tile (256 of up to 2 bytes an element)
// with 32-bit offsets from the tile's first.
constexpr int64_t kMaxStride = 1 << 22;

int check_mat(const Mat& m, bool optional) {
  if (!m.p) return optional ? PE_OK : fail(PE_ERR_INVALID_ARG, "%s is NULL", m.name);
  if (m.ld < m.cols || m.ld >= kMaxStride)
    return fail(PE_ERR_INVALID_ARG, "%s: row stride %lld outside [%lld, 2^22)", m.name, (long long)m.ld,
                (long long)m.cols);
  if ((uintptr_t)m.p % m.align || (m.rows > 1 && m.ld * m.es % m.align))
    return fail(PE_ERR_INVALID_ARG, "%s: address and row stride must be multiples of %d bytes", m.name, m.align);
  return PE_OK;
}

bool overlap(const Mat& a, const Mat& b) {
  if (!a.p || !b.p || (double)(uintptr_t)a.p >= b.end() || (double)(uintptr_t)b.p >= a.end()) return false;
  // Column ranges of one wider matrix share no byte although their rows interleave: b's columns lie `at` bytes
  // behind a's in rows of `stride` bytes.
  const int64_t stride = a.ld * a.es, len_a = a.cols * a.es, len_b = b.cols * b.es;
  if (stride != b.ld * b.es) return true;
  const int64_t at = ((int64_t)((uintptr_t)b.p - (uintptr_t)a.p) % stride + stride) % stride;
  return at < len_a || at + len_b > stride;
}
bool same(const Mat& a, const Mat& b) { return a.p == b.p && a.ld == b.ld && a.es == b.es && a.cols == b.cols; }

// Every output must be apart from every input and every other output, except
// that an output may be exactly the input named beside it (each element is
// read by the thread that later writes it).
struct Out { const Mat* m; std::initializer_list<const Mat*> may_be; };
int check_apart(std::initializer_list<Out> outs, std::initializer_list<const Mat*> ins) {
  for (const Out* o = outs.begin(); o != outs.end(); ++o) {
    for (const Mat* in : ins) {
      if (!overlap(*o->m, *in)) continue;
      bool ok = false;
      for (const Mat* q : o->may_be) ok = ok || (q == in && same(*o->m, *in));
      if (!ok) return fail(PE_ERR_INVALID_ARG, "%s overlaps %s", o->m->name, in->name);
    }
    for (const Out* q = outs.begin(); q != o; ++q)
      if (overlap(*o->m, *q->m)) return fail(PE_ERR_INVALID_ARG, "%s overlaps %s", o->m->name, q->m->name);
  }
  return PE_OK;
}

// Makes `device` current for the launches of one call and restores the caller's.
struct DeviceScope {
  int prev = -1;
  hipError_t err;
  explicit DeviceScope(int device) {
    err = hipGetDevice(&prev);
    if (err != hipSuccess) prev = -1;
    else if (prev == device) prev = -1;
    else err = hipSetDevice(device);
    if (err != hipSuccess) (void)hipGetLastError();   // reported here; the next call's launch must not find it
  }
  ~DeviceScope() {
    if (prev >= 0) (void)hipSetDevice(prev);
  }
};

#define PE_TRY(call)            \
  do {                          \
    const int rc_ = (call);     \
    if (rc_ != PE_OK) return rc_; \
  } while (0)

// A launch has fewer than 2^32 threads: 256 for each of T rows at most.
constexpr int kMaxRows = 1 << 24;

int check_dims(int device, int T, std::initializer_list<int> dims) {
  if (device < 0) return fail(PE_ERR_INVALID_ARG, "device %d is negative", device);
  if (T < 0 || T >= kMaxRows) return fail(PE_ERR_INVALID_ARG, "T=%d outside [0, 2^24)", T);
  for (int d : dims)
    if (d < 1) return fail(PE_ERR_INVALID_ARG, "dimensions must be positive");
  return PE_OK;
}

int check_wtype(int wtype, int K) {
  if (wtype == PE_W_FP8_B128) {
    if (K % 128) return fail(PE_ERR_INVALID_ARG, "block FP8 needs the summed dimension to be a multiple of 128");
  } else if (wtype == PE_W_BF16) {
    if (K % 8) return fail(PE_ERR_INVALID_ARG, "bf16 needs the summed dimension to be a multiple of 8");
  } else {
    return fail(PE_ERR_UNSUPPORTED, "the dense products take PE_W_BF16 and PE_W_FP8_B128 only");
  }
  return PE_OK;
}

int check_act(int act, bool none_ok) {
  if (act == PE_ACT_SILU || act == PE_ACT_GELU || (none_ok && act == PE_ACT_NONE)) return PE_OK;
  return fail(PE_ERR_INVALID_ARG, "unknown activation %d", act);
}

// Eight consecutive columns may be accessed as 16-byte vectors (8-byte ones of e4m3).
bool vec8(const Mat& m) {
  const int bytes = m.es == 1 ? 8 : 16;
  return !m.p || ((uintptr_t)m.p % bytes == 0 && m.ld * m.es % bytes == 0);
}

}  // namespace

extern "C" {

int pe_rmsnorm(int device, const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
               float eps, int T, int H, void* sum, int64_t lds, void* y, int64_t ldy, float* yscale, void* stream) {
  PE_TRY(check_dims(device, T, {H}));
  if (!(eps >= 0.f)) return fail(PE_ERR_INVALID_ARG, "eps must not be negative");
  if (H > PE_MAX_NORM_HIDDEN) return fail(PE_ERR_INVALID_ARG, "H=%d is larger than %d", H, PE_MAX_NORM_HIDDEN);
  if (yscale ? H % 128 : H % 8)
    return fail(PE_ERR_INVALID_ARG, "H must be a multiple of %d", yscale ? 128 : 8);
  if (T == 0) return PE_OK;
  const Mat mx{"x", x, T, H, ldx, 2, 16}, mr{"residual", residual, T, H, ldr, 2, 16};
  const Mat mw{"weight", weight, 1, H, H, 2, 16}, ms{"sum", sum, T, H, lds, 2, 16};
  const Mat my{"y", y, T, H, ldy, yscale ? 1 : 2, yscale ? 8 : 16};
  const Mat mq{"yscale", yscale, T, H / 128, H / 128, 4, 4};
  PE_TRY(check_mat(mx, false));
  PE_TRY(check_mat(mr, true));
  PE_TRY(check_mat(mw, false));
  PE_TRY(check_mat(ms, true));
  PE_TRY(check_mat(my, false));
  PE_TRY(check_mat(mq, true));
  PE_TRY(check_apart({{&ms, {&mx, &mr}}, {&my, {&mx, &mr}}, {&mq, {}}}, {&mx, &mr, &mw}));
  DeviceScope dev(device);
  PE_HIP(dev.err);
  pe::NormArgs a{};
  a.x = static_cast<const uint16_t*>(x); a.ldx = ldx;
  a.residual = static_cast<const uint16_t*>(residual); a.ldr = ldr;
  a.weight = static_cast<const uint16_t*>(weight);
  a.eps = eps; a.T = T; a.H = H;
  a.sum = static_cast<uint16_t*>(sum); a.lds = lds;
  a.y = y; a.ldy = ldy; a.yscale = yscale;
  pe::launch_rmsnorm(a, static_cast<hipStream_t>(stream));
  PE_HIP(hipGetLastError());
  return PE_OK;
}

int pe_route(int device, const float* logits, int64_t ldl, int T, int num_experts, int top_k, int scoring,
             int renormalize, float scale, int32_t* topk_ids, float* topk_w, void* stream) {
  const int E = num_experts, k = top_k;
  PE_TRY(check_dims(device, T, {E, k}));
  if (E > pe::kMaxExperts || k > E) return fail(PE_ERR_INVALID_ARG, "need top_k <= num_experts <= %d", pe::kMaxExperts);
  if (scoring != PE_SCORE_SOFTMAX && scoring != PE_SCORE_SIGMOID)
    return fail(PE_ERR_INVALID_ARG, "unknown scoring %d", scoring);
  if (T == 0) return PE_OK;
  const Mat ml{"logits", logits, T, E, ldl, 4, 4}, mi{"topk_ids", topk_ids, T, k, k, 4, 4};
  const Mat mw{"topk_w", topk_w, T, k, k, 4, 4};
  PE_TRY(check_mat(ml, false));
  PE_TRY(check_mat(mi, false));
  PE_TRY(check_mat(mw, false));
  PE_TRY(check_apart({{&mi, {}}, {&mw, {}}}, {&ml}));
  DeviceScope dev(device);
  PE_HIP(dev.err);
  pe::RouteArgs a{};
  a.logits = logits; a.ldl = ldl; a.T = T; a.E = E; a.k = k;
  a.sigmoid = scoring == PE_SCORE_SIGMOID;
  a.renorm = renormalize != 0;
  a.scale = scale;
  a.ids = topk_ids; a.w = topk_w;
  pe::launch_route(a, static_cast<hipStream_t>(stream));
  PE_HIP(hipGetLastError());
  return PE_OK;
}

int pe_linear(int device, int wtype, const void* x, int64_t ldx, const float* xscale, const void* w,
              const float* wscale, const void* bias, int act, const void* residual, int64_t ldr, int T, int N,
              int K, void* y, int64_t ldy, int ytype, void* stream) {
  PE_TRY(check_dims(device, T, {N, K}));
  PE_TRY(check_wtype(wtype, K));
  PE_TRY(check_act(act, true));
  if (ytype != PE_Y_BF16 && ytype != PE_Y_FP32) return fail(PE_ERR_INVALID_ARG, "unknown output type %d", ytype);
  if (T == 0) return PE_OK;
  const bool fp8 = wtype == PE_W_FP8_B128;
  const int es = fp8 ? 1 : 2, ys = ytype == PE_Y_FP32 ? 4 : 2;
  const Mat mx{"x", x, T, K, ldx, es, 16}, mw{"w", w, N, K, K, es, 16};
  const Mat mxs{"xscale", xscale, T, K / 128, K / 128, 4, 4};
  const Mat mws{"wscale", wscale, (N + 127) / 128, K / 128, K / 128, 4, 4};
  const Mat mb{"bias", bias, 1, N, N, 2, 2}, mr{"residual", residual, T, N, ldr, 2, 2};
  const Mat my{"y", y, T, N, ldy, ys, ys};
  PE_TRY(check_mat(mx, false));
  PE_TRY(check_mat(mw, false));
  if (fp8) {
    PE_TRY(check_mat(mxs, false));
    PE_TRY(check_mat(mws, false));
  } else if (xscale || wscale) {
    return fail(PE_ERR_INVALID_ARG, "bf16 operands take no scales");
  }
  PE_TRY(check_mat(mb, true));
  PE_TRY(check_mat(mr, true));
  PE_TRY(check_mat(my, false));
  PE_TRY(check_apart({{&my, {&mr}}}, {&mx, &mw, &mxs, &mws, &mb, &mr}));
  DeviceScope dev(device);
  PE_HIP(dev.err);
  pe::DenseArgs a{};
  a.a = x; a.lda = ldx; a.as = xscale;
  a.b = w; a.ldb = K; a.bs = wscale;
  a.T = T; a.N = N; a.K = K; a.act = act;
  a.bias = static_cast<const uint16_t*>(bias);
  a.residual = static_cast<const uint16_t*>(residual); a.ldr = ldr;
  a.y = y; a.ldy = ldy; a.y_f32 = ytype == PE_Y_FP32;
  a.vec = vec8(my) && vec8(mr) && (uintptr_t)bias % 16 == 0;
  pe::launch_dense(pe::DENSE_LINEAR, fp8, true, true, a, static_cast<hipStream_t>(stream));
  PE_HIP(hipGetLastError());
  return PE_OK;
}

int pe_glu(int device, int wtype, int act, const void* x, int64_t ldx, const float* xscale, const void* w13,
           const float* s13, int T, int hidden, int inter, void* h, int64_t ldh, float* hscale, void* gu,
           void* stream) {
  const int H = hidden, I = inter;
  PE_TRY(check_dims(device, T, {H, I}));
  PE_TRY(check_wtype(wtype, H));
  PE_TRY(check_act(act, false));
  const bool fp8 = wtype == PE_W_FP8_B128;
  if ((fp8 || hscale) ? I % 128 : I % 8)
    return fail(PE_ERR_INVALID_ARG, "inter must be a multiple of %d", (fp8 || hscale) ? 128 : 8);
  if (T == 0) return PE_OK;
  const int es = fp8 ? 1 : 2, hs = hscale ? 1 : 2;
  const Mat mx{"x", x, T, H, ldx, es, 16}, mw{"w13", w13, 2 * (int64_t)I, H, H, es, 16};
  const Mat mxs{"xscale", xscale, T, H / 128, H / 128, 4, 4};
  const Mat mws{"s13", s13, 2 * (int64_t)(I / 128), H / 128, H / 128, 4, 4};
  const Mat mh{"h", h, T, I, ldh, hs, hs}, mhs{"hscale", hscale, T, I / 128, I / 128, 4, 4};
  const Mat mg{"gu", gu, T, 2 * (int64_t)I, 2 * (int64_t)I, 2, 16};
  PE_TRY(check_mat(mx, false));
  PE_TRY(check_mat(mw, false));
  if (fp8) {
    PE_TRY(check_mat(mxs, false));
    PE_TRY(check_mat(mws, false));
  } else if (xscale || s13) {
    return fail(PE_ERR_INVALID_ARG, "bf16 operands take no scales");
  }
  PE_TRY(check_mat(mh, false));
  PE_TRY(check_mat(mhs, true));
  PE_TRY(check_mat(mg, true));
  PE_TRY(check_apart({{&mh, {}}, {&mhs, {}}, {&mg, {}}}, {&mx, &mw, &mxs, &mws}));
  DeviceScope dev(device);
  PE_HIP(dev.err);
  pe::DenseArgs a{};
  a.a = x; a.lda = ldx; a.as = xscale;
  a.b = w13; a.ldb = H; a.bs = s13;
  a.T = T; a.N = I; a.K = H; a.act = act;
  a.y = h; a.ldy = ldh; a.hs = hscale;
  a.gu = static_cast<uint16_t*>(gu);
  a.vec = vec8(mh);
  pe::launch_dense(pe::DENSE_GLU, fp8, true, true, a, static_cast<hipStream_t>(stream));
  PE_HIP(hipGetLastError());
  return PE_OK;
}

int pe_ffn_backward(int device, int act, const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* gu,
                    const void* w13, const void* w2, int T, int hidden, int inter, void* dgu, void* h, void* dx,
                    int64_t lddx, void* dw13, void* dw2, void* stream) {
  const int H = hidden, I = inter;
  PE_TRY(check_dims(device, T, {H, I}));
  PE_TRY(check_act(act, false));
  if (H % 8 || I % 8)
    return fail(PE_ERR_INVALID_ARG, "hidden and inter must be multiples of 8");
  if (H >= kMaxStride || I >= kMaxStride / 2)        // rows of dy and gu, also where T = 0 leaves those unread
    return fail(PE_ERR_INVALID_ARG, "hidden=%d or 2 * inter=2 * %d is not below 2^22", H, I);
  if (!dx && !dw13 && !dw2) return fail(PE_ERR_INVALID_ARG, "no gradient is asked for");
  const Mat mdy{"dy", dy, T, H, lddy, 2, 16}, mx{"x", x, T, H, ldx, 2, 16}, mgu{"gu", gu, T, 2 * (int64_t)I, 2 * (int64_t)I, 2, 16};
  const Mat mw13{"w13", w13, 2 * (int64_t)I, H, H, 2, 16}, mw2{"w2", w2, H, I, I, 2, 16};
  const Mat mdgu{"dgu", dgu, T, 2 * (int64_t)I, 2 * (int64_t)I, 2, 16}, mh{"h", h, T, I, I, 2, 16};
  const Mat mdx{"dx", dx, T, H, lddx, 2, 16}, mdw13{"dw13", dw13, 2 * (int64_t)I, H, H, 2, 16}, mdw2{"dw2", dw2, H, I, I, 2, 16};
  PE_TRY(check_mat(mdw13, true));
  PE_TRY(check_mat(mdw2, true));
  if (T > 0) {
    PE_TRY(check_mat(mdy, false));
    PE_TRY(check_mat(mx, !dw13));
    PE_TRY(check_mat(mgu, false));
    PE_TRY(check_mat(mw13, !dx));
    PE_TRY(check_mat(mw2, false));
    PE_TRY(check_mat(mdgu, false));
    PE_TRY(check_mat(mh, !dw2));
    PE_TRY(check_mat(mdx, true));
  }
  PE_TRY(check_apart({{&mdgu, {}}, {&mh, {}}, {&mdx, {}}, {&mdw13, {}}, {&mdw2, {}}}, {&mdy, &mx, &mgu, &mw13, &mw2}));
  DeviceScope dev(device);
  PE_HIP(dev.err);
  hipStream_t s = static_cast<hipStream_t>(stream);
  pe::DenseArgs a{};
  a.act = act;
  a.vec = 1;
  if (T > 0) {
    // dh = dy W2, and from it and the kept gate and up values their gradients and h
    a.a = dy; a.lda = lddy;
    a.b = w2; a.ldb = I;
    a.T = T; a.N = I; a.K = H;
    a.gu = static_cast<uint16_t*>(const_cast<void*>(gu));
    a.dgu = static_cast<uint16_t*>(dgu);
    a.y = dw2 ? h : nullptr; a.ldy = I;
    pe::launch_dense(pe::DENSE_DGLU, false, true, false, a, s);
    PE_HIP(hipGetLastError());
  }
  auto product = [&](const void* left, int64_t ld_l, const void* right, int64_t ld_r, int rows, int cols, int sum,
                     void* out, int64_t ld_o) {
    pe::DenseArgs p{};
    p.act = PE_ACT_NONE;
    p.vec = 1;
    p.a = left; p.lda = ld_l;
    p.b = right; p.ldb = ld_r;
    p.T = rows; p.N = cols; p.K = sum;
    p.y = out; p.ldy = ld_o;
    return p;
  };
  // with T = 0 the weight gradients are sums of nothing: zeros
  const pe::DenseArgs gx = product(dgu, 2 * (int64_t)I, w13, H, T, H, 2 * I, dx, lddx);
  const pe::DenseArgs g13 = product(dgu, 2 * (int64_t)I, x, ldx, 2 * I, H, T, dw13, H);
  const pe::DenseArgs g2 = product(dy, lddy, h, I, H, I, T, dw2, I);
  pe::launch_dense_grads(T > 0 && dx ? &gx : nullptr, dw13 ? &g13 : nullptr, dw2 ? &g2 : nullptr, s);
  PE_HIP(hipGetLastError());
  return PE_OK;
}

}  // extern "C"
