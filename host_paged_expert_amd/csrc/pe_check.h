// Argument checks shared by the C entry points of the operators that need no
// context, and the device of their launches.
#pragma once
#include <hip/hip_runtime.h>

#include <initializer_list>

#include "pe_error.h"

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
