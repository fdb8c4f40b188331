// C entry points of the operators around the step (norms, 8-bit rows, the
// linear layer on 8-bit rows): validation, then one or two launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "consts.hpp"
#include "launch.hpp"
#include "libmuon.h"
#include "linear8_plan.hpp"
#include "plan.hpp"
#include "timing.hpp"

using namespace muon;

namespace {

constexpr int64_t MAX_SIDE = (int64_t)1 << 30;
constexpr int64_t MAX_COLS = (int64_t)1 << 27;  // row operators: a launch per 64 columns stays within 2^32 threads
constexpr int64_t MAX_LD = (int64_t)1 << 40;    // row operators: 64-bit offsets
constexpr int64_t MAX_LD8 = (int64_t)1 << 21;   // linear layer: a tile's rows within 32-bit offsets
constexpr int64_t MAX_IN = 131071;              // 128 * 128 * in stays below 2^31

bool dtype_ok(int32_t d) { return d == MUON_F32 || d == MUON_BF16; }
size_t esize(int32_t d) { return d == MUON_F32 ? 4 : 2; }
bool side_ok(int64_t v) { return v >= 0 && v <= MAX_SIDE; }
bool cols_ok(int64_t v) { return v >= 0 && v <= MAX_COLS; }
bool ld_ok(int64_t ld, int64_t cols, int64_t most) { return ld >= cols && ld <= most; }
bool at(const void* p, size_t a) { return p && reinterpret_cast<uintptr_t>(p) % a == 0; }
bool at_or_null(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
int dev_dt(int32_t d) { return d == MUON_F32 ? DT_F32 : DT_BF16; }
char* ws_base(void* p) {
  const uintptr_t u = reinterpret_cast<uintptr_t>(p);
  return reinterpret_cast<char*>((u + WS_ALIGN - 1) / WS_ALIGN * WS_ALIGN);
}
muon_status done(hipError_t e) { return e == hipSuccess ? MUON_OK : MUON_E_HIP; }

// Workgroups of the norm's backward kernel = partial rows of its column sums.
int norm_parts(int64_t rows, int64_t cols) {
  // rows a workgroup takes at a time
  const int64_t per = cols <= 64 ? 32 : cols <= 256 ? 8 : cols <= 512 ? 4 : cols <= 768 ? 8 : cols <= 1024 ? 4 : 1;
  // More workgroups hide more of a row's latency, and each adds a partial row
  // that is written and read.  512 only where each takes at least two rounds
  // of rows, of at most 4 rows of at most 4096 columns (us, 256 against 512
  // workgroups: 16384 x 512 19.0 and 16.2, 8192 x 2048 34 and 27; but 8192 x 768
  // in rounds of 8 16.1 and 16.8, 8192 x 8192 81 and 88, 1000 x 4096 15.6 and
  // 19.1, 3000 x 1024 11.1 and 12.1, 1500 x 2048 13.0 and 14.0).
  const int64_t rounds = std::max<int64_t>(1, (rows + per - 1) / per);
  return (int)std::min<int64_t>(cols > 4096 || per >= 8 || rounds <= 1024 ? 256 : 512, rounds);
}
size_t norm_ws(int64_t rows, int64_t cols) {
  if (rows == 0 || cols == 0) return 0;
  return (size_t)norm_parts(rows, cols) * (size_t)cols * 2 * sizeof(float) + WS_ALIGN;
}

// How dy enters a gradient product: as it lies (0 planes to make), or as bf16
// planes, laid out in the workspace or, of fp32, cut in the product.
int dy_planes(const void* dy, int64_t lddy, int64_t out, int32_t dtype) {
  if (dtype == MUON_F32) return 3;
  return at_or_null(dy, 16) && lddy % 8 == 0 && out % 8 == 0 ? 0 : 1;
}

// Fills the shared part of the arguments; false if the grid does not fit.
bool linear8_args(const Linear8Plan& p, int64_t M, int64_t N, int64_t K, void* workspace, Linear8Args& a) {
  const int64_t tm = (M + p.tile - 1) / p.tile, tn = (N + p.tile - 1) / p.tile;
  if (tm * tn > (1 << 22)) return false;  // 512 threads each within 2^32
  a.M = (int32_t)M; a.N = (int32_t)N; a.K = (int32_t)K;
  a.tilesM = (int32_t)tm; a.tilesN = (int32_t)tn;
  a.splits = p.splits; a.per_split = p.per_split;
  a.whole = (int32_t)p.whole;
  a.ws = p.splits > 1 ? reinterpret_cast<float*>(ws_base(workspace) + p.ws_off) : nullptr;
  return true;
}

}  // namespace

extern "C" {

muon_status muon_rows8_quantize(const void* x, int64_t rows, int64_t cols, int64_t ldx, int32_t dtype, int8_t* q,
                                int64_t ldq, float* scale, void* stream) {
  if (!dtype_ok(dtype)) return MUON_E_DTYPE;
  if (!side_ok(rows) || !cols_ok(cols) || !ld_ok(ldx, cols, MAX_LD) || !ld_ok(ldq, cols, MAX_LD) || ldq % 16)
    return MUON_E_SHAPE;
  if (rows == 0) return MUON_OK;
  if (!at(scale, 4) || (cols > 0 && (!at(x, esize(dtype)) || !at(q, 16)))) return MUON_E_ARG;
  RowArgs a;
  std::memset(&a, 0, sizeof(a));
  a.x = x; a.ldx = ldx;
  a.q = q; a.ldq = ldq; a.scale = scale;
  a.rows = rows; a.cols = (int32_t)cols;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const double n = (double)rows * (double)cols;
  return done(timed(F_ROWS8, 0.0, n * (double)(esize(dtype) + 1), s,
                    [&] { return launch_row_forward(2, dev_dt(dtype), a, s); }));
}

muon_status muon_rows8_dequantize(const int8_t* q, int64_t ldq, const float* scale, int64_t rows, int64_t cols,
                                  void* y, int64_t ldy, int32_t dtype, void* stream) {
  if (!dtype_ok(dtype)) return MUON_E_DTYPE;
  if (!side_ok(rows) || !cols_ok(cols) || !ld_ok(ldy, cols, MAX_LD) || !ld_ok(ldq, cols, MAX_LD) || ldq % 16)
    return MUON_E_SHAPE;
  if (rows == 0 || cols == 0) return MUON_OK;
  if (!at(scale, 4) || !at(q, 16) || !at(y, esize(dtype))) return MUON_E_ARG;
  RestoreArgs a;
  std::memset(&a, 0, sizeof(a));
  a.q = q; a.ldq = ldq; a.scale = scale;
  a.y = y; a.ldy = ldy;
  a.rows = rows; a.cols = (int32_t)cols;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const double n = (double)rows * (double)cols;
  return done(timed(F_ROWS8, 0.0, n * (double)(esize(dtype) + 1), s,
                    [&] { return launch_row_restore(dev_dt(dtype), a, s); }));
}

muon_status muon_norm_forward(int32_t kind, const void* x, int64_t rows, int64_t cols, int64_t ldx, int32_t dtype,
                              const void* gamma, const void* beta, int32_t vec_dtype, float eps, void* y, int64_t ldy,
                              int8_t* q, int64_t ldq, float* scale, float* mean, float* rstd, void* stream) {
  if (kind != MUON_NORM_LAYER && kind != MUON_NORM_RMS) return MUON_E_METHOD;
  if (!dtype_ok(dtype) || !dtype_ok(vec_dtype)) return MUON_E_DTYPE;
  if (!side_ok(rows) || !cols_ok(cols) || !ld_ok(ldx, cols, MAX_LD) || (y && !ld_ok(ldy, cols, MAX_LD)) ||
      (q && (!ld_ok(ldq, cols, MAX_LD) || ldq % 16)))
    return MUON_E_SHAPE;
  if (!std::isfinite(eps) || eps < 0.f) return MUON_E_ARG;
  if (kind == MUON_NORM_RMS && mean) return MUON_E_ARG;
  if (rows == 0 || cols == 0) return MUON_OK;  // the address of an empty q may be null
  if ((q != nullptr) != (scale != nullptr) || (!y && !q && !mean && !rstd)) return MUON_E_ARG;
  if (!at(x, esize(dtype)) || !at(gamma, esize(vec_dtype)) || !at_or_null(beta, esize(vec_dtype)) ||
      !at_or_null(y, esize(dtype)) || !at_or_null(q, 16) || !at_or_null(scale, 4) || !at_or_null(mean, 4) ||
      !at_or_null(rstd, 4))
    return MUON_E_ARG;
  if (y == x && y && ldy != ldx) return MUON_E_ARG;
  RowArgs a;
  std::memset(&a, 0, sizeof(a));
  a.x = x; a.ldx = ldx;
  a.gamma = gamma; a.beta = beta; a.vec_dtype = dev_dt(vec_dtype);
  a.eps = eps;
  a.y = y; a.ldy = ldy;
  a.q = q; a.ldq = ldq; a.scale = scale;
  a.mean = mean; a.rstd = rstd;
  a.rows = rows; a.cols = (int32_t)cols;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const double n = (double)rows * (double)cols, es = (double)esize(dtype);
  return done(timed(F_NORM_FWD, 0.0, n * (es + (y ? es : 0.0) + (q ? 1.0 : 0.0)), s,
                    [&] { return launch_row_forward(kind, dev_dt(dtype), a, s); }));
}

muon_status muon_norm_backward_workspace_bytes(int64_t rows, int64_t cols, size_t* bytes) {
  if (!bytes) return MUON_E_ARG;
  if (!side_ok(rows) || !cols_ok(cols)) return MUON_E_SHAPE;
  *bytes = norm_ws(rows, cols);
  return MUON_OK;
}

muon_status muon_norm_backward(int32_t kind, const void* dy, int64_t lddy, const void* x, int64_t ldx, int64_t rows,
                               int64_t cols, int32_t dtype, const void* gamma, int32_t vec_dtype, const float* mean,
                               const float* rstd, void* dx, int64_t lddx, void* dgamma, void* dbeta,
                               int32_t accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  if (kind != MUON_NORM_LAYER && kind != MUON_NORM_RMS) return MUON_E_METHOD;
  if (!dtype_ok(dtype) || !dtype_ok(vec_dtype)) return MUON_E_DTYPE;
  if (!side_ok(rows) || !cols_ok(cols) || !ld_ok(lddy, cols, MAX_LD) || !ld_ok(ldx, cols, MAX_LD) ||
      !ld_ok(lddx, cols, MAX_LD))
    return MUON_E_SHAPE;
  const size_t es = esize(dtype), ve = esize(vec_dtype);
  if (kind == MUON_NORM_RMS && mean) return MUON_E_ARG;
  if (!at_or_null(dgamma, ve) || !at_or_null(dbeta, ve)) return MUON_E_ARG;
  if (cols == 0) return MUON_OK;
  if (rows > 0) {
    if (!at(dy, es) || !at(x, es) || !at(dx, es) || !at(gamma, ve) || !at(rstd, 4) || !at_or_null(mean, 4) ||
        (kind == MUON_NORM_LAYER && !mean))
      return MUON_E_ARG;
    if (dx == dy && lddx != lddy) return MUON_E_ARG;
  }
  const bool vecs = dgamma || dbeta;
  if (vecs && rows > 0 && (!workspace || workspace_bytes < norm_ws(rows, cols))) return MUON_E_WORKSPACE;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const int parts = rows > 0 ? norm_parts(rows, cols) : 0;
  float* part = vecs && rows > 0 ? reinterpret_cast<float*>(ws_base(workspace)) : nullptr;
  if (rows > 0) {
    NormBwdArgs a;
    std::memset(&a, 0, sizeof(a));
    a.dy = dy; a.lddy = lddy;
    a.x = x; a.ldx = ldx;
    a.gamma = gamma; a.vec_dtype = dev_dt(vec_dtype);
    a.mean = mean; a.rstd = rstd;
    a.dx = dx; a.lddx = lddx;
    a.partials = part;
    a.sum_dy = dbeta != nullptr;
    a.rows = rows; a.cols = (int32_t)cols;
    const double n = (double)rows * (double)cols;
    const hipError_t e = timed(F_NORM_BWD, 0.0, 3.0 * n * (double)es, s,
                               [&] { return launch_norm_backward(kind, dev_dt(dtype), a, parts, s); });
    if (e != hipSuccess) return MUON_E_HIP;
  }
  if (vecs) {
    JoinArgs j;
    std::memset(&j, 0, sizeof(j));
    j.partials = part;
    j.parts = parts;
    j.dgamma = dgamma; j.dbeta = dbeta;
    j.accumulate = accumulate;
    j.cols = cols;
    const hipError_t e =
        timed(F_NORM_BWD, 0.0, 0.0, s, [&] { return launch_norm_join(dev_dt(vec_dtype), j, s); });
    if (e != hipSuccess) return MUON_E_HIP;
  }
  return MUON_OK;
}

muon_status muon_linear8_workspace_bytes(int32_t pass, int64_t tokens, int64_t out, int64_t in, const void* dy,
                                         int64_t lddy, int32_t dy_dtype, size_t* bytes) {
  if (!bytes) return MUON_E_ARG;
  if (pass < MUON_LINEAR8_FORWARD || pass > MUON_LINEAR8_INPUT_GRAD) return MUON_E_METHOD;
  if (!side_ok(tokens) || !side_ok(out) || !side_ok(in) || (pass == MUON_LINEAR8_FORWARD && in > MAX_IN))
    return MUON_E_SHAPE;
  const bool grad = pass != MUON_LINEAR8_FORWARD;
  if (grad && !dtype_ok(dy_dtype)) return MUON_E_DTYPE;
  const int planes = grad ? dy_planes(dy, lddy, out, dy_dtype) : 0;
  *bytes = tokens && out && in ? linear8_plan(pass, tokens, out, in, planes).bytes : 0;
  return MUON_OK;
}

muon_status muon_linear8_forward(const int8_t* q, int64_t ldq, const float* scale, const int8_t* wq, int64_t ldw,
                                 const float* wscale, const void* bias, int32_t bias_dtype, int64_t tokens,
                                 int64_t out, int64_t in, void* y, int64_t ldy, int32_t dtype, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  if (!dtype_ok(dtype) || (bias && !dtype_ok(bias_dtype))) return MUON_E_DTYPE;
  if (!side_ok(tokens) || !side_ok(out) || !side_ok(in) || in > MAX_IN || !ld_ok(ldq, in, MAX_LD8) ||
      !ld_ok(ldw, in, MAX_LD8) || !ld_ok(ldy, out, MAX_LD8) || ldq % 16 || ldw % 16)
    return MUON_E_SHAPE;
  if (tokens == 0 || out == 0) return MUON_OK;
  if (!at(scale, 4) || !at(wscale, 4) || !at(y, esize(dtype)) || (bias && !at(bias, esize(bias_dtype))) ||
      (in > 0 && (!at(q, 16) || !at(wq, 16))))
    return MUON_E_ARG;
  const Linear8Plan p = linear8_plan(MUON_LINEAR8_FORWARD, tokens, out, in, 0);
  if (p.bytes && (!workspace || workspace_bytes < p.bytes)) return MUON_E_WORKSPACE;
  Linear8Args a;
  std::memset(&a, 0, sizeof(a));
  if (!linear8_args(p, tokens, out, in, workspace, a)) return MUON_E_SHAPE;
  a.A = q; a.lda = ldq; a.sa = scale;
  a.B = wq; a.ldb = ldw; a.sb = wscale;
  a.bias = bias; a.bias_dtype = dev_dt(bias_dtype);
  a.o = y; a.ldo = ldy;
  a.planes = 1;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const double f = 2.0 * (double)tokens * (double)out * (double)in;
  return done(timed(F_LINEAR8_Y, f, 0.0, s, [&] {
    if (in == 0) return launch_linear8_bias(dev_dt(dtype), a, s);
    return p.few ? launch_linear8_few(dev_dt(dtype), a, s) : launch_linear8_forward(p.tile, dev_dt(dtype), a, s);
  }));
}

static muon_status linear8_grad(bool weight, const void* dy, int64_t lddy, int32_t dy_dtype, const int8_t* q,
                                int64_t ldq, const float* scale, int64_t tokens, int64_t out, int64_t in, void* o,
                                int64_t ldo, int32_t o_dtype, int32_t accumulate, void* workspace,
                                size_t workspace_bytes, void* stream) {
  if (!dtype_ok(dy_dtype) || !dtype_ok(o_dtype)) return MUON_E_DTYPE;
  if (!side_ok(tokens) || !side_ok(out) || !side_ok(in) || !ld_ok(lddy, out, MAX_LD8) || !ld_ok(ldq, in, MAX_LD8) ||
      !ld_ok(ldo, in, MAX_LD8) || ldq % 16)
    return MUON_E_SHAPE;
  const int64_t rows = weight ? out : tokens, sum = weight ? tokens : out;
  if (rows == 0 || in == 0) return MUON_OK;
  if (!at(o, esize(o_dtype)) || (sum > 0 && (!at(dy, esize(dy_dtype)) || !at(q, 16) || !at(scale, 4))))
    return MUON_E_ARG;
  const int pass = weight ? MUON_LINEAR8_WEIGHT_GRAD : MUON_LINEAR8_INPUT_GRAD;
  const int planes = sum > 0 ? dy_planes(dy, lddy, out, dy_dtype) : 0;
  const Linear8Plan p = linear8_plan(pass, tokens, out, in, planes);
  if (p.bytes && (!workspace || workspace_bytes < p.bytes)) return MUON_E_WORKSPACE;
  Linear8Args a;
  std::memset(&a, 0, sizeof(a));
  if (!linear8_args(p, rows, in, sum, workspace, a)) return MUON_E_SHAPE;
  a.A = dy; a.lda = lddy;
  a.planes = planes ? planes : 1;
  PlanesArgs d;
  std::memset(&d, 0, sizeof(d));
  if (planes && !p.dy_f32) {
    d.dy = dy; d.ld = lddy;
    d.o = ws_base(workspace) + p.dy_off; d.ldo = p.lddy;
    d.plane = tokens * p.lddy;
    d.rows = tokens; d.cols = (int32_t)out;
    a.A = d.o; a.lda = p.lddy;
    a.plane = d.plane;
  }
  a.B = q; a.ldb = ldq; a.sb = scale;
  a.o = o; a.ldo = ldo;
  a.accumulate = accumulate;
  RestoreArgs x;
  std::memset(&x, 0, sizeof(x));
  if (p.expanded) {
    x.q = q; x.ldq = ldq; x.scale = scale;
    x.y = ws_base(workspace); x.ldy = p.ldx;
    x.rows = sum; x.cols = (int32_t)in;
    a.B = x.y; a.ldb = p.ldx;
  }
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const double f = 2.0 * (double)tokens * (double)out * (double)in;
  return done(timed(weight ? F_LINEAR8_DW : F_LINEAR8_DX, f, 0.0, s, [&] {
    if (planes && !p.dy_f32) {
      const hipError_t e = launch_linear8_planes(dev_dt(dy_dtype), d, s);
      if (e != hipSuccess) return e;
    }
    if (p.expanded) {
      const hipError_t e = launch_row_restore(DT_BF16, x, s);
      if (e != hipSuccess) return e;
    }
    return weight ? launch_linear8_dw(p.tile, p.expanded, p.dy_f32, dev_dt(o_dtype), a, s)
                  : launch_linear8_dx(p.tile, p.expanded, p.dy_f32, dev_dt(o_dtype), a, s);
  }));
}

muon_status muon_linear8_weight_grad(const void* dy, int64_t lddy, int32_t dy_dtype, const int8_t* q, int64_t ldq,
                                     const float* scale, int64_t tokens, int64_t out, int64_t in, void* dw,
                                     int64_t lddw, int32_t dw_dtype, int32_t accumulate, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  return linear8_grad(true, dy, lddy, dy_dtype, q, ldq, scale, tokens, out, in, dw, lddw, dw_dtype, accumulate,
                      workspace, workspace_bytes, stream);
}

muon_status muon_linear8_input_grad(const void* dy, int64_t lddy, int32_t dy_dtype, const int8_t* wq, int64_t ldw,
                                    const float* wscale, int64_t tokens, int64_t out, int64_t in, void* dx,
                                    int64_t lddx, int32_t dx_dtype, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  return linear8_grad(false, dy, lddy, dy_dtype, wq, ldw, wscale, tokens, out, in, dx, lddx, dx_dtype, 0, workspace,
                      workspace_bytes, stream);
}

}  // extern "C"
