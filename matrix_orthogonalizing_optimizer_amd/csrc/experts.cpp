// C entry points of the products grouped by expert: validation, then one or
// two launches.
#include <hip/hip_runtime.h>

#include <cstring>

#include "experts_plan.hpp"
#include "launch.hpp"
#include "libmuon.h"
#include "plan.hpp"
#include "timing.hpp"

using namespace muon;

static_assert(sizeof(ExpertsItem) == 32 && sizeof(ExpertsHead) <= 8192, "workspace layout");

namespace {

constexpr int64_t MAX_SIDE = (int64_t)1 << 30;
constexpr int64_t MAX_LD = (int64_t)1 << 21;       // a tile's rows within 32-bit offsets
constexpr int64_t MAX_STRIDE = (int64_t)1 << 42;   // between experts, 64-bit offsets
constexpr int64_t MAX_EXPERTS = (int64_t)1 << 16;
constexpr int64_t MAX_WORKGROUPS = (int64_t)1 << 22;  // 512 threads each within 2^32

bool dtype_ok(int32_t d) { return d == MUON_F32 || d == MUON_BF16; }
size_t esize(int32_t d) { return d == MUON_F32 ? 4 : 2; }
int dev_dt(int32_t d) { return d == MUON_F32 ? DT_F32 : DT_BF16; }
bool side_ok(int64_t v) { return v >= 0 && v <= MAX_SIDE; }
bool ld_ok(int64_t ld, int64_t cols) { return ld >= cols && ld <= MAX_LD; }
bool at(const void* p, size_t a) { return p && reinterpret_cast<uintptr_t>(p) % a == 0; }
bool pieces(const void* p, int64_t cols, int64_t ld) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && cols % 8 == 0 && ld % 8 == 0;
}

struct Matrix {
  const void* p;
  int64_t cols, ld;
};

// One pass.  r, s: its two operands of `rows` rows (the second one is w where
// pass is no weight gradient); o: the result.
muon_status experts_pass(int pass, const Matrix& r, const Matrix& s, int64_t stride, const int32_t* offsets, int64_t rows,
                         int64_t experts, int64_t out, int64_t in, int32_t dtype, void* o, int64_t ldo, int32_t odtype,
                         int32_t accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  const bool dw = pass == MUON_EXPERTS_WEIGHT_GRAD;
  if (!dtype_ok(dtype) || !dtype_ok(odtype)) return MUON_E_DTYPE;
  const int64_t ocols = pass == MUON_EXPERTS_FORWARD ? out : in;
  if (!side_ok(rows) || out < 0 || out > MAX_LD || in < 0 || in > MAX_LD || experts < 0 || experts > MAX_EXPERTS ||
      !ld_ok(r.ld, r.cols) ||
      !ld_ok(s.ld, s.cols) || !ld_ok(ldo, ocols) || stride > MAX_STRIDE)
    return MUON_E_SHAPE;
  // experts of w may not overlap in dw, and their rows lie in order
  if (experts > 1 && out > 0 && stride < (out - 1) * (dw ? ldo : s.ld) + in) return MUON_E_SHAPE;
  if (experts == 0 || ocols == 0 || (dw ? out == 0 : rows == 0)) return MUON_OK;
  const bool empty = dw ? rows == 0 : (pass == MUON_EXPERTS_FORWARD ? in : out) == 0;  // sums over nothing
  if (!at(offsets, 4) || !at(o, esize(odtype)) || (!empty && (!at(r.p, esize(dtype)) || !at(s.p, esize(dtype)))))
    return MUON_E_ARG;
  const bool direct = !empty && dtype == MUON_BF16 && pieces(r.p, r.cols, r.ld) && pieces(s.p, s.cols, s.ld) &&
                      (dw || stride % 8 == 0);
  const ExpertsPlan p = experts_plan(pass, rows, experts, out, in, dtype, direct);
  if (p.bytes && (!workspace || workspace_bytes < p.bytes)) return MUON_E_WORKSPACE;
  if (std::max(p.tiles * p.splits, p.joined * (p.tile * p.tile / 2048)) > MAX_WORKGROUPS) return MUON_E_SHAPE;
  ExpertsArgs a;
  std::memset(&a, 0, sizeof(a));
  a.A = r.p; a.lda = r.ld;
  a.B = s.p; a.ldb = s.ld;
  a.o = o; a.ldo = ldo;
  a.se = stride;
  a.offsets = offsets;
  a.rows = (int32_t)rows; a.experts = (int32_t)experts;
  a.M = (int32_t)out;
  a.N = (int32_t)ocols;
  a.K = (int32_t)(pass == MUON_EXPERTS_FORWARD ? in : out);
  a.tilesM = (int32_t)((out + p.tile - 1) / p.tile);
  a.tilesN = (int32_t)((ocols + p.tile - 1) / p.tile);
  a.splits = p.splits;
  a.accumulate = accumulate;
  if (p.bytes) {
    const uintptr_t u = reinterpret_cast<uintptr_t>(workspace);
    char* ws = reinterpret_cast<char*>((u + WS_ALIGN - 1) / WS_ALIGN * WS_ALIGN);
    a.ws = reinterpret_cast<float*>(ws + p.ws_off);
    if (p.big) a.head = reinterpret_cast<ExpertsHead*>(ws);
    if (p.big) a.items = reinterpret_cast<ExpertsItem*>(ws + p.items_off);
    a.cap = (int32_t)p.cap;
  }
  a.chunk = (int32_t)p.chunk;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const double f = 2.0 * (double)rows * (double)out * (double)in;
  const int fam = pass == MUON_EXPERTS_FORWARD ? F_EXPERTS_Y : dw ? F_EXPERTS_DW : F_EXPERTS_DX;
  const hipError_t e = timed(fam, f, 0.0, st, [&] {
    if (p.few) return launch_experts_few(dev_dt(dtype), dev_dt(odtype), a, st);
    if (p.big) {
      const auto go = pass == MUON_EXPERTS_FORWARD ? launch_experts_big_y : dw ? launch_experts_big_dw : launch_experts_big_dx;
      return go(dev_dt(odtype), a, st);
    }
    const auto go = pass == MUON_EXPERTS_FORWARD ? launch_experts_y : dw ? launch_experts_dw : launch_experts_dx;
    return go(direct, dev_dt(dtype), dev_dt(odtype), p.tiles, p.joined, a, st);
  });
  return e == hipSuccess ? MUON_OK : MUON_E_HIP;
}

}  // namespace

extern "C" {

muon_status muon_experts_workspace_bytes(int32_t pass, int64_t rows, int64_t experts, int64_t out, int64_t in,
                                         int32_t dtype, size_t* bytes) {
  if (!bytes) return MUON_E_ARG;
  if (pass < MUON_EXPERTS_FORWARD || pass > MUON_EXPERTS_INPUT_GRAD) return MUON_E_METHOD;
  if (!dtype_ok(dtype)) return MUON_E_DTYPE;
  // (a width is a leading dimension's least)
  if (!side_ok(rows) || out < 0 || out > MAX_LD || in < 0 || in > MAX_LD || experts < 0 || experts > MAX_EXPERTS)
    return MUON_E_SHAPE;
  // whichever way the operands are aligned
  *bytes = experts && out && in && rows
               ? std::max(experts_plan(pass, rows, experts, out, in, dtype, dtype == MUON_BF16).bytes,
                          experts_plan(pass, rows, experts, out, in, dtype, false).bytes)
               : 0;
  return MUON_OK;
}

muon_status muon_experts_forward(const void* x, int64_t ldx, const void* w, int64_t ldw, int64_t stride,
                                 const int32_t* offsets, int64_t rows, int64_t experts, int64_t out, int64_t in,
                                 int32_t dtype, void* y, int64_t ldy, int32_t y_dtype, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  return experts_pass(MUON_EXPERTS_FORWARD, {x, in, ldx}, {w, in, ldw}, stride, offsets, rows, experts, out, in, dtype, y,
                      ldy, y_dtype, 0, workspace, workspace_bytes, stream);
}

muon_status muon_experts_input_grad(const void* dy, int64_t lddy, const void* w, int64_t ldw, int64_t stride,
                                    const int32_t* offsets, int64_t rows, int64_t experts, int64_t out, int64_t in,
                                    int32_t dtype, void* dx, int64_t lddx, int32_t dx_dtype, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  return experts_pass(MUON_EXPERTS_INPUT_GRAD, {dy, out, lddy}, {w, in, ldw}, stride, offsets, rows, experts, out, in, dtype,
                      dx, lddx, dx_dtype, 0, workspace, workspace_bytes, stream);
}

muon_status muon_experts_weight_grad(const void* dy, int64_t lddy, const void* x, int64_t ldx, const int32_t* offsets,
                                     int64_t rows, int64_t experts, int64_t out, int64_t in, int32_t dtype, void* dw,
                                     int64_t lddw, int64_t stride, int32_t dw_dtype, int32_t accumulate, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  return experts_pass(MUON_EXPERTS_WEIGHT_GRAD, {dy, out, lddy}, {x, in, ldx}, stride, offsets, rows, experts, out, in, dtype,
                      dw, lddw, dw_dtype, accumulate, workspace, workspace_bytes, stream);
}

}  // extern "C"
