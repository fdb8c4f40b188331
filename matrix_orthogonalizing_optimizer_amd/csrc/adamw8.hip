// AdamW parameters with 8-bit moments: the part of a step that updates them,
// and the conversions of their moments.
#include "adamw8.hpp"

#include <cmath>
#include <cstring>

#include "launch.hpp"
#include "libmuon.h"
#include "plan.hpp"
#include "timing.hpp"

using namespace muon;

namespace muon {

// Above this a launch does not ask the caches to keep anything.  What fits the
// 256 MB cache partly comes out of it where it was just written (a step after
// step of 388 MB 67.4 us, streamed 74); what does not, gains (us, cached and
// streamed: 330 MB 59 and 60, 490 MB 90 and 92, 660 MB 121 and 115, 2.5 GB 455
// and 422, 5.3 GB 940 and 895).
constexpr double ADAMW8_STREAM_BYTES = 5.5e8;

// The descriptors travel in the launch's arguments: up to ADAMW8_TENSORS
// tensors a launch, and no table to upload before it.
hipError_t launch_adamw8(const PlanImpl& P, const muon_param_ptrs* ptrs, const muon_hparams& hp, hipStream_t s) {
  const uint32_t kMaxGrid = 1u << 22;  // 256 threads each within 2^32
  Adamw8Args a;
  std::memset(&a, 0, sizeof(a));
  a.one_minus_b1 = 1.f - hp.adam_beta1;
  a.one_minus_b2 = 1.f - hp.adam_beta2;
  a.eps = hp.adam_eps;
  a.keep = 1.f - hp.adam_lr * hp.adam_weight_decay;
  const double t = (double)hp.adam_step;
  const double bc1 = 1.0 - std::pow((double)hp.adam_beta1, t);
  const double bc2 = 1.0 - std::pow((double)hp.adam_beta2, t);
  a.step = (float)((double)hp.adam_lr * std::sqrt(bc2) / bc1);
  a.key = adamw8_key(hp.adam_step);
  double bytes = 0.0;
  uint32_t wgs = 0;
  auto go = [&]() -> hipError_t {
    if (a.tensors == 0) return hipSuccess;
    const hipError_t e = timed(F_ADAMW8, 0.0, bytes, s, [&] {
      for (uint32_t b0 = 0; b0 < wgs; b0 += kMaxGrid) {
        a.wg_base = b0;
        const dim3 g(wgs - b0 < kMaxGrid ? wgs - b0 : kMaxGrid), b(256);
        const bool stream = bytes > ADAMW8_STREAM_BYTES;
        if (a.eps < 0x1p-38f) {
          if (stream) hipLaunchKernelGGL((adamw8_kernel<true, true>), g, b, 0, s, a);
          else hipLaunchKernelGGL((adamw8_kernel<true, false>), g, b, 0, s, a);
        } else {
          if (stream) hipLaunchKernelGGL((adamw8_kernel<false, true>), g, b, 0, s, a);
          else hipLaunchKernelGGL((adamw8_kernel<false, false>), g, b, 0, s, a);
        }
        const hipError_t r = hipGetLastError();
        if (r != hipSuccess) return r;
      }
      return hipSuccess;
    });
    a.tensors = 0;
    wgs = 0;
    bytes = 0.0;
    return e;
  };
  for (int32_t p : P.adam8) {
    const muon_param_shape& sh = P.table[p];
    const int64_t numel = sh.rows * sh.cols;
    if (numel == 0) continue;
    // the planner keeps numel / per at 2^29 or less
    const int64_t per = (int64_t)ADAMW8_BLOCK * ADAMW8_WAVE_BLOCKS * 4;
    const uint32_t n = (uint32_t)((numel + per - 1) / per);
    if (a.tensors == ADAMW8_TENSORS || wgs > (1u << 30)) {
      const hipError_t e = go();
      if (e != hipSuccess) return e;
    }
    Adamw8Desc& d = a.desc[a.tensors];
    d.w = ptrs[p].param;
    d.g = ptrs[p].grad;
    d.m = reinterpret_cast<uint8_t*>(ptrs[p].exp_avg);
    d.v = reinterpret_cast<uint8_t*>(ptrs[p].exp_avg_sq);
    d.numel = numel;
    d.dtype = sh.dtype == MUON_F32 ? DT_F32 : DT_BF16;
    a.first[a.tensors++] = wgs;
    wgs += n;
    bytes += (double)numel * (sh.dtype == MUON_F32 ? 16.0 : 10.0);
  }
  return go();
}

}  // namespace muon

extern "C" {

muon_status muon_adamw8_state_bytes(int64_t numel, size_t* bytes) {
  if (!bytes) return MUON_E_ARG;
  if (numel < 0 || numel > ADAMW8_MAX_NUMEL) return MUON_E_SHAPE;
  const size_t blocks = ((size_t)numel + ADAMW8_BLOCK - 1) / ADAMW8_BLOCK;
  *bytes = blocks * ADAMW8_BLOCK + (blocks * 2 + 15) / 16 * 16;
  return MUON_OK;
}

static muon_status adamw8_convert(bool pack, float* x, void* state, int64_t numel, int32_t moment, int64_t step,
                                  void* stream) {
  if (moment != MUON_ADAMW8_FIRST && moment != MUON_ADAMW8_SECOND) return MUON_E_METHOD;
  if (numel < 0 || numel > ADAMW8_MAX_NUMEL) return MUON_E_SHAPE;
  if (numel == 0) return MUON_OK;
  if (!x || !state || reinterpret_cast<uintptr_t>(x) % 4 || reinterpret_cast<uintptr_t>(state) % 4) return MUON_E_ARG;
  Adamw8PackArgs a;
  std::memset(&a, 0, sizeof(a));
  a.x = x;
  a.state = static_cast<uint8_t*>(state);
  a.numel = numel;
  a.key = adamw8_key(step);
  const int64_t wgs = (numel + ADAMW8_BLOCK * 4 - 1) / (ADAMW8_BLOCK * 4);
  const dim3 g((unsigned)(wgs < 65536 ? wgs : 65536)), b(256);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const hipError_t e = timed(F_ADAMW8, 0.0, 5.0 * (double)numel, s, [&] {
    const bool second = moment == MUON_ADAMW8_SECOND;
    if (pack && second) hipLaunchKernelGGL((adamw8_pack_kernel<true>), g, b, 0, s, a);
    else if (pack) hipLaunchKernelGGL((adamw8_pack_kernel<false>), g, b, 0, s, a);
    else if (second) hipLaunchKernelGGL((adamw8_unpack_kernel<true>), g, b, 0, s, a);
    else hipLaunchKernelGGL((adamw8_unpack_kernel<false>), g, b, 0, s, a);
    return hipGetLastError();
  });
  return e == hipSuccess ? MUON_OK : MUON_E_HIP;
}

muon_status muon_adamw8_pack(const float* x, int64_t numel, int32_t moment, int64_t step, void* state, void* stream) {
  return adamw8_convert(true, const_cast<float*>(x), state, numel, moment, step, stream);
}

muon_status muon_adamw8_unpack(const void* state, int64_t numel, int32_t moment, float* x, void* stream) {
  return adamw8_convert(false, x, const_cast<void*>(state), numel, moment, 0, stream);
}

}  // extern "C"
