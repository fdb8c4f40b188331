// Host-side launchers of the libmuon kernels (implemented in the .hip files).
#pragma once

#include <hip/hip_runtime.h>

#include "kernel_args.hpp"
#include "libmuon.h"

namespace muon {

struct PlanImpl;

// GEMM launch for input dtype ti / output dtype to (DT_*), tile edge 128 or
// 256, symmetric-output flag, epilogue kind and operand layout (trans: both
// operands K-major, element (i, k) at p[k * ld + i]).  Returns
// hipErrorInvalidValue for a combination that is not instantiated.
hipError_t launch_gemm(int tile, int ti, int to, bool sym, int epi, bool trans, const GemmArgs& a, hipStream_t s);
hipError_t launch_gemm_bf16(int tile, int to, bool sym, int epi, bool trans, const GemmArgs& a, hipStream_t s);
hipError_t launch_gemm_f16(int tile, int to, bool sym, int epi, bool trans, const GemmArgs& a, hipStream_t s);
hipError_t launch_gemm_f32(int tile, int to, bool sym, int epi, bool trans, const GemmArgs& a, hipStream_t s);

hipError_t launch_momentum(int gdtype, int xdtype, bool tall, const MomArgs& a, int64_t blocks,
                           hipStream_t s);
hipError_t launch_norm_finalize(const float* partials, int32_t per_unit, float4* aux, int32_t units,
                                hipStream_t s);
hipError_t launch_adamw(const AdamArgs& a, int64_t total_blocks, hipStream_t s);
// The AdamW parameters of the plan with 8-bit moments.
hipError_t launch_adamw8(const PlanImpl& P, const muon_param_ptrs* ptrs, const muon_hparams& hp, hipStream_t s);
// Writes `bytes` (a multiple of 4) from host memory src to device memory dst
// (4-byte aligned) through the arguments of ceil(bytes / 3 KiB) small kernel
// launches on s; src may be reused as soon as the call returns.
hipError_t launch_upload(void* dst, const void* src, size_t bytes, hipStream_t s);

// Row operators.  kind: 0 layer norm, 1 RMS norm, 2 (forward only) no norm.
// dt: dtype of x / dy / y / dx.  parts: workgroups of the backward kernel,
// and rows of a.partials.
hipError_t launch_row_forward(int kind, int dt, const RowArgs& a, hipStream_t s);
hipError_t launch_row_restore(int dt, const RestoreArgs& a, hipStream_t s);
hipError_t launch_norm_backward(int kind, int dt, const NormBwdArgs& a, int parts, hipStream_t s);
hipError_t launch_norm_join(int vec_dtype, const JoinArgs& a, hipStream_t s);

// Linear layer on 8-bit rows.  tile: 128 or 256; odt: dtype of the result;
// expanded: a.B is the 8-bit operand turned into bf16 (256 tiles only).
hipError_t launch_linear8_forward(int tile, int odt, const Linear8Args& a, hipStream_t s);
hipError_t launch_linear8_few(int odt, const Linear8Args& a, hipStream_t s);  // at most 64 tokens
hipError_t launch_linear8_bias(int odt, const Linear8Args& a, hipStream_t s);  // no channels in
hipError_t launch_linear8_planes(int dt, const PlanesArgs& a, hipStream_t s);
hipError_t launch_linear8_dw(int tile, bool expanded, bool dy_f32, int odt, const Linear8Args& a, hipStream_t s);
hipError_t launch_linear8_dx(int tile, bool expanded, bool dy_f32, int odt, const Linear8Args& a, hipStream_t s);

// Products grouped by expert.  dt, odt: dtypes of the operands and of the
// result; direct: bf16 rows of whole 16-byte pieces; tiles: most that any
// offsets need (before they are split); joined: of them, those left in parts.
hipError_t launch_experts_y(bool direct, int dt, int odt, int64_t tiles, int64_t joined, const ExpertsArgs& a, hipStream_t s);
hipError_t launch_experts_big_y(int odt, const ExpertsArgs& a, hipStream_t s);  // tiles from lists (experts_big.hpp)
hipError_t launch_experts_big_dw(int odt, const ExpertsArgs& a, hipStream_t s);
hipError_t launch_experts_big_dx(int odt, const ExpertsArgs& a, hipStream_t s);
hipError_t launch_experts_few(int dt, int odt, const ExpertsArgs& a, hipStream_t s);  // forward, few rows an expert
hipError_t launch_experts_dw(bool direct, int dt, int odt, int64_t tiles, int64_t joined, const ExpertsArgs& a, hipStream_t s);
hipError_t launch_experts_dx(bool direct, int dt, int odt, int64_t tiles, int64_t joined, const ExpertsArgs& a, hipStream_t s);

}  // namespace muon
