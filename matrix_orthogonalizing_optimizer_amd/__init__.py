"""libmuon for AMD Instinct MI355X: the Muon optimizer step as hand-written
HIP kernels behind a C ABI (include/libmuon.h), and the operators that make
the gradients it reads (norms, activations kept as 8-bit rows, the linear
layer on them, matrix products grouped by expert), with a thin ctypes binding of the same names."""
from ._lib import (EXPORTED, MUON_BF16, MUON_COEFF_HYBRID, MUON_COEFF_QUINTIC,  # noqa: F401
                   MUON_ADAMW8_FIRST, MUON_ADAMW8_SECOND, MUON_F32, MUON_KIND_ADAMW, MUON_KIND_ADAMW8,
                   MUON_KIND_MUON, MUON_NS_AUTO, MUON_NS_GRAM, MUON_NS_GRAM_RESTART,
                   MUON_NS_STANDARD, MUON_LINEAR8_FORWARD, MUON_LINEAR8_INPUT_GRAD, MUON_LINEAR8_WEIGHT_GRAD,
                   MUON_NORM_LAYER, MUON_NORM_RMS, muon_linear8_forward, muon_linear8_input_grad,
                   muon_linear8_weight_grad, muon_linear8_workspace_bytes, muon_norm_backward,
                   muon_norm_backward_workspace_bytes, muon_norm_forward, muon_rows8_dequantize, muon_rows8_quantize,
                   MUON_SCALE_MOONLIGHT, MUON_SCALE_SPECTRAL, MUON_SCALE_UNIT_RMS, MuonError, Plan,
                   lib, make_hparams, MUON_EXPERTS_FORWARD, MUON_EXPERTS_INPUT_GRAD, MUON_EXPERTS_WEIGHT_GRAD,
                   muon_experts_forward, muon_experts_input_grad, muon_experts_weight_grad,
                   muon_experts_workspace_bytes, muon_adamw8_pack, muon_adamw8_state_bytes, muon_adamw8_unpack,
                   muon_ns_coefficients, muon_probe_copy, muon_probe_copy_lds, muon_probe_mfma,
                   muon_plan_buckets, muon_plan_create, muon_plan_units, muon_plan_workspace_bytes,
                   muon_status_string, muon_step, muon_timing_collect, muon_timing_enable,
                   muon_version, ns_orthogonalize, ns_orthogonalize_noalloc,
                   ns_orthogonalize_workspace_bytes)
