// Tiling constants shared by the host planner and the kernels.
#pragma once

namespace muon {
constexpr int KM_TR = 64;       // momentum kernel tile rows (parameter layout)
constexpr int KM_TC = 256;      // momentum kernel tile columns
constexpr int KMR_TR = 4;       // momentum kernel tile rows, tall units (row-contiguous tiles)
constexpr int KMR_TC = 512;     // momentum kernel tile columns, tall units
constexpr int ADAM_EPB = 4096;  // AdamW elements per workgroup
constexpr int ADAMW8_BLOCK = 256;     // elements that share one offset of the 8-bit moments
constexpr int ADAMW8_WAVE_BLOCKS = 2; // of them a wave updates
constexpr int ADAMW8_TENSORS = 76;    // tensors per launch: their descriptors fit its 4 KiB of arguments
constexpr long long ADAMW8_MAX_NUMEL = 1ll << 40;  // workgroups counted in 32 bits
constexpr int ROW_MAX_COLS = 16384;      // longest row the forward row operators keep in registers
constexpr int NORM_BWD_MAX_COLS = 8192;  // the same for the norm's backward pass, which holds two rows and two sums
}  // namespace muon
