// Argument blocks of the libmuon kernels (shared by launchers and kernels).
#pragma once

#include "consts.hpp"
#include "device_common.hpp"

namespace muon {

// Epilogues: C = alpha L R^T (SCALE); C = alpha L R^T + beta E + gamma I
// (POLY); the fused parameter update (FINAL).
enum : int32_t { EPI_SCALE = 0, EPI_POLY = 1, EPI_FINAL = 2 };
enum : int32_t { SEL_ONE = 0, SEL_INV_S = 1, SEL_INV_S2 = 2 };
enum : int32_t { FINAL_UPDATE = 0, FINAL_STORE = 1 };

struct GemmArgs {
  const void* L;   // M x K, K contiguous
  const void* R;   // N x K, K contiguous
  const void* E;   // epilogue addend (EPI_POLY), same layout as C
  void* C;         // direct output (M x N), or null; EPI_FINAL writes the parameters (TO = their dtype)
  void* C2;        // mirror output (N x M, the transpose), or null; C for a symmetric product
  int64_t ldl, ldr, lde, ldc, ldc2;
  int64_t sL, sR, sE, sC, sC2;  // per-unit strides in elements
  int32_t M, N, K;         // logical per-unit sizes
  int32_t units, tilesM, tilesN, tilesPerUnit, totalTiles;
  float alpha, beta, gamma;
  int32_t alphaSel;        // SEL_*: alpha is multiplied by aux[u].y or aux[u].z
  const float4* aux;       // per unit {s^2, 1/s, 1/s^2, 0}
  const UnitDesc* desc;    // EPI_FINAL: per-unit parameter pointers
  float lr, wd;            // EPI_FINAL
  int32_t finalMode;       // FINAL_UPDATE or FINAL_STORE
  int32_t wvec;            // EPI_FINAL: parameter / update_out rows are 16-byte aligned, ld % 8 == 0
};

// Momentum kernel (see elementwise.hpp).
struct MomArgs {
  const UnitDesc* desc;
  void* D;         // U in the parameter's own layout (rows x cols), or null
  void* T;         // U transposed (cols x rows), or null
  int64_t ldd, ldt;  // leading dimensions (multiples of 8)
  int64_t sD, sT;    // per-unit element strides
  float* partials; // one per workgroup
  int32_t rows, cols;      // unit shape in parameter layout
  int32_t tilesR, tilesC, tilesPerUnit;
  float mu;
  int32_t nesterov;
  int32_t vec_ok;  // every unit's g/mom rows are 16-byte aligned and cols % 8 == 0
};

// AdamW kernel (see elementwise.hpp).
struct AdamArgs {
  const AdamDesc* desc;
  int64_t block_base;  // first global block of this launch
  int32_t nparams;
  float one_minus_b1, one_minus_b2, eps, keep, step;
};

// AdamW on 8-bit moments (see adamw8.hpp).
struct Adamw8Desc {
  void* w;
  const void* g;
  uint8_t* m;
  uint8_t* v;
  int64_t numel;
  int32_t dtype;  // DT_F32 or DT_BF16, of w and g
  int32_t pad;
};
struct Adamw8Args {
  float one_minus_b1, one_minus_b2, eps, keep, step;
  uint32_t key;      // of the step's random bits
  int32_t tensors;
  uint32_t wg_base;  // first workgroup of this launch
  uint32_t first[ADAMW8_TENSORS];  // first workgroup of every tensor
  Adamw8Desc desc[ADAMW8_TENSORS];
};
static_assert(sizeof(Adamw8Args) <= 4096, "kernel arguments");
struct Adamw8PackArgs {
  float* x;
  uint8_t* state;
  int64_t numel;
  uint32_t key;
};

// Row operators (see row_ops.hpp).
struct RowArgs {
  const void* x;
  const void* gamma;  // vec_dtype; null when only quantizing
  const void* beta;   // or null
  void* y;            // or null
  int8_t* q;          // or null
  float* scale;
  float* mean;        // or null
  float* rstd;        // or null
  int64_t ldx, ldy, ldq, rows;
  int32_t cols;
  int32_t vec_dtype;
  float eps;
};
struct RestoreArgs {
  const int8_t* q;
  const float* scale;
  void* y;
  int64_t ldq, ldy, rows;
  int32_t cols;
};
struct NormBwdArgs {
  const void* dy;
  const void* x;
  const void* gamma;
  const float* mean;
  const float* rstd;
  void* dx;
  float* partials;  // [2][workgroups][cols], or null: no vector gradients
  int64_t lddy, ldx, lddx, rows;
  int32_t cols;
  int32_t vec_dtype;
  int32_t sum_dy;   // the bias gradient is asked for
};
struct JoinArgs {
  const float* partials;
  void* dgamma;
  void* dbeta;
  int32_t parts;
  int32_t accumulate;
  int64_t cols;
};

// Products of the linear layer on 8-bit rows (see linear8.hpp): C (M x N) as
// a sum over K of A B.
//   forward          A = q (tokens x in), B = w (out x in), both K-contiguous
//   weight gradient  A = dy (tokens x out, K-major), B = q (tokens x in, K-major)
//   input gradient   A = dy (tokens x out, K-contiguous), B = w (out x in, K-major)
struct Linear8Args {
  const void* A;
  const void* B;      // int8; bf16 where the 8-bit operand was expanded
  const float* sa;    // forward: one per row of C
  const float* sb;    // forward: one per column of C; gradients: one per summation index
  const void* bias;   // forward: one per column of C, or null
  void* o;            // C
  float* ws;          // partial tiles
  int64_t lda, ldb, ldo;
  int32_t M, N, K;
  int32_t tilesM, tilesN;
  int32_t whole;      // tiles computed whole; the others in `splits` parts (all whole if splits is 1)
  int32_t splits;
  int32_t per_split;  // K-stages (128 bytes of a row) per split
  int32_t bias_dtype;
  int32_t accumulate;
  int32_t planes;     // gradients: bf16 planes (or pieces cut in the product) of dy that sum to it
  int64_t plane;      // elements between them
};
// Products grouped by expert (see experts.hpp): C as a sum over K of A B, for
// the rows offsets[e] .. offsets[e + 1] - 1 of expert e.
//   forward          A = x (rows x in),  B = w (experts x out x in), C = y
//   input gradient   A = dy (rows x out), B = w, C = dx
//   weight gradient  A = dy, B = x, C = dw (experts x out x in)
struct ExpertsArgs {
  const void* A;
  const void* B;
  void* o;                 // C
  const int32_t* offsets;  // experts + 1
  float* ws;               // partial tiles
  int64_t lda, ldb, ldo;
  int64_t se;              // elements between experts of w or dw
  int32_t rows, experts;
  int32_t M;               // weight gradient: rows of an expert's C
  int32_t N;               // columns of C
  int32_t K;               // forward, input gradient
  int32_t tilesM, tilesN;  // of an expert's C (tilesM: weight gradient)
  int32_t splits;          // parts of every tile's K
  int32_t accumulate;      // weight gradient: added to C
  // large products: lists of the tiles (see experts_big.hpp)
  int32_t chunk;           // weight gradient: rows of an expert that a tile sums at once
  int32_t cap;             // tiles that a list has room for
  struct ExpertsHead* head;
  struct ExpertsItem* items;
};
// What one workgroup does of a large product: `size` rows (low half) and columns
// (high half) of an expert's C from row0, col0 on, over `count` rows from `begin` on.
struct __attribute__((aligned(32))) ExpertsItem {
  int32_t begin, count;
  int32_t row0, col0;
  int32_t size;
  int32_t expert;
  int32_t slot;  // partial tile it leaves in the workspace; -1: C itself
  int32_t pad;
};
constexpr int EXPERTS_SPLIT = 512;  // experts whose rows take several chunks, at most
struct ExpertsHead {
  int32_t count[8];  // items of each list
  int32_t splits;    // experts summed in chunks
  int32_t pad[7];
  int32_t taken[8][16];  // items that the list's workgroups have taken, a cache line each
  struct {
    int32_t expert, slot, chunks;  // partial tiles from slot on: [chunk][tile]
  } split[EXPERTS_SPLIT];
};

// dy as bf16 planes (see linear8_planes_kernel).
struct PlanesArgs {
  const void* dy;
  void* o;
  int64_t ld, ldo, plane;
  int64_t rows;
  int32_t cols;
};

// Host table -> device memory through kernel arguments: one launch carries
// up to BLOB_WORDS 32-bit words of a descriptor table, so no host staging
// buffer, no host-to-device copy and no wait on the host are involved.
constexpr int BLOB_WORDS = 768;  // 3 KiB of payload per launch
struct BlobArgs {
  uint32_t* dst;
  uint32_t nwords;
  uint32_t pad;
  uint32_t words[BLOB_WORDS];
};

}  // namespace muon
