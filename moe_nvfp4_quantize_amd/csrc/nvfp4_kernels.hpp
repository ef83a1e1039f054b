// nvfp4_kernels.hpp -- parameter blocks and launchers shared between the
// kernels (*.hip) and the C ABI layer (api.cpp).  Internal; not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "nvfp4_common.hpp"

namespace nvfp4 {

// ---------------------------------------------------------------- quantize
constexpr uint32_t kMaxPartials = 256;  // amax partials per matrix

// Arrival state of the single-read (resident) quantize kernel; lives at the
// start of the quantize workspace, which must be zero-filled before its first
// use.  Every completed launch leaves it ready for the next one.
constexpr uint32_t kMaxResidentWGs = 1024;
struct ResidentState {
  uint32_t parity;     // which slot array the current launch uses
  uint32_t done;       // workgroups finished in the current launch
  uint32_t fallbacks;  // workgroups whose wait expired (diagnostic; 0 when co-resident)
  // bound on each arrival wait, in polls; 0 (the zero-filled state) means the
  // built-in bound.  The kernels never write it: a caller may set a tiny bound
  // to force the expired-wait path (a test of that path).
  uint32_t spin_limit;
  // slot[p][w] = 0x80000000 | bits(max|x| of workgroup w): arrival flag and
  // value in one word, written and read with relaxed atomics
  uint32_t slot[2][kMaxResidentWGs];
};
constexpr size_t kResidentStateBytes = (sizeof(ResidentState) + 255) / 256 * 256;

struct QuantParams {
  const void *x;      // first element of matrix 0
  int64_t ld;         // row stride of x, elements
  int64_t x_mstride;  // elements between consecutive matrices
  uint32_t rows, nbpr, units;  // nbpr = cols/16, units = rows*nbpr
  FastDiv div_nbpr;
  uint8_t *q;  // [batch][rows][cols/2]
  uint8_t *s;  // [batch][rows][cols/16]
  float *g;    // [batch]
  int64_t q_mstride, s_mstride;  // bytes between matrices
  float *partials;               // [batch][P] workspace
  uint32_t P;                    // partials per matrix
  int static_global;
  int four6;  // block scale by the four-over-six rule (two-pass path)
  // quantize-dequantize: y [rows][ld_y] of the input type receives the decoded
  // values instead of q/s being written (nullptr: plain quantize)
  void *y;
  int64_t ld_y;
  // FP8 W8A8: q [rows][cols] receives one E4M3 code per element, the scale is
  // amax / 448, s is not written
  int fp8;
};

uint32_t quantize_partials_per_matrix(uint64_t units);
// st: resident-kernel state (nullptr: two-pass path only)
hipError_t launch_quantize(QuantParams p, bool bf16, bool vec, uint32_t batch, ResidentState *st,
                           hipStream_t stream);

// -------------------------------------------------------------------- GEMM
struct GemmParams {
  const uint8_t *a_q, *a_s;
  const float *a_g;
  const uint8_t *b_q, *b_s;
  const float *b_g;
  uint32_t M, N, K;
  void *c;
  int64_t ldc;
  // grouped (MoE) mode
  uint32_t a_rows;                // rows of A (the gather's source rows)
  const int32_t *src_row;         // nullable row gather
  const int32_t *expert_offsets;  // [E+1]
  uint32_t E;
  int64_t b_mstride_q, b_mstride_s;  // bytes between expert matrices
  // NVFP4 output of the SiLU-gate epilogue (static global scale h_g)
  uint8_t *h_q, *h_s;
  const float *h_g;
};

enum class OutType { F32, BF16 };
enum class Epilogue { None, SiluGate, SiluGateNvfp4 };

hipError_t launch_gemm(const GemmParams &p, OutType out, hipStream_t stream);
// whether the fused SiLU-gate -> NVFP4 epilogue can run these operands
bool grouped_nvfp4_out_supported(const GemmParams &p);
hipError_t launch_grouped_gemm(const GemmParams &p, uint32_t R, OutType out, Epilogue epi,
                               hipStream_t stream);

// --------------------------------------------------------------- FP8 GEMM
// C [M][N] (ldc) = (a_g b_g) * A B^T with A [M][K] and B [N][K] dense
// row-major E4M3FN bytes (row stride K), K % 16 == 0, 16-byte aligned bases.
struct Fp8GemmParams {
  const uint8_t *a_q;
  const float *a_g;
  const uint8_t *b_q;
  const float *b_g;
  uint32_t M, N, K;
  void *c;
  int64_t ldc;
};

// whether the direct-to-LDS kernel runs these operands (else the plain one)
bool fp8_gemm_dma_ok(const Fp8GemmParams &p);
hipError_t launch_fp8_gemm(const Fp8GemmParams &p, OutType out, hipStream_t stream);

// ------------------------------------------------------- block-scaled FP8
struct Fp8BlockQuantParams {
  const void *x;
  int64_t ld;  // row stride of x, elements
  uint32_t rows, cols;
  uint32_t block_rows;  // 1 or 128
  uint32_t blocks;      // scales: ceil(rows / block_rows) * ceil(cols / 128)
  FastDiv div_kb;       // by ceil(cols / 128)
  uint8_t *q;           // [rows][cols]
  float *s;             // [ceil(rows / block_rows)][ceil(cols / 128)]
};

hipError_t launch_fp8_block_quantize(const Fp8BlockQuantParams &p, bool bf16, bool vec, hipStream_t stream);

struct Fp8BlockGemmParams {
  const uint8_t *a_q;  // [M][K]
  const float *a_s;    // [M][ceil(K / 128)]
  const uint8_t *b_q;  // [N][K]
  const float *b_s;    // [ceil(N / 128)][ceil(K / 128)]
  uint32_t M, N, K;
  void *c;
  int64_t ldc;
};

hipError_t launch_fp8_block_gemm(const Fp8BlockGemmParams &p, OutType out, hipStream_t stream);

// --------------------------------------------------------------------- MoE
size_t route_workspace_bytes(int64_t T, int32_t E, int32_t k);
hipError_t launch_route(const float *logits, int64_t T, int32_t E, int32_t k, int32_t *topk_ids,
                        float *topk_w, int32_t *offsets, int32_t *src_row, int32_t *inv,
                        void *workspace, hipStream_t stream);
hipError_t launch_combine(const void *y, bool y_bf16, const float *w, const int32_t *inv, int64_t T,
                          int32_t k, int64_t H, void *out, bool out_bf16, hipStream_t stream);

// The routed-expert layer for few tokens.  The caller fills the first part;
// launch_moe_decode lays out the workspace and fills the rest.
struct MoeDecodeParams {
  const void *x;
  int64_t ld_x;         // elements
  const float *logits;  // [T][E]
  uint32_t T, E, k, H, I;
  const uint8_t *gu_q, *gu_s;  // [E][2I][H/2], [E][2I][H/16]
  const float *gu_g;           // [E]
  const uint8_t *d_q, *d_s;    // [E][H][I/2], [E][H][I/16]
  const float *d_g;            // [E]
  void *out;
  int64_t ld_out;

  uint32_t S;                  // slots T k
  uint32_t tiles_i, tiles_h;   // row tiles of I and H (a launch's own)
  uint32_t topk_blocks;        // workgroups of the prep kernel that route
  int32_t *ids;                // [S] expert of slot t k + j
  float *w;                    // [S] routing weight
  int32_t *xe;                 // [T] x's power of two
  _Float16 *xp;                // [2][T][H] f16 planes of x
  _Float16 *h;                 // [2][S][I] f16 planes of h
  int8_t *he;                  // [S][he_ld] h's powers, a block of 16 each
  int64_t he_ld;               // I / 16 rounded up to 4
  float *y;                    // [S][H] weighted products
};

constexpr uint32_t kMaxDecodeTokens = 128;
size_t moe_decode_workspace_bytes(int64_t T, int32_t E, int32_t k, int64_t H, int64_t I);
hipError_t launch_moe_decode(MoeDecodeParams p, bool x_bf16, bool gu_aligned, bool d_aligned, bool out_bf16,
                             void *workspace, hipStream_t stream);

}  // namespace nvfp4
