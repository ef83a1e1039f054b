// fp8_block_gemm.hip -- FP8 (E4M3) GEMM with one scale per block of 128 on gfx950.
//
//   C[m][n] = sum_b a_s[m][b] * b_s[n / 128][b]
//                   * sum_{k in block b} e4m3(A[m][k]) * e4m3(B[n][k])
// A [M][K] activations with a scale per row and 128 columns, B [N][K] weights
// with a scale per 128 x 128 tile, both row-major E4M3FN bytes.  The scales are
// float32, which the matrix instructions cannot carry (their own block scales
// are powers of two), so each 128-column block is multiplied from a zero
// accumulator and joined to the running sum by one float32 FMA per output with
// the product of its two scales.
//
// Which matrix instruction: the FP8 MFMAs of gfx950 (the block-scaled and the
// older unscaled ones alike) add neighbouring products with about 14 bits below
// the largest of them (448 * 448 + 14.06 comes out as 448 * 448 + 8; products
// further apart in K add exactly), which leaves 1.4e-5 of a result of 128 random
// products.  That vanishes in a bf16 result (2^-9), which uses them; a float32
// result takes the operands exactly to f16 (E4M3 has 4 significant bits and
// exponents inside f16's) and the f16 MFMA, whose sums are good to float32, at
// half the matrix rate.
#include "nvfp4_common.hpp"
#include "nvfp4_format.hpp"
#include "nvfp4_kernels.hpp"

#include <type_traits>

namespace nvfp4 {

namespace {

typedef float float4v __attribute__((ext_vector_type(4)));
typedef float float16v __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef _Float16 half8v __attribute__((ext_vector_type(8)));

// 32 E4M3 bytes of a lane's row, as the matrix instruction takes them
struct Fp8Frag {
  u32x4 lo, hi;
};

__device__ __forceinline__ i32x8 joined(const Fp8Frag &f) {
  return __builtin_bit_cast(i32x8, __builtin_shufflevector(f.lo, f.hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// bytes [8j, 8j + 8) as f16 (exact)
__device__ __forceinline__ half8v halves(const Fp8Frag &f, int j) {
  const u32x4 w = j < 2 ? f.lo : f.hi;
  const uint32_t a = w[2 * (j % 2)], b = w[2 * (j % 2) + 1];
  const half2v p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, false);
  const half2v p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, true);
  const half2v p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, false);
  const half2v p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, true);
  return (half8v){p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// acc += a x b over 64 of K, 32 x 32 (lane half h holds bytes [32h, 32h + 32)
// of its row of either operand: any K order that both share)
template <bool EXACT>
__device__ __forceinline__ float16v mul32(const Fp8Frag &a, const Fp8Frag &b, float16v acc) {
  if constexpr (EXACT) {
#pragma unroll
    for (int j = 0; j < 4; ++j) acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(halves(a, j), halves(b, j), acc, 0, 0, 0);
    return acc;
  } else {
    // both operands E4M3 (formats 0), unit block scales (E8M0 127)
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(joined(a), joined(b), acc, 0, 0, 0, 127, 0, 127);
  }
}

// acc += a x b over 128 of K, 16 x 16 (lane quarter q holds bytes [32q, 32q + 32))
template <bool EXACT>
__device__ __forceinline__ float4v mul16(const Fp8Frag &a, const Fp8Frag &b, float4v acc) {
  if constexpr (EXACT) {
#pragma unroll
    for (int j = 0; j < 4; ++j) acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(halves(a, j), halves(b, j), acc, 0, 0, 0);
    return acc;
  } else {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(joined(a), joined(b), acc, 0, 0, 0, 127, 0, 127);
  }
}

template <typename OutT>
__device__ __forceinline__ OutT to_out(float v);
template <>
__device__ __forceinline__ float to_out<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t to_out<uint16_t>(float v) { return (uint16_t)float_to_bf16_bits(v); }

template <typename OutT>
constexpr bool kExact = sizeof(OutT) == 4;

// bytes [k, k + 32) of a row, zero past K (K % 16 == 0: a 16-byte piece is all
// in or all out)
__device__ __forceinline__ Fp8Frag load_frag(const uint8_t *row, uint64_t k, uint64_t K) {
  Fp8Frag f = {{0, 0, 0, 0}, {0, 0, 0, 0}};
  if (k < K) f.lo = *reinterpret_cast<const u32x4 *>(row + k);
  if (k + 16 < K) f.hi = *reinterpret_cast<const u32x4 *>(row + k + 16);
  return f;
}

// Plain kernel (any K % 16 == 0, 64-bit offsets): a 64 x 64 tile per workgroup,
// one 32 x 32 MFMA tile per wave, operands loaded from global memory into
// registers 16 bytes at a time (zero past K).  The weight fragment goes first,
// so a lane's accumulators are one row of C and its scale one factor.
template <typename OutT>
__global__ __launch_bounds__(256) void block_gemm_plain_kernel(Fp8BlockGemmParams p) {
  const uint32_t tid = threadIdx.x, wave = tid / 64, lane = tid % 64;
  const uint32_t l32 = lane % 32, lh = lane / 32;
  const uint32_t tiles_n = (p.N + 63) / 64;
  const uint32_t row0 = (blockIdx.x / tiles_n) * 64 + (wave / 2) * 32;
  const uint32_t col0 = (blockIdx.x % tiles_n) * 64 + (wave % 2) * 32;
  const uint64_t K = p.K;
  const uint32_t KB = (p.K + 127) / 128;
  const uint32_t m = min(row0 + l32, p.M - 1), n = min(col0 + l32, p.N - 1);
  const uint8_t *ar = p.a_q + (uint64_t)m * K, *br = p.b_q + (uint64_t)n * K;
  const float *as = p.a_s + (uint64_t)m * KB;
  const float *bs = p.b_s + (uint64_t)(min(col0, p.N - 1) / 128) * KB;  // 32 columns lie in one scale row
  float16v acc = {};
  for (uint32_t kb = 0; kb < KB; ++kb) {
    float16v part = {};
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint64_t k = (uint64_t)kb * 128 + 64 * t + 32 * lh;
      part = mul32<kExact<OutT>>(load_frag(br, k, K), load_frag(ar, k, K), part);
    }
    const float f = as[kb] * bs[kb];
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[r] = __builtin_fmaf(part[r], f, acc[r]);
  }
  // accumulator 4q + e of lane (l32, lh): row l32, column 8q + 4 lh + e
  OutT *Cp = static_cast<OutT *>(p.c);
  const uint32_t row = row0 + l32;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const uint32_t col = col0 + 8 * (r / 4) + 4 * lh + (r % 4);
    if (row < p.M && col < p.N) Cp[(int64_t)row * p.ldc + col] = to_out<OutT>(acc[r]);
  }
}

template <typename OutT>
hipError_t launch_typed(const Fp8BlockGemmParams &p, hipStream_t stream) {
  const uint64_t grid = (uint64_t)((p.M + 63) / 64) * ((p.N + 63) / 64);
  if (grid > 0x7FFFFFFFull) return hipErrorInvalidValue;
  block_gemm_plain_kernel<OutT><<<(uint32_t)grid, 256, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_block_gemm(const Fp8BlockGemmParams &p, OutType out, hipStream_t stream) {
  if (p.M == 0 || p.N == 0) return hipSuccess;
  return out == OutType::F32 ? launch_typed<float>(p, stream) : launch_typed<uint16_t>(p, stream);
}

}  // namespace nvfp4
