// fp8_block_quantize.hip -- block-scaled FP8 (E4M3) quantize on gfx950.
//
// The FP8 sibling of the per-tensor quantizer with one float32 scale per block
// of 128 columns, over one row (activations) or 128 rows (weights):
//   s = max(amax(block) / 448, 2^-126), 1 for a block of zeros;
//   q = the E4M3 code nearest the quotient x / s, ties to even.
// The code is decided by the real quotient, not by its float32 rounding: a
// quotient that only rounds onto a midpoint of two codes still goes to the side
// it lies on, so the result does not depend on how the division is carried out.
// With y = fl(x / s) (a reciprocal and two FMAs) the remainder e = x - y s is
// exact in one FMA, and its sign says on which side of y the quotient lies: y's
// last bit is set towards it (rounding to odd), after which rounding to E4M3's
// four significant bits is a rounding of the quotient itself.
//
// Bound: HBM, one read of x, one write of the codes.  16 elements per lane (two
// or four 16-byte loads, one 16-byte store), so a row's block is eight lanes and
// its maximum three lane exchanges; a 128 x 128 tile is one workgroup that keeps
// its elements in registers while their maximum crosses the waves through LDS.
#include "nvfp4_common.hpp"
#include "nvfp4_format.hpp"
#include "nvfp4_kernels.hpp"

namespace nvfp4 {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr float kMinScale = 0x1p-126f;  // the smallest normal float

template <typename T, bool VEC>
__device__ __forceinline__ void load16(const T *p, float v[16]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u32x4 w;
      if constexpr (VEC) w = *reinterpret_cast<const u32x4 *>(p + 4 * j);
      else
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = f2u(p[4 * j + e]);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * j + e] = u2f(w[e]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if constexpr (VEC) {
        const u32x4 w = *reinterpret_cast<const u32x4 *>(p + 8 * j);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[8 * j + 2 * e] = bf16_lo(w[e]);
          v[8 * j + 2 * e + 1] = bf16_hi(w[e]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[8 * j + e] = u2f((uint32_t)p[8 * j + e] << 16);
      }
    }
  }
}

__device__ __forceinline__ float amax16(const float v[16]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(v[i]));
  return m;
}

__device__ __forceinline__ float block_decode_scale(float amax) {
  return amax == 0.0f ? 1.0f : fmaxf(amax / kE4M3Max, kMinScale);
}

// Blocks of very small values are worked on 2^64 larger (an exact scaling of x
// and s alike), so that the remainder below never underflows.
__device__ __forceinline__ u32x4 encode16(const float v[16], float s) {
  const float up = s < 0x1p-60f ? 0x1p64f : 1.0f;
  s *= up;
  const float rs = 1.0f / s;
  float y[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float a = fabsf(v[i]) * up;
    const float t = div_rn(a, s, rs);
    const float e = __builtin_fmaf(-t, s, a);
    uint32_t u = f2u(t);
    u -= e < 0.0f ? 1u : 0u;
    u |= e != 0.0f ? 1u : 0u;
    y[i] = u2f(u | (f2u(v[i]) & 0x80000000u));
  }
  u32x4 o;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * j], y[4 * j + 1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * j + 2], y[4 * j + 3], w, true);
    o[j] = (uint32_t)w;
  }
  return o;
}

// One scale per row and 128 columns: eight lanes per block, U blocks per lane
// (their loads are in flight together).  Measured: bf16 8192 x 5120 in 24.9 us (128
// MB moved, 5.1 TB/s, where a large copy moves 5.2); 1 x 5120 in 2.8 us, a launch.
template <typename T, bool VEC, int U>
__global__ __launch_bounds__(256) void block_quantize_rows_kernel(Fp8BlockQuantParams p) {
  const uint32_t l8 = threadIdx.x % 8;
  const uint32_t g0 = blockIdx.x * (32u * U) + threadIdx.x / 8;
  float v[U][16];
  uint32_t row[U], kb[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint32_t g = min(g0 + 32u * i, p.blocks - 1);
    row[i] = p.div_kb.div(g);
    kb[i] = g - row[i] * p.div_kb.d;
    const uint32_t col = kb[i] * 128 + l8 * 16;
#pragma unroll
    for (int e = 0; e < 16; ++e) v[i][e] = 0.0f;
    if (col < p.cols) load16<T, VEC>((const T *)p.x + (int64_t)row[i] * p.ld + col, v[i]);
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    float m = amax16(v[i]);
    m = fmaxf(m, __shfl_xor(m, 1, 64));
    m = fmaxf(m, __shfl_xor(m, 2, 64));
    m = fmaxf(m, __shfl_xor(m, 4, 64));
    const float s = block_decode_scale(m);
    const u32x4 c = encode16(v[i], s);
    const uint32_t g = g0 + 32u * i, col = kb[i] * 128 + l8 * 16;
    if (g >= p.blocks) continue;
    if (col < p.cols) *reinterpret_cast<u32x4 *>(p.q + (int64_t)row[i] * p.cols + col) = c;
    if (l8 == 0) p.s[g] = s;
  }
}

// One scale per 128 x 128 tile: thread t holds 16 columns of rows t / 8 + 32 i.
// Measured: bf16 25600 x 5120 in 77.6 us (393 MB, 5.1 TB/s).
template <typename T, bool VEC>
__global__ __launch_bounds__(256) void block_quantize_tiles_kernel(Fp8BlockQuantParams p) {
  const uint32_t tr = p.div_kb.div(blockIdx.x), kb = blockIdx.x - tr * p.div_kb.d;
  const uint32_t col = kb * 128 + (threadIdx.x % 8) * 16, r0 = tr * 128 + threadIdx.x / 8;
  float v[4][16];
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int e = 0; e < 16; ++e) v[i][e] = 0.0f;
    if (r0 + 32 * i < p.rows && col < p.cols)
      load16<T, VEC>((const T *)p.x + (int64_t)(r0 + 32 * i) * p.ld + col, v[i]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) m = fmaxf(m, amax16(v[i]));
  const float s = block_decode_scale(block_max(m));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const u32x4 c = encode16(v[i], s);
    if (r0 + 32 * i < p.rows && col < p.cols)
      *reinterpret_cast<u32x4 *>(p.q + (int64_t)(r0 + 32 * i) * p.cols + col) = c;
  }
  if (threadIdx.x == 0) p.s[blockIdx.x] = s;
}

template <typename T, bool VEC>
hipError_t launch_t(const Fp8BlockQuantParams &p, hipStream_t stream) {
  if (p.block_rows == 1) {
    constexpr int U = 2;
    block_quantize_rows_kernel<T, VEC, U><<<(p.blocks + 32 * U - 1) / (32 * U), 256, 0, stream>>>(p);
  } else {
    block_quantize_tiles_kernel<T, VEC><<<p.blocks, 256, 0, stream>>>(p);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_block_quantize(const Fp8BlockQuantParams &p, bool bf16, bool vec, hipStream_t stream) {
  if (p.blocks == 0) return hipSuccess;
  if (bf16) return vec ? launch_t<uint16_t, true>(p, stream) : launch_t<uint16_t, false>(p, stream);
  return vec ? launch_t<float, true>(p, stream) : launch_t<float, false>(p, stream);
}

}  // namespace nvfp4
