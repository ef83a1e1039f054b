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
// older unscaled ones alike) add the products of eight consecutive K at a common
// scale, each cut below 2^-13 of 2^(sum of the exponents) of the largest (448 *
// 448 + 14.06 comes out as 448 * 448 + 8; products further apart in K add
// exactly), which leaves 1.4e-5 of a result of 128 random products.  That
// vanishes in a bf16 result (2^-9), which uses them; a float32 result takes the
// operands exactly to f16 (E4M3 has 4 significant bits and exponents inside
// f16's) and the f16 MFMA, whose sums are good to float32, at half the matrix rate.
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

// A 32 x 64 operand of the 32 x 32 products (lane half h holds bytes [32h, 32h + 32)
// of its row of either operand: any K order that both share): the bytes
// themselves, or, for float32 results, their f16 values, converted once.
template <bool EXACT>
struct Operand {
  i32x8 v;
  __device__ __forceinline__ explicit Operand(const Fp8Frag &f) : v(joined(f)) {}
};
template <>
struct Operand<true> {
  half8v v[4];
  __device__ __forceinline__ explicit Operand(const Fp8Frag &f) : v{halves(f, 0), halves(f, 1), halves(f, 2), halves(f, 3)} {}
};

// acc += a x b
__device__ __forceinline__ float16v mul32(const Operand<true> &a, const Operand<true> &b, float16v acc) {
#pragma unroll
  for (int j = 0; j < 4; ++j) acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(a.v[j], b.v[j], acc, 0, 0, 0);
  return acc;
}
__device__ __forceinline__ float16v mul32(const Operand<false> &a, const Operand<false> &b, float16v acc) {
  // both operands E4M3 (formats 0), unit block scales (E8M0 127)
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a.v, b.v, acc, 0, 0, 0, 127, 0, 127);
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

// A row or a few (and, with 64-bit offsets, any number): bound by one read of B.  A
// workgroup owns 16 columns of 16 rows of C and its NW waves take the 128-column
// blocks of K in turn, U blocks' loads in flight together, straight into registers
// (M = 1 reads the same lines of A in every lane group).  The waves' sums are
// joined through LDS in wave order.  Measured: 1 x 151936 x 2048 in 51 us (311 MB, 6.1
// TB/s: part of it from the last-level cache), 1 x 4096 x 14336 in 14.1 us (4.2).  (16
// waves of 2: 67 and 14.6, half of them idle at K 2048; 8 of 4: 66 and 16.6.)
template <int NW, int U, typename OutT>
__global__ __launch_bounds__(NW * 64) void block_gemm_rows_kernel(Fp8BlockGemmParams p) {
  __shared__ __attribute__((aligned(16))) float red[NW][16][20];
  const uint32_t tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / 64), lane = tid % 64;
  const uint32_t l16 = lane % 16, lq = lane / 16;
  const uint32_t n0 = blockIdx.x * 16, m0 = blockIdx.y * 16;
  const uint64_t K = p.K;
  const uint32_t KB = (p.K + 127) / 128;
  const uint64_t m = min(m0 + l16, p.M - 1);
  const uint8_t *br = p.b_q + (uint64_t)min(n0 + l16, p.N - 1) * K, *ar = p.a_q + m * K;
  const float *as = p.a_s + m * KB;
  const float *bs = p.b_s + (uint64_t)(n0 / 128) * KB;  // 16 columns lie in one scale row
  float4v acc = {0, 0, 0, 0};
  for (uint32_t kb0 = wave; kb0 < KB; kb0 += NW * U) {
    Fp8Frag fb[U], fa[U];
    float f[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t kb = kb0 + NW * u;
      const uint64_t k = (uint64_t)kb * 128 + 32 * lq;
      fb[u] = load_frag(br, k, K);
      fa[u] = load_frag(ar, k, K);
      f[u] = kb < KB ? as[kb] * bs[kb] : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float4v part = mul16<kExact<OutT>>(fb[u], fa[u], (float4v){0, 0, 0, 0});
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[r] = __builtin_fmaf(part[r], f[u], acc[r]);
    }
  }
  // accumulator r of lane (l16, lq): row l16, column 4 lq + r
  *reinterpret_cast<float4v *>(&red[wave][l16][4 * lq]) = acc;
  __syncthreads();
  OutT *Cp = static_cast<OutT *>(p.c);
  if (tid < 256) {
    const uint32_t r = tid / 16, n = tid % 16;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) v += red[w][r][n];
    if (m0 + r < p.M && n0 + n < p.N) Cp[(int64_t)(m0 + r) * p.ldc + n0 + n] = to_out<OutT>(v);
  }
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float float2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));

// Swizzle of the eight 16-byte pieces of a 128-byte LDS row: piece c of row r is
// stored at c ^ swz128(r).  A 16-byte read is served 16 lanes at a time, which in
// the fragment reads are 16 consecutive rows at one piece: r % 2 gives the half
// of a 256-byte window and swz128 a different piece of it for every two rows.
__device__ __forceinline__ uint32_t swz128(uint32_t r) { return (r >> 1) & 7u; }

// Few rows or few tiles: a (32 FM) x (32 FN) tile of C per workgroup, whose NW
// waves take the 128-column blocks of K in turn, each alone: it fetches its blocks
// of A and B straight into NST stages of LDS of its own (1 KB a transfer, whole
// 128-byte lines), reads the fragments back and multiplies, without a barrier
// before the waves' sums are joined through LDS, in wave order, at the end.  The
// work is bound by how fast a compute unit takes in its (32 FM + 32 FN) K bytes,
// which the depth of the stages (not registers) keeps in flight.  The resources
// end at the matrix's last row: rows past it cost nothing.  Measured: 32 x 25600 x
// 5120 in 30 us (133 MB, 4.4 TB/s); 1 x 5120 x 5120 in 7.4 us (26 MB, 3.5 TB/s); 1000 x 1552 x 2064 float32 in 15 us.
template <int FM, int FN, int NW, int NST, typename OutT>
__global__ __launch_bounds__(NW * 64, 1) void block_gemm_strip_kernel(Fp8BlockGemmParams p) {
  using Op = Operand<kExact<OutT>>;
  constexpr int BM = 32 * FM, BN = 32 * FN;
  static_assert(128 % BN == 0, "a tile's columns lie in one scale row");
  constexpr int TA = BM / 8, TB = BN / 8, TS = (BM + 63) / 64, TN = TA + TB + TS;
  constexpr int OFF_B = BM * 128, OFF_S = OFF_B + BN * 128, STAGE = OFF_S + TS * 256;
  constexpr int RED = BN + 4;  // floats per row of a wave's sums
  constexpr int LDS = NW * NST * STAGE > NW * BM * RED * 4 ? NW * NST * STAGE : NW * BM * RED * 4;
  static_assert(LDS <= 160 * 1024 && (NST - 1) * TN < 64, "LDS, wait count");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[LDS];

  const uint32_t tid = threadIdx.x;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(tid / 64), lane = tid % 64;
  const uint32_t K = p.K, KB = (K + 127) / 128;
  const uint32_t tiles_m = (p.M + BM - 1) / BM, tiles_n = (p.N + BN - 1) / BN;
  uint32_t tm, tn;
  dense_tile(blockIdx.x, tiles_m, tiles_n, &tm, &tn);
  const uint32_t row0 = tm * BM, col0 = tn * BN;

  typedef __amdgpu_buffer_rsrc_t Rsrc;
  auto rsrc = [](const void *base, uint32_t bytes) -> Rsrc {
    return __builtin_amdgcn_make_buffer_rsrc((void *)base, (short)0, (int)bytes, 0x00020000);
  };
  const uint32_t rows_a = min(p.M - row0, (uint32_t)BM), rows_b = min(p.N - col0, (uint32_t)BN);
  const uint8_t *const ta = p.a_q + (size_t)row0 * K, *const tb = p.b_q + (size_t)col0 * K;
  const float *const ts = p.a_s + (size_t)row0 * KB;
  // transfer j of an operand: tile rows 8 j + lane / 8, physical piece lane % 8;
  // the swizzle repeats every 16 rows: two phases
  uint32_t piece[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) piece[e] = ((lane % 8) ^ swz128(8 * e + lane / 8)) * 16;
  const uint32_t first = (lane / 8) * K;
  uint8_t *ring = smem + wave * NST * STAGE;
  auto issue = [&](uint32_t buf, uint32_t kb) {
    uint8_t *st = ring + buf * STAGE;
    const int so = (int)(kb * 128);
    const uint32_t on = kb < KB ? 1u : 0u;  // past the last block: empty resources, nothing is fetched
    const Rsrc rA = rsrc(ta, on * rows_a * K), rB = rsrc(tb, on * rows_b * K), rS = rsrc(ts, on * rows_a * KB * 4);
    uint32_t v[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) v[e] = first + (kb * 128 + piece[e] < K ? piece[e] : 0u);
#pragma unroll
    for (int j = 0; j < TB; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rB, (lds_void *)(st + OFF_B + j * 1024), 16, (int)(v[j % 2] + j * 8 * K),
                                               so, 0, 0);
#pragma unroll
    for (int j = 0; j < TA; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rA, (lds_void *)(st + j * 1024), 16, (int)(v[j % 2] + j * 8 * K), so, 0,
                                               0);
#pragma unroll
    for (int j = 0; j < TS; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rS, (lds_void *)(st + OFF_S + j * 256), 4, (int)((j * 64 + lane) * KB * 4),
                                               (int)(kb * 4), 0, 0);
  };

  typedef const float __attribute__((address_space(4))) cfloat;
  cfloat *bs = (cfloat *)(uintptr_t)(p.b_s + (size_t)(col0 / 128) * KB);
  const uint32_t l32 = lane % 32, lh = lane / 32;
  uint32_t off[2][2];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int h = 0; h < 2; ++h) off[t][h] = l32 * 128 + ((4 * t + 2 * lh + h) ^ swz128(l32)) * 16;
  auto frag = [&](const uint8_t *at, int t, uint32_t left) {
    Fp8Frag f;
    f.lo = *reinterpret_cast<const u32x4 *>(at + off[t][0]);
    f.hi = *reinterpret_cast<const u32x4 *>(at + off[t][1]);
    if (left < 128) {  // uniform: the last block of a K that is no multiple of 128
      const uint32_t c = (4 * t + 2 * lh) * 16;
      if (c >= left) f.lo = (u32x4){0, 0, 0, 0};
      if (c + 16 >= left) f.hi = (u32x4){0, 0, 0, 0};
    }
    return f;
  };

  float16v acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = (float16v){};
  // the wave's blocks: wave, wave + NW, ... (past the last one transfers are still
  // counted, so that one wait count serves every turn)
#pragma unroll
  for (int st = 0; st < NST; ++st) issue(st, wave + st * NW);
  uint32_t buf = 0;
  for (uint32_t kb = wave; kb < KB; kb += NW) {
    const float sb = bs[kb];
    wait_vm<(NST - 1) * TN>();
    asm volatile("" ::: "memory");
    const uint8_t *st = ring + buf * STAGE;
    const uint32_t left = K - kb * 128;
    Fp8Frag a[FM][2], b[FN][2];
    float f[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i) f[i] = *reinterpret_cast<const float *>(st + OFF_S + (i * 32 + l32) * 4);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int i = 0; i < FM; ++i) a[i][t] = frag(st + i * 4096, t, left);
#pragma unroll
      for (int j = 0; j < FN; ++j) b[j][t] = frag(st + OFF_B + j * 4096, t, left);
    }
    wait_lgkm0();  // the stage has been read: it takes the block NST turns ahead
    asm volatile("" ::: "memory");
    issue(buf, kb + NST * NW);
    buf = buf + 1 == NST ? 0 : buf + 1;
#pragma unroll
    for (int i = 0; i < FM; ++i) f[i] *= sb;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const Op b0(b[j][0]), b1(b[j][1]);
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        float16v part = mul32(b0, Op(a[i][0]), (float16v){});
        part = mul32(b1, Op(a[i][1]), part);
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = __builtin_fmaf(part[r], f[i], acc[i][j][r]);
      }
    }
  }
  wait_vm<0>();
  __syncthreads();  // every transfer has landed: the stages become the waves' sums
  float *red = reinterpret_cast<float *>(smem);
  // accumulator 4q + e of lane (l32, lh): row l32, column 8q + 4 lh + e
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<u32x4 *>(red + (wave * BM + i * 32 + l32) * RED + j * 32 + 8 * q + 4 * lh) =
            (u32x4){f2u(acc[i][j][4 * q]), f2u(acc[i][j][4 * q + 1]), f2u(acc[i][j][4 * q + 2]),
                    f2u(acc[i][j][4 * q + 3])};
  __syncthreads();
  OutT *Cp = static_cast<OutT *>(p.c);
  for (uint32_t c = tid; c < rows_a * (BN / 4); c += NW * 64) {
    const uint32_t m = c / (BN / 4), n = c % (BN / 4) * 4;
    float4v v = *reinterpret_cast<const float4v *>(red + m * RED + n);
#pragma unroll
    for (int w = 1; w < NW; ++w) {
      const float4v o = *reinterpret_cast<const float4v *>(red + (w * BM + m) * RED + n);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += o[e];
    }
    OutT *gp = Cp + (int64_t)(row0 + m) * p.ldc + col0 + n;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < rows_b) gp[e] = to_out<OutT>(v[e]);
  }
}

// Many rows: a BM x BN tile per workgroup, NWM x NWN waves of 64 x WN each.
//  * One step is one 128-column block: its tiles of A and B (128 bytes a row) and
//    A's scales go from global memory straight into LDS (buffer loads, 1 KB a
//    transfer), NST stages, fetched NST steps ahead.  The resources end at the
//    matrix's last row, so rows past it read nothing and need no clamp.
//  * Fragments are double buffered in registers: those of step s + 1 are read
//    from LDS behind the matrix instructions of step s.  They may live in the
//    accumulation half of the register file (matrix instructions and LDS reads
//    reach it), while the sums, which the vector unit adds to, live in the other
//    (this file is compiled with -amdgpu-mfma-vgpr-form for that).
//  * The float32 join costs one FMA per output and block on the vector unit
//    beside two matrix instructions per 32 x 32 outputs: the FMAs of one column
//    fragment run under the matrix instructions of the next.
//  * The weight fragment goes first, so a lane's accumulators are runs of four
//    columns of one row: its scale is one factor, and the epilogue stages 8- or
//    16-byte pieces through LDS and stores 16 bytes a lane.
//  * K % 128 != 0: the last block's pieces past K are zeroed as they are read
//    (their transfers are pointed at the row's first piece).
// Measured: 8192 x 25600 x 5120 to bf16 in 1.22 ms (1.76 PFLOP/s; the per-tensor FP8
// GEMM, which joins nothing, 0.94), bound by the float32 joins beside the matrix
// instructions (with operands that stay in the cache 1.03); 128 x 151936 x 2048 in
// 88 us (350 MB, 4.0 TB/s).
template <int BM, int BN, int NWM, int NWN, int NST, bool VSTORE, typename OutT>
__global__ __launch_bounds__(NWM *NWN * 64, 1) void block_gemm_tile_kernel(Fp8BlockGemmParams p) {
  constexpr int NW = NWM * NWN, WM = BM / NWM, WN = BN / NWN, FM = WM / 32, FN = WN / 32;
  static_assert(WM == 64, "a wave's 64 row scales are one transfer");
  static_assert(128 % WN == 0, "a wave's columns lie in one scale row");
  constexpr int TA = BM / 8 / NW, TB = BN / 8 / NW;  // transfers of 8 rows per wave and step
  constexpr int TN = TA + TB + 1;
  constexpr int OFF_B = BM * 128, OFF_S = OFF_B + BN * 128, STAGE = OFF_S + NW * 256;
  using Op = Operand<kExact<OutT>>;
  static_assert(NST * STAGE <= 160 * 1024, "LDS");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[NST * STAGE];

  const uint32_t tid = threadIdx.x;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(tid / 64), lane = tid % 64;
  const uint32_t K = p.K, KB = (K + 127) / 128;
  const uint32_t tiles_m = (p.M + BM - 1) / BM, tiles_n = (p.N + BN - 1) / BN;
  uint32_t tm, tn;
  dense_tile(blockIdx.x, tiles_m, tiles_n, &tm, &tn);
  const uint32_t row0 = tm * BM, col0 = tn * BN;
  const uint32_t wm = wave / NWN, wn = wave % NWN;

  typedef __amdgpu_buffer_rsrc_t Rsrc;
  auto rsrc = [](const void *base, uint32_t bytes) -> Rsrc {
    return __builtin_amdgcn_make_buffer_rsrc((void *)base, (short)0, (int)bytes, 0x00020000);
  };
  const uint32_t rows_a = min(p.M - row0, (uint32_t)BM), rows_b = min(p.N - col0, (uint32_t)BN);
  const uint8_t *const ta = p.a_q + (size_t)row0 * K, *const tb = p.b_q + (size_t)col0 * K;
  const float *const ts = p.a_s + (size_t)row0 * KB;
  // transfer j of an operand: tile rows (j NW + wave) * 8 + lane / 8, physical
  // piece lane % 8 (the swizzle repeats every 16 rows: the same for every j when
  // 8 NW is a multiple of 16)
  static_assert(NW % 2 == 0, "swizzle phase");
  const uint32_t trow = wave * 8 + lane / 8;
  const uint32_t piece = ((lane % 8) ^ swz128(trow)) * 16;
  const uint32_t first = trow * K;
  const uint32_t srow = (wm * 64 + lane) * KB * 4;
  const uint32_t size_a = rows_a * K, size_b = rows_b * K, size_s = rows_a * KB * 4;
  // the transfers of block kb into stage buf; q-th of TN
  auto issue = [&](uint32_t buf, uint32_t kb, int q) {
    uint8_t *st = smem + buf * STAGE;
    const uint32_t v = first + (kb * 128 + piece < K ? piece : 0u);
    const int so = (int)(kb * 128);
    const bool on = kb < KB;  // past the last block: empty resources, nothing is fetched
    const Rsrc rA = rsrc(ta, on ? size_a : 0u), rB = rsrc(tb, on ? size_b : 0u), rS = rsrc(ts, on ? size_s : 0u);
    if (q < TA)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rA, (lds_void *)(st + (q * NW + wave) * 1024), 16,
                                               (int)(v + q * (NW * 8) * K), so, 0, 0);
    else if (q < TA + TB)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rB, (lds_void *)(st + OFF_B + ((q - TA) * NW + wave) * 1024), 16,
                                               (int)(v + (q - TA) * (NW * 8) * K), so, 0, 0);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rS, (lds_void *)(st + OFF_S + wave * 256), 4, (int)srow, (int)(kb * 4),
                                               0, 0);
  };

  const uint32_t l32 = lane % 32, lh = lane / 32;
  struct Frags {
    Fp8Frag a[FM][2], b[FN][2];
    float s[FM];
    float sb;
  };
  // pieces 4t + 2 lh + h (t: half of the block) of fragment rows; row groups of
  // 32 share a swizzle phase
  uint32_t oa[2][2], ob[2][2];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t c = ((4 * t + 2 * lh + h) ^ swz128(l32)) * 16;
      oa[t][h] = (wm * WM + l32) * 128 + c;
      ob[t][h] = OFF_B + (wn * WN + l32) * 128 + c;
    }
  // B's scales are uniform over a wave: scalar loads (constant address space),
  // outside the vector loads' count
  typedef const float __attribute__((address_space(4))) cfloat;
  cfloat *bs = (cfloat *)(uintptr_t)(p.b_s + (size_t)(min(col0 + wn * WN, p.N - 1) / 128) * KB);
  // the d-th of ND reads of a stage (at byte st of LDS) into x
  constexpr int ND = 5 * FM + 4 * FN;
  auto read = [&](uint32_t st, Frags &x, int d) {
    if (d < FM) {
      x.s[d] = *reinterpret_cast<const float *>(smem + st + OFF_S + wave * 256 + (d * 32 + l32) * 4);
      return;
    }
    d -= FM;
    const bool isA = d < 4 * FM;
    if (!isA) d -= 4 * FM;
    const int g = d / 4, t = d / 2 % 2, h = d % 2;
    Fp8Frag &f = isA ? x.a[g][t] : x.b[g][t];
    const u32x4 v = *reinterpret_cast<const u32x4 *>(smem + st + (isA ? oa[t][h] : ob[t][h]) + g * 4096);
    if (h == 0) f.lo = v;
    else f.hi = v;
  };
  // pieces past the last `left` bytes of a block
  auto cut = [&](Frags &x, uint32_t left) {
    auto one = [&](Fp8Frag &f, int t) {
      const uint32_t c = (4 * t + 2 * lh) * 16;
      if (c >= left) f.lo = (u32x4){0, 0, 0, 0};
      if (c + 16 >= left) f.hi = (u32x4){0, 0, 0, 0};
    };
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int i = 0; i < FM; ++i) one(x.a[i][t], t);
#pragma unroll
      for (int j = 0; j < FN; ++j) one(x.b[j][t], t);
    }
  };

  float16v acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  // Unit u = (column fragment u / FM, row fragment u % FM) of a block: two matrix
  // instructions.  Its FMAs run under the next unit's (the last unit's under the
  // next block's first), so they never wait for a result.
  constexpr int NU = FM * FN;
  float16v part[2];
  float pf = 0.0f;  // factor of the unit whose FMAs are due
  auto join_unit = [&](int u, const float16v &v, float f, int from, int to) {
    const int i = u % FM, j = u / FM;
#pragma unroll
    for (int r = from; r < to; ++r) acc[i][j][r] = __builtin_fmaf(v[r], f, acc[i][j][r]);
  };
  // under(u) runs behind unit u's first matrix instruction
  auto multiply = [&](const Frags &x, auto under) {
    static_assert(NU % 2 == 0, "the part buffers alternate over units and blocks");
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int i = u % FM, j = u / FM;
      part[u % 2] = mul32(Op(x.b[j][0]), Op(x.a[i][0]), (float16v){});
      __builtin_amdgcn_sched_barrier(0);
      under(u);
      join_unit((u + NU - 1) % NU, part[(u + 1) % 2], pf, 0, 6);
      __builtin_amdgcn_sched_barrier(0);
      part[u % 2] = mul32(Op(x.b[j][1]), Op(x.a[i][1]), part[u % 2]);
      __builtin_amdgcn_sched_barrier(0);
      join_unit((u + NU - 1) % NU, part[(u + 1) % 2], pf, 6, 16);
      pf = x.s[i] * x.sb;
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // Step s: its fragments are in registers; stage s + 1 has landed (own
  // transfers waited for, then the barrier for everyone's), and buffer s % NST is
  // free (its reads were waited for before the barrier): it takes block s + NST.
  // Past the end transfers fetch nothing but are still counted, so that one wait
  // count serves every step.
#pragma unroll
  for (int st = 0; st < NST; ++st)
#pragma unroll
    for (int q = 0; q < TN; ++q) issue(st, st, q);
  wait_vm<(NST - 1) * TN>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  Frags x[2];
#pragma unroll
  for (int d = 0; d < ND; ++d) read(0, x[0], d);
  x[0].sb = bs[0];
  part[1] = (float16v){};
  uint32_t cur = 0;  // s % NST
  auto step = [&](uint32_t s, auto tag) {
    constexpr int C = decltype(tag)::value;
    wait_vm<(NST - 2) * TN>();
    wait_lgkm0();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    const uint32_t nxt = cur + 1 == NST ? 0 : cur + 1;
    const uint32_t kb = s + NST;
    x[C ^ 1].sb = bs[min(s + 1, KB - 1)];
    multiply(x[C], [&](int u) {
#pragma unroll
      for (int d = 0; d < ND; ++d)
        if (d * NU / ND == u) read(nxt * STAGE, x[C ^ 1], d);
#pragma unroll
      for (int q = 0; q < TN; ++q)
        if (q * NU / TN == u) issue(cur, kb, q);
    });
    cur = nxt;
  };
  uint32_t s = 0;
  const uint32_t whole = K / 128;
  for (; s + 2 <= whole; s += 2) {
    step(s, std::integral_constant<int, 0>());
    step(s + 1, std::integral_constant<int, 1>());
  }
  wait_lgkm0();
  if (s < whole) {  // one more whole block
    step(s, std::integral_constant<int, 0>());
    wait_lgkm0();
    if (s + 1 < KB) {
      cut(x[1], K - whole * 128);
      multiply(x[1], [](int) {});
    }
  } else if (s < KB) {
    cut(x[0], K - whole * 128);
    multiply(x[0], [](int) {});
  }
  join_unit(NU - 1, part[1], pf, 0, 16);
  // every transfer has landed and every wave is past its last read: all of LDS
  // is free for the epilogue
  wait_vm<0>();
  wait_lgkm0();
  __syncthreads();

  // ---------------------------------------------------------------- epilogue
  // Accumulator 4q + e of lane (l32, lh): row l32, column 8q + 4 lh + e of the
  // fragment.  Each wave stages 32 rows x WN columns at a time in its own part of
  // LDS, 16-byte chunks of row t rotated by t / (rows per 256 bytes), then reads
  // every chunk back and writes it out 16 bytes a lane.
  constexpr int ROW_BYTES = WN * (int)sizeof(OutT);
  constexpr int CPR = ROW_BYTES / 16;
  constexpr int RW = ROW_BYTES >= 256 ? 1 : 256 / ROW_BYTES;
  static_assert(NW * 32 * ROW_BYTES <= NST * STAGE, "epilogue staging must fit");
  uint8_t *slab = smem + wave * 32 * ROW_BYTES;
  auto at = [&](uint32_t t, uint32_t c) { return t * ROW_BYTES + ((c + t / RW) % CPR) * 16; };
  OutT *Cp = static_cast<OutT *>(p.c);
  const uint32_t ccol0 = col0 + wn * WN;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
#pragma unroll
    for (int j = 0; j < FN; ++j) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float v0 = acc[i][j][4 * q], v1 = acc[i][j][4 * q + 1];
        const float v2 = acc[i][j][4 * q + 2], v3 = acc[i][j][4 * q + 3];
        if constexpr (sizeof(OutT) == 2) {
          const float2v f01 = {v0, v1}, f23 = {v2, v3};
          const u32x2 pk = {__builtin_bit_cast(uint32_t, __builtin_convertvector(f01, bf16x2v)),
                            __builtin_bit_cast(uint32_t, __builtin_convertvector(f23, bf16x2v))};
          *reinterpret_cast<u32x2 *>(slab + at(l32, 4 * j + q) + lh * 8) = pk;
        } else {
          const u32x4 fv = {f2u(v0), f2u(v1), f2u(v2), f2u(v3)};
          *reinterpret_cast<u32x4 *>(slab + at(l32, 8 * j + 2 * q + lh)) = fv;
        }
      }
    }
    // the slab is this wave's own: ordering inside the wave suffices
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    constexpr int VEC = 16 / (int)sizeof(OutT);
    constexpr int NIT = 32 * CPR / 64;
    const uint32_t rbase = row0 + wm * WM + i * 32;
    u32x4 chunk[NIT];
#pragma unroll
    for (int it = 0; it < NIT; ++it) {
      const uint32_t c = lane + it * 64;
      chunk[it] = *reinterpret_cast<const u32x4 *>(slab + at(c / CPR, c % CPR));
    }
#pragma unroll
    for (int it = 0; it < NIT; ++it) {
      const uint32_t c = lane + it * 64;
      const uint32_t row = rbase + c / CPR, col = ccol0 + (c % CPR) * VEC;
      if (row >= p.M) continue;
      OutT *gp = Cp + (int64_t)row * p.ldc + col;
      if (VSTORE && col + VEC <= p.N) {
        *reinterpret_cast<u32x4 *>(gp) = chunk[it];
      } else {
        OutT sv[VEC];
        __builtin_memcpy(sv, &chunk[it], 16);
        for (int e = 0; e < VEC; ++e)
          if (col + e < p.N) gp[e] = sv[e];
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

template <int FM, int FN, int NW, int NST, typename OutT>
hipError_t launch_strip(const Fp8BlockGemmParams &p, hipStream_t stream) {
  const uint32_t grid = ((p.M + 32 * FM - 1) / (32 * FM)) * ((p.N + 32 * FN - 1) / (32 * FN));
  block_gemm_strip_kernel<FM, FN, NW, NST, OutT><<<grid, NW * 64, 0, stream>>>(p);
  return hipGetLastError();
}

template <int BM, int BN, int NWM, int NWN, int NST, typename OutT>
hipError_t launch_tile(const Fp8BlockGemmParams &p, hipStream_t stream) {
  const bool vstore = ((uintptr_t)p.c % 16 == 0) && (p.ldc * (int64_t)sizeof(OutT)) % 16 == 0;
  const uint32_t grid = ((p.M + BM - 1) / BM) * ((p.N + BN - 1) / BN);
  if (vstore) block_gemm_tile_kernel<BM, BN, NWM, NWN, NST, true, OutT><<<grid, NWM * NWN * 64, 0, stream>>>(p);
  else block_gemm_tile_kernel<BM, BN, NWM, NWN, NST, false, OutT><<<grid, NWM * NWN * 64, 0, stream>>>(p);
  return hipGetLastError();
}

template <typename OutT>
hipError_t launch_rows(const Fp8BlockGemmParams &p, hipStream_t stream) {
  const uint64_t grid_m = ((uint64_t)p.M + 15) / 16;
  if (grid_m > 65535) return hipErrorInvalidValue;
  block_gemm_rows_kernel<8, 2, OutT><<<dim3((p.N + 15) / 16, (uint32_t)grid_m), 512, 0, stream>>>(p);
  return hipGetLastError();
}

// Which kernel, and which tile: the largest one that still gives most compute
// units a workgroup (tiles >= 0.6 of them), since a unit takes its operands in at
// a bounded rate (about 45 GB/s each) and a larger tile takes in less per output.
// Measured with K = 5120 (us, this choice first, then the neighbours it beat):
//   M x N         tile            us     others
//   1024 x 5120   128 x 256       44.5   128 x 128 56.8, 64 x 64 53
//   512 x 5120    128 x 128       26.7   128 x 256 48, 64 x 64 32.6
//   256 x 5120    64 x 128        23.0   128 x 128 30, 64 x 64 22.7
//   128 x 25600   128 x 128       47.2   128 x 256 58, 64 x 64 57
//   128 x 5120    64 x 64         14.5   128 x 128 28, 32 x 64 16.4
//   64 x 25600    64 x 128        37.2   64 x 64 42
//   64 x 5120     32 x 64         10.8   64 x 64 15.2, 32 x 32 13.3
//   32 x 25600    32 x 128        30.8   32 x 64 33.5
//   32 x 5120     32 x 32         9.5    32 x 64 11.0
//   1 x 5120      32 x 32         7.4    rows 9.0
// Up to four rows whose 32-column tiles would leave units idle go by 16 columns straight
// from memory (the rows kernel), and so does a single row while K is one turn of its
// waves (us, rows / tiles, N x K):
//   1 row:  2048 x 2048 4.0 / 5.1, 4096 x 14336 14.1 / 20.6, 1024 x 5120 5.5 / 6.8,
//           25600 x 2048 12.1 / 13.1, 151936 x 2048 51.2 / 59.2, 5120 x 25600 37.2 / 32.3
//   4 rows: 2048 x 2048 4.2 / 5.1, 4096 x 14336 13.9 / 17.4, 25600 x 2048 13.8 / 13.1
//   16:     2048 x 2048 4.9 / 5.0, 25600 x 2048 19.1 / 13.9
// A float32 result (f16 products, converted operands) skips 64 x 128: 1000 x 1552
// x 2064 takes 15.5 with 64 x 64 and 22.7 with 64 x 128.
template <typename OutT>
hipError_t launch_typed(const Fp8BlockGemmParams &p, hipStream_t stream) {
  // the tiles' resources hold up to 256 rows: 32-bit offsets
  if ((uint64_t)p.K * 256 >= (1ull << 32)) return launch_rows<OutT>(p, stream);
  const uint64_t enough = device_cu_count() * 3 / 5;
  auto fills = [&](uint64_t bm, uint64_t bn) { return ((p.M + bm - 1) / bm) * ((p.N + bn - 1) / bn) >= enough; };
  if ((p.M <= 4 && !fills(32, 32)) || (p.M == 1 && p.K <= 2048)) return launch_rows<OutT>(p, stream);
  if (p.M > 64) {
    if (fills(128, 256)) return launch_tile<128, 256, 2, 2, 3, OutT>(p, stream);
    if (fills(128, 128)) return launch_tile<128, 128, 2, 2, 3, OutT>(p, stream);
  }
  if (p.M > 32) {
    if constexpr (!kExact<OutT>)
      if (fills(64, 128)) return launch_tile<64, 128, 1, 2, 3, OutT>(p, stream);
    if (fills(64, 64)) return launch_strip<2, 2, 4, 1, OutT>(p, stream);
    if (fills(32, 64)) return launch_strip<1, 2, 8, 1, OutT>(p, stream);
  } else if (fills(32, 128)) {
    return launch_strip<1, 4, 2, 2, OutT>(p, stream);
  }
  return launch_strip<1, 1, 8, 1, OutT>(p, stream);
}

}  // namespace

hipError_t launch_fp8_block_gemm(const Fp8BlockGemmParams &p, OutType out, hipStream_t stream) {
  if (p.M == 0 || p.N == 0) return hipSuccess;
  return out == OutType::F32 ? launch_typed<float>(p, stream) : launch_typed<uint16_t>(p, stream);
}

}  // namespace nvfp4
