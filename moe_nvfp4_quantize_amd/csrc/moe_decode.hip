// moe_decode.hip -- the whole routed-expert layer for few tokens on gfx950.
//
//   ids, w = top-k of the router logits, softmax over the k selected;
//   h_j    = SiLU(Wg[e_j] x) * (Wu[e_j] x)          for each of a token's k experts
//   out    = sum_j w_j Wd[e_j] h_j
// with NVFP4 expert weights (e2m1 * e4m3 * g_e) and the activations as they are:
// with few tokens the layer is bound by reading the selected experts' weights
// (0.5625 bytes an element, once each), so 4-bit activations would save nothing
// and the two quantizations of moe_layer (and what they round away) fall out.
//
// Launches, none of which waits for another on the host:
//   1. prep: a wave per token finds its experts; a workgroup per token writes x as
//      f16 (below).
//   2. gate_up: one workgroup per (expert, 16 rows of h); its waves split the hidden
//      dimension and join through LDS; SiLU gate; h to the workspace as f16.  Where
//      experts have many tokens: 64 rows, a wave for 16, and the columns shared.
//   3. down: one workgroup per (expert, 64 RT rows of out), its products times the
//      routing weight to the workspace, and
//   4. combine: the sum over a token's experts, in slot order.
//      Up to kOwnSlots slots: instead one kernel whose workgroups own 16 rows of out,
//      their waves taking the slots in turn, joined in wave order.
// Measured (kernels alone, us): 32 tokens, 512 experts top-10, H 4096, I 1024, bf16
// (1.7 GB of weights): prep 6, gate_up 226 (5.0 TB/s; a large copy moves 5.2), down 133
// (4.2), combine 5.  4 tokens of the same layer: 5.4, 38.8 (4.7), 25.4 (3.6), 4.7.  One
// token, 128 experts top-8, H 2048, I 768: 3.1, 6.8 (2.1), own 6.9 (1.0): there
// the latency of dependent loads bounds each launch, not their bytes.
// No atomics anywhere: the same result every time.  No list of experts is built:
// a workgroup is given a slot and leaves if an earlier slot has the same expert
// (or, with more slots than experts, an expert, and leaves if no slot has it), and
// finds the tokens of its expert by comparing all slots, a few ballots.
//
// Products: f16 MFMA (16 weight rows x 16 columns x 32 of K) with float32
// accumulation.  A weight e2m1 * e4m3 is exact in f16 (as in gemm.hip) and decodes
// in eight packed instructions per eight codes; bf16, which needs the products
// formed in float32, took sixteen and 30% longer for the layer.  Activations come
// to f16 under a power of two of their own, which the result is multiplied by in
// float32: x per token, its largest value in [2^14, 2^15); h per 16 rows of a
// slot, where gate_up has it in hand, and down brings a slot's blocks to its
// largest one's power as it reads them.  What a value loses by that is below
// 2^-39 of its row's largest.  A float32 value is two f16 planes whose sum it is to
// 2^-22, each a column of its own; h is one plane (2^-11) where the output is
// rounded to bf16 (2^-8) anyway.
#include "nvfp4_common.hpp"
#include "nvfp4_format.hpp"
#include "nvfp4_kernels.hpp"
#include "moe_select.hpp"

namespace nvfp4 {

namespace {

typedef float float4v __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef _Float16 half8v __attribute__((ext_vector_type(8)));

constexpr int CH = 256;  // K elements per wave step: 64 per lane quarter

// ------------------------------------------------------------------- route

// maximum over the wave, in every lane (scalar): rows of 16 by rotations, then
// the rows by broadcasts
template <int CTRL>
__device__ __forceinline__ float dpp_max(float v) {
  const int o = __builtin_amdgcn_update_dpp((int)f2u(v), (int)f2u(v), CTRL, 0xf, 0xf, false);
  return fmaxf(v, u2f((uint32_t)o));
}
__device__ __forceinline__ float wave_max_uniform(float v) {
  v = dpp_max<0x121>(v);  // row_ror:1
  v = dpp_max<0x122>(v);
  v = dpp_max<0x124>(v);
  v = dpp_max<0x128>(v);
  v = dpp_max<0x142>(v);  // row_bcast:15
  v = dpp_max<0x143>(v);  // row_bcast:31
  return u2f((uint32_t)__builtin_amdgcn_readlane((int)f2u(v), 63));
}

// Top-k of one row by one wave: lane l holds logits l * PL .. l * PL + PL - 1, a taken
// or missing one as NaN (a maximum passes over it; a NaN logit ranks as -infinity).
// Each round takes the wave's largest: equal logits go to the lowest lane and, in
// it, to the lowest index, the lower expert id.  Lane j < k returns the j-th expert
// and its routing weight.
template <int PL>
__device__ __forceinline__ void topk_row(const float *row, uint32_t E, uint32_t k, int32_t *id, float *w) {
  const uint32_t lane = threadIdx.x % 64;
  float v[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const uint32_t e = lane * PL + i;
    v[i] = e < E ? router_logit(row[e]) : __builtin_nanf("");
  }
  float sel_v = 0.0f;
  int32_t sel_e = 0;
  for (uint32_t j = 0; j < k; ++j) {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < PL; ++i) m = fmaxf(m, v[i]);
    const float top = wave_max_uniform(m);
    // k <= E: some lane still has a logit, and a NaN equals nothing
    const uint32_t win = (uint32_t)__builtin_ctzll(__ballot(m == top));
    int32_t at = 0;
#pragma unroll
    for (int i = PL - 1; i >= 0; --i) at = v[i] == top ? i : at;
    const int32_t wi = __builtin_amdgcn_readlane(at, win);
    const int32_t gone = lane == win ? wi : -1;
#pragma unroll
    for (int i = 0; i < PL; ++i) v[i] = i == gone ? __builtin_nanf("") : v[i];
    if (lane == j) {
      sel_v = top;
      sel_e = (int32_t)(win * PL) + wi;
    }
  }
  const float top = __shfl(sel_v, 0, 64);
  const float ex = lane < k ? expf(sel_v - top) : 0.0f;
  float sum = ex;
  for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 64);
  *id = sel_e;
  *w = ex / sum;
}

__device__ __forceinline__ void topk_any(const float *row, uint32_t E, uint32_t k, int32_t *id, float *w) {
  if (E <= 128) topk_row<2>(row, E, k, id, w);
  else if (E <= 256) topk_row<4>(row, E, k, id, w);
  else if (E <= 512) topk_row<8>(row, E, k, id, w);
  else topk_row<16>(row, E, k, id, w);
}

// float32 -> P f16 planes whose sum it is
template <int P>
__device__ __forceinline__ void split(float v, _Float16 out[P]) {
  out[0] = (_Float16)v;
  if constexpr (P == 2) out[1] = (_Float16)(v - (float)out[0]);
}

// the power p with amax 2^-p in [2^14, 2^15); kNoPower where amax is 0
constexpr int32_t kNoPower = -128;
__device__ __forceinline__ int32_t power_of(float amax) {
  return amax == 0.0f ? kNoPower : max(__builtin_amdgcn_frexp_expf(amax) - 15, kNoPower + 1);
}

// The first p.topk_blocks workgroups: routing, a wave per token.  The others: a
// token's x, as P f16 planes of stride H and its power.
template <int P>
__global__ __launch_bounds__(256) void decode_prep_kernel(MoeDecodeParams p) {
  if (blockIdx.x < p.topk_blocks) {
    const uint32_t t = blockIdx.x * 4 + threadIdx.x / 64, lane = threadIdx.x % 64;
    if (t >= p.T) return;
    int32_t id;
    float w;
    topk_any(p.logits + (int64_t)t * p.E, p.E, p.k, &id, &w);
    if (lane < p.k) {
      p.ids[t * p.k + lane] = id;
      p.w[t * p.k + lane] = w;
    }
    return;
  }
  // eight elements a thread and turn (H % 16 == 0); rows up to 4096 stay in registers
  const uint32_t t = blockIdx.x - p.topk_blocks;
  auto load = [&](uint32_t h, float v[8]) {
    if constexpr (P == 1) {
      u32x4 w;
      __builtin_memcpy(&w, (const uint16_t *)p.x + (int64_t)t * p.ld_x + h, 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
      }
    } else {
      __builtin_memcpy(v, (const float *)p.x + (int64_t)t * p.ld_x + h, 32);
    }
  };
  auto largest = [](const float v[8], float m) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
    return m;
  };
  constexpr uint32_t U = 2, TURN = 256 * 8;
  const uint32_t h0 = threadIdx.x * 8;
  float v[U][8] = {};
#pragma unroll
  for (uint32_t i = 0; i < U; ++i)
    if (h0 + i * TURN < p.H) load(h0 + i * TURN, v[i]);
  float m = 0.0f;
#pragma unroll
  for (uint32_t i = 0; i < U; ++i) m = largest(v[i], m);
  for (uint32_t h = h0 + U * TURN; h < p.H; h += TURN) {
    float x[8];
    load(h, x);
    m = largest(x, m);
  }
  const int32_t e = power_of(block_max(m));
  if (threadIdx.x == 0) p.xe[t] = e;
  auto store = [&](uint32_t h, const float x[8]) {
    _Float16 o[8][P];
#pragma unroll
    for (int i = 0; i < 8; ++i) split<P>(__builtin_ldexpf(x[i], -e), o[i]);
#pragma unroll
    for (int pl = 0; pl < P; ++pl) {
      half8v w;
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = o[i][pl];
      *reinterpret_cast<half8v *>(p.xp + ((int64_t)pl * p.T + t) * p.H + h) = w;
    }
  };
#pragma unroll
  for (uint32_t i = 0; i < U; ++i)
    if (h0 + i * TURN < p.H) store(h0 + i * TURN, v[i]);
  for (uint32_t h = h0 + U * TURN; h < p.H; h += TURN) {
    float x[8];
    load(h, x);
    store(h, x);
  }
}

// ---------------------------------------------------------------- products

// 8 E2M1 codes (one dword) times their block scale -> 8 exact f16.  An E4M3 byte
// moved up by 7 bits is the f16 encoding of the scale / 256, which the code
// conversion's power of two makes up for.
__device__ __forceinline__ half8v decode8(uint32_t w, _Float16 s) {
  const half2v s2 = {s, s};
  const half2v p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 256.0f, 0) * s2;
  const half2v p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 256.0f, 1) * s2;
  const half2v p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 256.0f, 2) * s2;
  const half2v p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 256.0f, 3) * s2;
  return (half8v){p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// Swizzle of the eight 16-byte pieces of a 128-byte LDS row: piece c of row r is stored
// at c ^ swz128(r), so 16 rows read at one piece are free of conflicts (every two rows
// share a window of 256 bytes)
__device__ __forceinline__ uint32_t swz128(uint32_t r) { return (r >> 1) & 7u; }

// What a lane holds of 16 weight rows for one 256-wide step: 64 codes of its row
// and their 4 block scales.
struct Codes {
  u32x4 lo, hi;
  uint32_t s;
};

// A lane's 64 elements [k, k + 64) of its row, at whatever alignment the row has: a
// whole step (every lane in) by wide loads, the last one block by block of 16, each
// all in or all out (K % 16 == 0).
__device__ __forceinline__ Codes load_codes(const uint8_t *q, const uint8_t *s, uint32_t k, uint32_t K, bool whole) {
  Codes c;
  c.lo = c.hi = (u32x4){0, 0, 0, 0};
  c.s = 0;
  if (whole) {
    __builtin_memcpy(&c.lo, q + k / 2, 16);
    __builtin_memcpy(&c.hi, q + k / 2 + 16, 16);
    __builtin_memcpy(&c.s, s + k / 16, 4);
  } else {
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      if (k + 16 * b < K) {
        uint32_t w[2];
        __builtin_memcpy(w, q + k / 2 + 8 * b, 8);
        if (b < 2) {
          c.lo[2 * b] = w[0];
          c.lo[2 * b + 1] = w[1];
        } else {
          c.hi[2 * b - 4] = w[0];
          c.hi[2 * b - 3] = w[1];
        }
        c.s |= (uint32_t)s[k / 16 + b] << (8 * b);
      }
    }
  }
  return c;
}

// the j-th of a step's eight 16-row fragments
__device__ __forceinline__ half8v weights(const Codes &c, int j) {
  const half2v even = __builtin_bit_cast(half2v, (c.s & 0x00FF00FFu) << 7);         // blocks 0 and 2
  const half2v odd = __builtin_bit_cast(half2v, ((c.s >> 8) & 0x00FF00FFu) << 7);   // blocks 1 and 3
  const int b = j / 2;
  return decode8(j < 4 ? c.lo[j] : c.hi[j - 4], b % 2 ? odd[b / 2] : even[b / 2]);
}

// A lane's column in column tile i: its row of f16 values, and, for h, the powers
// of its blocks of 16 and the power that the sums are under so far.
struct ColumnData {
  const _Float16 *row;
  const int8_t *powers;
  int32_t top;
  bool in;
};

// A step's columns: the fragments of 256 elements from k0 and, for h, their powers.
template <int NT, bool POWERS>
struct Columns {
  half8v f[NT][8];
  uint32_t w[NT];
  __device__ __forceinline__ void load(const ColumnData (&x)[NT], uint32_t k, uint32_t K) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u32x4 v = {0, 0, 0, 0};
        if (x[i].in && k + 8 * j < K) v = *reinterpret_cast<const u32x4 *>(x[i].row + k + 8 * j);
        f[i][j] = __builtin_bit_cast(half8v, v);
      }
      if constexpr (POWERS) load_powers(x[i], i, k, K);
    }
  }
  // a row of powers is padded to 4 bytes, so the four of 64 elements are one load
  __device__ __forceinline__ void load_powers(const ColumnData &x, int i, uint32_t k, uint32_t K) {
    w[i] = x.in && k < K ? *reinterpret_cast<const uint32_t *>(x.powers + k / 16) : 0x80808080u;
  }
  // each block to the largest power met so far, the sums with it (as a running
  // maximum carries a softmax)
  template <int NM>
  __device__ __forceinline__ void align(ColumnData (&x)[NT], uint32_t k, uint32_t K, float4v (&acc)[NM][NT]) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      int32_t e[4], top = x[i].top;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        e[b] = k + 16 * b < K ? (int32_t)(int8_t)(w[i] >> (8 * b)) : kNoPower;
        top = max(top, e[b]);
      }
      top = max(top, __shfl_xor(top, 16, 64));  // the column's other quarters
      top = max(top, __shfl_xor(top, 32, 64));
#pragma unroll
      for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[m][i][r] = __builtin_ldexpf(acc[m][i][r], x[i].top - top);
      x[i].top = top;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const _Float16 h = __builtin_amdgcn_ldexph((_Float16)1.0f, e[b] - top);  // 0 below 2^-24
#pragma unroll
        for (int j = 2 * b; j < 2 * b + 2; ++j) f[i][j] *= (half8v){h, h, h, h, h, h, h, h};
      }
    }
  }
};

template <int NM, int NT, bool POWERS>
__device__ __forceinline__ void multiply(const Codes (&c)[NM], const Columns<NT, POWERS> &x, float4v (&acc)[NM][NT]) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      const half8v w = weights(c[m], j);
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[m][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w, x.f[i][j], acc[m][i], 0, 0, 0);
    }
}

// A wave's 16-row tiles of NM matrices, a step of codes at a time (q and s: matrix
// m's codes and scales, from its tile's first row on).
//  ALIGNED: fetch() starts a step's way into LDS (ring: NM kTile bytes of the wave's
//  own), take() reads it back once it has landed: a transfer takes eight rows' whole
//  128 bytes, where loads in the matrix instruction's order touch 16 rows with every
//  16 lanes, 64 line lookups for the 1 KB that 8 lines hold (the header's 32
//  tokens: 385 us with those, 354 with whole lines).
//  Otherwise fetch() loads straight into registers, at any alignment.
constexpr uint32_t kTile = 16 * 128 + 16 * 16;  // codes, then scales
template <int NM, bool ALIGNED>
struct Tiles {
  const uint8_t *q[NM], *s[NM];
  uint8_t *ring;
  uint32_t K;
  Codes next[ALIGNED ? 1 : NM];

  __device__ __forceinline__ void fetch(uint32_t k0) {
    const uint32_t lane = threadIdx.x % 64;
    if constexpr (ALIGNED) {
      const uint32_t row = lane / 8, sw = swz128(row);  // (row + 8 has the phase sw ^ 4)
#pragma unroll
      for (int m = 0; m < NM; ++m) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t piece = lane % 8 ^ (sw ^ (h ? 4u : 0u));
          if (k0 + piece * 32 < K)
            __builtin_amdgcn_global_load_lds((glb_void *)(q[m] + (uint64_t)(row + 8 * h) * (K / 2) + k0 / 2 + piece * 16),
                                             (lds_void *)(ring + m * kTile + h * 1024), 16, 0, 0);
        }
        if (k0 + lane % 4 * 64 < K)
          __builtin_amdgcn_global_load_lds((glb_void *)(s[m] + (uint64_t)(lane / 4) * (K / 16) + k0 / 16 + lane % 4 * 4),
                                           (lds_void *)(ring + m * kTile + 2048), 4, 0, 0);
      }
    } else {
      const uint32_t l16 = lane % 16, k = k0 + lane / 16 * 64;
#pragma unroll
      for (int m = 0; m < NM; ++m)
        next[m] = load_codes(q[m] + (uint64_t)l16 * (K / 2), s[m] + (uint64_t)l16 * (K / 16), k, K, k0 + CH <= K);
    }
  }
  // after a wait for the step's loads; ends when LDS has been read
  __device__ __forceinline__ void take(uint32_t k0, Codes (&c)[NM]) {
    const uint32_t lane = threadIdx.x % 64, l16 = lane % 16, lq = lane / 16;
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      if constexpr (ALIGNED) {
        const uint8_t *at = ring + m * kTile;
        c[m].lo = *reinterpret_cast<const u32x4 *>(at + l16 * 128 + (2 * lq ^ swz128(l16)) * 16);
        c[m].hi = *reinterpret_cast<const u32x4 *>(at + l16 * 128 + ((2 * lq + 1) ^ swz128(l16)) * 16);
        // past K the columns are finite, and so is any code; a scale need not be
        c[m].s = k0 + lq * 64 < K ? *reinterpret_cast<const uint32_t *>(at + 2048 + l16 * 16 + lq * 4) : 0u;
      } else {
        c[m] = next[m];
      }
    }
    wait_lgkm0();
    asm volatile("" ::: "memory");
  }
};

// acc[m] += 16 rows of matrix m x one tile of 16 columns, over the steps k0 = first,
// first + turn, ... of 256 each; the columns straight from memory.
template <int NM, bool ALIGNED, bool POWERS>
__device__ __forceinline__ void products(Tiles<NM, ALIGNED> &w, ColumnData (&x)[1], uint32_t first, uint32_t turn,
                                         float4v (&acc)[NM][1]) {
  const uint32_t lq = (threadIdx.x % 64) / 16, K = w.K;
  if (ALIGNED && first < K) w.fetch(first);
  for (uint32_t k0 = first; k0 < K; k0 += turn) {
    if constexpr (!ALIGNED) w.fetch(k0);
    Columns<1, POWERS> col;
    col.load(x, k0 + lq * 64, K);
    if constexpr (ALIGNED) {
      wait_vm<0>();  // this step's codes (and columns)
      asm volatile("" ::: "memory");
    }
    Codes c[NM];
    w.take(k0, c);
    if (ALIGNED && k0 + turn < K) w.fetch(k0 + turn);  // behind this step's products
    if constexpr (POWERS) col.align(x, k0 + lq * 64, K, acc);
    multiply(c, col, acc);
  }
}

// The same for NT tiles of columns and all four waves in step: the workgroup brings
// a step of its columns (512 bytes each) into LDS once, two columns a transfer, two
// buffers at cols (NT 16 KB), and every wave reads the fragments there, conflict free:
// piece p of column c is stored at p ^ (c % 16).  row(c): column c's values, or null
// where there is none (what LDS holds there reaches only its own column of the
// result).
template <int NM, int NT, bool ALIGNED, bool POWERS, typename Row>
__device__ __forceinline__ void products_many(Tiles<NM, ALIGNED> &w, ColumnData (&x)[NT], Row row, uint8_t *cols,
                                              float4v (&acc)[NM][NT]) {
  const uint32_t lane = threadIdx.x % 64, l16 = lane % 16, lq = lane / 16, K = w.K;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const _Float16 *from[NT * 2];
#pragma unroll
  for (int i = 0; i < NT * 2; ++i) from[i] = row((i * 4 + wave) * 2 + lane / 32);
  auto bring = [&](uint32_t buf, uint32_t k0) {
#pragma unroll
    for (int i = 0; i < NT * 2; ++i) {
      const uint32_t t = i * 4 + wave, c = t * 2 + lane / 32;
      const uint32_t piece = lane % 32 ^ c % 16;
      // a piece past K would meet zero weights: the column's first one stands in
      const uint32_t k = k0 + piece * 8 < K ? k0 + piece * 8 : 0u;
      if (from[i])
        __builtin_amdgcn_global_load_lds((glb_void *)(from[i] + k), (lds_void *)(cols + buf * NT * 8192 + t * 1024), 16, 0,
                                         0);
    }
  };
  uint32_t buf = 0;
  bring(0, 0);
  w.fetch(0);
  for (uint32_t k0 = 0; k0 < K; k0 += CH) {
    const uint32_t k = k0 + lq * 64;
    wait_vm<0>();  // this wave's part of the step
    asm volatile("" ::: "memory");
    Codes c[NM];
    w.take(k0, c);  // (and the wave's reads of the other buffer are done)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (k0 + CH < K) {
      bring(buf ^ 1, k0 + CH);
      w.fetch(k0 + CH);
    }
    Columns<NT, POWERS> col;
    const uint8_t *st = cols + buf * NT * 8192;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        col.f[i][j] = *reinterpret_cast<const half8v *>(st + (i * 16 + l16) * 512 + ((lq * 8 + j) ^ l16) * 16);
      if constexpr (POWERS) col.load_powers(x[i], i, k, K);
    }
    if constexpr (POWERS) col.align(x, k, K, acc);
    multiply(c, col, acc);
    buf ^= 1;
  }
}

__device__ __forceinline__ float silu(float z) {
  return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-z * 1.44269504088896341f));
}

// P planes per token share the 16 columns
template <int P>
constexpr uint32_t kTokens = 16 / P;

// The tokens of an expert: ranks [from, from + N) of the slots that have it, in
// slot order, into list[0 .. N) (the wave's own LDS); returns how many slots have
// it in all, and the first one.
__device__ __forceinline__ uint32_t find_tokens(const int32_t *ids, uint32_t S, int32_t e, uint32_t from, uint32_t N,
                                                uint32_t *list, uint32_t *first) {
  const uint32_t lane = threadIdx.x % 64;
  uint32_t n = 0;
  *first = S;
  for (uint32_t s0 = 0; s0 < S; s0 += 512) {
    int32_t id[8];  // in flight together
#pragma unroll
    for (int i = 0; i < 8; ++i) id[i] = s0 + i * 64 + lane < S ? ids[s0 + i * 64 + lane] : -1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (s0 + i * 64 >= S) break;
      const unsigned long long m = __ballot(id[i] == e);
      if (m == 0) continue;
      const uint32_t s = s0 + i * 64 + lane;
      if (n == 0) *first = s0 + i * 64 + (uint32_t)__builtin_ctzll(m);
      const uint32_t rank = n + (uint32_t)__popcll(m & ((1ull << lane) - 1ull));
      if (id[i] == e && rank >= from && rank < from + N) list[rank - from] = s;
      n += (uint32_t)__popcll(m);
    }
  }
  // written and read by the same wave
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  return n;
}

// A lane's column of tile i of a pass over N tokens of which cnt exist: token
// i * TP + l16 % TP, plane l16 / TP.
template <int P>
struct Column {
  uint32_t slot;
  bool in;
  __device__ __forceinline__ Column(const uint32_t *list, uint32_t i, uint32_t cnt) {
    const uint32_t l16 = threadIdx.x % 16, c = i * kTokens<P> + l16 % kTokens<P>;
    in = c < cnt;
    slot = in ? list[c] : 0u;
  }
};

// Slots up to which one kernel does down and combine.  Beyond, it reads a shared
// expert's rows once per slot and its few workgroups hold less in flight.  Whole
// layer, us, one kernel / two (k of E experts, T tokens, H 2048, I 768): 8 slots (T1
// k8) 17.1 / 18.9, 16 (T2 k8) 21.3 / 21.9, 16 (T16 k1) 20.4 / 20.9, 24 (T3 k8) 26.0 /
// 25.6, 32 (T4 k8) 31.9 / 28.6, 32 (T32 k1) 30.5 / 27.3; H 4096, I 1024: 16 37.1 / 40.3
constexpr uint32_t kOwnSlots = 16;

// Which expert a workgroup works for, and its tokens.
struct Work {
  int32_t e;
  uint32_t total;  // 0: none
  __device__ __forceinline__ Work(const MoeDecodeParams &p, uint32_t item, uint32_t N, uint32_t *list) {
    e = __builtin_amdgcn_readfirstlane(p.S <= p.E ? p.ids[item] : (int32_t)item);
    uint32_t first;
    total = find_tokens(p.ids, p.S, e, 0, N, list, &first);
    if (p.S <= p.E && first != item) total = 0;  // the same in every wave
  }
};

// the tiles of gate rows and up rows from r0 on (I % 16 == 0: a tile is whole, or past
// I, and reads the last one again)
template <bool ALIGNED>
__device__ __forceinline__ void gate_up_tiles(const MoeDecodeParams &p, int32_t e, uint32_t r0, uint8_t *ring,
                                              Tiles<2, ALIGNED> &w) {
  w.K = p.H;
  w.ring = ring;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const uint64_t row = ((uint64_t)e * 2 + m) * p.I + min(r0, p.I - 16);
    w.q[m] = p.gu_q + row * (p.H / 2);
    w.s[m] = p.gu_s + row * (p.H / 16);
  }
}

template <int RT, bool ALIGNED>
__device__ __forceinline__ void down_tiles(const MoeDecodeParams &p, int32_t e, uint32_t r0, uint8_t *ring,
                                           Tiles<RT, ALIGNED> &w) {
  w.K = p.I;
  w.ring = ring;
#pragma unroll
  for (int m = 0; m < RT; ++m) {
    const uint64_t row = (uint64_t)e * p.H + min(r0 + m * 16, p.H - 16);
    w.q[m] = p.d_q + row * (p.I / 2);
    w.s[m] = p.d_s + row * (p.I / 16);
  }
}

// PX planes of x, PH planes of h; 16 rows of h a workgroup, one tile of columns a pass
template <int PX, int PH, bool ALIGNED>
__global__ __launch_bounds__(256) void decode_gate_up_kernel(MoeDecodeParams p) {
  constexpr uint32_t N = kTokens<PX>, NW = 4;
  // the waves' steps of codes, then their sums [wave][gate, up][column][row]
  constexpr uint32_t RED = NW * 2 * 16 * 20 * 4, RING = ALIGNED ? NW * 2 * kTile : 0;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[RED > RING ? RED : RING];
  float(*red)[2][16][20] = reinterpret_cast<float(*)[2][16][20]>(smem);
  __shared__ uint32_t lists[NW][N];
  const uint32_t tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / 64), lane = tid % 64;
  const uint32_t l16 = lane % 16, lq = lane / 16;
  const uint32_t item = blockIdx.x / p.tiles_i, r0 = (blockIdx.x % p.tiles_i) * 16;
  uint32_t *list = lists[wave];
  const Work work(p, item, N, list);
  if (work.total == 0) return;
  const uint32_t I = p.I;
  Tiles<2, ALIGNED> w;
  gate_up_tiles(p, work.e, r0, smem + wave * 2 * kTile, w);
  const float g = p.gu_g[work.e];
  for (uint32_t t0 = 0; t0 < work.total; t0 += N) {
    uint32_t first;
    if (t0 > 0) find_tokens(p.ids, p.S, work.e, t0, N, list, &first);
    const uint32_t cnt = min(work.total - t0, N);
    const Column<PX> c(list, 0, cnt);
    ColumnData x[1];
    x[0].row = p.xp + ((int64_t)(l16 / N) * p.T + c.slot / p.k) * p.H;
    x[0].in = c.in;
    float4v acc[2][1] = {{{0, 0, 0, 0}}, {{0, 0, 0, 0}}};
    if (t0 > 0) __syncthreads();  // the last pass's sums have been read: LDS takes codes again
    products<2, ALIGNED, false>(w, x, wave * CH, NW * CH, acc);
    __syncthreads();  // every wave is done with its codes
#pragma unroll
    for (int m = 0; m < 2; ++m) *reinterpret_cast<float4v *>(&red[wave][m][l16][4 * lq]) = acc[m][0];
    __syncthreads();
    const uint32_t tc = tid / 16, r = tid % 16;
    if (tc < cnt) {
      float zg = 0.0f, zu = 0.0f;
#pragma unroll
      for (int pl = 0; pl < PX; ++pl)
#pragma unroll
        for (uint32_t v = 0; v < NW; ++v) {
          zg += red[v][0][pl * N + tc][r];
          zu += red[v][1][pl * N + tc][r];
        }
      const uint32_t slot = list[tc];
      const int32_t xe = p.xe[slot / p.k];
      const float h = silu(__builtin_ldexpf(zg * g, xe)) * __builtin_ldexpf(zu * g, xe);
      // the 16 rows are a row of 16 lanes: their power is one exchange away
      float top = fabsf(h);
      top = dpp_max<0x121>(top);
      top = dpp_max<0x122>(top);
      top = dpp_max<0x124>(top);
      top = dpp_max<0x128>(top);
      const int32_t he = power_of(top);
      _Float16 o[PH];
      split<PH>(__builtin_ldexpf(h, -he), o);
#pragma unroll
      for (int pl = 0; pl < PH; ++pl) p.h[((int64_t)pl * p.S + slot) * I + r0 + r] = o[pl];
      if (r == 0) p.he[(int64_t)slot * p.he_ld + r0 / 16] = (int8_t)he;
    }
  }
}

// the planes of a token side by side
template <int PH>
__device__ __forceinline__ float4v join_planes(float4v v) {
  const uint32_t lane = threadIdx.x % 64;
  float4v o = v;
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int pl = 1; pl < PH; ++pl) o[r] += __shfl(v[r], (int)(lane + pl * kTokens<PH>) & 63, 64);
  return o;
}

// Many tokens an expert: 64 rows of h a workgroup, 16 a wave, NT tiles of columns a
// pass, which the waves share.
template <int PX, int PH, int NT, bool ALIGNED>
__global__ __launch_bounds__(256) void decode_gate_up_many_kernel(MoeDecodeParams p) {
  constexpr uint32_t TP = kTokens<PX>, N = NT * TP, NW = 4;
  __shared__ __attribute__((aligned(1024))) uint8_t cols[NT * 16384];
  __shared__ __attribute__((aligned(1024))) uint8_t ring[ALIGNED ? NW * 2 * kTile : 16];
  __shared__ uint32_t lists[NW][N];
  const uint32_t tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / 64), lane = tid % 64;
  const uint32_t l16 = lane % 16, lq = lane / 16;
  const uint32_t item = blockIdx.x / p.tiles_i, r0 = (blockIdx.x % p.tiles_i) * 64 + wave * 16;
  uint32_t *list = lists[wave];
  const Work work(p, item, N, list);
  if (work.total == 0) return;
  Tiles<2, ALIGNED> w;
  gate_up_tiles(p, work.e, r0, ring + (ALIGNED ? wave * 2 * kTile : 0), w);
  const float g = p.gu_g[work.e];
  for (uint32_t t0 = 0; t0 < work.total; t0 += N) {
    uint32_t first;
    if (t0 > 0) {
      find_tokens(p.ids, p.S, work.e, t0, N, list, &first);
      __syncthreads();  // every wave is done with the last pass's columns
    }
    const uint32_t cnt = min(work.total - t0, N);
    ColumnData x[NT];
    float4v acc[2][NT];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[m][i] = (float4v){0, 0, 0, 0};
    products_many<2, NT, ALIGNED, false>(
        w, x,
        [&](uint32_t c) -> const _Float16 * {
          const uint32_t t = c / 16 * TP + c % TP;
          return t < cnt ? p.xp + ((int64_t)(c % 16 / TP) * p.T + list[t] / p.k) * p.H : nullptr;
        },
        cols, acc);
    if (r0 >= p.I) continue;  // (after the pass's barriers)
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const float4v zg = join_planes<PX>(acc[0][i]), zu = join_planes<PX>(acc[1][i]);
      const Column<PX> c(list, i, cnt);
      const int32_t xe = c.in ? p.xe[c.slot / p.k] : 0;
      float h[4], top = 0.0f;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        h[r] = silu(__builtin_ldexpf(zg[r] * g, xe)) * __builtin_ldexpf(zu[r] * g, xe);
        top = fmaxf(top, fabsf(h[r]));
      }
      // a column's 16 rows are in its four lane quarters
      top = fmaxf(top, __shfl_xor(top, 16, 64));
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      const int32_t he = power_of(top);
      if (l16 < TP && c.in) {  // plane 0 holds the sums
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          _Float16 o[PH];
          split<PH>(__builtin_ldexpf(h[r], -he), o);
#pragma unroll
          for (int pl = 0; pl < PH; ++pl) p.h[((int64_t)pl * p.S + c.slot) * p.I + r0 + 4 * lq + r] = o[pl];
        }
        if (lq == 0) p.he[(int64_t)c.slot * p.he_ld + r0 / 16] = (int8_t)he;
      }
    }
  }
}

// the sums of a column tile, times the routing weight, to y
template <int PH, int RT, int NT>
__device__ __forceinline__ void store_y(const MoeDecodeParams &p, const float4v (&acc)[RT][NT], int i, uint32_t slot,
                                        const ColumnData &h, float g, uint32_t r0) {
  const uint32_t lane = threadIdx.x % 64, l16 = lane % 16, lq = lane / 16;
  const float f = h.in ? g * p.w[slot] : 0.0f;
#pragma unroll
  for (int m = 0; m < RT; ++m) {
    float4v v = join_planes<PH>(acc[m][i]);
    if (l16 < kTokens<PH> && h.in && r0 + m * 16 < p.H) {  // plane 0
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = __builtin_ldexpf(v[r] * f, h.top);
      *reinterpret_cast<float4v *>(p.y + (int64_t)slot * p.H + r0 + m * 16 + 4 * lq) = v;
    }
  }
}

// y[slot][H] = w (Wd h), 64 RT rows of one expert: a wave per 16 RT, one tile of
// columns a pass
template <int PH, int RT, bool ALIGNED>
__global__ __launch_bounds__(256) void decode_down_kernel(MoeDecodeParams p) {
  constexpr uint32_t N = kTokens<PH>, NW = 4;
  __shared__ __attribute__((aligned(1024))) uint8_t ring[ALIGNED ? NW * RT * kTile : 16];
  __shared__ uint32_t lists[NW][N];
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), l16 = threadIdx.x % 16;
  const uint32_t item = blockIdx.x / p.tiles_h, r0 = (blockIdx.x % p.tiles_h) * (64 * RT) + wave * (16 * RT);
  if (r0 >= p.H) return;  // no barriers below
  uint32_t *list = lists[wave];
  const Work work(p, item, N, list);
  if (work.total == 0) return;
  Tiles<RT, ALIGNED> w;
  down_tiles<RT>(p, work.e, r0, ring + (ALIGNED ? wave * RT * kTile : 0), w);
  const float g = p.d_g[work.e];
  for (uint32_t t0 = 0; t0 < work.total; t0 += N) {
    uint32_t first;
    if (t0 > 0) find_tokens(p.ids, p.S, work.e, t0, N, list, &first);
    const Column<PH> c(list, 0, min(work.total - t0, N));
    ColumnData h[1];
    h[0].row = p.h + ((int64_t)(l16 / N) * p.S + c.slot) * p.I;
    h[0].powers = p.he + (int64_t)c.slot * p.he_ld;
    h[0].in = c.in;
    h[0].top = kNoPower;
    float4v acc[RT][1];
#pragma unroll
    for (int m = 0; m < RT; ++m) acc[m][0] = (float4v){0, 0, 0, 0};
    products<RT, ALIGNED, true>(w, h, 0, CH, acc);
    store_y<PH>(p, acc, 0, c.slot, h[0], g, r0);
  }
}

template <int PH, int NT, int RT, bool ALIGNED>
__global__ __launch_bounds__(256) void decode_down_many_kernel(MoeDecodeParams p) {
  constexpr uint32_t TP = kTokens<PH>, N = NT * TP, NW = 4;
  __shared__ __attribute__((aligned(1024))) uint8_t cols[NT * 16384];
  __shared__ __attribute__((aligned(1024))) uint8_t ring[ALIGNED ? NW * RT * kTile : 16];
  __shared__ uint32_t lists[NW][N];
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const uint32_t item = blockIdx.x / p.tiles_h, r0 = (blockIdx.x % p.tiles_h) * (64 * RT) + wave * (16 * RT);
  uint32_t *list = lists[wave];
  const Work work(p, item, N, list);
  if (work.total == 0) return;
  Tiles<RT, ALIGNED> w;
  down_tiles<RT>(p, work.e, r0, ring + (ALIGNED ? wave * RT * kTile : 0), w);
  const float g = p.d_g[work.e];
  for (uint32_t t0 = 0; t0 < work.total; t0 += N) {
    uint32_t first;
    if (t0 > 0) {
      find_tokens(p.ids, p.S, work.e, t0, N, list, &first);
      __syncthreads();  // every wave is done with the last pass's columns
    }
    const uint32_t cnt = min(work.total - t0, N);
    ColumnData h[NT];
    uint32_t slot[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const Column<PH> c(list, i, cnt);
      slot[i] = c.slot;
      h[i].powers = p.he + (int64_t)c.slot * p.he_ld;
      h[i].in = c.in;
      h[i].top = kNoPower;
    }
    float4v acc[RT][NT];
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[m][i] = (float4v){0, 0, 0, 0};
    products_many<RT, NT, ALIGNED, true>(
        w, h,
        [&](uint32_t c) -> const _Float16 * {
          const uint32_t t = c / 16 * TP + c % TP;
          return t < cnt ? p.h + ((int64_t)(c % 16 / TP) * p.S + list[t]) * p.I : nullptr;
        },
        cols, acc);
#pragma unroll
    for (int i = 0; i < NT; ++i) store_y<PH>(p, acc, i, slot[i], h[i], g, r0);
  }
}

// out[t] = the sum of its slots' rows, in slot order; H % 16 == 0: four columns a thread
template <typename OutT>
__global__ __launch_bounds__(64) void decode_combine_kernel(MoeDecodeParams p) {
  const uint32_t h = (blockIdx.x * 64 + threadIdx.x) * 4, t = blockIdx.y;
  if (h >= p.H) return;
  const float *y = p.y + (int64_t)t * p.k * p.H + h;
  float4v v = {0, 0, 0, 0};
#pragma unroll 8
  for (uint32_t j = 0; j < p.k; ++j) {
    const float4v o = *reinterpret_cast<const float4v *>(y + (int64_t)j * p.H);
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] += o[r];
  }
  OutT *out = static_cast<OutT *>(p.out) + (int64_t)t * p.ld_out + h;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if constexpr (sizeof(OutT) == 4) out[r] = v[r];
    else out[r] = (OutT)float_to_bf16_bits(v[r]);
  }
}

// Few slots: down and combine in one kernel.  A workgroup owns 16 rows of out; its
// waves take (slot, part of K) in turn, a slot's column (or planes) alone in the
// products, and add to sums of their own in LDS.
template <int PH, bool ALIGNED, typename OutT>
__global__ __launch_bounds__(1024) void decode_own_kernel(MoeDecodeParams p) {
  constexpr uint32_t NW = 16, TP = kTokens<PH>;
  __shared__ __attribute__((aligned(16))) float sum[NW][kOwnSlots][16];
  __shared__ __attribute__((aligned(1024))) uint8_t ring[ALIGNED ? NW * kTile : 16];
  const uint32_t tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / 64), lane = tid % 64;
  const uint32_t l16 = lane % 16, lq = lane / 16;
  const uint32_t r0 = blockIdx.x * 16, K = p.I;
  if (tid < p.T * 16)
#pragma unroll
    for (uint32_t w = 0; w < NW; ++w) sum[w][tid / 16][tid % 16] = 0.0f;
  __syncthreads();
  // parts of K: as many as leave every wave something to do, at most one a step
  const uint32_t steps = (K + CH - 1) / CH;
  const uint32_t parts = min(max(NW / p.S, 1u), steps);
  for (uint32_t unit = wave; unit < p.S * parts; unit += NW) {
    const uint32_t slot = unit / parts, part = unit % parts;
    const int32_t e = p.ids[slot];
    Tiles<1, ALIGNED> w;
    down_tiles<1>(p, e, r0, ring + (ALIGNED ? wave * kTile : 0), w);
    const float fac = p.d_g[e] * p.w[slot];
    ColumnData h[1];
    h[0].in = l16 % TP == 0;  // a column for each plane
    h[0].row = p.h + ((int64_t)(l16 / TP) * p.S + slot) * K;
    h[0].powers = p.he + (int64_t)slot * p.he_ld;
    h[0].top = kNoPower;
    float4v a[1][1] = {{{0, 0, 0, 0}}};
    products<1, ALIGNED, true>(w, h, part * CH, parts * CH, a);
    const float4v acc = join_planes<PH>(a[0][0]);
    if (l16 == 0) {
      float4v *at = reinterpret_cast<float4v *>(&sum[wave][slot / p.k][4 * lq]);
      float4v v = *at;
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] += __builtin_ldexpf(acc[r] * fac, h[0].top);
      *at = v;
    }
  }
  __syncthreads();
  if (tid < p.T * 16) {
    const uint32_t t = tid / 16, r = tid % 16;
    float v = 0.0f;
#pragma unroll
    for (uint32_t w = 0; w < NW; ++w) v += sum[w][t][r];
    OutT *out = static_cast<OutT *>(p.out) + (int64_t)t * p.ld_out + r0 + r;
    if constexpr (sizeof(OutT) == 4) *out = v;
    else *out = (OutT)float_to_bf16_bits(v);
  }
}

// Column tiles a pass, from the tokens an expert has on average: 1 (the columns
// straight from memory), or 2 or 4 (through LDS, shared).  One more pass reads the
// weights again, one tile too many costs registers and LDS.  Whole layer, us, with
// 1 / 2 / 4 tiles (H 2048, I 768, 16 experts, bf16: 16 tokens a tile; a token's slots
// spread unevenly, so a mean of half a tile fills one):
//   tokens an expert 4: 24.0 / 30.6 / 40.8    8: 26.2 / 30.7 / 40.5
//   12: 33.2 / 31.5 / 41.7   16: 40.2 / 32.6 / 42.5   32: 59.9 / 52.0 / 46.1
// float32 (8 tokens a tile), H 4096, I 1024: 4: 52.0 / 57.5 / 82.0
//   8: 79 / 60.2 / 85.5   16: 130 / 95.1 / 91.9
template <int P>
int column_tiles(const MoeDecodeParams &p) {
  const uint32_t mean = p.S / min(p.S, p.E);
  return mean * 2 <= kTokens<P> ? 1 : mean <= kTokens<P> ? 2 : 4;
}

template <int PX, int PH, bool ALIGNED>
void launch_gate_up(MoeDecodeParams p, hipStream_t stream) {
  const int nt = column_tiles<PX>(p);
  p.tiles_i = nt == 1 ? p.I / 16 : (p.I + 63) / 64;
  const uint32_t grid = p.tiles_i * min(p.S, p.E);
  if (nt == 1) decode_gate_up_kernel<PX, PH, ALIGNED><<<grid, 256, 0, stream>>>(p);
  else if (nt == 2) decode_gate_up_many_kernel<PX, PH, 2, ALIGNED><<<grid, 256, 0, stream>>>(p);
  else decode_gate_up_many_kernel<PX, PH, 4, ALIGNED><<<grid, 256, 0, stream>>>(p);
}

template <int PH, int RT, bool ALIGNED>
void launch_down_rt(MoeDecodeParams p, hipStream_t stream) {
  p.tiles_h = (p.H + 64 * RT - 1) / (64 * RT);
  const uint32_t grid = p.tiles_h * min(p.S, p.E);
  const int nt = column_tiles<PH>(p);
  if (nt == 1) decode_down_kernel<PH, RT, ALIGNED><<<grid, 256, 0, stream>>>(p);
  else if (nt == 2) decode_down_many_kernel<PH, 2, RT, ALIGNED><<<grid, 256, 0, stream>>>(p);
  else decode_down_many_kernel<PH, 4, RT, ALIGNED><<<grid, 256, 0, stream>>>(p);
}

template <int PH, bool ALIGNED, typename OutT>
hipError_t launch_down(const MoeDecodeParams &p, hipStream_t stream) {
  if (p.S <= kOwnSlots) {
    decode_own_kernel<PH, ALIGNED, OutT><<<p.H / 16, 1024, 0, stream>>>(p);
    return hipGetLastError();
  }
  // Two row tiles a wave keep twice the bytes in flight and read the columns half as
  // often; one while that leaves a compute unit fewer than three workgroups of 64 rows.
  // Whole layer, us, one / two (T x E x k x H x I, workgroups of one tile):
  //   128x8x2x2048x768      256   35.7 / 37.8
  //   40x4x4x4096x1024      256   51.0 / 53.8
  //   64x16x4x2048x768      512   33.0 / 33.5     128x16x4x2048x768  512  46.0 / 40.5
  //   3x64x8x2048x768       768   26.4 / 26.7     37x24x5x2064x784   768  49.2 / 46.0
  //   64x32x4x2048x768     1024   40.0 / 37.8
  //   8x64x8x2048x768      2048   40.9 / 39.3
  //   32x512x10x4096x1024 15300    386 / 358
  if ((uint64_t)(p.H / 64) * min(p.S, p.E) >= 3 * device_cu_count()) launch_down_rt<PH, 2, ALIGNED>(p, stream);
  else launch_down_rt<PH, 1, ALIGNED>(p, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  decode_combine_kernel<OutT><<<dim3((p.H + 255) / 256, p.T), 64, 0, stream>>>(p);
  return hipGetLastError();
}

template <int PX, int PH, typename OutT>
hipError_t launch_products(const MoeDecodeParams &p, bool gu_aligned, bool d_aligned, hipStream_t stream) {
  if (gu_aligned) launch_gate_up<PX, PH, true>(p, stream);
  else launch_gate_up<PX, PH, false>(p, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return d_aligned ? launch_down<PH, true, OutT>(p, stream) : launch_down<PH, false, OutT>(p, stream);
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

// the workspace's parts, in order, from its base
struct DecodeParts {
  size_t ids, w, xe, xp, h, he, y, total;
  int64_t he_ld;
  DecodeParts(size_t T, size_t k, size_t H, size_t I) {
    const size_t S = T * k;
    size_t at = 0;
    auto take = [&](size_t bytes) {
      const size_t r = at;
      at += align256(bytes);
      return r;
    };
    he_ld = (int64_t)((I / 16 + 3) / 4 * 4);
    ids = take(S * 4);
    w = take(S * 4);
    xe = take(T * 4);
    xp = take(2 * T * H * 2);
    h = take(2 * S * I * 2);
    he = take(S * (size_t)he_ld);
    y = take(S * H * 4);
    total = at;
  }
};

}  // namespace

size_t moe_decode_workspace_bytes(int64_t T, int32_t /*E*/, int32_t k, int64_t H, int64_t I) {
  return DecodeParts((size_t)T, (size_t)k, (size_t)H, (size_t)I).total;
}

hipError_t launch_moe_decode(MoeDecodeParams p, bool x_bf16, bool gu_aligned, bool d_aligned, bool out_bf16,
                             void *workspace, hipStream_t stream) {
  if (p.T == 0) return hipSuccess;
  p.S = p.T * p.k;
  uint8_t *const ws = static_cast<uint8_t *>(workspace);
  const DecodeParts at(p.T, p.k, p.H, p.I);
  p.ids = reinterpret_cast<int32_t *>(ws + at.ids);
  p.w = reinterpret_cast<float *>(ws + at.w);
  p.xe = reinterpret_cast<int32_t *>(ws + at.xe);
  p.xp = reinterpret_cast<_Float16 *>(ws + at.xp);
  p.h = reinterpret_cast<_Float16 *>(ws + at.h);
  p.he = reinterpret_cast<int8_t *>(ws + at.he);
  p.y = reinterpret_cast<float *>(ws + at.y);
  p.he_ld = at.he_ld;
  p.topk_blocks = (p.T + 3) / 4;
  if (x_bf16) decode_prep_kernel<1><<<p.topk_blocks + p.T, 256, 0, stream>>>(p);
  else decode_prep_kernel<2><<<p.topk_blocks + p.T, 256, 0, stream>>>(p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (x_bf16)
    return out_bf16 ? launch_products<1, 1, uint16_t>(p, gu_aligned, d_aligned, stream)
                    : launch_products<1, 2, float>(p, gu_aligned, d_aligned, stream);
  return out_bf16 ? launch_products<2, 1, uint16_t>(p, gu_aligned, d_aligned, stream)
                  : launch_products<2, 2, float>(p, gu_aligned, d_aligned, stream);
}

}  // namespace nvfp4
