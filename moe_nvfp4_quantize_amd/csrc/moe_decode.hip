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
//   1. prep (more than kFuseT tokens, or x to be split): a wave per token finds its
//      experts; x is split into planes (below) where the products need it.
//   2. gate_up: one workgroup per (expert, 16 rows of h); its waves split the hidden
//      dimension and join through LDS; SiLU gate; h to the workspace.  With up to
//      kFuseT tokens every workgroup finds the tokens' experts itself.
//   3. down: one workgroup per (expert, 64 rows of out), its products times the
//      routing weight to the workspace, and
//   4. combine: the sum over a token's experts, in slot order.
//      Up to kOwnSlots slots: instead one kernel whose workgroups own 16 rows of out,
//      their waves taking the slots in turn, joined in wave order.
// No atomics anywhere: the same result every time.  No list of experts is built:
// a workgroup is given a slot and leaves if an earlier slot has the same expert
// (or, with more slots than experts, an expert, and leaves if no slot has it), and
// finds the tokens of its expert by comparing all slots, a few ballots.
//
// Products: bf16 MFMA (16 weight rows x 16 columns x 32 of K) with float32
// accumulation.  A weight e2m1 * e4m3 has at most 6 significant bits, so it is
// exact in bf16.  A float32 operand is split into bf16 planes whose sum it is
// (three planes: exactly; two: to 2^-18), each plane a column of its own: with
// few tokens an expert's columns are mostly free, so the planes cost no further
// matrix instruction.  Three planes are used for float32 results, two planes of h
// where the output is rounded to bf16 (2^-9) anyway.
#include "nvfp4_common.hpp"
#include "nvfp4_format.hpp"
#include "nvfp4_kernels.hpp"
#include "moe_select.hpp"

namespace nvfp4 {

namespace {

typedef float float2v __attribute__((ext_vector_type(2)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

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

// Top-k of one row by one wave: lane l holds logits l * PL .. l * PL + PL - 1, sorted
// (stable, so equal logits keep the lower id first); each round the wave's largest
// head wins, equal heads going to the lowest lane, and that lane drops it.  Lane
// j < k returns the j-th expert and its routing weight.
template <int PL>
__device__ __forceinline__ void topk_row(const float *row, uint32_t E, uint32_t k, int32_t *id, float *w) {
  const uint32_t lane = threadIdx.x % 64;
  float v[PL];
  int32_t x[PL];  // index inside the lane; 64: no logit (sorted last, never taken: k <= E)
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const uint32_t e = lane * PL + i;
    v[i] = e < E ? router_logit(row[e]) : -INFINITY;
    x[i] = e < E ? i : 64;
  }
  // odd-even transposition: neighbours only, so equal logits never pass each other
#pragma unroll
  for (int r = 0; r < PL; ++r)
#pragma unroll
    for (int i = r % 2; i + 1 < PL; i += 2) {
      const bool sw = topk_before(v[i + 1], x[i + 1], v[i], x[i]);
      const float a = v[i], b = v[i + 1];
      const int32_t c = x[i], d = x[i + 1];
      v[i] = sw ? b : a;
      v[i + 1] = sw ? a : b;
      x[i] = sw ? d : c;
      x[i + 1] = sw ? c : d;
    }
  float sel_v = 0.0f;
  int32_t sel_e = 0;
  for (uint32_t j = 0; j < k; ++j) {
    const float top = wave_max_uniform(v[0]);
    const unsigned long long at = __ballot(x[0] < 64 && v[0] == top);
    const uint32_t win = (uint32_t)__builtin_ctzll(at);
    const int32_t wi = __builtin_amdgcn_readlane(x[0], win);
    if (lane == win) {
#pragma unroll
      for (int i = 0; i + 1 < PL; ++i) {
        v[i] = v[i + 1];
        x[i] = x[i + 1];
      }
      v[PL - 1] = -INFINITY;
      x[PL - 1] = 64;
    }
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

// float32 -> P bf16 planes whose sum it is: each plane but the last of two is
// cut (not rounded), so that what remains is exact
template <int P>
__device__ __forceinline__ void split(float v, uint16_t out[P]) {
  if constexpr (P == 1) {
    out[0] = (uint16_t)float_to_bf16_bits(v);
  } else if constexpr (P == 2) {
    out[0] = (uint16_t)float_to_bf16_bits(v);
    out[1] = (uint16_t)float_to_bf16_bits(v - u2f((uint32_t)out[0] << 16));
  } else {
    const float a = u2f(f2u(v) & 0xFFFF0000u), r = v - a;
    const float b = u2f(f2u(r) & 0xFFFF0000u), c = r - b;
    out[0] = (uint16_t)(f2u(a) >> 16);
    out[1] = (uint16_t)(f2u(b) >> 16);
    out[2] = (uint16_t)(f2u(c) >> 16);
  }
}

// The first p.topk_blocks workgroups: routing, a wave per token.  The others: x into
// bf16 planes of stride H, 256 elements each: float32 x (P = 3) or bf16 x whose rows
// are not 16-byte aligned (P = 1).
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
  const uint32_t b = blockIdx.x - p.topk_blocks, per = (p.H + 255) / 256;
  const uint32_t t = b / per, h = (b % per) * 256 + threadIdx.x;
  if (h >= p.H) return;
  uint16_t o[P];
  if constexpr (P == 1) o[0] = ((const uint16_t *)p.x)[(int64_t)t * p.ld_x + h];
  else split<P>(((const float *)p.x)[(int64_t)t * p.ld_x + h], o);
#pragma unroll
  for (int i = 0; i < P; ++i) p.xp[((int64_t)i * p.T + t) * p.H + h] = o[i];
}

// ---------------------------------------------------------------- products

// 8 E2M1 codes (one dword) times the block scale s -> 8 exact bf16: converted to
// float32 in pairs, multiplied (exact: 6 significant bits), and the high halves
// packed
__device__ __forceinline__ bf16x8 decode8(uint32_t w, float s) {
  uint32_t o[4];
  auto pair = [&](float2v v) {
    return __builtin_amdgcn_perm(f2u(v[1] * s), f2u(v[0] * s), 0x07060302u);
  };
  o[0] = pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0));
  o[1] = pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1));
  o[2] = pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2));
  o[3] = pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3));
  return __builtin_bit_cast(bf16x8, (u32x4){o[0], o[1], o[2], o[3]});
}

// What a lane holds of 16 weight rows for one 256-wide step: 64 codes of its row
// and their 4 block scales.
struct Codes {
  u32x4 lo, hi;
  uint32_t s;
};

// A lane's 64 elements [k, k + 64) of its row.
//  ALIGNED (K % 64 == 0, 16-byte aligned codes, 4-byte aligned scales): all in or
//  all out.  Otherwise a whole step (all lanes in) takes the same loads at whatever
//  alignment the row has, and the last step goes block by block of 16, each all in
//  or all out (K % 16 == 0).
template <bool ALIGNED>
__device__ __forceinline__ Codes load_codes(const uint8_t *q, const uint8_t *s, uint32_t k, uint32_t K, bool whole) {
  Codes c;
  c.lo = c.hi = (u32x4){0, 0, 0, 0};
  c.s = 0;
  if constexpr (ALIGNED) {
    if (k < K) {
      c.lo = *reinterpret_cast<const u32x4 *>(q + k / 2);
      c.hi = *reinterpret_cast<const u32x4 *>(q + k / 2 + 16);
      c.s = *reinterpret_cast<const uint32_t *>(s + k / 16);
    }
  } else if (whole) {
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

// a lane's column: elements [k + 8j, k + 8j + 8) of one bf16 row
__device__ __forceinline__ bf16x8 load_column(const uint16_t *x, bool in, uint32_t k, uint32_t K, int j) {
  u32x4 v = {0, 0, 0, 0};
  if (in && k + 8 * j < K) v = *reinterpret_cast<const u32x4 *>(x + k + 8 * j);
  return __builtin_bit_cast(bf16x8, v);
}

template <int J>
__device__ __forceinline__ float scale_at(uint32_t s) { return __builtin_amdgcn_cvt_f32_fp8((int)s, J); }

// the j-th of a step's eight 16-row fragments
__device__ __forceinline__ bf16x8 weights(const Codes &c, int j) {
  const uint32_t w = j < 4 ? c.lo[j] : c.hi[j - 4];
  const float s = j < 2 ? scale_at<0>(c.s) : j < 4 ? scale_at<1>(c.s) : j < 6 ? scale_at<2>(c.s) : scale_at<3>(c.s);
  return decode8(w, s);
}

__device__ __forceinline__ float silu(float z) {
  return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-z * 1.44269504088896341f));
}

// P bf16 planes per token share the 16 columns: 16, 8 or 5 tokens at a time
template <int P>
constexpr uint32_t kTokens = P == 1 ? 16 : P == 2 ? 8 : 5;

// The tokens of an expert: ranks [from, from + N) of the slots that have it, in
// slot order, into list[0 .. N) (the wave's own LDS); returns how many slots have
// it in all, and the first one.
__device__ __forceinline__ uint32_t find_tokens(const int32_t *ids, uint32_t S, int32_t e, uint32_t from, uint32_t N,
                                                uint32_t *list, uint32_t *first) {
  const uint32_t lane = threadIdx.x % 64;
  uint32_t n = 0;
  *first = S;
  for (uint32_t s0 = 0; s0 < S; s0 += 64) {
    const uint32_t s = s0 + lane;
    const bool mine = s < S && ids[s] == e;
    const unsigned long long m = __ballot(mine);
    if (m == 0) continue;
    if (n == 0) *first = s0 + (uint32_t)__builtin_ctzll(m);
    const uint32_t rank = n + (uint32_t)__popcll(m & ((1ull << lane) - 1ull));
    if (mine && rank >= from && rank < from + N) list[rank - from] = s;
    n += (uint32_t)__popcll(m);
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
    in = l16 / kTokens<P> < (uint32_t)P && c < cnt;
    slot = in ? list[c] : 0u;
  }
};

constexpr uint32_t kFuseT = 4;    // tokens up to which gate_up routes by itself
constexpr uint32_t kOwnSlots = 16;  // slots up to which one kernel does down and combine

// PX planes of x, PH planes of h, NT tiles of 16 columns a pass
template <int PX, int PH, int NT, bool ALIGNED, bool FUSE>
__global__ __launch_bounds__(256) void decode_gate_up_kernel(MoeDecodeParams p) {
  constexpr uint32_t TP = kTokens<PX>, N = NT * TP, NW = 4;
  __shared__ __attribute__((aligned(16))) float red[NW][2][NT * 16][20];  // [wave][gate, up][column][row]
  __shared__ uint32_t lists[NW][N];
  __shared__ int32_t own_ids[FUSE ? kFuseT * 32 : 1];
  const uint32_t tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / 64), lane = tid % 64;
  const uint32_t l16 = lane % 16, lq = lane / 16;
  const uint32_t item = blockIdx.x / p.tiles_i, r0 = (blockIdx.x % p.tiles_i) * 16;
  const int32_t *ids = p.ids;
  if constexpr (FUSE) {
    if (wave < p.T) {
      int32_t id;
      float w;
      topk_any(p.logits + (int64_t)wave * p.E, p.E, p.k, &id, &w);
      if (lane < p.k) {
        own_ids[wave * p.k + lane] = id;
        if (blockIdx.x == 0) {  // for the kernels behind this one
          p.ids[wave * p.k + lane] = id;
          p.w[wave * p.k + lane] = w;
        }
      }
    }
    __syncthreads();
    ids = own_ids;
  }
  const int32_t e = __builtin_amdgcn_readfirstlane(p.S <= p.E ? ids[item] : (int32_t)item);
  uint32_t *list = lists[wave];
  uint32_t first;
  const uint32_t total = find_tokens(ids, p.S, e, 0, N, list, &first);
  if (total == 0 || (p.S <= p.E && first != item)) return;  // the same in every wave
  const uint32_t K = p.H, I = p.I;
  const uint64_t row = (uint64_t)e * 2 * I + r0 + l16;  // I % 16 == 0: whole row tiles
  const uint8_t *gq = p.gu_q + row * (K / 2), *gs = p.gu_s + row * (K / 16);
  const uint8_t *uq = gq + (uint64_t)I * (K / 2), *us = gs + (uint64_t)I * (K / 16);
  const float g = p.gu_g[e];
  for (uint32_t t0 = 0; t0 < total; t0 += N) {
    if (t0 > 0) find_tokens(ids, p.S, e, t0, N, list, &first);
    const uint32_t cnt = min(total - t0, N);
    const uint16_t *x[NT];
    bool in[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const Column<PX> c(list, i, cnt);
      in[i] = c.in;
      x[i] = p.xs + (int64_t)(l16 / TP) * p.x_plane + (int64_t)(c.slot / p.k) * p.x_ld;
    }
    float4v ag[NT], au[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) ag[i] = au[i] = (float4v){0, 0, 0, 0};
    for (uint32_t k0 = wave * CH; k0 < K; k0 += NW * CH) {
      const uint32_t k = k0 + lq * 64;
      const bool whole = k0 + CH <= K;
      const Codes cg = load_codes<ALIGNED>(gq, gs, k, K, whole), cu = load_codes<ALIGNED>(uq, us, k, K, whole);
      bf16x8 f[NT][8];
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) f[i][j] = load_column(x[i], in[i], k, K, j);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bf16x8 wg = weights(cg, j), wu = weights(cu, j);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          ag[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wg, f[i][j], ag[i], 0, 0, 0);
          au[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wu, f[i][j], au[i], 0, 0, 0);
        }
      }
    }
    __syncthreads();  // the last pass's sums have been read
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      *reinterpret_cast<float4v *>(&red[wave][0][i * 16 + l16][4 * lq]) = ag[i];
      *reinterpret_cast<float4v *>(&red[wave][1][i * 16 + l16][4 * lq]) = au[i];
    }
    __syncthreads();
    for (uint32_t c = tid / 16; c < cnt; c += 16) {
      const uint32_t r = tid % 16;
      float zg = 0.0f, zu = 0.0f;
#pragma unroll
      for (int pl = 0; pl < PX; ++pl)
#pragma unroll
        for (uint32_t w = 0; w < NW; ++w) {
          const uint32_t col = c / TP * 16 + pl * TP + c % TP;
          zg += red[w][0][col][r];
          zu += red[w][1][col][r];
        }
      uint16_t o[PH];
      split<PH>(silu(zg * g) * (zu * g), o);
#pragma unroll
      for (int pl = 0; pl < PH; ++pl) p.h[((int64_t)pl * p.S + list[c]) * I + r0 + r] = o[pl];
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

// y[slot][H] = w (Wd h), 64 rows of one expert: a wave per 16
template <int PH, int NT, bool ALIGNED>
__global__ __launch_bounds__(256) void decode_down_kernel(MoeDecodeParams p) {
  constexpr uint32_t TP = kTokens<PH>, N = NT * TP, NW = 4;
  __shared__ uint32_t lists[NW][N];
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
  const uint32_t l16 = lane % 16, lq = lane / 16;
  const uint32_t item = blockIdx.x / p.tiles_h, r0 = (blockIdx.x % p.tiles_h) * 64 + wave * 16;
  const uint32_t K = p.I, H = p.H;
  if (r0 >= H) return;  // H % 16 == 0: a wave's rows are all in or all out; no barriers below
  const int32_t e = __builtin_amdgcn_readfirstlane(p.S <= p.E ? p.ids[item] : (int32_t)item);
  uint32_t *list = lists[wave];
  uint32_t first;
  const uint32_t total = find_tokens(p.ids, p.S, e, 0, N, list, &first);
  if (total == 0 || (p.S <= p.E && first != item)) return;
  const uint64_t row = (uint64_t)e * H + r0 + l16;
  const uint8_t *dq = p.d_q + row * (K / 2), *ds = p.d_s + row * (K / 16);
  const float g = p.d_g[e];
  for (uint32_t t0 = 0; t0 < total; t0 += N) {
    if (t0 > 0) find_tokens(p.ids, p.S, e, t0, N, list, &first);
    const uint32_t cnt = min(total - t0, N);
    const uint16_t *h[NT];
    bool in[NT];
    uint32_t slot[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const Column<PH> c(list, i, cnt);
      in[i] = c.in;
      slot[i] = c.slot;
      h[i] = p.h + ((int64_t)(l16 / TP) * p.S + c.slot) * K;
    }
    float4v acc[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i] = (float4v){0, 0, 0, 0};
    for (uint32_t k0 = 0; k0 < K; k0 += CH) {
      const uint32_t k = k0 + lq * 64;
      const Codes cd = load_codes<ALIGNED>(dq, ds, k, K, k0 + CH <= K);
      bf16x8 f[NT][8];
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) f[i][j] = load_column(h[i], in[i], k, K, j);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bf16x8 w = weights(cd, j);
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, f[i][j], acc[i], 0, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      float4v v = join_planes<PH>(acc[i]);
      if (l16 < TP && in[i]) {  // plane 0
        const float f = g * p.w[slot[i]];
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] *= f;
        *reinterpret_cast<float4v *>(p.y + (int64_t)slot[i] * H + r0 + 4 * lq) = v;
      }
    }
  }
}

// out[t] = the sum of its slots' rows, in slot order; H % 16 == 0: four columns a thread
template <typename OutT>
__global__ __launch_bounds__(256) void decode_combine_kernel(MoeDecodeParams p) {
  const uint32_t h = (blockIdx.x * 256 + threadIdx.x) * 4, t = blockIdx.y;
  if (h >= p.H) return;
  const float *y = p.y + (int64_t)t * p.k * p.H + h;
  float4v v = {0, 0, 0, 0};
#pragma unroll 4
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
  const uint32_t tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / 64), lane = tid % 64;
  const uint32_t l16 = lane % 16, lq = lane / 16;
  const uint32_t r0 = blockIdx.x * 16, K = p.I, H = p.H;
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
    const uint64_t row = (uint64_t)e * H + r0 + l16;
    const uint8_t *dq = p.d_q + row * (K / 2), *ds = p.d_s + row * (K / 16);
    const float fac = p.d_g[e] * p.w[slot];
    const bool in = l16 % TP == 0 && l16 / TP < (uint32_t)PH;
    const uint16_t *h = p.h + ((int64_t)(l16 / TP) * p.S + slot) * K;
    float4v acc = {0, 0, 0, 0};
    for (uint32_t k0 = part * CH; k0 < K; k0 += parts * CH) {
      const uint32_t k = k0 + lq * 64;
      const Codes cd = load_codes<ALIGNED>(dq, ds, k, K, k0 + CH <= K);
      bf16x8 f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = load_column(h, in, k, K, j);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(weights(cd, j), f[j], acc, 0, 0, 0);
    }
    acc = join_planes<PH>(acc);
    if (l16 == 0) {
      float4v *at = reinterpret_cast<float4v *>(&sum[wave][slot / p.k][4 * lq]);
      float4v v = *at;
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] += acc[r] * fac;
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

// column tiles a pass, from the tokens an expert has on average: one more pass
// reads the weights again (from L2), one tile too many costs registers
template <int P>
int column_tiles(const MoeDecodeParams &p) {
  const uint32_t mean = p.S / min(p.S, p.E);
  return mean * 2 <= kTokens<P> ? 1 : mean <= kTokens<P> ? 2 : 4;
}

template <int PX, int PH, bool ALIGNED>
void launch_gate_up(const MoeDecodeParams &p, bool fuse, hipStream_t stream) {
  const uint32_t grid = p.tiles_i * min(p.S, p.E);
  if constexpr (PX == 1) {
    if (fuse) {
      decode_gate_up_kernel<PX, PH, 1, ALIGNED, true><<<grid, 256, 0, stream>>>(p);
      return;
    }
  }
  const int nt = column_tiles<PX>(p);
  if (nt == 1) decode_gate_up_kernel<PX, PH, 1, ALIGNED, false><<<grid, 256, 0, stream>>>(p);
  else if (nt == 2) decode_gate_up_kernel<PX, PH, 2, ALIGNED, false><<<grid, 256, 0, stream>>>(p);
  else decode_gate_up_kernel<PX, PH, 4, ALIGNED, false><<<grid, 256, 0, stream>>>(p);
}

template <int PH, bool ALIGNED, typename OutT>
hipError_t launch_down(const MoeDecodeParams &p, hipStream_t stream) {
  if (p.S <= kOwnSlots) {
    decode_own_kernel<PH, ALIGNED, OutT><<<p.H / 16, 1024, 0, stream>>>(p);
    return hipGetLastError();
  }
  const uint32_t grid = p.tiles_h * min(p.S, p.E);
  const int nt = column_tiles<PH>(p);
  if (nt == 1) decode_down_kernel<PH, 1, ALIGNED><<<grid, 256, 0, stream>>>(p);
  else if (nt == 2) decode_down_kernel<PH, 2, ALIGNED><<<grid, 256, 0, stream>>>(p);
  else decode_down_kernel<PH, 4, ALIGNED><<<grid, 256, 0, stream>>>(p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  decode_combine_kernel<OutT><<<dim3((p.H + 1023) / 1024, p.T), 256, 0, stream>>>(p);
  return hipGetLastError();
}

template <int PX, int PH, typename OutT>
hipError_t launch_products(const MoeDecodeParams &p, bool fuse, bool gu_aligned, bool d_aligned, hipStream_t stream) {
  if (gu_aligned) launch_gate_up<PX, PH, true>(p, fuse, stream);
  else launch_gate_up<PX, PH, false>(p, fuse, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return d_aligned ? launch_down<PH, true, OutT>(p, stream) : launch_down<PH, false, OutT>(p, stream);
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

size_t moe_decode_workspace_bytes(int64_t T, int32_t /*E*/, int32_t k, int64_t H, int64_t I) {
  const size_t S = (size_t)T * k;
  return 2 * align256(S * 4) + align256(3 * (size_t)T * H * 2) + align256(3 * S * (size_t)I * 2) +
         align256(S * (size_t)H * 4);
}

hipError_t launch_moe_decode(MoeDecodeParams p, bool x_bf16, bool x_vec, bool gu_aligned, bool d_aligned,
                             bool out_bf16, void *workspace, hipStream_t stream) {
  if (p.T == 0) return hipSuccess;
  p.S = p.T * p.k;
  p.tiles_i = p.I / 16;
  p.tiles_h = (p.H + 63) / 64;
  uint8_t *at = static_cast<uint8_t *>(workspace);
  auto take = [&](size_t bytes) {
    uint8_t *r = at;
    at += align256(bytes);
    return r;
  };
  p.ids = reinterpret_cast<int32_t *>(take((size_t)p.S * 4));
  p.w = reinterpret_cast<float *>(take((size_t)p.S * 4));
  p.xp = reinterpret_cast<uint16_t *>(take(3 * (size_t)p.T * p.H * 2));
  p.h = reinterpret_cast<uint16_t *>(take(3 * (size_t)p.S * p.I * 2));
  p.y = reinterpret_cast<float *>(take((size_t)p.S * p.H * 4));
  const bool copy = !x_bf16 || !x_vec;
  p.xs = copy ? p.xp : static_cast<const uint16_t *>(p.x);
  p.x_ld = copy ? (int64_t)p.H : p.ld_x;
  p.x_plane = (int64_t)p.T * p.H;
  const bool fuse = p.T <= kFuseT && !copy;
  if (!fuse) {
    p.topk_blocks = (p.T + 3) / 4;
    const uint32_t grid = p.topk_blocks + (copy ? p.T * ((p.H + 255) / 256) : 0u);
    if (x_bf16) decode_prep_kernel<1><<<grid, 256, 0, stream>>>(p);
    else decode_prep_kernel<3><<<grid, 256, 0, stream>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (x_bf16)
    return out_bf16 ? launch_products<1, 2, uint16_t>(p, fuse, gu_aligned, d_aligned, stream)
                    : launch_products<1, 3, float>(p, fuse, gu_aligned, d_aligned, stream);
  return out_bf16 ? launch_products<3, 2, uint16_t>(p, fuse, gu_aligned, d_aligned, stream)
                  : launch_products<3, 3, float>(p, fuse, gu_aligned, d_aligned, stream);
}

}  // namespace nvfp4
