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
// Three launches, none of which waits for another on the host:
//   1. route: one workgroup; a wave per token finds its experts; a bit mask of
//      the tokens per expert then gives every active expert's list of slots.
//   2. gate_up: one workgroup per (active expert, 16 rows of h); its waves split
//      the hidden dimension and join through LDS; SiLU gate; h to the workspace.
//   3. down: one workgroup per 16 rows of out; its waves take the active experts
//      in turn, each adding its products, times the routing weight, to sums of
//      its own in LDS, which are joined in wave order (no atomics: the same
//      result every time).
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

constexpr int kMaxE = 1024;
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

// Top-k of one row by one wave: lane l holds logits l * PL .. l * PL + PL - 1, so
// equal logits go to the lowest lane and, inside it, to the lowest index.  Lane
// j < k returns the j-th expert and its routing weight.
template <int PL>
__device__ __forceinline__ void topk_row(const float *row, uint32_t E, uint32_t k, int32_t *id, float *w) {
  const uint32_t lane = threadIdx.x % 64;
  float v[PL];
  uint32_t open = 0;
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const uint32_t e = lane * PL + i;
    v[i] = e < E ? router_logit(row[e]) : -INFINITY;
    open |= (e < E ? 1u : 0u) << i;
  }
  float sel_v = 0.0f;
  int32_t sel_e = 0;
  for (uint32_t j = 0; j < k; ++j) {
    float bv = -INFINITY;
    int32_t bi = PL;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const bool take = ((open >> i) & 1u) & topk_before(v[i], i, bv, bi);
      bv = take ? v[i] : bv;
      bi = take ? i : bi;
    }
    const float top = wave_max_uniform(bv);
    // k <= E: some lane has an open logit; those without take no part
    const unsigned long long at = __ballot(open != 0 && bv == top);
    const uint32_t win = (uint32_t)__builtin_ctzll(at);
    const int32_t wi = __builtin_amdgcn_readlane(bi, win);
    if (lane == win) open &= ~(1u << wi);
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

__global__ __launch_bounds__(1024) void decode_route_kernel(MoeDecodeParams p) {
  __shared__ unsigned long long mask[2][kMaxE];  // tokens (64 a word) of each expert
  __shared__ int32_t first[kMaxE];               // first list entry of each expert
  __shared__ int32_t part[2][16];
  const uint32_t tid = threadIdx.x, wave = tid / 64, lane = tid % 64;
  mask[0][tid] = 0ull;
  mask[1][tid] = 0ull;
  __syncthreads();
  for (uint32_t t = wave; t < p.T; t += 16) {
    int32_t id;
    float w;
    topk_any(p.logits + (int64_t)t * p.E, p.E, p.k, &id, &w);
    if (lane < p.k) {
      p.ids[t * p.k + lane] = id;
      p.w[t * p.k + lane] = w;
      atomicOr(&mask[t / 64][id], 1ull << (t % 64));
    }
  }
  __syncthreads();
  // thread e: expert e's tokens and whether it is active, scanned over the experts
  const int32_t n = __popcll(mask[0][tid]) + __popcll(mask[1][tid]);
  int32_t rows = n, act = n > 0;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int32_t a = __shfl_up(rows, off, 64), b = __shfl_up(act, off, 64);
    if (lane >= (uint32_t)off) {
      rows += a;
      act += b;
    }
  }
  if (lane == 63) {
    part[0][wave] = rows;
    part[1][wave] = act;
  }
  __syncthreads();
  for (uint32_t v = 0; v < wave; ++v) {
    rows += part[0][v];
    act += part[1][v];
  }
  first[tid] = rows - n;
  if (n > 0) p.active[act - 1] = make_int4((int)tid, rows - n, n, 0);
  if (tid == 1023) p.n_active[0] = act;
  __syncthreads();
  // slot (t, j) goes after the expert's earlier tokens
  for (uint32_t t = wave; t < p.T; t += 16) {
    if (lane >= p.k) continue;
    const int32_t e = p.ids[t * p.k + lane];
    const unsigned long long below = (1ull << (t % 64)) - 1ull;
    int32_t r = first[e] + __popcll(mask[t / 64][e] & below);
    if (t >= 64) r += __popcll(mask[0][e]);
    p.list[r] = (int32_t)(t * p.k + lane);
  }
}

// x into bf16 planes of stride H: float32 x (three planes) and bf16 x whose rows
// are not 16-byte aligned (one)
template <int P>
__global__ __launch_bounds__(256) void decode_planes_kernel(MoeDecodeParams p) {
  const uint32_t t = blockIdx.y, h = blockIdx.x * 256 + threadIdx.x;
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

// Row r0 + l16 of a [rows][K] matrix, elements [k, k + 64).
// FAST (K % 64 == 0, aligned bases): the 64 elements are all in or all out.
// Otherwise block by block of 16, each all in or all out (K % 16 == 0).
template <bool FAST>
__device__ __forceinline__ Codes load_codes(const uint8_t *q, const uint8_t *s, bool row_in, uint32_t k, uint32_t K) {
  Codes c;
  c.lo = c.hi = (u32x4){0, 0, 0, 0};
  c.s = 0;
  if constexpr (FAST) {
    if (row_in && k < K) {
      c.lo = *reinterpret_cast<const u32x4 *>(q + k / 2);
      c.hi = *reinterpret_cast<const u32x4 *>(q + k / 2 + 16);
      c.s = *reinterpret_cast<const uint32_t *>(s + k / 16);
    }
  } else {
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      if (row_in && k + 16 * b < K) {
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

// a lane's column: elements [k, k + 64) of one bf16 row, eight fragments
template <bool FAST>
__device__ __forceinline__ void load_column(const uint16_t *x, bool in, uint32_t k, uint32_t K, bf16x8 f[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    u32x4 v = {0, 0, 0, 0};
    if (in && (FAST ? k : k + 8 * j) < K) v = *reinterpret_cast<const u32x4 *>(x + k + 8 * j);
    f[j] = __builtin_bit_cast(bf16x8, v);
  }
}

template <int J>
__device__ __forceinline__ float scale_at(uint32_t s) { return __builtin_amdgcn_cvt_f32_fp8((int)s, J); }

// acc += 16 weight rows x 16 columns over one 256-wide step
__device__ __forceinline__ float4v multiply(const Codes &c, const bf16x8 f[8], float4v acc) {
  const float s0 = scale_at<0>(c.s), s1 = scale_at<1>(c.s), s2 = scale_at<2>(c.s), s3 = scale_at<3>(c.s);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t w = j < 4 ? c.lo[j] : c.hi[j - 4];
    const float s = j < 2 ? s0 : j < 4 ? s1 : j < 6 ? s2 : s3;
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(decode8(w, s), f[j], acc, 0, 0, 0);
  }
  return acc;
}

__device__ __forceinline__ float silu(float z) {
  return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-z * 1.44269504088896341f));
}

// P bf16 planes per token share the 16 columns: 16, 8 or 5 tokens at a time
template <int P>
constexpr uint32_t kTokens = P == 1 ? 16 : P == 2 ? 8 : 5;

// PX planes of x, PH planes of h
template <int PX, int PH, bool FAST>
__global__ __launch_bounds__(256) void decode_gate_up_kernel(MoeDecodeParams p) {
  constexpr uint32_t TP = kTokens<PX>, NW = 4;
  __shared__ __attribute__((aligned(16))) float red[NW][2][16][20];  // [wave][gate, up][column][row]
  const uint32_t tid = threadIdx.x, wave = tid / 64, lane = tid % 64, l16 = lane % 16, lq = lane / 16;
  const uint32_t item = blockIdx.x / p.tiles_i, r0 = (blockIdx.x % p.tiles_i) * 16;
  if (item >= (uint32_t)p.n_active[0]) return;
  const int4 it = p.active[item];
  const uint32_t K = p.H, I = p.I;
  const uint64_t row = (uint64_t)it.x * 2 * I + r0 + l16;  // I % 16 == 0: whole row tiles
  const uint8_t *gq = p.gu_q + row * (K / 2), *gs = p.gu_s + row * (K / 16);
  const uint8_t *uq = gq + (uint64_t)I * (K / 2), *us = gs + (uint64_t)I * (K / 16);
  const float g = p.gu_g[it.x];
  for (uint32_t t0 = 0; t0 < (uint32_t)it.z; t0 += TP) {
    const uint32_t cnt = min((uint32_t)it.z - t0, TP);
    const uint32_t plane = l16 / TP, c = l16 % TP;
    const bool col_in = plane < PX && c < cnt;
    const uint32_t slot = col_in ? (uint32_t)p.list[it.y + t0 + c] : 0u;
    const uint16_t *x = p.xs + (int64_t)plane * p.x_plane + (int64_t)(slot / p.k) * p.x_ld;
    float4v ag = {}, au = {};
    for (uint32_t k0 = wave * CH; k0 < K; k0 += NW * CH) {
      const uint32_t k = k0 + lq * 64;
      const Codes cg = load_codes<FAST>(gq, gs, true, k, K), cu = load_codes<FAST>(uq, us, true, k, K);
      bf16x8 f[8];
      load_column<FAST>(x, col_in, k, K, f);
      ag = multiply(cg, f, ag);
      au = multiply(cu, f, au);
    }
    __syncthreads();  // the last pass's sums have been read
    *reinterpret_cast<float4v *>(&red[wave][0][l16][4 * lq]) = ag;
    *reinterpret_cast<float4v *>(&red[wave][1][l16][4 * lq]) = au;
    __syncthreads();
    const uint32_t tc = tid / 16, r = tid % 16;
    if (tc < cnt) {
      float zg = 0.0f, zu = 0.0f;
#pragma unroll
      for (int pl = 0; pl < PX; ++pl)
#pragma unroll
        for (uint32_t w = 0; w < NW; ++w) {
          zg += red[w][0][pl * TP + tc][r];
          zu += red[w][1][pl * TP + tc][r];
        }
      uint16_t o[PH];
      split<PH>(silu(zg * g) * (zu * g), o);
      const uint32_t s = (uint32_t)p.list[it.y + t0 + tc];
#pragma unroll
      for (int pl = 0; pl < PH; ++pl) p.h[((int64_t)pl * p.S + s) * I + r0 + r] = o[pl];
    }
  }
}

template <int PH, bool FAST, int NW, int TMAX, typename OutT>
__global__ __launch_bounds__(NW * 64) void decode_down_kernel(MoeDecodeParams p) {
  constexpr uint32_t TP = kTokens<PH>;
  __shared__ __attribute__((aligned(16))) float sum[NW][TMAX][16];
  const uint32_t tid = threadIdx.x, wave = tid / 64, lane = tid % 64, l16 = lane % 16, lq = lane / 16;
  const uint32_t r0 = blockIdx.x * 16, K = p.I, H = p.H;
  for (uint32_t i = tid; i < NW * p.T * 16; i += NW * 64)
    sum[i / (p.T * 16)][i / 16 % p.T][i % 16] = 0.0f;
  __syncthreads();
  const uint32_t n = (uint32_t)p.n_active[0];
  const uint32_t plane = l16 / TP, c = l16 % TP;
  for (uint32_t item = wave; item < n; item += NW) {
    const int4 it = p.active[item];
    const uint64_t row = (uint64_t)it.x * H + r0 + l16;
    const uint8_t *dq = p.d_q + row * (K / 2), *ds = p.d_s + row * (K / 16);
    const float g = p.d_g[it.x];
    for (uint32_t t0 = 0; t0 < (uint32_t)it.z; t0 += TP) {
      const uint32_t cnt = min((uint32_t)it.z - t0, TP);
      const bool col_in = plane < PH && c < cnt;
      const uint32_t slot = col_in ? (uint32_t)p.list[it.y + t0 + c] : 0u;
      const uint16_t *h = p.h + ((int64_t)plane * p.S + slot) * K;
      float4v acc = {};
      for (uint32_t k0 = 0; k0 < K; k0 += CH) {
        const uint32_t k = k0 + lq * 64;
        const Codes cd = load_codes<FAST>(dq, ds, true, k, K);
        bf16x8 f[8];
        load_column<FAST>(h, col_in, k, K, f);
        acc = multiply(cd, f, acc);
      }
      // the planes of a token side by side, then added to the wave's own sums
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float v = acc[r];
#pragma unroll
        for (int pl = 1; pl < PH; ++pl) v += __shfl(acc[r], (int)(lane + pl * TP) & 63, 64);
        acc[r] = v;
      }
      if (plane == 0 && c < cnt) {
        float4v *at = reinterpret_cast<float4v *>(&sum[wave][slot / p.k][4 * lq]);
        const float f = g * p.w[slot];
        float4v v = *at;
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] += acc[r] * f;
        *at = v;
      }
    }
  }
  __syncthreads();
  OutT *out = static_cast<OutT *>(p.out);
  for (uint32_t i = tid; i < p.T * 16; i += NW * 64) {
    const uint32_t t = i / 16, r = i % 16;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) v += sum[w][t][r];
    if constexpr (sizeof(OutT) == 4) out[(int64_t)t * p.ld_out + r0 + r] = v;
    else out[(int64_t)t * p.ld_out + r0 + r] = (OutT)float_to_bf16_bits(v);
  }
}

template <int PH, bool FAST, typename OutT>
void launch_down(const MoeDecodeParams &p, hipStream_t stream) {
  const uint32_t grid = p.H / 16;
  if (p.T <= 16) decode_down_kernel<PH, FAST, 16, 16, OutT><<<grid, 1024, 0, stream>>>(p);
  else if (p.T <= 64) decode_down_kernel<PH, FAST, 8, 64, OutT><<<grid, 512, 0, stream>>>(p);
  else decode_down_kernel<PH, FAST, 8, 128, OutT><<<grid, 512, 0, stream>>>(p);
}

template <int PX, int PH>
hipError_t launch_products(const MoeDecodeParams &p, bool gu_fast, bool d_fast, bool out_bf16, hipStream_t stream) {
  const uint32_t grid = p.tiles_i * min(p.S, p.E);
  if (gu_fast) decode_gate_up_kernel<PX, PH, true><<<grid, 256, 0, stream>>>(p);
  else decode_gate_up_kernel<PX, PH, false><<<grid, 256, 0, stream>>>(p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (out_bf16) {
    if (d_fast) launch_down<PH, true, uint16_t>(p, stream);
    else launch_down<PH, false, uint16_t>(p, stream);
  } else {
    if (d_fast) launch_down<PH, true, float>(p, stream);
    else launch_down<PH, false, float>(p, stream);
  }
  return hipGetLastError();
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

size_t moe_decode_workspace_bytes(int64_t T, int32_t E, int32_t k, int64_t H, int64_t I) {
  const size_t S = (size_t)T * k;
  return align256(4) + align256(S * 4) * 3 + align256((size_t)E * 16) + align256(3 * (size_t)T * H * 2) +
         align256(3 * S * (size_t)I * 2);
}

hipError_t launch_moe_decode(MoeDecodeParams p, bool x_bf16, bool x_vec, bool gu_fast, bool d_fast, bool out_bf16,
                             void *workspace, hipStream_t stream) {
  if (p.T == 0) return hipSuccess;
  p.S = p.T * p.k;
  p.tiles_i = p.I / 16;
  uint8_t *at = static_cast<uint8_t *>(workspace);
  auto take = [&](size_t bytes) {
    uint8_t *r = at;
    at += align256(bytes);
    return r;
  };
  p.n_active = reinterpret_cast<int32_t *>(take(4));
  p.ids = reinterpret_cast<int32_t *>(take((size_t)p.S * 4));
  p.w = reinterpret_cast<float *>(take((size_t)p.S * 4));
  p.list = reinterpret_cast<int32_t *>(take((size_t)p.S * 4));
  p.active = reinterpret_cast<int4 *>(take((size_t)p.E * 16));
  p.xp = reinterpret_cast<uint16_t *>(take(3 * (size_t)p.T * p.H * 2));
  p.h = reinterpret_cast<uint16_t *>(take(3 * (size_t)p.S * p.I * 2));
  const bool copy = !x_bf16 || !x_vec;
  p.xs = copy ? p.xp : static_cast<const uint16_t *>(p.x);
  p.x_ld = copy ? (int64_t)p.H : p.ld_x;
  p.x_plane = (int64_t)p.T * p.H;
  if (copy) {
    const dim3 grid((p.H + 255) / 256, p.T);
    if (x_bf16) decode_planes_kernel<1><<<grid, 256, 0, stream>>>(p);
    else decode_planes_kernel<3><<<grid, 256, 0, stream>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  decode_route_kernel<<<1, 1024, 0, stream>>>(p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (x_bf16)
    return out_bf16 ? launch_products<1, 2>(p, gu_fast, d_fast, true, stream)
                    : launch_products<1, 3>(p, gu_fast, d_fast, false, stream);
  return out_bf16 ? launch_products<3, 2>(p, gu_fast, d_fast, true, stream)
                  : launch_products<3, 3>(p, gu_fast, d_fast, false, stream);
}

}  // namespace nvfp4
