// A whole mixture-of-experts layer for a few tokens (T <= 16) on gfx950.
//
//   logits[t, e] = x[t] . Wr[e] + bias[e]          ids, w = top-k softmax of them
//   g = x[t] . W_gate[e, d],  u = x[t] . W_up[e, d]
//   hw[t, e, d] = (sum of w over t's slots that name e) * SiLU(g) * u
//   y[t, c] = R( sum over t's experts e ascending of hw[t, e] . W_down[e, c] )
//
// Bound: the weights of the distinct experts, read once. With so few tokens
// every matrix product is a stream of weight rows against at most 16 rows of
// activations, one v_mfma 16x16x32 tile high, so the kernels are built around
// the stream and the dispatch tables, the sorted rows, expert_out and the
// separate reduce of the general path all go away:
//
//   few_logits_kernel   one workgroup an expert, all tokens: sums in fp64 (the
//                       products of 16-bit and fp32 values are exact there), so
//                       ids do not hang on a summation order; fp64 vector FMAs
//                       run at the fp32 rate and the kernel waits for memory.
//   few_gate_up_kernel  every workgroup repeats the top-k selection in its
//                       prologue (a few LDS-sized arrays; cheaper than a launch
//                       and a pass through memory), finds the distinct experts
//                       and takes (expert, 16 columns) items in turn. Its 4
//                       waves split the reduction; partial sums meet in LDS.
//   few_down_kernel     a workgroup takes 64 columns of y and a share of the
//                       distinct experts: row t of the MFMA tile is token t, so
//                       its accumulators hold parts of y and no pass combines
//                       expert rows; few_combine_kernel adds up the shares.
//
// Both GEMM kernels run one uninterrupted stream of chunks (64 bytes of each
// of 16 weight rows = 1 KB a load) through a register ring that crosses item
// and expert borders. MFMA rows of tokens that an expert does not serve read
// zeros through the buffer's bounds check (no memory is touched) and are left
// out where sums are added up (a select: nothing of an expert, not even a
// NaN, reaches a token that it does not serve).
//
// Precision: hw stays in 32 bits between the kernels. bf16, FP8 and MXFP4
// weights meet it as a pair of bf16 (16 significant bits; a single bf16 would
// double the error variance of a bf16 y), fp16 weights meet it in fp32 on
// v_mfma_f32_16x16x4 (fp16 pairs would overflow past 65504; at 16 rows the
// fp32 instruction still outruns the weight stream: 8 x 32 cycles per 1 KB a
// wave, 16 B/clk/CU against the 10 that HBM delivers). FP8 codes are exact in
// 16 bits; MXFP4 codes times their E8M0 scale are exact in bf16, so fp16
// activations against MXFP4 weights are split into two bf16 (exact).

#include "common.hpp"
#include "launch.hpp"

namespace moe {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));

constexpr int kRows = 16;                        // tokens of one call at most
constexpr int kMaxE = 1024;
constexpr int kMaxP = kRows * 64;                // routed pairs at most
constexpr int kGateUpThreads = 256;
constexpr int kW16 = 0, kWFp8 = 1, kWMx = 2;     // weight formats

// Reduction elements in 16 bytes of one weight row.
template <int F>
constexpr int lane_elems() {
  return F == kW16 ? 8 : (F == kWFp8 ? 16 : 32);
}

struct FewArgs {
  const void* x;
  const uint8_t *wg, *wu, *wd;
  const void *sg, *su, *sd;       // FP8: fp32 per row; MXFP4: E8M0 per 32 elements
  const float* logits;            // nullptr: ids and weights are given
  int32_t* ids;
  float* weights;
  uint8_t* hw;                    // [P, D] fp32, or two [P, D] bf16 (high, low parts)
  float* parts;                   // [parts, T, H] sums of few_down_kernel's expert groups
  void* y;
  int T, H, D, E, K, renorm;
};

// ---------------------------------------------------------------- router --

// Logits of expert blockIdx.x for tokens TT * blockIdx.y and on: every thread
// strides over the row four elements at a time, fp64 sums go lane -> wave ->
// workgroup.
template <int DT, int TT>
__global__ __launch_bounds__(256) void few_logits_kernel(const uint16_t* __restrict__ x,
                                                         const float* __restrict__ wr,
                                                         const float* __restrict__ bias, int T,
                                                         int H, int E, float* __restrict__ logits) {
  __shared__ double part[4][TT];
  const int e = blockIdx.x, tid = threadIdx.x, t0 = blockIdx.y * TT;
  x += static_cast<int64_t>(t0) * H;
  T -= t0;
  double acc[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) acc[t] = 0.0;
  const float* row = wr + static_cast<int64_t>(e) * H;
#pragma unroll 2
  for (int c = tid * 4; c < H; c += 1024) {
    const float4 w = *reinterpret_cast<const float4*>(row + c);
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const int tt = t < T ? t : 0;
      const u32x2 v = *reinterpret_cast<const u32x2*>(x + static_cast<int64_t>(tt) * H + c);
      acc[t] = fma(static_cast<double>(to_float<DT>(v.x & 0xffffu)), static_cast<double>(w.x), acc[t]);
      acc[t] = fma(static_cast<double>(to_float<DT>(v.x >> 16)), static_cast<double>(w.y), acc[t]);
      acc[t] = fma(static_cast<double>(to_float<DT>(v.y & 0xffffu)), static_cast<double>(w.z), acc[t]);
      acc[t] = fma(static_cast<double>(to_float<DT>(v.y >> 16)), static_cast<double>(w.w), acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < TT; ++t) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) acc[t] += __shfl_xor(acc[t], off);
    if ((tid & 63) == 0) part[tid >> 6][t] = acc[t];
  }
  __syncthreads();
  if (tid < T && tid < TT) {
    double s = part[0][tid] + part[1][tid] + part[2][tid] + part[3][tid];
    if (bias) s += static_cast<double>(bias[e]);
    logits[static_cast<int64_t>(t0 + tid) * E + e] = static_cast<float>(s);
  }
}

// ------------------------------------------------------------- selection --

// Unsigned keys in the order of the floats (-0 as +0); 0 means "none".
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);
  const uint32_t k = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return k ? k : 1u;
}

__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// The wave's largest value, in every lane: rows of 16 by DPP shifts, then
// across the rows (lanes without a source read 0).
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#define MOE_DPP_MAX(ctrl, rows)                                                                   \
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), ctrl, rows, \
                                                               0xf, false)))
  MOE_DPP_MAX(0x111, 0xf);   // row_shr:1
  MOE_DPP_MAX(0x112, 0xf);
  MOE_DPP_MAX(0x114, 0xf);
  MOE_DPP_MAX(0x118, 0xf);
  MOE_DPP_MAX(0x142, 0xa);   // row_bcast:15 into rows 1 and 3
  MOE_DPP_MAX(0x143, 0xc);   // row_bcast:31 into rows 2 and 3
#undef MOE_DPP_MAX
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 63));
}

// The wave's sum, in every lane, the same way (lanes without a source add 0).
__device__ __forceinline__ float wave_sum(float v) {
#define MOE_DPP_ADD(ctrl, rows)                                                                      \
  v += __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_update_dpp(                            \
      0, static_cast<int>(__float_as_uint(v)), ctrl, rows, 0xf, false)))
  MOE_DPP_ADD(0x111, 0xf);
  MOE_DPP_ADD(0x112, 0xf);
  MOE_DPP_ADD(0x114, 0xf);
  MOE_DPP_ADD(0x118, 0xf);
  MOE_DPP_ADD(0x142, 0xa);
  MOE_DPP_ADD(0x143, 0xc);
#undef MOE_DPP_ADD
  return __uint_as_float(static_cast<uint32_t>(
      __builtin_amdgcn_readlane(static_cast<int>(__float_as_uint(v)), 63)));
}

// Top-k of one token by one wave: lane L holds experts L * NPL .. + NPL - 1,
// so the lowest lane with the maximum holds the lowest expert index. (Several
// tokens side by side in one wave measured slower: the larger code has to be
// fetched by every CU before its first weight load.)
template <int NPL>
__device__ __forceinline__ void select_topk(const float* logits, int E, int K, int renorm, int lane,
                                            int* sid, float* sw) {
  uint32_t key[NPL], best;
  int best_j;
#pragma unroll
  for (int j = 0; j < NPL; ++j) {
    const int e = lane * NPL + j;
    key[j] = e < E ? order_key(logits[e]) : 0u;
  }
  auto rescan = [&]() __attribute__((always_inline)) {
    best = key[0];
    best_j = 0;
#pragma unroll
    for (int j = 1; j < NPL; ++j) {
      const bool more = key[j] > best;
      best = more ? key[j] : best;
      best_j = more ? j : best_j;
    }
  };
  rescan();
  const float top = key_value(wave_max(best));
  float z = 0.0f;
#pragma unroll
  for (int j = 0; j < NPL; ++j) z += key[j] ? expf(key_value(key[j]) - top) : 0.0f;
  z = wave_sum(z);
  float mine = 0.0f;            // lane k keeps the k-th selection (K <= 64)
  int mine_id = 0;
  for (int k = 0; k < K; ++k) {
    const uint32_t m = wave_max(best);
    const int src = __builtin_ctzll(__ballot(best == m));
    const int id = __builtin_amdgcn_readlane(lane * NPL + best_j, src);
    mine = lane == k ? key_value(m) : mine;
    mine_id = lane == k ? id : mine_id;
#pragma unroll
    for (int j = 0; j < NPL; ++j) key[j] = lane * NPL + j == id ? 0u : key[j];
    rescan();
  }
  float p = lane < K ? expf(mine - top) / z : 0.0f;
  if (renorm) p = p / wave_sum(p);
  if (lane < K) {
    sid[lane] = mine_id;
    sw[lane] = p;
  }
}

// What the workgroups of both GEMM kernels know of the routing.
struct Plan {
  int sid[kMaxP];              // expert of each slot, -1 = masked
  uint32_t mask[kMaxE];        // tokens of each expert
  uint16_t list[kMaxE];        // the distinct experts, ascending
  int count;
};

// mask, list and count from sid (written before, by any thread).
__device__ __forceinline__ void build_plan(Plan& s, int P, int K, int E, int tid, int threads) {
  for (int e = tid; e < E; e += threads) s.mask[e] = 0u;
  __syncthreads();
  for (int p = tid; p < P; p += threads) {
    if (s.sid[p] >= 0) atomicOr(&s.mask[s.sid[p]], 1u << (p / K));
  }
  __syncthreads();
  if (tid < 64) {
    int n = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const bool used = e0 + tid < E && s.mask[e0 + tid] != 0u;
      const uint64_t b = __ballot(used);
      if (used) s.list[n + __popcll(b & ((1ull << tid) - 1))] = static_cast<uint16_t>(e0 + tid);
      n += __popcll(b);
    }
    if (tid == 0) s.count = n;
  }
  __syncthreads();
}

// --------------------------------------------------------------- operands --

// 16 bytes at byte `lane_off + wave_off` of a buffer; zeros, without touching
// memory, where the sum is past its size (kNoRow: rows that do not exist).
constexpr uint32_t kNoRow = 0x80000000u;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, static_cast<int>(bytes), 0x00027000);
}
__device__ __forceinline__ u32x4 buffer_load16(__amdgpu_buffer_rsrc_t b, uint32_t lane_off, int wave_off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, static_cast<int>(lane_off), wave_off, 0));
}

// A value that is the same in all lanes, in a scalar register.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

template <int DT>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (DT == kBF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  } else {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
}

// 16 bytes of a weight row -> its 16-bit MFMA operands of 8 elements each
// (dtype DT; MXFP4 always bf16, scaled by 2^(sc - 127)).
template <int DT, int F>
__device__ __forceinline__ void decode(u32x4 w, uint32_t sc, u32x4* out) {
  if constexpr (F == kW16) {
    out[0] = w;
  } else if constexpr (F == kWFp8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t v;
      if constexpr (DT == kBF16) {
        v = (i & 1) ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i >> 1], 1.0f, true))
                    : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i >> 1], 1.0f, false));
      } else {
        v = (i & 1) ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[i >> 1], 1.0f, true))
                    : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[i >> 1], 1.0f, false));
      }
      out[i >> 2][i & 3] = v;
    }
  } else {
    const float s = __uint_as_float(sc << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      out[i][0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], s, 0));
      out[i][1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], s, 1));
      out[i][2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], s, 2));
      out[i][3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], s, 3));
    }
  }
}

// v = high + low in bf16, |v - high - low| <= 2^-17 |v|.
__device__ __forceinline__ void split_bf16(float v, uint32_t& hi, uint32_t& lo) {
  hi = float_to_bf16(v);
  // a value that rounds to infinity (or is not finite) has no remainder
  const float r = v - bf16_to_float(hi);
  lo = fabsf(r) <= 3.0e38f ? float_to_bf16(r) : 0u;
}

// Eight fp16 values as two bf16 operands (exact: 11 significant bits).
__device__ __forceinline__ void split_f16x8(u32x4 x, u32x4& hi, u32x4& lo) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h0, l0, h1, l1;
    split_bf16(f16_to_float(x[i] & 0xffffu), h0, l0);
    split_bf16(f16_to_float(x[i] >> 16), h1, l1);
    hi[i] = h0 | (h1 << 16);
    lo[i] = l0 | (l1 << 16);
  }
}

// ---------------------------------------------------------------- gate/up --

// hw in fp32 (fp16 weights) or as bf16 parts.
template <int DT, int F>
constexpr bool hw_fp32() {
  return DT == kF16 && F == kW16;
}

// One step of a wave: a pair of chunks (both halves of the 128-byte lines of 16
// NT gate and up rows) and the tokens' x.
template <int F, int NT>
struct GateUpSlot {
  u32x4 g[NT][2], u[NT][2];
  u32x4 x[2][lane_elems<F>() / 8];
  u32x2 sg[NT], su[NT];         // FP8: the rows' fp32 scales (in .x); MXFP4: the pair's 8 E8M0 bytes
};

// The E8M0 byte of lane group lg in half k of a pair's 8.
__device__ __forceinline__ uint32_t pair_scale(const u32x2& s, int k, int lg) {
  return ((k ? s.y : s.x) >> (8 * lg)) & 0xffu;
}

// Column tiles of 16 that a wave works on at once, ring depth in pairs and waves
// per SIMD. x is read once for all tiles: with 4-bit weights its loads would
// outnumber the weights' two to one at one tile (8 tokens on MXFP4 weights of
// the 256 x 7168 x 2048 layer: 261 us, 184 us with two, 202 us with four). 16-bit
// weights stream at 5.9 TB/s with one tile and four workgroups on a CU (16 tokens
// 1008 us for 5.98 GB). Rings of 2, 3 and 4 pairs: one token 83.0, 81.7, 84.5 us,
// on the 128 x 2048 x 768 layer 17.0, 16.5, 18.7 us.
template <int F>
struct GateUpShape {
  static constexpr int kTiles = F == kW16 ? 1 : 2;
  static constexpr int kDepth = F == kW16 ? 3 : 2;
  static constexpr int kWaves = F == kW16 ? 4 : 2;
};

template <int DT, int F>
__global__ __launch_bounds__(kGateUpThreads, GateUpShape<F>::kWaves) void few_gate_up_kernel(FewArgs a) {
  constexpr int EL = lane_elems<F>(), NX = EL / 8;
  constexpr int S = GateUpShape<F>::kDepth, NT = GateUpShape<F>::kTiles;
  __shared__ Plan plan;
  __shared__ float sw[kMaxP];
  __shared__ f32x4 red[2][4][2 * NT][64];
  const int tid = threadIdx.x, wave = uniform(tid >> 6), lane = tid & 63, lr = lane & 15, lg = lane >> 4;
  const int P = a.T * a.K;

  if (a.logits) {
    for (int t = wave; t < a.T; t += 4) {
      const float* l = a.logits + static_cast<int64_t>(t) * a.E;
      if (a.E > 256) select_topk<16>(l, a.E, a.K, a.renorm, lane, plan.sid + t * a.K, sw + t * a.K);
      else select_topk<4>(l, a.E, a.K, a.renorm, lane, plan.sid + t * a.K, sw + t * a.K);
    }
  } else {
    for (int p = tid; p < P; p += kGateUpThreads) {
      const int id = a.ids[p];
      plan.sid[p] = id >= 0 && id < a.E ? id : -1;
      sw[p] = a.weights ? a.weights[p] : 1.0f;
    }
  }
  build_plan(plan, P, a.K, a.E, tid, kGateUpThreads);
  if (a.logits && blockIdx.x == 0) {
    for (int p = tid; p < P; p += kGateUpThreads) {
      a.ids[p] = plan.sid[p];
      a.weights[p] = sw[p];
    }
  }

  const int tiles = a.D / (16 * NT);
  const int items = plan.count * tiles;
  if (static_cast<int>(blockIdx.x) >= items) return;
  // This wave's steps of every item: pairs of chunks (128 bytes a row) wave, wave + 4, ...
  const int pairs = a.H / (8 * EL);
  const int n = (pairs - wave + 3) / 4;
  const int64_t row_bytes = static_cast<int64_t>(a.H / EL) * 16;
  const int64_t blocks = a.H / 32;

  // Where the next chunk to load lies: wave-uniform bases (scalar registers)
  // and fixed 32-bit lane offsets.
  int l_item = blockIdx.x, l_c = 0;
  const uint8_t *pg = nullptr, *pu = nullptr, *qg = nullptr, *qu = nullptr;
  const uint32_t w_off = static_cast<uint32_t>(lr * row_bytes) + lg * 16;
  const uint32_t s_off = F == kWFp8 ? lr * 4 : static_cast<uint32_t>(lr * blocks);
  const int64_t tile_bytes = 16 * row_bytes;
  uint32_t x_off = 0;
  auto aim = [&]() __attribute__((always_inline)) {
    const int e = uniform(plan.list[l_item / tiles]);
    const int64_t row = static_cast<int64_t>(e) * a.D + (l_item % tiles) * (16 * NT);
    pg = a.wg + row * row_bytes;
    pu = a.wu + row * row_bytes;
    if constexpr (F != kW16) {
      qg = static_cast<const uint8_t*>(a.sg) + row * (F == kWFp8 ? 4 : blocks);
      qu = static_cast<const uint8_t*>(a.su) + row * (F == kWFp8 ? 4 : blocks);
    }
    const uint32_t m = static_cast<uint32_t>(uniform(static_cast<int>(plan.mask[e])));
    x_off = (m >> lr) & 1 ? static_cast<uint32_t>(lr * a.H + lg * EL) * 2 : kNoRow;
  };
  const __amdgpu_buffer_rsrc_t xb = buffer_of(a.x, static_cast<int64_t>(a.T) * a.H * 2);
  GateUpSlot<F, NT> ring[S];
  auto load = [&](GateUpSlot<F, NT>& s) __attribute__((always_inline)) {
    // Both halves of a line right after one another: with other loads between
    // them the second one stalls the first-level cache on the pending line.
    const int64_t c = 4 * l_c + wave;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const uint8_t *g = pg + t * tile_bytes + c * 128, *u = pu + t * tile_bytes + c * 128;
      s.g[t][0] = *reinterpret_cast<const u32x4*>(g + w_off);
      s.g[t][1] = *reinterpret_cast<const u32x4*>(g + w_off + 64);
      s.u[t][0] = *reinterpret_cast<const u32x4*>(u + w_off);
      s.u[t][1] = *reinterpret_cast<const u32x4*>(u + w_off + 64);
      if constexpr (F == kWFp8) {
        s.sg[t].x = *reinterpret_cast<const uint32_t*>(qg + t * 64 + s_off);
        s.su[t].x = *reinterpret_cast<const uint32_t*>(qu + t * 64 + s_off);
      } else if constexpr (F == kWMx) {
        s.sg[t] = *reinterpret_cast<const u32x2*>(qg + t * 16 * blocks + c * 8 + s_off);
        s.su[t] = *reinterpret_cast<const u32x2*>(qu + t * 16 * blocks + c * 8 + s_off);
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int i = 0; i < NX; ++i) {
        s.x[k][i] = buffer_load16(xb, x_off + 16 * i, static_cast<int>(c) * (16 * EL) + k * (8 * EL));
      }
    }
    if (++l_c == n) {
      // past the last item the last pair is read again (in bounds, never used)
      if (l_item + static_cast<int>(gridDim.x) < items) {
        l_item += gridDim.x;
        l_c = 0;
        aim();
      } else {
        l_c = n - 1;
      }
    }
  };

  int item = blockIdx.x, buf = 0;
  f32x4 accg[NT] = {}, accu[NT] = {};
  float scale_g[NT], scale_u[NT];
  // The item's sums are complete: add up the waves' parts and store hw.
  auto finish = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      red[buf][wave][2 * t][lane] = accg[t];
      red[buf][wave][2 * t + 1][lane] = accu[t];
      accg[t] = accu[t] = f32x4{};
    }
    wait_lds();
    barrier_no_wait();
    const int e = uniform(plan.list[item / tiles]);
    const int t = lg * 4 + wave;     // thread (wave i, lane l): register i of lane l, row 4 (l / 16) + i
    const bool live = (plan.mask[e] >> t) & 1;
    int p = 0;
    float w = 0.0f;
    if (live) {
      for (int k = a.K - 1; k >= 0; --k) {
        if (plan.sid[t * a.K + k] == e) {
          p = t * a.K + k;
          w += sw[p];
        }
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float g = 0.0f, u = 0.0f;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        g += reinterpret_cast<const float*>(&red[buf][v][2 * nt][lane])[wave];
        u += reinterpret_cast<const float*>(&red[buf][v][2 * nt + 1][lane])[wave];
      }
      if constexpr (F == kWFp8) {
        g *= scale_g[nt];
        u *= scale_u[nt];
      }
      const float v = w * (silu(g) * u);
      const int64_t at = static_cast<int64_t>(p) * a.D + (item % tiles) * (16 * NT) + nt * 16 + lr;
      if (live) {
        if constexpr (hw_fp32<DT, F>()) {
          reinterpret_cast<float*>(a.hw)[at] = v;
        } else {
          uint32_t hi, lo;
          split_bf16(v, hi, lo);
          uint16_t* h = reinterpret_cast<uint16_t*>(a.hw);
          h[at] = static_cast<uint16_t>(hi);
          h[static_cast<int64_t>(P) * a.D + at] = static_cast<uint16_t>(lo);
        }
      }
    }
    buf ^= 1;   // the other buffer: a wave still reading this one has not passed the next barrier
    item += gridDim.x;
  };

  if (n == 0) {                      // fewer pairs than waves: this one only adds zeros
    while (item < items) {
      if constexpr (F == kWFp8) {
        const int64_t row = static_cast<int64_t>(plan.list[item / tiles]) * a.D + (item % tiles) * (16 * NT) + lr;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          scale_g[t] = static_cast<const float*>(a.sg)[row + 16 * t];
          scale_u[t] = static_cast<const float*>(a.su)[row + 16 * t];
        }
      }
      finish();
    }
    return;
  }
  aim();
#pragma unroll
  for (int s = 0; s < S; ++s) load(ring[s]);
  int c = 0;
  auto step = [&](auto U) __attribute__((always_inline)) {
    constexpr int s = decltype(U)::value;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      u32x4 xl[F == kWMx && DT == kF16 ? NX : 1];     // fp16 x in two bf16 parts
      if constexpr (F == kWMx && DT == kF16) {
#pragma unroll
        for (int i = 0; i < NX; ++i) {
          const u32x4 x = ring[s].x[k][i];
          split_f16x8(x, ring[s].x[k][i], xl[i]);
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        u32x4 wg[NX], wu[NX];
        decode<DT, F>(ring[s].g[t][k], pair_scale(ring[s].sg[t], k, lg), wg);
        decode<DT, F>(ring[s].u[t][k], pair_scale(ring[s].su[t], k, lg), wu);
#pragma unroll
        for (int i = 0; i < NX; ++i) {
          if constexpr (F == kWMx && DT == kF16) {
            accg[t] = mfma16<kBF16>(ring[s].x[k][i], wg[i], accg[t]);
            accu[t] = mfma16<kBF16>(ring[s].x[k][i], wu[i], accu[t]);
            accg[t] = mfma16<kBF16>(xl[i], wg[i], accg[t]);
            accu[t] = mfma16<kBF16>(xl[i], wu[i], accu[t]);
          } else {
            accg[t] = mfma16<DT>(ring[s].x[k][i], wg[i], accg[t]);
            accu[t] = mfma16<DT>(ring[s].x[k][i], wu[i], accu[t]);
          }
        }
      }
    }
    if constexpr (F == kWFp8) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        scale_g[t] = __uint_as_float(ring[s].sg[t].x);
        scale_u[t] = __uint_as_float(ring[s].su[t].x);
      }
    }
    load(ring[s]);
    if (++c == n) {
      c = 0;
      finish();
    }
  };
  // Whole turns of the ring without a condition around a load (one would make
  // the compiler wait for more loads than it has to), then the rest.
  const int mine = (items - static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
  const int steps = mine * n;
  for (int i = 0; i < steps / S; ++i) static_for<S>(step);
  static_for<S>([&](auto U) __attribute__((always_inline)) {
    if (decltype(U)::value < steps % S) step(U);
  });
}

// ------------------------------------------------------------------- down --

// Column tiles of 16 that a wave works on at once, waves of a workgroup and
// ring depth in pairs. The hidden values of a chunk take 2 (16-bit weights), 4
// (FP8) or 8 (MXFP4) loads against one of the weights, so they are read once
// for four (eight) tiles; the experts are then split over workgroups instead of
// the columns, and a last kernel adds up the parts. 256 x 7168 x 2048 layer
// against one tile a wave: 16 tokens 610 -> 509 us (5.9 TB/s), one token 56 ->
// 47 us, 8 tokens on MXFP4 223 -> 103 us (four tiles: 116). The last kernel
// takes 4 to 5 us, most of it its launch; adding up in this one by the last
// workgroup of each column tile needs a fence over the XCDs in every workgroup
// and took 59 us against 10.6 + 3.9 on the 128 x 2048 x 768 layer.
template <int F>
constexpr int kDownTiles = F == kWMx ? 8 : 4;
constexpr int kDownWaves = 4;
constexpr int kDownFill = 512;            // workgroups that run at once: two on a CU
template <int F>
constexpr int kDownDepth = F == kW16 ? 3 : (F == kWFp8 ? 2 : 1);

template <int F>
struct DownSlot {
  u32x4 w[kDownTiles<F>][2];
  u32x4 h[2][lane_elems<F>() / 4];   // hw: fp32 (8 elements in 2), or the high parts, then the low parts
  u32x2 s[kDownTiles<F>];
};

template <int DT, int F>
__global__ __launch_bounds__(64 * kDownWaves, 2) void few_down_kernel(FewArgs a) {
  constexpr int EL = lane_elems<F>(), NX = EL / 8, S = kDownDepth<F>, NT = kDownTiles<F>, NW = kDownWaves;
  __shared__ Plan plan;
  __shared__ uint16_t pair[kMaxE * kRows];   // hw row of (distinct expert, token)
  __shared__ f32x4 red[NW][NT][64];
  const int tid = threadIdx.x, wave = uniform(tid >> 6), lane = tid & 63, lr = lane & 15, lg = lane >> 4;
  const int P = a.T * a.K;
  for (int p = tid; p < P; p += 64 * NW) {
    const int id = a.ids[p];
    plan.sid[p] = id >= 0 && id < a.E ? id : -1;
  }
  build_plan(plan, P, a.K, a.E, tid, 64 * NW);
  for (int i = tid; i < plan.count * kRows; i += 64 * NW) {
    const int e = plan.list[i / kRows];
    const uint32_t m = plan.mask[e];
    const int t = i % kRows;
    int p = kMaxP;                                  // not one of this expert's tokens
    if ((m >> t) & 1) {
      for (int k = a.K - 1; k >= 0; --k) {
        if (plan.sid[t * a.K + k] == e) p = t * a.K + k;
      }
    }
    pair[i] = static_cast<uint16_t>(p);
  }
  __syncthreads();

  const int col0 = blockIdx.x * (16 * NT);
  const int pairs = a.D / (8 * EL);                 // 128-byte pieces of a weight row
  const int64_t row_bytes = static_cast<int64_t>(a.D / EL) * 16;
  const int64_t blocks = a.D / 32;
  // This wave's share of the (expert, piece) stream.
  const int64_t total = static_cast<int64_t>(plan.count) * pairs;
  const int parts = gridDim.y * NW, part = blockIdx.y * NW + wave;
  const int u0 = static_cast<int>(total * part / parts);
  const int u1 = static_cast<int>(total * (part + 1) / parts);

  f32x4 sum[NT] = {}, acc[NT] = {};
  if (u0 < u1) {
    int l_j = u0 / pairs, l_c = u0 % pairs, l_left = u1 - u0;
    const uint8_t *pw = nullptr, *q = nullptr;
    const uint32_t w_off = static_cast<uint32_t>(lr * row_bytes) + lg * 16;
    const uint32_t s_off = F == kWFp8 ? lr * 4 : static_cast<uint32_t>(lr * blocks);
    const int64_t half = static_cast<int64_t>(P) * a.D * 2;
    const __amdgpu_buffer_rsrc_t hb = buffer_of(a.hw, hw_fp32<DT, F>() ? 2 * half : half);
    const __amdgpu_buffer_rsrc_t lb = buffer_of(a.hw + half, half);
    uint32_t h_off = 0;
    auto aim = [&]() __attribute__((always_inline)) {
      const int64_t row = static_cast<int64_t>(uniform(plan.list[l_j])) * a.H + col0;
      pw = a.wd + row * row_bytes;
      if constexpr (F != kW16) q = static_cast<const uint8_t*>(a.sd) + row * (F == kWFp8 ? 4 : blocks);
      const int p = pair[l_j * kRows + lr];
      h_off = p < kMaxP ? static_cast<uint32_t>(p * a.D + lg * EL) * (hw_fp32<DT, F>() ? 4 : 2) : kNoRow;
    };
    DownSlot<F> ring[S];
    auto load = [&](DownSlot<F>& s) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint8_t* w = pw + t * (16 * row_bytes) + static_cast<int64_t>(l_c) * 128;
        s.w[t][0] = *reinterpret_cast<const u32x4*>(w + w_off);
        s.w[t][1] = *reinterpret_cast<const u32x4*>(w + w_off + 64);
        if constexpr (F == kWFp8) s.s[t].x = *reinterpret_cast<const uint32_t*>(q + t * 64 + s_off);
        else if constexpr (F == kWMx) s.s[t] = *reinterpret_cast<const u32x2*>(q + t * 16 * blocks + l_c * 8 + s_off);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if constexpr (hw_fp32<DT, F>()) {
#pragma unroll
          for (int i = 0; i < 2; ++i) s.h[k][i] = buffer_load16(hb, h_off + 16 * i, (2 * l_c + k) * (16 * EL));
        } else {
#pragma unroll
          for (int i = 0; i < NX; ++i) {
            s.h[k][i] = buffer_load16(hb, h_off + 16 * i, (2 * l_c + k) * (8 * EL));
            s.h[k][NX + i] = buffer_load16(lb, h_off + 16 * i, (2 * l_c + k) * (8 * EL));
          }
        }
      }
      if (--l_left > 0) {
        if (++l_c == pairs) {
          l_c = 0;
          ++l_j;
          aim();
        }
      }          // else: the last pair is read again (in bounds, never used)
    };
    aim();
#pragma unroll
    for (int s = 0; s < S; ++s) load(ring[s]);
    int j = u0 / pairs, c = u0 % pairs, left = u1 - u0;
    auto step = [&](auto U) __attribute__((always_inline)) {
      constexpr int s = decltype(U)::value;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if constexpr (hw_fp32<DT, F>()) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t w = ring[s].w[t][k][i >> 1];
              acc[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(ring[s].h[k][i >> 2][i & 3]),
                                                            f16_to_float((i & 1) ? (w >> 16) : (w & 0xffffu)), acc[t],
                                                            0, 0, 0);
            }
          } else {
            u32x4 w[NX];
            decode<kBF16, F>(ring[s].w[t][k], pair_scale(ring[s].s[t], k, lg), w);
#pragma unroll
            for (int i = 0; i < NX; ++i) {
              acc[t] = mfma16<kBF16>(ring[s].h[k][i], w[i], acc[t]);
              acc[t] = mfma16<kBF16>(ring[s].h[k][NX + i], w[i], acc[t]);
            }
          }
        }
      }
      float scale[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) scale[t] = F == kWFp8 ? __uint_as_float(ring[s].s[t].x) : 1.0f;
      load(ring[s]);
      --left;
      if (++c == pairs || left == 0) {      // this wave's part of expert j is complete
        c = 0;
        const uint32_t m = static_cast<uint32_t>(uniform(plan.mask[plan.list[j]])) >> (lg * 4);
        ++j;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[t][i] += (m >> i) & 1 ? acc[t][i] * scale[t] : 0.0f;
          acc[t] = f32x4{};
        }
      }
    };
    const int mine = left;
    for (int i = 0; i < mine / S; ++i) static_for<S>(step);
    static_for<S>([&](auto U) __attribute__((always_inline)) {
      if (decltype(U)::value < mine % S) step(U);
    });
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) red[wave][t][lane] = sum[t];
  __syncthreads();
  const int t = lg * 4 + wave;             // register `wave` of lane `lane`
  if (t < a.T) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w) v += reinterpret_cast<const float*>(&red[w][nt][lane])[wave];
      const int64_t at = static_cast<int64_t>(t) * a.H + col0 + nt * 16 + lr;
      if (gridDim.y == 1) {
        static_cast<uint16_t*>(a.y)[at] = static_cast<uint16_t>(from_float<DT>(v));
      } else {
        a.parts[static_cast<int64_t>(blockIdx.y) * a.T * a.H + at] = v;
      }
    }
  }
}

// y = R(the sum of `count` parts [T, H], in order), four values a thread.
template <int DT>
__global__ __launch_bounds__(256) void few_combine_kernel(const float* __restrict__ parts, int count,
                                                          int64_t n, uint16_t* __restrict__ y) {
  const int64_t at = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (at >= n) return;
  f32x4 v = {};
#pragma unroll 4
  for (int g = 0; g < count; ++g) v += *reinterpret_cast<const f32x4*>(parts + g * n + at);
  *reinterpret_cast<u32x2*>(y + at) = u32x2{from_float<DT>(v[0]) | (from_float<DT>(v[1]) << 16),
                                           from_float<DT>(v[2]) | (from_float<DT>(v[3]) << 16)};
}

// ----------------------------------------------------------------- launch --

template <int DT>
void launch_logits(const FewProblem& p, hipStream_t st) {
  const uint16_t* x = static_cast<const uint16_t*>(p.x);
  auto go = [&](auto TT) {
    constexpr int tt = decltype(TT)::value;
    hipLaunchKernelGGL((few_logits_kernel<DT, tt>), dim3(p.E, (p.T + tt - 1) / tt), dim3(256), 0, st, x,
                       p.w_router, p.bias, p.T, p.H, p.E, p.logits);
  };
  if (p.T == 1) go(int_c<1>{});
  else if (p.T == 2) go(int_c<2>{});
  else go(int_c<4>{});
}

template <int DT, int F>
hipError_t launch_typed(const FewProblem& p, hipStream_t st) {
  FewArgs a{p.x, static_cast<const uint8_t*>(p.wg), static_cast<const uint8_t*>(p.wu),
            static_cast<const uint8_t*>(p.wd), p.sg, p.su, p.sd, nullptr, p.ids, p.weights,
            static_cast<uint8_t*>(p.hw), p.parts, p.y, p.T, p.H, p.D, p.E, p.K, p.renorm};
  if (p.w_router) {
    launch_logits<DT>(p, st);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    a.logits = p.logits;
  }
  // Items of the most experts there can be.
  const int most = p.T * p.K < p.E ? p.T * p.K : p.E;
  const int64_t items = static_cast<int64_t>(most) * (p.D / (16 * GateUpShape<F>::kTiles));
  constexpr int kFill = 256 * GateUpShape<F>::kWaves;     // workgroups that run at once
  const int grid = static_cast<int>(items < kFill ? items : kFill);
  hipLaunchKernelGGL((few_gate_up_kernel<DT, F>), dim3(grid), dim3(kGateUpThreads), 0, st, a);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const int tiles = p.H / (16 * kDownTiles<F>);
  const int64_t pieces = static_cast<int64_t>(most) * (p.D / (8 * lane_elems<F>()));
  int parts = kDownFill / tiles;
  // at least two pieces a wave; one part writes y itself
  if (parts > pieces / (2 * kDownWaves)) parts = static_cast<int>(pieces / (2 * kDownWaves));
  if (parts < 1) parts = 1;
  hipLaunchKernelGGL((few_down_kernel<DT, F>), dim3(tiles, parts), dim3(64 * kDownWaves), 0, st, a);
  err = hipGetLastError();
  if (err != hipSuccess || parts == 1) return err;
  const int64_t n = static_cast<int64_t>(p.T) * p.H;
  hipLaunchKernelGGL(few_combine_kernel<DT>, dim3(static_cast<unsigned>((n + 1023) / 1024)), dim3(256), 0,
                     st, p.parts, parts, n, static_cast<uint16_t*>(p.y));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_few(const FewProblem& p, hipStream_t st) {
  switch (p.fmt) {
    case kFewW16: return p.dtype == kBF16 ? launch_typed<kBF16, kW16>(p, st) : launch_typed<kF16, kW16>(p, st);
    case kFewFp8: return p.dtype == kBF16 ? launch_typed<kBF16, kWFp8>(p, st) : launch_typed<kF16, kWFp8>(p, st);
    default: return p.dtype == kBF16 ? launch_typed<kBF16, kWMx>(p, st) : launch_typed<kF16, kWMx>(p, st);
  }
}

}  // namespace moe
