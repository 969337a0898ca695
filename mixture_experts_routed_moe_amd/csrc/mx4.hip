// Microscaled 4-bit experts on both sides: MXFP4 weights against MXFP4
// activations on v_mfma_scale_f32_16x16x128_f8f6f4 (E2M1 elements, one E8M0
// scale per 32 along the reduction, as the OCP Microscaling specification
// v1.0 defines them).
//
//   gate/up: g = xq W_gate^T, u = xq W_up^T (fp32), hq, hs = MXFP4(SiLU(g) * u)
//   down:    expert_out = R(hq W_down^T)
//
// The hidden values go from the fp32 accumulators to MXFP4 codes in the
// epilogue: they are rounded once, and neither a 16-bit h nor a quantising
// pass over it exists (at T = 4096, H = 7168, D = 2048 that pass moved 134 MB
// twice).
//
// Operands. The weights are the MFMA's first operand and the activations its
// second, so a lane's result registers hold 4 neighbouring output columns of
// ONE row, and the 32-column block that shares a scale lies in the 4 lanes of
// a row and two tiles: its largest magnitude takes 7 in-lane maxima and two
// exchanges. Lane group g (of 16 lanes) holds elements 32g .. 32g + 31 of the
// instruction's 128: a load instruction reads 64 contiguous bytes of each of
// 16 rows, and the two halves of a 128-byte line are loaded right after one
// another. (With the 32x32x64 instruction a load reads 16-byte pieces of 32
// lines and each line is asked for four times; the first-level cache stalls on
// a line that is still on its way: T = 4096 gate/up 1376 us, T = 512 890 us
// against FIG1 and FIG2 here.)
//
// Scales: a lane's byte of a row's 4 is moved down by a shift, 16 bytes (two
// pairs of chunks) of a row are loaded at once: rows of scales are short
// strips of lines, and with one load a chunk each line was fetched again for
// every chunk.
//
// Bound: the weight stream (a prefill expert of ~128 rows needs 8 x 16 cycles
// of MFMA a 1 KB weight load, a third of the time HBM takes to deliver it).
// Weights go from memory into a register ring; a workgroup of 4 waves shares
// the activation rows through double-buffered LDS, staged through registers as
// many pairs ahead as the weights are loaded (loads complete in order: waiting
// for a late-issued activation would wait for every weight before it). One
// pass takes up to 16 * NBMAX rows, so an expert's weights are read once.

#include "common.hpp"
#include "launch.hpp"

namespace moe {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kPair = 256;                // reduction elements of a pair of chunks
constexpr int kRowBytes = kPair / 2;      // of one row: a 128-byte line
constexpr int kLdsRow = kRowBytes + 16;   // padded: 8 rows' 16-byte reads cover all banks
constexpr int kBlk = 32;
constexpr int kPairScales = kPair / kBlk;
constexpr int kTiles = 4;                 // weight tiles of 16 rows a wave

// A (weights) and B (activations) E2M1: format code 4, four of the eight
// operand registers in use; the lowest byte of each scale register.
__device__ __forceinline__ f32x4 mfma_mx4(const u32x4& a, const u32x4& b, uint32_t sa, uint32_t sb,
                                          f32x4 c) {
  const i32x8 aa = {static_cast<int>(a.x), static_cast<int>(a.y), static_cast<int>(a.z),
                    static_cast<int>(a.w), 0, 0, 0, 0};
  const i32x8 bb = {static_cast<int>(b.x), static_cast<int>(b.y), static_cast<int>(b.z),
                    static_cast<int>(b.w), 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(aa, bb, c, 4, 4, 0, static_cast<int>(sa), 0,
                                                           static_cast<int>(sb));
}

struct Mx4Args {
  const uint8_t* a;         // gate/up: xq [T, kd/2]; down: hq [P, kd/2]
  const uint8_t* as;        // E8M0 [rows, kd/32]
  const uint8_t *b0, *b1;   // [E, n, kd/2]
  const uint8_t *s0, *s1;   // [E, n, kd/32]
  uint8_t *hq, *hs;         // gate/up: [P, n/2], [P, n/32]
  uint16_t* out;            // down: [P, n]
  const int32_t* sorted_token;
  const int32_t* group_sizes;
  const int32_t* group_offsets;
  const int32_t* group_padded_offsets;
  const int32_t* block_expert;
  const int32_t* active_blocks;
  const int32_t* active_count;
  int n, kd, block_m, n_tiles, tokens;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, static_cast<int>(bytes), 0x00027000);
}
// 16 bytes at lane_off + wave_off; what lies past the buffer reads as zeros
// (the second pair of scales of a row's last pair).
__device__ __forceinline__ u32x4 buffer_load16(__amdgpu_buffer_rsrc_t b, uint32_t lane_off, int wave_off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, static_cast<int>(lane_off), wave_off, 0));
}

template <int NS>
struct Mx4Slot {
  u32x4 w[kTiles][2];       // the lane's weight rows, both halves of the line
  u32x4 a[NS];              // this thread's 16 bytes of activation rows tid / 8 + 32 q
};

template <int NBMAX>
struct Mx4Lds {
  static constexpr int kRows = (16 * NBMAX + 31) / 32 * 32;
  uint8_t row[2][kRows][kLdsRow];
  u32x4 scale[2][kThreads];   // 16 bytes of row tid, two pairs; one a thread (rows past the pass
                              // among them): a branch in the step would let the compiler sink the
                              // MFMAs past the next loads
};

// Where a pass reads: wave-uniform addresses that walk along the reduction, and
// fixed 32-bit lane offsets.
struct Mx4Walk {
  const uint8_t* w[kTiles];           // the weight tiles' first rows
  const uint8_t* a;                   // activations
  __amdgpu_buffer_rsrc_t s01, s23, as;  // scales of weight tiles 0 and 1, 2 and 3, of the activations
};

// One pass over the reduction for NB groups of 16 activation rows. a_off /
// as_off: this thread's staging offsets. Pairs are taken two at a time (one
// 16-byte load of scales); np >= 1 of them.
template <int NB, int NBMAX, int S>
__device__ __forceinline__ void mx4_pass(Mx4Walk p, uint32_t w_off, uint32_t s_off, int tile_scales,
                                         const uint32_t* a_off, uint32_t as_off, int np, int tid,
                                         int lr, int lg, Mx4Lds<NBMAX>& lds, f32x4 (*acc)[kTiles]) {
  static_assert(S == 2 || S == 4, "a slot's parity is its pair's");
  constexpr int NS = (NB + 1) / 2;
#pragma unroll
  for (int q = 0; q < NB; ++q) {
#pragma unroll
    for (int t = 0; t < kTiles; ++t) acc[q][t] = f32x4{};
  }
  Mx4Slot<NS> ring[S];
  u32x4 sw[kTiles], sw_next[kTiles], sa_next;
  int left = np - 1;
  auto load = [&](Mx4Slot<NS>& s) __attribute__((always_inline)) {
    // activations first: they are waited for a step earlier
#pragma unroll
    for (int q = 0; q < NS; ++q) s.a[q] = *reinterpret_cast<const u32x4*>(p.a + a_off[q]);
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      s.w[t][0] = *reinterpret_cast<const u32x4*>(p.w[t] + w_off);
      s.w[t][1] = *reinterpret_cast<const u32x4*>(p.w[t] + w_off + 64);
    }
    // Past the end the last pair is read again (in bounds, never used): every
    // step issues the same loads, which the compiler's wait counts rely on.
    const int64_t on = left > 0 ? kRowBytes : 0;
    --left;
    p.a += on;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) p.w[t] += on;
  };
  auto load_scales = [&](int pair) __attribute__((always_inline)) {
    const int at = (pair < np ? pair : 0) * kPairScales;
    sa_next = buffer_load16(p.as, as_off, at);
    sw_next[0] = buffer_load16(p.s01, s_off, at);
    sw_next[1] = buffer_load16(p.s01, s_off, at + tile_scales);
    sw_next[2] = buffer_load16(p.s23, s_off, at);
    sw_next[3] = buffer_load16(p.s23, s_off, at + tile_scales);
  };
  auto stage = [&](const Mx4Slot<NS>& s, int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < NS; ++q) {
      *reinterpret_cast<u32x4*>(&lds.row[buf][(tid >> 3) + 32 * q][(tid & 7) * 16]) = s.a[q];
    }
  };
  load_scales(0);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int s = 0; s < S; ++s) {
    load(ring[s]);
    __builtin_amdgcn_sched_barrier(0);
  }
  stage(ring[0], 0);
  lds.scale[0][tid] = sa_next;
#pragma unroll
  for (int t = 0; t < kTiles; ++t) sw[t] = sw_next[t];
  wait_lds();
  barrier_no_wait();

  // Pair `pair` of slot u; PH: its place in the group of two pairs; g: the group's LDS buffer.
  auto step = [&](int pair, auto U, int g) __attribute__((always_inline)) {
    constexpr int u = decltype(U)::value, ph = u & 1;
    if constexpr (ph == 0) load_scales(pair + 2);
    u32x2 sb[NB];                          // this pair's scale words of each activation row
    constexpr int F = 2 * NB;              // fragments: half k, row group q
    u32x4 frag[3];
    auto read = [&](int f) __attribute__((always_inline)) {
      const int k = f / NB, q = f % NB;
      if (k == 0) sb[q] = reinterpret_cast<const u32x2*>(&lds.scale[g][16 * q + lr])[ph];
      return *reinterpret_cast<const u32x4*>(&lds.row[ph][16 * q + lr][k * 64 + lg * 16]);
    };
    frag[0] = read(0);
    if constexpr (F > 1) frag[1] = read(1);
    __builtin_amdgcn_sched_barrier(0);
    uint32_t wa[2][kTiles];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      wa[0][t] = sw[t][2 * ph] >> (8 * lg);
      wa[1][t] = sw[t][2 * ph + 1] >> (8 * lg);
    }
    static_for<F>([&](auto I) __attribute__((always_inline)) {
      constexpr int f = decltype(I)::value, k = f / NB, q = f % NB;
      if constexpr (f + 2 < F) frag[(f + 2) % 3] = read(f + 2);
      const uint32_t sc = sb[q][k] >> (8 * lg);
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        acc[q][t] = mfma_mx4(ring[u].w[t][k], frag[f % 3], wa[k][t], sc, acc[q][t]);
      }
      // Keep reads and MFMAs in this order: left free, the compiler sinks the
      // MFMAs past the next step's loads and copies the ring.
      __builtin_amdgcn_sched_barrier(0);
    });
    stage(ring[(u + 1) % S], ph ^ 1);
    if constexpr (ph == 1) {
      lds.scale[g ^ 1][tid] = sa_next;
#pragma unroll
      for (int t = 0; t < kTiles; ++t) sw[t] = sw_next[t];
    }
    load(ring[u]);
    wait_lds();
    barrier_no_wait();
  };
  int c0 = 0;
  for (; c0 + S <= np; c0 += S) {
    static_for<S>([&](auto U) __attribute__((always_inline)) {
      constexpr int u = decltype(U)::value;
      step(c0 + u, U, ((c0 + u) >> 1) & 1);
    });
  }
  const int rest = np - c0;
  static_for<S>([&](auto U) __attribute__((always_inline)) {
    constexpr int u = decltype(U)::value;
    if (u < rest) step(c0 + u, U, ((c0 + u) >> 1) & 1);
  });
}

// hq / hs of one 16-row group: lane (lr, lg) holds columns 4 lg + 0..3 of both
// 16-column tiles for activation row lr.
__device__ __forceinline__ void store_mxfp4(const f32x4* g, const f32x4* u, int lg, bool live,
                                            uint8_t* codes, uint8_t* scale) {
  float v[8];
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = silu(g[i >> 2][i & 3]) * u[i >> 2][i & 3];
    amax = fmaxf(amax, fabsf(v[i]));
  }
  amax = fmaxf(amax, __shfl_xor(amax, 16));
  amax = fmaxf(amax, __shfl_xor(amax, 32));
  const int e = mx_scale_exp(amax, 2);
  const float X = ldexpf(1.0f, e - 127);
  uint32_t q0 = 0u;                         // tile 0's four codes, then tile 1's
#pragma unroll
  for (int i = 0; i < 8; ++i) q0 |= float_to_fp4e2m1(v[i] / X) << (4 * i);
  const uint32_t q1 = __shfl_xor(q0, 16), q2 = __shfl_xor(q0, 32), q3 = __shfl_xor(q0, 48);
  if (live && lg == 0) {                    // lane group 0: q1, q2, q3 are groups 1, 2, 3
    *reinterpret_cast<u32x4*>(codes) = u32x4{(q0 & 0xffffu) | (q1 << 16), (q2 & 0xffffu) | (q3 << 16),
                                             (q0 >> 16) | (q1 & 0xffff0000u), (q2 >> 16) | (q3 & 0xffff0000u)};
    *scale = static_cast<uint8_t>(e);
  }
}

// gate/up: wave w owns columns 128 nt + 32 w + 0..31 of W_gate (tiles 0, 1) and
// W_up (tiles 2, 3); down: columns 256 nt + 64 w + 0..63 of W_down.
template <int DT, bool GATEUP, int NBMAX, int S, int WAVES>
__global__ __launch_bounds__(kThreads, WAVES) void mx4_grouped_kernel(Mx4Args g) {
  __shared__ __attribute__((aligned(16))) Mx4Lds<NBMAX> lds;
  const int total = g.active_count[0] * g.n_tiles;
  const int per_xcd = (total + 7) >> 3;
  const int natural = (blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);
  if (static_cast<int>(blockIdx.x >> 3) >= per_xcd || natural >= total) return;
  const int ab = natural / g.n_tiles;
  const int nt = natural - ab * g.n_tiles;
  const int bx = g.active_blocks[ab];
  const int e = g.block_expert[bx];
  const int row_in_group = bx * g.block_m - g.group_padded_offsets[e];
  const int rows = min(g.block_m, g.group_sizes[e] - row_in_group);
  if (rows <= 0) return;
  const int64_t m_start = g.group_offsets[e] + row_in_group;

  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = tid & 15, lg = (tid >> 4) & 3;
  const int64_t half = g.kd / 2, kb = g.kd / kBlk;
  const int col0 = GATEUP ? nt * 128 + wave * 32 : nt * 256 + wave * 64;
  const int64_t wrow = static_cast<int64_t>(e) * g.n + col0;
  Mx4Walk walk;
  if constexpr (GATEUP) {
    walk.w[0] = g.b0 + wrow * half;
    walk.w[2] = g.b1 + wrow * half;
    walk.s01 = buffer_of(g.s0 + wrow * kb, 32 * kb);
    walk.s23 = buffer_of(g.s1 + wrow * kb, 32 * kb);
  } else {
    walk.w[0] = g.b0 + wrow * half;
    walk.w[2] = walk.w[0] + 32 * half;
    walk.s01 = buffer_of(g.s0 + wrow * kb, 32 * kb);
    walk.s23 = buffer_of(g.s0 + (wrow + 32) * kb, 32 * kb);
  }
  walk.w[1] = walk.w[0] + 16 * half;
  walk.w[3] = walk.w[2] + 16 * half;
  const uint32_t w_off = static_cast<uint32_t>(lr * half) + lg * 16;
  const uint32_t s_off = static_cast<uint32_t>(lr * kb);
  const int np = g.kd / kPair;

  // passes of equal height
  const int passes = (rows + 16 * NBMAX - 1) / (16 * NBMAX);
  const int height = ((rows + passes - 1) / passes + 15) / 16 * 16;
  for (int r0 = 0; r0 < rows; r0 += height) {
    if (r0 > 0) __syncthreads();
    const int rows_pass = min(height, rows - r0);
    auto source = [&](int r) __attribute__((always_inline)) {
      if (r >= rows_pass) r = 0;                  // in bounds; its results are never stored
      return static_cast<int64_t>(GATEUP ? g.sorted_token[m_start + r0 + r] : r);
    };
    constexpr int kStage = (NBMAX + 1) / 2;
    uint32_t a_off[kStage];
#pragma unroll
    for (int q = 0; q < kStage; ++q) {
      a_off[q] = static_cast<uint32_t>(source((tid >> 3) + 32 * q) * half) + (tid & 7) * 16;
    }
    const uint32_t as_off = static_cast<uint32_t>(source(tid) * kb);
    const int64_t first = GATEUP ? 0 : m_start + r0;
    walk.a = g.a + first * half;
    walk.as = buffer_of(g.as + first * kb, (GATEUP ? g.tokens : rows_pass) * kb);
    f32x4 acc[NBMAX][kTiles];
    auto run = [&](auto NBC) __attribute__((always_inline)) {
      constexpr int nb = decltype(NBC)::value;
      mx4_pass<nb, NBMAX, S>(walk, w_off, s_off, static_cast<int>(16 * kb), a_off, as_off, np, tid, lr, lg, lds, acc);
#pragma unroll
      for (int q = 0; q < nb; ++q) {
        const int row = 16 * q + lr;
        const bool live = row < rows_pass;
        const int64_t at = m_start + r0 + row;
        if constexpr (GATEUP) {
          store_mxfp4(acc[q], acc[q] + 2, lg, live, g.hq + at * (g.n / 2) + col0 / 2,
                      g.hs + at * (g.n / kBlk) + col0 / kBlk);
        } else if (live) {
#pragma unroll
          for (int t = 0; t < kTiles; ++t) {
            const f32x4& v = acc[q][t];
            const u32x2 o = {from_float<DT>(v[0]) | (from_float<DT>(v[1]) << 16),
                             from_float<DT>(v[2]) | (from_float<DT>(v[3]) << 16)};
            *reinterpret_cast<u32x2*>(g.out + at * g.n + col0 + 16 * t + 4 * lg) = o;
          }
        }
      }
    };
    // the row groups of this pass, 1 or rounded up to an even number
    const int groups = (rows_pass + 15) >> 4;
    if (groups == 1) {
      run(int_c<1>{});
    } else {
      static_for<NBMAX / 2>([&](auto I) __attribute__((always_inline)) {
        constexpr int nb = 2 * decltype(I)::value + 2;
        if ((groups + 1) / 2 * 2 == nb) run(int_c<nb>{});
      });
    }
  }
}

template <int DT, bool GATEUP>
hipError_t launch_grouped(const Mx4GemmProblem& p, const moe_tables& t, hipStream_t stream) {
  Mx4Args g{p.a, p.as, p.b0, p.b1, p.s0, p.s1, p.hq, p.hs, static_cast<uint16_t*>(p.out),
            t.sorted_token, t.group_sizes, t.group_offsets, t.group_padded_offsets, t.block_expert,
            t.active_blocks, t.active_count, p.n, p.kd, t.block_m, p.n / (GATEUP ? 128 : 256), t.T};
  const int64_t total = static_cast<int64_t>(t.num_blocks) * g.n_tiles;
  const dim3 grid(static_cast<unsigned>((total + 7) / 8 * 8));
  auto go = [&](auto NB, auto S, auto WAVES) {
    hipLaunchKernelGGL((mx4_grouped_kernel<DT, GATEUP, decltype(NB)::value, decltype(S)::value, decltype(WAVES)::value>),
                       grid, dim3(kThreads), 0, stream, g);
  };
  if (t.block_m == 16) {
    go(int_c<1>{}, int_c<2>{}, int_c<2>{});
  } else if (t.block_m == 32) {
    go(int_c<2>{}, int_c<2>{}, int_c<2>{});
  } else if (t.block_m == 64) {
    go(int_c<4>{}, int_c<2>{}, int_c<2>{});
  } else if (t.block_m == 128) {
    go(int_c<8>{}, int_c<2>{}, int_c<1>{});
  } else {
    go(int_c<12>{}, int_c<2>{}, int_c<1>{});
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gate_up_mx4(const Mx4GemmProblem& p, const moe_tables& t, hipStream_t stream) {
  return launch_grouped<kBF16, true>(p, t, stream);
}

hipError_t launch_down_mx4(const Mx4GemmProblem& p, const moe_tables& t, hipStream_t stream) {
  if (p.dtype == kBF16) return launch_grouped<kBF16, false>(p, t, stream);
  return launch_grouped<kF16, false>(p, t, stream);
}

}  // namespace moe
