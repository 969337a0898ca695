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
// against 938 and 679 here.)
//
// Scales: a row's bytes are loaded 64 at a time (eight pairs of chunks), go
// through LDS, and a lane moves its byte of each 4 down by a shift. Rows of
// scales are short strips of lines that the first-level cache does not keep
// between two pairs: loaded 8 or 16 bytes at a time they cost T = 512 gate/up
// 818 or 737 us, against 694 us so (679 with the single buffer below).
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
#include "mx_codes.hpp"

namespace moe {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kPair = 256;                // reduction elements of a pair of chunks
constexpr int kRowBytes = kPair / 2;      // of one row: a 128-byte line
constexpr int kLdsRow = kRowBytes + 16;   // padded: 8 rows' 16-byte reads cover all banks
constexpr int kBlk = 32;
constexpr int kPairScales = kPair / kBlk;
constexpr int kStrip = 8;                 // pairs whose scales are loaded at once: 64 bytes a row
constexpr int kScaleRow = 64 + 16;        // of them in LDS, padded

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

// Shape of a workgroup: NW waves, TILES weight tiles of 16 rows a wave, passes
// of up to 16 NBMAX activation rows.
template <int NW, int TILES, int NBMAX>
struct Mx4Shape {
  static constexpr int kThreads = 64 * NW;
  static constexpr int kStageRows = kThreads / 8;      // activation rows staged by one load a thread
  static constexpr int stages(int nb) { return (16 * nb + kStageRows - 1) / kStageRows; }
  static constexpr int kRows = stages(NBMAX) * kStageRows;
  static constexpr int scale_loads(int nb) { return (16 * nb + kThreads / 4 - 1) / (kThreads / 4); }
  static constexpr int kScaleRows = scale_loads(NBMAX) * (kThreads / 4);
  static constexpr int kWeightRows = kThreads / 64 * 16 * TILES;
  // A wave alone writes and reads its weights' scales, so one buffer of them is
  // enough and lighter on LDS (two -> one: T = 512 697 + 418 -> 679 + 411 us,
  // T = 1024 in blocks of 64 723 + 441 -> 715 + 436). Two leave the compiler more
  // room between a strip's writes and its reads, which tall passes need (T =
  // 4096: 938 + 613 us, with one 1088 + 734) and single groups gain a little
  // from (128 x 2048 x 768, T = 67: gate/up 42.8, 43.7 us).
  static constexpr int kWeightBufs = NBMAX == 1 || NBMAX >= 8 ? 2 : 1;
};

template <int NS, int TILES>
struct Mx4Slot {
  u32x4 w[TILES][2];        // the lane's weight rows, both halves of the line
  u32x4 a[NS];              // this thread's 16 bytes of activation rows tid / 8 + kStageRows q
};

template <typename SH>
struct Mx4Lds {
  uint8_t row[2][SH::kRows][kLdsRow];
  uint8_t as[2][SH::kScaleRows][kScaleRow];    // scales of the activation rows
  uint8_t ws[SH::kWeightBufs][SH::kWeightRows][kScaleRow];   // and of every wave's weight rows
};

// Where a pass reads: wave-uniform addresses that walk along the reduction, and
// fixed 32-bit lane offsets.
template <int TILES>
struct Mx4Walk {
  const uint8_t* w[TILES];            // the weight tiles' first rows
  const uint8_t* a;                   // activations
  __amdgpu_buffer_rsrc_t s0, s1, as;  // scales of the lower and upper half of the weight tiles, of the activations
};

// One pass over the reduction for NB groups of 16 activation rows. a_off /
// as_off: this thread's staging offsets; np >= 1 pairs.
template <int NB, typename SH, int TILES, int S>
__device__ __forceinline__ void mx4_pass(Mx4Walk<TILES> p, uint32_t w_off, uint32_t s_off, int tile_scales,
                                         const uint32_t* a_off, const uint32_t* as_off, int np, int tid,
                                         int lr, int lg, Mx4Lds<SH>& lds, f32x4 (*acc)[TILES]) {
  constexpr int NS = SH::stages(NB), H = TILES / 2;
#pragma unroll
  for (int q = 0; q < NB; ++q) {
#pragma unroll
    for (int t = 0; t < TILES; ++t) acc[q][t] = f32x4{};
  }
  Mx4Slot<NS, TILES> ring[S];
  u32x4 sw_next[TILES], sa_next[SH::scale_loads(NB)];
  const int wave = tid >> 6;
  int left = np - 1;
  auto load = [&](Mx4Slot<NS, TILES>& s) __attribute__((always_inline)) {
    // activations first: they are waited for a step earlier
#pragma unroll
    for (int q = 0; q < NS; ++q) s.a[q] = *reinterpret_cast<const u32x4*>(p.a + a_off[q]);
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      s.w[t][0] = *reinterpret_cast<const u32x4*>(p.w[t] + w_off);
      s.w[t][1] = *reinterpret_cast<const u32x4*>(p.w[t] + w_off + 64);
    }
    // Past the end the last pair is read again (in bounds, never used): every
    // step issues the same loads, which the compiler's wait counts rely on.
    const int64_t on = left > 0 ? kRowBytes : 0;
    --left;
    p.a += on;
#pragma unroll
    for (int t = 0; t < TILES; ++t) p.w[t] += on;
  };
  // Scales of the strip of eight pairs from `pair` on: lane group lg 16 bytes of each weight row,
  // four threads a row of the activations.
  auto load_scales = [&](int pair) __attribute__((always_inline)) {
    const int at = (pair < np ? pair : 0) * kPairScales;
#pragma unroll
    for (int q = 0; q < SH::scale_loads(NB); ++q) sa_next[q] = buffer_load16(p.as, as_off[q], at);
#pragma unroll
    for (int t = 0; t < H; ++t) {
      sw_next[t] = buffer_load16(p.s0, s_off, at + t * tile_scales);
      sw_next[H + t] = buffer_load16(p.s1, s_off, at + t * tile_scales);
    }
  };
  auto stage_scales = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < SH::scale_loads(NB); ++q) {
      *reinterpret_cast<u32x4*>(&lds.as[buf][(tid >> 2) + SH::kThreads / 4 * q][(tid & 3) * 16]) = sa_next[q];
    }
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      *reinterpret_cast<u32x4*>(&lds.ws[buf % SH::kWeightBufs][(wave * TILES + t) * 16 + lr][lg * 16]) = sw_next[t];
    }
  };
  auto stage = [&](const Mx4Slot<NS, TILES>& s, int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < NS; ++q) {
      *reinterpret_cast<u32x4*>(&lds.row[buf][(tid >> 3) + SH::kStageRows * q][(tid & 7) * 16]) = s.a[q];
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
  stage_scales(0);
  wait_lds();
  barrier_no_wait();

  // Pair V of a strip, in slot V % S; g: the strip's LDS buffer of scales.
  auto step = [&](int pair, auto VV, int g) __attribute__((always_inline)) {
    constexpr int V = decltype(VV)::value, u = V % S, ph = V & 1;
    if constexpr (V == 0) load_scales(pair + kStrip);
    u32x2 sb[NB];                          // this pair's scale words of each activation row
    constexpr int F = 2 * NB;              // fragments: half k, row group q
    u32x4 frag[3];
    auto read = [&](int f) __attribute__((always_inline)) {
      const int k = f / NB, q = f % NB;
      if (k == 0) sb[q] = *reinterpret_cast<const u32x2*>(&lds.as[g][16 * q + lr][V * kPairScales]);
      return *reinterpret_cast<const u32x4*>(&lds.row[ph][16 * q + lr][k * 64 + lg * 16]);
    };
    frag[0] = read(0);
    if constexpr (F > 1) frag[1] = read(1);
    __builtin_amdgcn_sched_barrier(0);
    uint32_t wa[2][TILES];
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      const u32x2 sw = *reinterpret_cast<const u32x2*>(&lds.ws[g % SH::kWeightBufs][(wave * TILES + t) * 16 + lr][V * kPairScales]);
      wa[0][t] = sw.x >> (8 * lg);
      wa[1][t] = sw.y >> (8 * lg);
    }
    static_for<F>([&](auto I) __attribute__((always_inline)) {
      constexpr int f = decltype(I)::value, k = f / NB, q = f % NB;
      if constexpr (f + 2 < F) frag[(f + 2) % 3] = read(f + 2);
      const uint32_t sc = sb[q][k] >> (8 * lg);
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        acc[q][t] = mfma_mx4(ring[u].w[t][k], frag[f % 3], wa[k][t], sc, acc[q][t]);
      }
      // Keep reads and MFMAs in this order: left free, the compiler sinks the
      // MFMAs past the next step's loads and copies the ring.
      __builtin_amdgcn_sched_barrier(0);
    });
    stage(ring[(u + 1) % S], ph ^ 1);
    if constexpr (V == kStrip - 1) stage_scales(g ^ 1);
    load(ring[u]);
    wait_lds();
    barrier_no_wait();
  };
  int c0 = 0, g = 0;
  for (; c0 + kStrip <= np; c0 += kStrip, g ^= 1) {
    static_for<kStrip>([&](auto V) __attribute__((always_inline)) { step(c0 + decltype(V)::value, V, g); });
  }
  const int rest = np - c0;
  static_for<kStrip - 1>([&](auto V) __attribute__((always_inline)) {
    if (decltype(V)::value < rest) step(c0 + decltype(V)::value, V, g);
  });
}

// SiLU by the hardware's exp2 and reciprocal (1 ulp each; the argument's
// rounding makes it |g| 2^-24 relative): the result is rounded to 4 bits, and
// the library's expf and division took a tenth of the T = 4096 kernel.
__device__ __forceinline__ float silu_fast(float g) {
  return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * g));
}

// Wave w of a workgroup owns, with C = 8 TILES columns: gate/up columns (nt NW +
// w) C + 0..C-1 of W_gate (the lower half of its tiles) and W_up (the upper
// half); down columns 2 C (nt NW + w) + 0..2C-1 of W_down.
template <int DT, bool GATEUP, int NBMAX, int NW, int TILES, int S, int WAVES>
__global__ __launch_bounds__(64 * NW, WAVES) void mx4_grouped_kernel(Mx4Args g) {
  using SH = Mx4Shape<NW, TILES, NBMAX>;
  constexpr int H = TILES / 2;
  static_assert(H == 2, "a wave's gate and up tiles cover one 32-column block");
  __shared__ __attribute__((aligned(16))) Mx4Lds<SH> lds;
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
  const int col0 = (nt * NW + wave) * (GATEUP ? 16 * H : 16 * TILES);
  const int64_t wrow = static_cast<int64_t>(e) * g.n + col0;
  Mx4Walk<TILES> walk;
  const uint8_t* upper = GATEUP ? g.b1 + wrow * half : g.b0 + (wrow + 16 * H) * half;
#pragma unroll
  for (int t = 0; t < H; ++t) {
    walk.w[t] = g.b0 + (wrow + 16 * t) * half;
    walk.w[H + t] = upper + 16 * t * half;
  }
  walk.s0 = buffer_of(g.s0 + wrow * kb, 16 * H * kb);
  walk.s1 = buffer_of(GATEUP ? g.s1 + wrow * kb : g.s0 + (wrow + 16 * H) * kb, 16 * H * kb);
  const uint32_t w_off = static_cast<uint32_t>(lr * half) + lg * 16;
  const uint32_t s_off = static_cast<uint32_t>(lr * kb) + lg * 16;
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
    constexpr int kStages = SH::stages(NBMAX);
    uint32_t a_off[kStages];
#pragma unroll
    for (int q = 0; q < kStages; ++q) {
      a_off[q] = static_cast<uint32_t>(source((tid >> 3) + SH::kStageRows * q) * half) + (tid & 7) * 16;
    }
    uint32_t as_off[SH::scale_loads(NBMAX)];
#pragma unroll
    for (int q = 0; q < SH::scale_loads(NBMAX); ++q) {
      as_off[q] = static_cast<uint32_t>(source((tid >> 2) + SH::kThreads / 4 * q) * kb) + (tid & 3) * 16;
    }
    const int64_t first = GATEUP ? 0 : m_start + r0;
    walk.a = g.a + first * half;
    walk.as = buffer_of(g.as + first * kb, (GATEUP ? g.tokens : rows_pass) * kb);
    f32x4 acc[NBMAX][TILES];
    auto run = [&](auto NBC) __attribute__((always_inline)) {
      constexpr int nb = decltype(NBC)::value;
      mx4_pass<nb, SH, TILES, S>(walk, w_off, s_off, static_cast<int>(16 * kb), a_off, as_off, np, tid, lr, lg, lds, acc);
      if constexpr (GATEUP) {
        // The hidden values take the gate's registers; a 32-column block is the wave's two tiles of a
        // row, its amax over the row's 4 lanes.
#pragma unroll
        for (int q = 0; q < nb; ++q) {
          const int row = 16 * q + lr;
          float amax = 0.0f;
#pragma unroll
          for (int t = 0; t < H; ++t) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              acc[q][t][i] = silu_fast(acc[q][t][i]) * acc[q][H + t][i];
              amax = fmaxf(amax, fabsf(acc[q][t][i]));
            }
          }
          amax = fmaxf(amax, __shfl_xor(amax, 16));
          amax = fmaxf(amax, __shfl_xor(amax, 32));
          const int e8 = mx_scale_exp(amax, 2);
          const float X = ldexpf(1.0f, e8 - 127);
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = acc[q][i >> 2][i & 3];
          const uint32_t q0 = pk8_fp4e2m1(v, X);           // 16 bits a tile
          const uint32_t q1 = __shfl_xor(q0, 16), q2 = __shfl_xor(q0, 32), q3 = __shfl_xor(q0, 48);
          if (row < rows_pass && lg == 0) {     // lane group 0 collects the row: q1, q2, q3 are groups 1, 2, 3
            const int64_t at = m_start + r0 + row;
            uint8_t* codes = g.hq + at * (g.n / 2) + col0 / 2;
            const uint32_t c0 = (q0 & 0xffffu) | (q1 << 16), c1 = (q2 & 0xffffu) | (q3 << 16);
            *reinterpret_cast<u32x4*>(codes) = u32x4{c0, c1, (q0 >> 16) | (q1 & 0xffff0000u), (q2 >> 16) | (q3 & 0xffff0000u)};
            g.hs[at * (g.n / kBlk) + col0 / kBlk] = static_cast<uint8_t>(e8);
          }
        }
      } else {
#pragma unroll
        for (int q = 0; q < nb; ++q) {
          const int row = 16 * q + lr;
          if (row >= rows_pass) continue;
          uint16_t* out = g.out + (m_start + r0 + row) * g.n + col0 + 4 * lg;
#pragma unroll
          for (int t = 0; t < TILES; ++t) {
            const f32x4& v = acc[q][t];
            *reinterpret_cast<u32x2*>(out + 16 * t) = u32x2{from_float<DT>(v[0]) | (from_float<DT>(v[1]) << 16),
                                                            from_float<DT>(v[2]) | (from_float<DT>(v[3]) << 16)};
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

template <int DT, bool GATEUP, int NBMAX, int NW, int TILES, int S, int WAVES>
hipError_t launch_shape(Mx4Args g, const moe_tables& t, hipStream_t stream) {
  g.n_tiles = g.n / (NW * TILES * (GATEUP ? 8 : 16));
  const int64_t total = static_cast<int64_t>(t.num_blocks) * g.n_tiles;
  const dim3 grid(static_cast<unsigned>((total + 7) / 8 * 8));
  hipLaunchKernelGGL((mx4_grouped_kernel<DT, GATEUP, NBMAX, NW, TILES, S, WAVES>), grid, dim3(64 * NW), 0, stream, g);
  return hipGetLastError();
}

template <int DT, bool GATEUP>
hipError_t launch_grouped(const Mx4GemmProblem& p, const moe_tables& t, hipStream_t stream) {
  const Mx4Args g{p.a, p.as, p.b0, p.b1, p.s0, p.s1, p.hq, p.hs, static_cast<uint16_t*>(p.out),
                  t.sorted_token, t.group_sizes, t.group_offsets, t.group_padded_offsets, t.block_expert,
                  t.active_blocks, t.active_count, p.n, p.kd, t.block_m, 0, t.T};
  switch (t.block_m) {
    case 16: return launch_shape<DT, GATEUP, 1, 4, 4, 2, 2>(g, t, stream);
    case 32: return launch_shape<DT, GATEUP, 2, 4, 4, 2, 2>(g, t, stream);
    case 64: return launch_shape<DT, GATEUP, 4, 4, 4, 2, 2>(g, t, stream);
    case 128: return launch_shape<DT, GATEUP, 8, 4, 4, 2, 1>(g, t, stream);
    default: return launch_shape<DT, GATEUP, 12, 4, 4, 2, 1>(g, t, stream);
  }
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
