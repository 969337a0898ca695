// Microscaled 4-bit experts on both sides: MXFP4 weights against MXFP4
// activations on v_mfma_scale_f32_32x32x64_f8f6f4 (E2M1 elements, one E8M0
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
// second, so a lane's result registers hold 16 output columns of ONE row: the
// 32-column block that shares a scale lies in the two halves of a lane pair,
// and its largest magnitude takes 15 in-lane maxima and one exchange. A lane
// half h holds elements 32h .. 32h + 31 of the instruction's 64; the reduction
// runs in chunks of 256 elements in which half h owns elements 128h .. 128h +
// 127 of its rows (64 contiguous bytes), k-slice t (0..3) takes bytes 16t of
// each half, and byte t of each half's 4-byte scale word.
//
// Bound: the weight stream (a prefill expert of ~128 rows needs 4 x 32 cycles
// of MFMA a 1 KB weight load, a third of the time HBM takes to deliver it).
// Weights go from memory into a register ring; a workgroup of 4 waves shares
// the activation rows through double-buffered LDS, staged through registers as
// many chunks ahead as the weights are loaded (loads complete in order:
// waiting for a late-issued activation would wait for every weight before it).
// One pass takes up to 32 * NAMAX rows, so an expert's weights are read once.

#include "common.hpp"
#include "launch.hpp"

namespace moe {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kThreads = 256;
constexpr int kCK = 256;                  // reduction elements per chunk
constexpr int kRowBytes = kCK / 2;        // of one row
constexpr int kLdsRow = kRowBytes + 16;   // padded: 8 rows' 16-byte reads cover all banks
constexpr int kBlk = 32;

// A (weights) and B (activations) E2M1: format code 4, four of the eight
// operand registers in use; byte T of each scale word.
template <int T>
__device__ __forceinline__ f32x16 mfma_mx4(const u32x4& a, const u32x4& b, uint32_t sa, uint32_t sb,
                                           f32x16 c) {
  const i32x8 aa = {static_cast<int>(a.x), static_cast<int>(a.y), static_cast<int>(a.z),
                    static_cast<int>(a.w), 0, 0, 0, 0};
  const i32x8 bb = {static_cast<int>(b.x), static_cast<int>(b.y), static_cast<int>(b.z),
                    static_cast<int>(b.w), 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(aa, bb, c, 4, 4, T, static_cast<int>(sa), T,
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
  int n, kd, block_m, n_tiles;
};

template <int NA>
struct Mx4Slot {
  u32x4 w[2][4];            // the lane's two weight rows, its half's 64 bytes
  uint32_t sw[2];
  u32x4 a[NA];              // this thread's 16 bytes of activation rows tid / 8 + 32 q
  u32x2 sa;                 // the scale bytes of activation row tid
};

template <int NAMAX>
struct Mx4Lds {
  uint8_t row[2][32 * NAMAX][kLdsRow];
  u32x2 scale[2][kThreads];   // one a thread, rows past the pass among them: a
                              // branch in the step would let the compiler sink
                              // the MFMAs past the next loads
};

// Where a pass reads: wave-uniform addresses that walk along the reduction, and
// fixed 32-bit lane offsets.
struct Mx4Walk {
  const uint8_t *w0, *w1, *s0, *s1;   // the two weight tiles' first rows, their scales
  const uint8_t *a, *as;              // activations, their scales
};

// One pass over the reduction for NA groups of 32 activation rows. a_off /
// as_off: this thread's staging offsets.
template <int NA, int NAMAX, int S>
__device__ __forceinline__ void mx4_pass(Mx4Walk p, uint32_t w_off, uint32_t s_off,
                                         const uint32_t* a_off, uint32_t as_off, int nch, int tid,
                                         int lr, int lh, Mx4Lds<NAMAX>& lds, f32x16* acc) {
#pragma unroll
  for (int q = 0; q < 2 * NA; ++q) acc[q] = f32x16{};
  Mx4Slot<NA> ring[S];
  int left = nch - 1;
  auto load = [&](Mx4Slot<NA>& s) __attribute__((always_inline)) {
    // activations first: they are waited for a step earlier
#pragma unroll
    for (int q = 0; q < NA; ++q) s.a[q] = *reinterpret_cast<const u32x4*>(p.a + a_off[q]);
    s.sa = *reinterpret_cast<const u32x2*>(p.as + as_off);
    s.sw[0] = *reinterpret_cast<const uint32_t*>(p.s0 + s_off);
    s.sw[1] = *reinterpret_cast<const uint32_t*>(p.s1 + s_off);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s.w[0][i] = *reinterpret_cast<const u32x4*>(p.w0 + w_off + 16 * i);
      s.w[1][i] = *reinterpret_cast<const u32x4*>(p.w1 + w_off + 16 * i);
    }
    // Past the end the last chunk is read again (in bounds, never used): every
    // step issues the same loads, which the compiler's wait counts rely on.
    const int64_t on = left > 0 ? 1 : 0;
    --left;
    p.a += on * kRowBytes;
    p.w0 += on * kRowBytes;
    p.w1 += on * kRowBytes;
    p.as += on * (kCK / kBlk);
    p.s0 += on * (kCK / kBlk);
    p.s1 += on * (kCK / kBlk);
  };
  auto stage = [&](const Mx4Slot<NA>& s, int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < NA; ++q) {
      *reinterpret_cast<u32x4*>(&lds.row[buf][(tid >> 3) + 32 * q][(tid & 7) * 16]) = s.a[q];
    }
    lds.scale[buf][tid] = s.sa;
  };
#pragma unroll
  for (int s = 0; s < S; ++s) {
    load(ring[s]);
    __builtin_amdgcn_sched_barrier(0);
  }
  stage(ring[0], 0);
  wait_lds();
  barrier_no_wait();
  auto step = [&](int c, auto U) __attribute__((always_inline)) {
    constexpr int u = decltype(U)::value;
    const int buf = c & 1;
    uint32_t sa[NA];
#pragma unroll
    for (int q = 0; q < NA; ++q) {
      const u32x2 v = lds.scale[buf][32 * q + lr];
      sa[q] = lh ? v.y : v.x;
    }
    static_for<4>([&](auto TT) __attribute__((always_inline)) {
      constexpr int t = decltype(TT)::value;
#pragma unroll
      for (int q = 0; q < NA; ++q) {
        const u32x4 b = *reinterpret_cast<const u32x4*>(&lds.row[buf][32 * q + lr][lh * 64 + t * 16]);
        acc[2 * q] = mfma_mx4<t>(ring[u].w[0][t], b, ring[u].sw[0], sa[q], acc[2 * q]);
        acc[2 * q + 1] = mfma_mx4<t>(ring[u].w[1][t], b, ring[u].sw[1], sa[q], acc[2 * q + 1]);
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    stage(ring[(u + 1) % S], buf ^ 1);
    load(ring[u]);
    wait_lds();
    barrier_no_wait();
  };
  int c0 = 0;
  for (; c0 + S <= nch; c0 += S) {
    static_for<S>([&](auto U) __attribute__((always_inline)) { step(c0 + decltype(U)::value, U); });
  }
  const int rest = nch - c0;
  static_for<S>([&](auto U) __attribute__((always_inline)) {
    if (decltype(U)::value < rest) step(c0 + decltype(U)::value, U);
  });
}

// hq / hs of one 32-row group: lane (lr, lh) holds columns 8 j + 4 lh + 0..3
// (j = 0..3) of activation row lr; its partner lane ^ 32 the block's rest.
__device__ __forceinline__ void store_mxfp4(const f32x16& g, const f32x16& u, int lh, bool live,
                                            uint8_t* codes, uint8_t* scale) {
  float v[16];
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    v[i] = silu(g[i]) * u[i];
    amax = fmaxf(amax, fabsf(v[i]));
  }
  amax = fmaxf(amax, __shfl_xor(amax, 32));
  const int e = mx_scale_exp(amax, 2);
  const float X = ldexpf(1.0f, e - 127);
  uint32_t q[2] = {0u, 0u};                 // columns j = 0, 1 and j = 2, 3
#pragma unroll
  for (int i = 0; i < 16; ++i) q[i >> 3] |= float_to_fp4e2m1(v[i] / X) << (4 * (i & 7));
  // half 0 collects bytes 0..7 of the block (j = 0, 1), half 1 bytes 8..15
  const uint32_t mine = q[lh], other = __shfl_xor(q[lh ^ 1], 32);
  const uint32_t lo = lh ? other : mine, hi = lh ? mine : other;   // the first / second four of each eight
  const u32x2 out = {(lo & 0xffffu) | (hi << 16), (lo >> 16) | (hi & 0xffff0000u)};
  if (live) {
    *reinterpret_cast<u32x2*>(codes + lh * 8) = out;
    if (lh == 0) *scale = static_cast<uint8_t>(e);
  }
}

// gate/up: wave w owns columns 128 nt + 32 w + 0..31 of W_gate and W_up; down:
// columns 256 nt + 64 w + 0..63 of W_down.
template <int DT, bool GATEUP, int NAMAX, int S>
__global__ __launch_bounds__(kThreads, NAMAX <= 2 ? 2 : 1) void mx4_grouped_kernel(Mx4Args g) {
  __shared__ __attribute__((aligned(16))) Mx4Lds<NAMAX> lds;
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
  const int lr = tid & 31, lh = (tid >> 5) & 1;
  const int64_t kd = g.kd, kb = kd / kBlk;
  const int col0 = GATEUP ? nt * 128 + wave * 32 : nt * 256 + wave * 64;
  const int64_t wrow = static_cast<int64_t>(e) * g.n + col0;
  const uint8_t* w0 = g.b0 + wrow * (kd / 2);
  const uint8_t* w1 = GATEUP ? g.b1 + wrow * (kd / 2) : w0 + 32 * (kd / 2);
  const uint8_t* s0 = g.s0 + wrow * kb;
  const uint8_t* s1 = GATEUP ? g.s1 + wrow * kb : s0 + 32 * kb;
  const uint32_t w_off = static_cast<uint32_t>(lr * (g.kd / 2)) + lh * 64;
  const uint32_t s_off = static_cast<uint32_t>(lr * (g.kd / kBlk)) + lh * 4;
  const int nch = g.kd / kCK;

  // passes of equal height
  const int passes = (rows + 32 * NAMAX - 1) / (32 * NAMAX);
  const int height = ((rows + passes - 1) / passes + 31) / 32 * 32;
  for (int r0 = 0; r0 < rows; r0 += height) {
    if (r0 > 0) __syncthreads();
    const int rows_pass = min(height, rows - r0);
    auto source = [&](int r) __attribute__((always_inline)) {
      if (r >= rows_pass) r = 0;                  // in bounds; its results are never stored
      return static_cast<int64_t>(GATEUP ? g.sorted_token[m_start + r0 + r] : r);
    };
    uint32_t a_off[NAMAX];
#pragma unroll
    for (int q = 0; q < NAMAX; ++q) {
      a_off[q] = static_cast<uint32_t>(source((tid >> 3) + 32 * q) * (kd / 2)) + (tid & 7) * 16;
    }
    const uint32_t as_off = static_cast<uint32_t>(source(tid) * kb);
    const int64_t first = GATEUP ? 0 : m_start + r0;
    const Mx4Walk walk{w0, w1, s0, s1, g.a + first * (kd / 2), g.as + first * kb};
    f32x16 acc[2 * NAMAX];
    auto run = [&](auto NAC) __attribute__((always_inline)) {
      constexpr int na = decltype(NAC)::value;
      mx4_pass<na, NAMAX, S>(walk, w_off, s_off, a_off, as_off, nch, tid, lr, lh, lds, acc);
#pragma unroll
      for (int q = 0; q < na; ++q) {
        const int row = 32 * q + lr;
        const bool live = row < rows_pass;
        const int64_t at = m_start + r0 + row;
        if constexpr (GATEUP) {
          store_mxfp4(acc[2 * q], acc[2 * q + 1], lh, live, g.hq + at * (g.n / 2) + col0 / 2,
                      g.hs + at * (g.n / kBlk) + col0 / kBlk);
        } else if (live) {
#pragma unroll
          for (int w = 0; w < 2; ++w) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const f32x16& v = acc[2 * q + w];
              const u32x2 o = {from_float<DT>(v[4 * j]) | (from_float<DT>(v[4 * j + 1]) << 16),
                               from_float<DT>(v[4 * j + 2]) | (from_float<DT>(v[4 * j + 3]) << 16)};
              *reinterpret_cast<u32x2*>(g.out + at * g.n + col0 + 32 * w + 8 * j + 4 * lh) = o;
            }
          }
        }
      }
    };
    const int active = (rows_pass + 31) >> 5;
    static_for<NAMAX>([&](auto I) {
      constexpr int na = decltype(I)::value + 1;
      if (active == na) run(int_c<na>{});
    });
  }
}

template <int DT, bool GATEUP>
hipError_t launch_grouped(const Mx4GemmProblem& p, const moe_tables& t, hipStream_t stream) {
  Mx4Args g{p.a, p.as, p.b0, p.b1, p.s0, p.s1, p.hq, p.hs, static_cast<uint16_t*>(p.out),
            t.sorted_token, t.group_sizes, t.group_offsets, t.group_padded_offsets, t.block_expert,
            t.active_blocks, t.active_count, p.n, p.kd, t.block_m, p.n / (GATEUP ? 128 : 256)};
  const int64_t total = static_cast<int64_t>(t.num_blocks) * g.n_tiles;
  const dim3 grid(static_cast<unsigned>((total + 7) / 8 * 8));
  if (t.block_m <= 32) {
    hipLaunchKernelGGL((mx4_grouped_kernel<DT, GATEUP, 1, 3>), grid, dim3(kThreads), 0, stream, g);
  } else if (t.block_m == 64) {
    hipLaunchKernelGGL((mx4_grouped_kernel<DT, GATEUP, 2, 2>), grid, dim3(kThreads), 0, stream, g);
  } else if (t.block_m == 128) {
    hipLaunchKernelGGL((mx4_grouped_kernel<DT, GATEUP, 4, 4>), grid, dim3(kThreads), 0, stream, g);
  } else {
    hipLaunchKernelGGL((mx4_grouped_kernel<DT, GATEUP, 6, 3>), grid, dim3(kThreads), 0, stream, g);
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
