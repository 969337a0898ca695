// The norms around a block on gfx950: the norm of a block's output, its gate
// and residual scale, the residual sum, the norm in front of the next block
// and that block's activation quantiser, in one pass over the rows.
//
// For every row (token) t of H values, in fp32 from the loads to the stores:
//   v    = y[t], or sum over k ascending with pos[t,k] >= 0 of
//          w[t,k] * expert_out[pos[t,k]]            (the experts' combine)
//   b    = v * rstd(v) * gamma_post                 (v itself without gamma_post)
//   r    = residual[t] + (alpha * gate) * b         -> residual_out, one rounding
//   n    = r * rstd(r) * gamma_pre                  -> h, one rounding
//   codes, scales = the quantised form of n
// with rstd(u) = 1 / sqrt(mean(u^2) + eps). n is computed from the unrounded
// r and quantised unrounded: every output is rounded once.
//
// Bound: bytes. A row is read once (residual, and y or its K expert rows) and
// held in registers across both norms; gamma and a channel gate stay in L2.
// One workgroup owns one row: thread j holds the V consecutive values at
// (i * threads + j) * V, i < NV. The sums of squares go lane -> wave
// (shuffles) -> workgroup (LDS, every thread adds the waves' partial sums in
// the same order), so results do not depend on the launch. V = 8 where every
// row starts on the vector's boundary, V = 1 otherwise (odd row lengths,
// bases off a 16-byte boundary). bf16 on both sides, H = 7168: T = 4096 52.6 us
// (236 MB, 4.5 of the 4.8 TB/s that a copy reaches), one row 3.9 us (latency).

#include "common.hpp"
#include "launch.hpp"
#include "mx_codes.hpp"

namespace moe {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kSlots = 8;          // expert rows whose loads are issued together

template <int DT>
constexpr int elem_bytes() {
  return DT == kF32 ? 4 : 2;
}

// V consecutive values at element index i, widened to fp32.
template <int DT, int V>
__device__ __forceinline__ void load_vals(const void* base, int64_t i, float* f) {
  if constexpr (V == 1) {
    if constexpr (DT == kF32) f[0] = static_cast<const float*>(base)[i];
    else f[0] = to_float<DT>(static_cast<const uint16_t*>(base)[i]);
  } else if constexpr (DT == kF32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
    const float4 a = p[0], b = p[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else {
    const u32x4 q = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(base) + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = to_float<DT>(q[j] & 0xffffu);
      f[2 * j + 1] = to_float<DT>(q[j] >> 16);
    }
  }
}

template <int DT, int V>
__device__ __forceinline__ void store_vals(void* base, int64_t i, const float* f) {
  if constexpr (V == 1) {
    if constexpr (DT == kF32) static_cast<float*>(base)[i] = f[0];
    else static_cast<uint16_t*>(base)[i] = static_cast<uint16_t>(from_float<DT>(f[0]));
  } else if constexpr (DT == kF32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
    p[0] = make_float4(f[0], f[1], f[2], f[3]);
    p[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    u32x4 q;
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = from_float<DT>(f[2 * j]) | (from_float<DT>(f[2 * j + 1]) << 16);
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(base) + i) = q;
  }
}

// The workgroup's sum (or maximum) of one value a thread; `part` holds one
// value a wave and is used for one reduction only.
template <bool MAX>
__device__ __forceinline__ float block_reduce(float v, float* part, int waves) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    const float o = __shfl_xor(v, off);
    v = MAX ? fmaxf(v, o) : v + o;
  }
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  v = part[0];
  for (int i = 1; i < waves; ++i) v = MAX ? fmaxf(v, part[i]) : v + part[i];
  return v;
}

template <int DT, int RDT, int V, int NV, bool REDUCE>
__global__ __launch_bounds__(kMaxThreads) void block_norm_kernel(NormProblem a) {
  __shared__ float part[3][kMaxThreads / 64];
  const int64_t t = blockIdx.x;
  const int threads = blockDim.x;
  const int waves = threads >> 6;
  const int tid = threadIdx.x;
  const int64_t base = t * a.H;
  const float inv_h = 1.0f / static_cast<float>(a.H);

  // Columns past H: their loads go to the row's last vector, their values are
  // zeros (a select where they enter r, nothing is computed around branches).
  int col[NV];
  bool live[NV];
  float v[NV][V], r[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    col[i] = (i * threads + tid) * V;
    live[i] = col[i] < a.H;
    col[i] = live[i] ? col[i] : a.H - V;
    load_vals<RDT, V>(a.res, base + col[i], r[i]);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      r[i][j] = live[i] ? r[i][j] : 0.0f;
      v[i][j] = 0.0f;
    }
  }

  if (REDUCE || a.y) {
    if constexpr (REDUCE) {
      const int32_t* pt = a.pos + t * a.K;
      const float* wt = a.w ? a.w + t * a.K : nullptr;
      for (int k0 = 0; k0 < a.K; k0 += kSlots) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          float f[kSlots][V];
          int32_t p[kSlots];
#pragma unroll
          for (int s = 0; s < kSlots; ++s) {
            p[s] = k0 + s < a.K ? pt[k0 + s] : -1;
            if (p[s] >= a.rows) p[s] = -1;   // past the rows: skipped, never read
            if (p[s] >= 0) load_vals<DT, V>(a.y, static_cast<int64_t>(p[s]) * a.H + col[i], f[s]);
          }
#pragma unroll
          for (int s = 0; s < kSlots; ++s) {
            if (p[s] < 0) continue;
            const float wk = wt ? wt[k0 + s] : 1.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) v[i][j] = __builtin_fmaf(wk, f[s][j], v[i][j]);
          }
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        load_vals<DT, V>(a.y, base + col[i], v[i]);
      }
    }

    float rstd = 1.0f;
    if (a.gamma_post) {
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < V; ++j) ss = live[i] ? __builtin_fmaf(v[i][j], v[i][j], ss) : ss;
      }
      ss = block_reduce<false>(ss, part[0], waves);
      rstd = 1.0f / sqrtf(ss * inv_h + a.eps);
    }
    float scale = a.alpha;
    if (a.gate_kind == MOE_GATE_TOKEN) scale *= static_cast<const float*>(a.gate)[t];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float g[V];
      if (a.gamma_post) {
        load_vals<kF32, V>(a.gamma_post, col[i], g);
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] = v[i][j] * rstd * g[j];
      }
      if (a.gate_kind == MOE_GATE_CHANNEL) {
        load_vals<kF32, V>(a.gate, col[i], g);
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] *= g[j];
      } else if (a.gate_kind == MOE_GATE_FULL) {
        load_vals<DT, V>(a.gate, base + col[i], g);
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] *= g[j];
      }
#pragma unroll
      for (int j = 0; j < V; ++j) r[i][j] = live[i] ? __builtin_fmaf(scale, v[i][j], r[i][j]) : 0.0f;
      if (a.res_out && live[i]) store_vals<RDT, V>(a.res_out, base + col[i], r[i]);
    }
  }
  if (!a.gamma_pre) return;

  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int j = 0; j < V; ++j) ss = __builtin_fmaf(r[i][j], r[i][j], ss);   // zeros past H
  }
  ss = block_reduce<false>(ss, part[1], waves);
  const float rstd = 1.0f / sqrtf(ss * inv_h + a.eps);
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float g[V];
    load_vals<kF32, V>(a.gamma_pre, col[i], g);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      r[i][j] = live[i] ? r[i][j] * rstd * g[j] : 0.0f;
      amax = fmaxf(amax, fabsf(r[i][j]));
    }
    if (a.h && live[i]) store_vals<DT, V>(a.h, base + col[i], r[i]);
  }
  if (a.quant == MOE_QUANT_NONE) return;

  if (a.quant == MOE_QUANT_FP8 || a.quant == MOE_QUANT_INT8) {
    // One scale a row: amax / (the largest code), 1 for an all-zero row.
    amax = block_reduce<true>(amax, part[2], waves);
    const bool fp8 = a.quant == MOE_QUANT_FP8;
    const float s = amax > 0.0f ? amax / (fp8 ? 448.0f : 127.0f) : 1.0f;
    if (tid == 0) static_cast<float*>(a.scales)[t] = s;
    uint8_t* out = static_cast<uint8_t*>(a.codes) + base;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      uint32_t q[(V + 3) / 4] = {};
      if (fp8) {
        if constexpr (V == 8) {
#pragma unroll
          for (int j = 0; j < 8; j += 4) {
            q[j >> 2] = pk4_fp8e4m3(r[i][j] / s, r[i][j + 1] / s, r[i][j + 2] / s, r[i][j + 3] / s);
          }
        } else {
          q[0] = float_to_fp8e4m3(r[i][0] / s);
        }
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float c = fminf(fmaxf(rintf(r[i][j] / s), -127.0f), 127.0f);
          q[j >> 2] |= (static_cast<uint32_t>(static_cast<int>(c)) & 0xffu) << (8 * (j & 3));
        }
      }
      if (!live[i]) continue;
      if constexpr (V == 8) *reinterpret_cast<u32x2*>(out + col[i]) = u32x2{q[0], q[1]};
      else out[col[i]] = static_cast<uint8_t>(q[0]);
    }
    return;
  }
  // MX formats: a 32-block is four neighbouring lanes' vectors (H a multiple
  // of 32, so a block is never cut by the end of the row).
  if constexpr (V == 8) {
    const bool fp4 = a.quant == MOE_QUANT_MXFP4;
    const int64_t nb = a.H / 32;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float m = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(r[i][j]));
      m = fmaxf(m, __shfl_xor(m, 1));
      m = fmaxf(m, __shfl_xor(m, 2));
      if (!live[i]) continue;
      const int e = mx_scale_exp(m, fp4 ? 2 : 8);
      if ((tid & 3) == 0) static_cast<uint8_t*>(a.scales)[t * nb + col[i] / 32] = static_cast<uint8_t>(e);
      const float X = ldexpf(1.0f, e - 127);
      if (fp4) {
        const uint32_t q = pk8_fp4e2m1(r[i], X);
        reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.codes) + (base + col[i]) / 2)[0] = q;
      } else {
        const u32x2 q = {pk4_fp8e4m3(r[i][0] / X, r[i][1] / X, r[i][2] / X, r[i][3] / X),
                         pk4_fp8e4m3(r[i][4] / X, r[i][5] / X, r[i][6] / X, r[i][7] / X)};
        *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(a.codes) + base + col[i]) = q;
      }
    }
  }
}

template <int DT, int RDT, int V, int NV>
hipError_t launch_nv(const NormProblem& a, hipStream_t stream) {
  const int vecs = (a.H + V - 1) / V;
  const int threads = ((vecs + NV - 1) / NV + 63) / 64 * 64;
  if (a.pos) {
    hipLaunchKernelGGL((block_norm_kernel<DT, RDT, V, NV, true>), dim3(a.T), dim3(threads), 0, stream, a);
  } else {
    hipLaunchKernelGGL((block_norm_kernel<DT, RDT, V, NV, false>), dim3(a.T), dim3(threads), 0, stream, a);
  }
  return hipGetLastError();
}

template <int DT, int RDT>
hipError_t launch_typed(const NormProblem& a, hipStream_t stream) {
  // single values: as many threads as a workgroup holds (bf16, graph of twenty
  // calls: T = 900, H = 7001 23.0 us; T = 300, H = 16383 23.9 us; one row of 7001 6.6 us)
  if (!a.vec && a.H <= 2 * kMaxThreads) return launch_nv<DT, RDT, 1, 2>(a, stream);
  if (!a.vec && a.H <= 8 * kMaxThreads) return launch_nv<DT, RDT, 1, 8>(a, stream);
  if (!a.vec) return launch_nv<DT, RDT, 1, 16>(a, stream);     // up to 16384 values
  // Two vectors a thread where rows are long and there are more of them than
  // CUs: more, smaller workgroups then overlap their reductions' waits. H =
  // 7168: T = 4096 58.8 -> 53.4 us (4.4 TB/s), the combine of 512 x 8 rows 19.1
  // -> 16.4; but one token 3.8 -> 4.4, and T = 777 of H = 2048 9.2 -> 10.1.
  // (Four vectors: 57.3, 22.8, 5.6, 12.1.)
  const bool two = a.H > 8 * kMaxThreads || (a.H > 4 * kMaxThreads && a.T >= 256);
  return two ? launch_nv<DT, RDT, 8, 2>(a, stream) : launch_nv<DT, RDT, 8, 1>(a, stream);
}

}  // namespace

hipError_t launch_block_norm(const NormProblem& a, hipStream_t stream) {
  if (a.dtype == kF32) return launch_typed<kF32, kF32>(a, stream);
  if (a.dtype == kBF16) {
    return a.res_dtype == kF32 ? launch_typed<kBF16, kF32>(a, stream) : launch_typed<kBF16, kBF16>(a, stream);
  }
  return a.res_dtype == kF32 ? launch_typed<kF16, kF32>(a, stream) : launch_typed<kF16, kF16>(a, stream);
}

}  // namespace moe
