// gate.hip - the gate of the router on given logits, with the tokens each
// expert got and the balance loss, and its gradient.
//
//   p = softmax(z) over the experts (a logit of -inf: not available)
//   ids = the k largest, ties to the lower id; w = p[ids], or p[ids] / sum
//   c_e = tokens whose ids name e, n = tokens routed, S_e = sum of p_e over them
//   loss = E / (k n^2) sum_e c_e S_e
//
// Gradient, with the counts taken as constants, b_e = dloss E c_e / (k n^2):
//   plain weights        dz_e = p_e (b_e - B - D) + [e = ids_j] w_j dw_j
//   renormalised weights dz_e = p_e (b_e - B)     + [e = ids_j] w_j (dw_j - D)
//   B = sum_e p_e b_e, D = sum_j w_j dw_j
// (p_e dw_j = w_j dw_j at e = ids_j for plain weights; renormalised weights are
// a softmax over the chosen logits alone).
//
// Bound: HBM for long batches (4 T E bytes in, for the gradient 4 T E out).
#include "device.hpp"
#include "kernels.hpp"

namespace moe {
namespace {

constexpr int kGateWaves = 4;     // of the gradient's workgroup

// e^x for x <= 0 as 2^(x log2 e): the product's rounding error and the constant's
// are put back (without them the error grows with |x|)
__device__ __forceinline__ float exp_neg(float x) {
  constexpr float kL2e = 1.44269502f, kL2eLo = 1.92596299e-8f;
  const float t = x * kL2e;
  const float r = fmaf(x, kL2e, -t) + x * kL2eLo;
  const float e = __builtin_amdgcn_exp2f(t);
  // below e^-200 the result is 0 in fp32, and r may be an infinity or NaN
  return x < -200.f ? 0.f : fmaf(e, r * 0.693147181f, e);
}

// maximum, sum, "or" over the 16 lanes of a DPP row, in every lane of it
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, dpp_f<kDppXor1>(v));
  v = fmaxf(v, dpp_f<kDppXor2>(v));
  v = fmaxf(v, dpp_f<kDppHalfMirror>(v));
  return fmaxf(v, dpp_f<kDppMirror>(v));
}
__device__ __forceinline__ float row_sum(float v) {
  v += dpp_f<kDppXor1>(v);
  v += dpp_f<kDppXor2>(v);
  v += dpp_f<kDppHalfMirror>(v);
  return v + dpp_f<kDppMirror>(v);
}
__device__ __forceinline__ uint32_t row_max_u32(uint32_t v) {
  v = max(v, dpp_u<kDppXor1>(v));
  v = max(v, dpp_u<kDppXor2>(v));
  v = max(v, dpp_u<kDppHalfMirror>(v));
  return max(v, dpp_u<kDppMirror>(v));
}
__device__ __forceinline__ uint32_t row_min_u32(uint32_t v) {
  v = min(v, dpp_u<kDppXor1>(v));
  v = min(v, dpp_u<kDppXor2>(v));
  v = min(v, dpp_u<kDppHalfMirror>(v));
  return min(v, dpp_u<kDppMirror>(v));
}

// A wave takes four tokens at once, 16 lanes each: the reductions stay inside
// a DPP row (four instructions for four tokens; a token per wave needs them and
// the steps between rows for each one).  Lane l of a row holds the logits of
// experts 64 c + 4 l + (0..3), c < C.  Round by round the largest key and the
// lowest id that holds it are taken out.
//
// Statistics: choices are counted in LDS (integers: any order); the sums of p
// stay in registers over a wave's tokens and are added over its rows, then over
// the workgroup's waves, in a fixed order: one partial row per workgroup.
//
// Bound by its vector instructions: a round looks at each of a lane's keys twice,
// 2 k E operations a token.  T = 16384, E = 256, k = 6: 12.3 us against 3.4 us of
// bytes; T = 200, E = 128: 6.0 us, nearly all of it latency (4 waves a workgroup
// instead of 16: the same).
template <int C, int WAVES, int KB, bool STATS>
__global__ __launch_bounds__(WAVES * 64) void gate_kernel(GateArgs a) {
  constexpr int V = 4 * C;                            // logits per lane
  __shared__ float ls[STATS ? WAVES * C * 64 : 1];
  __shared__ int lc[STATS ? C * 64 + 1 : 1];          // and the tokens routed
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane & 15;
  if (STATS) {
    for (int i = threadIdx.x; i <= C * 64; i += WAVES * 64) lc[i] = 0;
    __syncthreads();
  }
  const bool vec = a.E % 4 == 0 && (uintptr_t)a.z % 16 == 0;
  float S[V];
#pragma unroll
  for (int i = 0; i < V; ++i) S[i] = 0.f;
  for (int64_t t0 = ((int64_t)wave * gridDim.x + blockIdx.x) * 4; t0 < a.T;
       t0 += (int64_t)gridDim.x * WAVES * 4) {
    const int64_t t = t0 + (lane >> 4);
    bool in = t < a.T;
    float v[V];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int e = 64 * c + 4 * l;
      const float* src = a.z + t * a.E + e;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * c + i] = -INFINITY;
      if (vec) {
        if (in && e < a.E) {
          const float4 f = *reinterpret_cast<const float4*>(src);
          v[4 * c] = f.x; v[4 * c + 1] = f.y; v[4 * c + 2] = f.z; v[4 * c + 3] = f.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (in && e + i < a.E) v[4 * c + i] = src[i];
      }
    }
    if (a.mask) in = in && a.mask[in ? t : 0];        // padding: as a row of -inf
    float m = -INFINITY;
    uint32_t nan = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      v[i] = in ? v[i] : -INFINITY;
      v[i] += 0.f;                                    // a logit of -0 ranks with +0
      nan |= v[i] != v[i];
      m = fmaxf(m, v[i]);
    }
    m = row_max(m);
    // a row with no expert available (or masked, or past the end) is not routed
    const bool routed = in && (m > -INFINITY || row_max_u32(nan));
    // the maximum a row subtracts: any finite one will do where nothing is routed
    const float sub = routed ? m : 0.f;
    uint32_t key[V];
    float ps = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      key[i] = v[i] > -INFINITY ? fkey(v[i]) : 0u;    // 0: never chosen (-inf, NaN)
      v[i] = exp_neg(v[i] - sub);
      ps += v[i];
    }
    const float inv = 1.0f / row_sum(ps);             // not routed: infinite, not used
    if (STATS) {
#pragma unroll
      for (int i = 0; i < V; ++i) S[i] += routed ? v[i] * inv : 0.f;
      if (routed && l == 0) atomicAdd(&lc[C * 64], 1);
    }
    int rid[KB];
    float rw[KB], wsum = 0.f;
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      rid[b] = -1;
      rw[b] = 0.f;
      for (int j = 0; j < 16 && 16 * b + j < a.k; ++j) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) best = max(best, key[i]);
        const uint32_t gm = row_max_u32(best);
        uint32_t id = 0xffffffffu;
#pragma unroll
        for (int i = V - 1; i >= 0; --i)
          if (key[i] == gm) id = 64 * (i / 4) + 4 * l + i % 4;
        id = row_min_u32(id);
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (64u * (i / 4) + 4 * l + i % 4 == id) key[i] = 0u;
        const bool have = gm != 0u;                   // an expert is left
        const float e = have ? exp_neg(fkey_value(gm) - sub) : 0.f;
        wsum += e;
        if (l == j) {
          rid[b] = have ? (int)id : -1;
          rw[b] = e;
          if (STATS && have) atomicAdd(&lc[id], 1);
        }
      }
    }
    if (t < a.T) {
#pragma unroll
      for (int b = 0; b < KB; ++b)
        if (16 * b + l < a.k) {
          // a NaN in the row makes its weights NaN through inv
          const float w = a.renorm ? rw[b] / (wsum + 0.f * inv) : rw[b] * inv;
          a.ids[t * a.k + 16 * b + l] = routed ? rid[b] : -1;
          a.w[t * a.k + 16 * b + l] = routed && rid[b] >= 0 ? w : 0.f;
        }
    }
  }
  if (STATS) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      S[i] += __shfl_xor(S[i], 16, kWave);
      S[i] += __shfl_xor(S[i], 32, kWave);
    }
    if (lane < 16) {
#pragma unroll
      for (int c = 0; c < C; ++c)
        *reinterpret_cast<v4f*>(&ls[wave * C * 64 + 64 * c + 4 * l]) =
            v4f{S[4 * c], S[4 * c + 1], S[4 * c + 2], S[4 * c + 3]};
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += WAVES * 64) {
      float s = 0.f;
      for (int w = 0; w < WAVES; ++w) s += ls[w * C * 64 + e];
      a.part_s[(int64_t)blockIdx.x * a.E + e] = s;
      a.part_c[(int64_t)blockIdx.x * a.E + e] = lc[e];
    }
    if (threadIdx.x == 0) {
      a.part_n[blockIdx.x] = lc[C * 64];
      if (blockIdx.x == 0) *a.ticket = 0u;            // for gate_reduce_kernel, the next launch
    }
  }
}

// Partial rows -> counts and the loss.  A workgroup takes 16 experts, 64 threads
// of each every 64th row; the last workgroup to finish adds the workgroups' shares
// of the loss in order.  Bound by latency: 3.9 us for 256 rows of 256 experts (64
// experts a workgroup: 4.1), 4 us for 13 rows of 128 (one workgroup for all: 5.2).
constexpr int kReduceExperts = 16, kReduceSlices = 64;

__global__ __launch_bounds__(kReduceExperts * kReduceSlices) void gate_reduce_kernel(GateArgs a,
                                                                                     int parts) {
  __shared__ float ss[kReduceSlices][kReduceExperts];
  __shared__ int sc[kReduceSlices][kReduceExperts];
  __shared__ int sn[kReduceSlices * kReduceExperts / 64];
  const int l = threadIdx.x & 15, q = threadIdx.x >> 4, lane = threadIdx.x & 63;
  const int e = blockIdx.x * kReduceExperts + l;
  float s = 0.f;
  int c = 0, n = 0;
  if (e < a.E) {
#pragma unroll 4
    for (int b = q; b < parts; b += kReduceSlices) {
      s += a.part_s[(int64_t)b * a.E + e];
      c += a.part_c[(int64_t)b * a.E + e];
    }
  }
  for (int b = threadIdx.x; b < parts; b += kReduceSlices * kReduceExperts) n += a.part_n[b];
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) n += __shfl_xor(n, off, kWave);
  // four slices of a wave, then the waves
  s += __shfl_xor(s, 16, kWave);
  s += __shfl_xor(s, 32, kWave);
  c += __shfl_xor(c, 16, kWave);
  c += __shfl_xor(c, 32, kWave);
  if (lane < 16) {
    ss[q / 4][l] = s;
    sc[q / 4][l] = c;
  }
  if (lane == 0) sn[threadIdx.x >> 6] = n;
  __syncthreads();
  if (threadIdx.x >= 64) return;
  n = 0;
  s = 0.f;
  c = 0;
#pragma unroll
  for (int w = 0; w < kReduceSlices / 4; ++w) {
    n += sn[w];
    s += ss[w][l];
    c += sc[w][l];
  }
  if (a.counts) {
    if (lane < 16 && e < a.E) a.counts[e] = c;
    if (blockIdx.x == 0 && lane == 0) a.counts[a.E] = n;
  }
  if (!a.loss) return;
  const float share = row_sum(e < a.E ? (float)c * s : 0.f);
  int last = 0;
  if (lane == 0) {
    __hip_atomic_store(&a.share[blockIdx.x], share, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    last = __hip_atomic_fetch_add(a.ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
           gridDim.x - 1;
  }
  if (!__builtin_amdgcn_readfirstlane(last)) return;
  // at most 64 workgroups (1024 experts): a lane each, added in a fixed order
  float v = 0.f;
  if (lane < (int)gridDim.x)
    v = __hip_atomic_load(&a.share[lane], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const float total = wave_sum_dpp(v);
  if (lane == 0) {
    const float d = (float)a.k * (float)n * (float)n;
    *a.loss = n > 0 ? total * (float)a.E / d : 0.f;
  }
}

// Four tokens per wave, as in gate_kernel; lane j of a row holds the token's
// choices j, j + 16, ..  Their terms meet the others in LDS: a comparison of each
// of a lane's experts with each choice cost more than the rest together.
// Bound by HBM and, at this size, by the launch: T = 16001, E = 256, k = 6 11.8 us,
// 2.9 TB/s (6.6 us at the rate of a long copy).
template <int C, int KB>
__global__ __launch_bounds__(kGateWaves * 64) void gate_backward_kernel(GateBackward a) {
  constexpr int V = 4 * C;
  __shared__ v4f s_dz[kGateWaves][4][C * 16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane & 15, row = lane >> 4;
  const bool vec = a.E % 4 == 0 && ((uintptr_t)a.z | (uintptr_t)a.dz) % 16 == 0;
  float p[V], w[KB], dw[KB], b[V];
  int id[KB];
  auto load = [&](int64_t t) {
    const bool in = t < a.T;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int e = 64 * c + 4 * l;
      const float* src = a.z + t * a.E + e;
#pragma unroll
      for (int i = 0; i < 4; ++i) p[4 * c + i] = -INFINITY;
      if (vec) {
        if (in && e < a.E) {
          const float4 v = *reinterpret_cast<const float4*>(src);
          p[4 * c] = v.x; p[4 * c + 1] = v.y; p[4 * c + 2] = v.z; p[4 * c + 3] = v.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (in && e + i < a.E) p[4 * c + i] = src[i];
      }
    }
#pragma unroll
    for (int k = 0; k < KB; ++k) {
      const int64_t at = t * a.k + 16 * k + l;
      const bool has = in && 16 * k + l < a.k;
      id[k] = has ? a.ids[at] : -1;
      w[k] = has && a.dw ? a.w[at] : 0.f;
      dw[k] = has && a.dw ? a.dw[at] : 0.f;
    }
  };
  int64_t t0 = ((int64_t)blockIdx.x * kGateWaves + wave) * 4;
  load(t0 + row);                                     // before the wait for the counts
  {
    const float n = a.dloss ? (float)a.counts[a.E] : 0.f;
    const float f = n > 0.f ? *a.dloss * (float)a.E / ((float)a.k * n * n) : 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = 64 * (i / 4) + 4 * l + i % 4;
      b[i] = a.dloss && e < a.E ? f * (float)a.counts[e] : 0.f;
    }
  }
  for (;;) {
    const int64_t t = t0 + row;
    const bool in = t < a.T;
    float D = 0.f;
#pragma unroll
    for (int k = 0; k < KB; ++k) {
      if (id[k] < 0 || id[k] >= a.E) w[k] = dw[k] = 0.f;
      D += w[k] * dw[k];
    }
    D = row_sum(D);
    // not routed: the first choice is negative (lane 0 of the row has it)
    const bool routed = __shfl(id[0], lane & 48, kWave) >= 0;
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, p[i]);
    m = row_max(m);
    const float top = routed ? m : 0.f;
    float ps = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      p[i] = exp_neg(p[i] - top);
      ps += p[i];
    }
    const float inv = 1.0f / row_sum(ps);
    float pb = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      p[i] *= inv;
      pb += p[i] * b[i];
    }
    const float B = row_sum(pb), sub = a.renorm ? B : B + D;
    v4f r[C];
#pragma unroll
    for (int i = 0; i < V; ++i) r[i / 4][i % 4] = routed ? p[i] * (b[i] - sub) : 0.f;
    if (a.dw) {
      // one wave's LDS accesses are done in order; the compiler must keep them so
#pragma unroll
      for (int c = 0; c < C; ++c) s_dz[wave][row][16 * c + l] = r[c];
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      float* mine = reinterpret_cast<float*>(s_dz[wave][row]);
#pragma unroll
      for (int k = 0; k < KB; ++k)
        if (routed && id[k] >= 0 && id[k] < a.E)
          __hip_atomic_fetch_add(mine + id[k], w[k] * (a.renorm ? dw[k] - D : dw[k]),
                                 __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
      for (int c = 0; c < C; ++c) r[c] = s_dz[wave][row][16 * c + l];
    }
    if (in) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int e = 64 * c + 4 * l;
        float* dst = a.dz + t * a.E + e;
        if (vec) {
          if (e < a.E) *reinterpret_cast<v4f*>(dst) = r[c];
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (e + i < a.E) dst[i] = r[c][i];
        }
      }
    }
    t0 += (int64_t)gridDim.x * kGateWaves * 4;
    if (t0 >= a.T) return;
    load(t0 + row);
  }
}

template <int C, int WAVES, int KB>
hipError_t run_gate_k(const GateArgs& a, int grid, hipStream_t st) {
  if (a.counts || a.loss)
    hipLaunchKernelGGL((gate_kernel<C, WAVES, KB, true>), dim3(grid), dim3(WAVES * 64), 0, st, a);
  else
    hipLaunchKernelGGL((gate_kernel<C, WAVES, KB, false>), dim3(grid), dim3(WAVES * 64), 0, st, a);
  return hipGetLastError();
}

template <int C, int WAVES>
hipError_t run_gate(const GateArgs& a, int grid, hipStream_t st) {
  return a.k <= 16 ? run_gate_k<C, WAVES, 1>(a, grid, st) : run_gate_k<C, WAVES, 4>(a, grid, st);
}

}  // namespace

hipError_t launch_gate(const GateArgs& a, hipStream_t st) {
  const int grid = gate_parts(a.T);
  // waves per workgroup: as many as the registers of a lane's logits allow
  hipError_t err = a.E <= 64    ? run_gate<1, 16>(a, grid, st)
                   : a.E <= 128 ? run_gate<2, 16>(a, grid, st)
                   : a.E <= 256 ? run_gate<4, 16>(a, grid, st)
                   : a.E <= 512 ? run_gate<8, 8>(a, grid, st)
                                : run_gate<16, 4>(a, grid, st);
  if (err != hipSuccess || !(a.counts || a.loss)) return err;
  hipLaunchKernelGGL(gate_reduce_kernel, dim3((a.E + kReduceExperts - 1) / kReduceExperts),
                     dim3(kReduceExperts * kReduceSlices), 0, st, a, grid);
  return hipGetLastError();
}

template <int C>
hipError_t run_backward(const GateBackward& a, hipStream_t st) {
  // four tokens a wave, up to eight waves a SIMD (T >= 1, up to 2^31 - 1)
  const int quads = (a.T - 1) / 4 + 1, most = 8192;
  const dim3 g(((quads < most ? quads : most) + kGateWaves - 1) / kGateWaves), b(kGateWaves * 64);
  if (a.k <= 16) hipLaunchKernelGGL((gate_backward_kernel<C, 1>), g, b, 0, st, a);
  else hipLaunchKernelGGL((gate_backward_kernel<C, 4>), g, b, 0, st, a);
  return hipGetLastError();
}

hipError_t launch_gate_backward(const GateBackward& a, hipStream_t st) {
  return a.E <= 64    ? run_backward<1>(a, st)
         : a.E <= 128 ? run_backward<2>(a, st)
         : a.E <= 256 ? run_backward<4>(a, st)
         : a.E <= 512 ? run_backward<8>(a, st)
                      : run_backward<16>(a, st);
}

}  // namespace moe
