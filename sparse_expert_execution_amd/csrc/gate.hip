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

constexpr int kGateWaves = 4;

// Sum over the tokens of a workgroup of p_e and of the choices, in registers
// (a lane owns experts lane + 64 i), then over its waves in LDS: one partial
// row per workgroup, so the sums have a fixed order and need no atomics.
template <int M, bool STATS>
__global__ __launch_bounds__(kGateWaves * 64) void gate_kernel(GateArgs a) {
  __shared__ float ls[STATS ? kGateWaves * M * 64 : 1];
  __shared__ int lc[STATS ? kGateWaves * M * 64 : 1];
  __shared__ int ln[kGateWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float S[M];
  int C[M];
#pragma unroll
  for (int i = 0; i < M; ++i) { S[i] = 0.f; C[i] = 0; }
  int routed = 0;
  for (int64_t t = (int64_t)blockIdx.x * kGateWaves + wave; t < a.T;
       t += (int64_t)gridDim.x * kGateWaves) {
    int my_id = -1;
    float my_w = 0.f;
    bool live = !a.mask || a.mask[t];
    if (live) {
      float v[M];
      uint32_t key[M];
      float m = -INFINITY;
      bool nan = false;
#pragma unroll
      for (int i = 0; i < M; ++i) {
        const int e = lane + 64 * i;
        // + 0: a logit of -0 ranks with +0
        v[i] = e < a.E ? a.z[t * a.E + e] + 0.f : -INFINITY;
        nan |= v[i] != v[i];
        key[i] = v[i] > -INFINITY ? fkey(v[i]) : 0u;   // 0: never chosen (-inf, NaN)
        m = fmaxf(m, v[i]);
      }
      m = wave_max_dpp(m);
      if (m == -INFINITY && __ballot(nan) == 0) {
        live = false;                                  // no expert is available
      } else {
        float p[M], ps = 0.f;
#pragma unroll
        for (int i = 0; i < M; ++i) {
          p[i] = lane + 64 * i < a.E ? expf(v[i] - m) : 0.f;
          ps += p[i];
        }
        const float inv = 1.0f / wave_sum_dpp(ps);
        float wsum = 0.f;
        for (int j = 0; j < a.k; ++j) {
          uint32_t lb = 0;
          int li = 0;
#pragma unroll
          for (int i = 0; i < M; ++i)
            if (key[i] > lb) { lb = key[i]; li = i; }
          const uint32_t gm = wave_max_u32_dpp(lb);
          if (gm == 0) break;
          uint64_t win = __ballot(lb == gm);
          int id = 0x7fffffff;
          while (win) {
            const int l = __builtin_ctzll(win);
            const int cand = l + 64 * __builtin_amdgcn_readlane(li, l);
            id = cand < id ? cand : id;
            win &= win - 1;
          }
#pragma unroll
          for (int i = 0; i < M; ++i)
            if (lane + 64 * i == id) {
              key[i] = 0u;
              if (STATS) ++C[i];
            }
          const float e = expf(fkey_value(gm) - m);
          wsum += e;
          if (lane == j) { my_w = e; my_id = id; }
        }
        // without an expert to choose (a row of NaN) the ids stay -1; a NaN in
        // the row makes its weights NaN through inv
        my_w = my_id < 0 ? 0.f : a.renorm ? my_w / (wsum + 0.f * inv) : my_w * inv;
        if (STATS) {
#pragma unroll
          for (int i = 0; i < M; ++i) S[i] += p[i] * inv;
          ++routed;
        }
      }
    }
    if (lane < a.k) {
      a.ids[t * a.k + lane] = live ? my_id : -1;
      a.w[t * a.k + lane] = live ? my_w : 0.f;
    }
  }
  if (STATS) {
#pragma unroll
    for (int i = 0; i < M; ++i) {
      ls[(wave * M + i) * 64 + lane] = S[i];
      lc[(wave * M + i) * 64 + lane] = C[i];
    }
    if (lane == 0) ln[wave] = routed;
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kGateWaves * 64) {
      float s = 0.f;
      int c = 0;
#pragma unroll
      for (int w = 0; w < kGateWaves; ++w) {
        s += ls[w * M * 64 + e];
        c += lc[w * M * 64 + e];
      }
      a.part_s[(int64_t)blockIdx.x * a.E + e] = s;
      a.part_c[(int64_t)blockIdx.x * a.E + e] = c;
    }
    if (threadIdx.x == 0) {
      int r = 0;
#pragma unroll
      for (int w = 0; w < kGateWaves; ++w) r += ln[w];
      a.part_n[blockIdx.x] = r;
      if (blockIdx.x == 0) *a.ticket = 0u;             // for gate_reduce_kernel, the next launch
    }
  }
}

// Partial rows -> counts and the loss.  A workgroup takes 64 experts (4 slices
// of the rows each); the last one to finish adds the workgroups' shares of
// the loss in order.
__global__ __launch_bounds__(256) void gate_reduce_kernel(GateArgs a, int parts) {
  __shared__ float ss[4][64];
  __shared__ int sc[4][64];
  __shared__ int sn[4];
  const int lane = threadIdx.x & 63, q = threadIdx.x >> 6;
  const int e = blockIdx.x * 64 + lane;
  float s = 0.f;
  int c = 0, n = 0;
  if (e < a.E)
    for (int b = q; b < parts; b += 4) {
      s += a.part_s[(int64_t)b * a.E + e];
      c += a.part_c[(int64_t)b * a.E + e];
    }
  for (int b = threadIdx.x; b < parts; b += 256) n += a.part_n[b];
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) n += __shfl_xor(n, off, kWave);
  ss[q][lane] = s;
  sc[q][lane] = c;
  if (lane == 0) sn[q] = n;
  __syncthreads();
  if (q != 0) return;
  n = sn[0] + sn[1] + sn[2] + sn[3];
  s = (ss[0][lane] + ss[1][lane]) + (ss[2][lane] + ss[3][lane]);
  c = sc[0][lane] + sc[1][lane] + sc[2][lane] + sc[3][lane];
  if (a.counts) {
    if (e < a.E) a.counts[e] = c;
    if (blockIdx.x == 0 && lane == 0) a.counts[a.E] = n;
  }
  if (!a.loss) return;
  const float share = wave_sum_dpp(e < a.E ? (float)c * s : 0.f);
  if (lane == 0) {
    __hip_atomic_store(&a.share[blockIdx.x], share, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const bool last = __hip_atomic_fetch_add(a.ticket, 1u, __ATOMIC_ACQ_REL,
                                             __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
    if (last) {
      float total = 0.f;
      for (unsigned b = 0; b < gridDim.x; ++b)
        total += __hip_atomic_load(&a.share[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      const float d = (float)a.k * (float)n * (float)n;
      *a.loss = n > 0 ? total * (float)a.E / d : 0.f;
    }
  }
}

// One wave per token.
template <int M>
__global__ __launch_bounds__(kGateWaves * 64) void gate_backward_kernel(GateBackward a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float b[M];
  {
    float f = 0.f;
    if (a.dloss) {
      const float n = (float)a.counts[a.E];
      f = n > 0.f ? *a.dloss * (float)a.E / ((float)a.k * n * n) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < M; ++i) {
      const int e = lane + 64 * i;
      b[i] = a.dloss && e < a.E ? f * (float)a.counts[e] : 0.f;
    }
  }
  for (int64_t t = (int64_t)blockIdx.x * kGateWaves + wave; t < a.T;
       t += (int64_t)gridDim.x * kGateWaves) {
    int id = -1;
    float w = 0.f, dw = 0.f;
    if (lane < a.k) {
      id = a.ids[t * a.k + lane];
      if (a.dw && id >= 0) { w = a.w[t * a.k + lane]; dw = a.dw[t * a.k + lane]; }
    }
    float* dz = a.dz + t * a.E;
    if (__builtin_amdgcn_readfirstlane(id) < 0) {      // not routed
#pragma unroll
      for (int i = 0; i < M; ++i)
        if (lane + 64 * i < a.E) dz[lane + 64 * i] = 0.f;
      continue;
    }
    float p[M], m = -INFINITY, ps = 0.f;
#pragma unroll
    for (int i = 0; i < M; ++i) {
      const int e = lane + 64 * i;
      p[i] = e < a.E ? a.z[t * a.E + e] : -INFINITY;
      m = fmaxf(m, p[i]);
    }
    m = wave_max_dpp(m);
#pragma unroll
    for (int i = 0; i < M; ++i) {
      p[i] = lane + 64 * i < a.E ? expf(p[i] - m) : 0.f;
      ps += p[i];
    }
    const float inv = 1.0f / wave_sum_dpp(ps);
    float pb = 0.f;
#pragma unroll
    for (int i = 0; i < M; ++i) {
      p[i] *= inv;
      pb += p[i] * b[i];
    }
    const float B = wave_sum_dpp(pb), D = wave_sum_dpp(w * dw);
    const float sub = a.renorm ? B : B + D;
    const float add = a.renorm ? w * (dw - D) : w * dw;
    float r[M];
#pragma unroll
    for (int i = 0; i < M; ++i) r[i] = p[i] * (b[i] - sub);
    if (a.dw)
      for (int j = 0; j < a.k; ++j) {
        const int e = __builtin_amdgcn_readlane(id, j);
        const float v = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(add), j));
#pragma unroll
        for (int i = 0; i < M; ++i)
          if (lane + 64 * i == e) r[i] += v;
      }
#pragma unroll
    for (int i = 0; i < M; ++i)
      if (lane + 64 * i < a.E) dz[lane + 64 * i] = r[i];
  }
}

template <int M>
hipError_t run_gate(const GateArgs& a, int grid, hipStream_t st) {
  if (a.counts || a.loss)
    hipLaunchKernelGGL((gate_kernel<M, true>), dim3(grid), dim3(kGateWaves * 64), 0, st, a);
  else
    hipLaunchKernelGGL((gate_kernel<M, false>), dim3(grid), dim3(kGateWaves * 64), 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gate(const GateArgs& a, hipStream_t st) {
  const int grid = gate_parts(a.T);
  hipError_t err = a.E <= 64    ? run_gate<1>(a, grid, st)
                   : a.E <= 128 ? run_gate<2>(a, grid, st)
                   : a.E <= 256 ? run_gate<4>(a, grid, st)
                   : a.E <= 512 ? run_gate<8>(a, grid, st)
                                : run_gate<16>(a, grid, st);
  if (err != hipSuccess || !(a.counts || a.loss)) return err;
  hipLaunchKernelGGL(gate_reduce_kernel, dim3((a.E + 63) / 64), dim3(256), 0, st, a, grid);
  return hipGetLastError();
}

hipError_t launch_gate_backward(const GateBackward& a, hipStream_t st) {
  const int waves = a.T < 8192 ? a.T : 8192;
  const dim3 g((waves + kGateWaves - 1) / kGateWaves), b(kGateWaves * 64);
  if (a.E <= 64) hipLaunchKernelGGL(gate_backward_kernel<1>, g, b, 0, st, a);
  else if (a.E <= 128) hipLaunchKernelGGL(gate_backward_kernel<2>, g, b, 0, st, a);
  else if (a.E <= 256) hipLaunchKernelGGL(gate_backward_kernel<4>, g, b, 0, st, a);
  else if (a.E <= 512) hipLaunchKernelGGL(gate_backward_kernel<8>, g, b, 0, st, a);
  else hipLaunchKernelGGL(gate_backward_kernel<16>, g, b, 0, st, a);
  return hipGetLastError();
}

}  // namespace moe
