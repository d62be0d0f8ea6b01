// q4_experts.hip - decode of experts held as 4-bit integer matrices (q4.hpp):
// gate and up with SwiGLU, then down with the weighted combine, two launches.
//
//   h_p  = silu(W_g x_t) * (W_u x_t)        p = (t, j), expert ids[p]
//   y_t  = sum_j w_tj W_d h_tj  (+ the shared expert, weight 1)
//
// Bound: HBM, the bytes of the distinct experts.  Both kernels read each
// chosen expert once for up to 16 of its tokens (the columns of one matrix
// instruction); tokens past 16 read it again, from cache.
#include "q4.hpp"

namespace moe {
namespace {

using namespace q4;

// ---- gate / up --------------------------------------------------------------
// grid.y names a pair p (the last one the shared expert); the first pair of an
// expert takes all pairs of that expert, the others leave at once.  The list
// of its pairs is kept for the down kernel.  8 waves: (8 / KS) row tiles x KS
// slices of H, partial sums met in LDS in slice order.
constexpr int kGuWaves = 8;

template <int G>
__global__ __launch_bounds__(kGuWaves * 64) void q4_gate_up_kernel(Q4Experts a) {
  __shared__ v4f red[kGuWaves][2][64];
  __shared__ int16_t list[kQ4MaxPairs];
  __shared__ int wcount[kGuWaves];
  __shared__ int not_first;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int p = blockIdx.y;
  int n_cols, slot = -1;
  const uint8_t* block;
  if (p < a.P) {
    const int e = a.ids[p];
    if (e >= 0 && e < a.E) slot = a.slot_of ? a.slot_of[e] : e;
    if (threadIdx.x == 0) not_first = 0;
    const int i = threadIdx.x;
    const bool match = slot >= 0 && i < a.P && a.ids[i] == e;
    const uint64_t b = __ballot(match);
    if (lane == 0) wcount[wave] = __popcll(b);
    __syncthreads();
    if (match && i < p) not_first = 1;
    int base = 0, total = 0;
#pragma unroll
    for (int v = 0; v < kGuWaves; ++v) {
      if (v < wave) base += wcount[v];
      total += wcount[v];
    }
    if (match) list[base + __popcll(b & ((1ull << lane) - 1))] = (int16_t)i;
    __syncthreads();
    n_cols = not_first ? 0 : total;                  // 0 where the expert is not resident
    block = a.pool + (int64_t)slot * a.expert_bytes;
  } else {
    n_cols = a.T;
    block = a.shared;
  }
  if (blockIdx.x == 0) {
    if (threadIdx.x == 0) a.units[p] = make_int2(n_cols, slot);
    if (p < a.P)
      for (int i = threadIdx.x; i < n_cols; i += kGuWaves * 64)
        a.lists[(int64_t)p * a.P + i] = list[i];
  }
  if (n_cols == 0) return;

  const int KS = 1 << a.log_ks_gu, slice = wave & (KS - 1), set = wave >> a.log_ks_gu;
  const int sets = kGuWaves >> a.log_ks_gu, tiles = a.I / 16, nkb = (a.H + 127) / 128;
  const int tile = min((int)blockIdx.x * sets + set, tiles - 1);
  const int q = lane >> 4;
  const Matrix mg{block + a.off[0], block + a.off[1], nullptr, nkb};
  const Matrix mu{block + a.off[2], block + a.off[3], nullptr, nkb};

  for (int c0 = 0; c0 < n_cols; c0 += 16) {
    const int c = c0 + (lane & 15);
    const bool live = c < n_cols;
    int token = 0;
    if (live) token = p < a.P ? list[c] / a.k : c;
    const uint16_t* xrow = a.x + (int64_t)token * a.H;
    v4f ag = v4f{0.f, 0.f, 0.f, 0.f}, au = ag;
    auto load_x = [&](u32x4 (&x)[4], int kb) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int k = 128 * kb + 32 * s + 8 * q;
        x[s] = u32x4{0, 0, 0, 0};
        if (live && k < a.H) x[s] = *reinterpret_cast<const u32x4*>(xrow + k);
      }
    };
    Tile<G, false> tg, tu;
    u32x4 xr[4];
    if (slice < nkb) {
      load_tile<G, false>(tg, mg, tile, slice);
      load_tile<G, false>(tu, mu, tile, slice);
      load_x(xr, slice);
    }
    for (int kb = slice; kb < nkb; kb += KS) {
      Tile<G, false> ng, nu;
      u32x4 nx[4];
      const int kn = kb + KS;
      if (kn < nkb) {
        load_tile<G, false>(ng, mg, tile, kn);
        load_tile<G, false>(nu, mu, tile, kn);
        load_x(nx, kn);
      }
      bf16x8 x[1][4], w[4];
      v4f cs[128 / G];
#pragma unroll
      for (int s = 0; s < 4; ++s) x[0][s] = frag(xr[s]);
      group_sums<G, 1>(cs, x);
      tile_weights<G, false>(w, tg);
      mul_tile<G, false, 1>(ag, tg, w, x, cs);
      tile_weights<G, false>(w, tu);
      mul_tile<G, false, 1>(au, tu, w, x, cs);
      tg = ng;
      tu = nu;
#pragma unroll
      for (int s = 0; s < 4; ++s) xr[s] = nx[s];
    }
    __syncthreads();                                  // the previous columns are read
    red[wave][0][lane] = ag;
    red[wave][1][lane] = au;
    __syncthreads();
    for (int i = threadIdx.x; i < sets * 64; i += kGuWaves * 64) {
      const int l = i & 63, st = i >> 6;
      v4f g = v4f{0.f, 0.f, 0.f, 0.f}, u = g;
      for (int s = 0; s < KS; ++s) {
        g += red[(st << a.log_ks_gu) + s][0][l];
        u += red[(st << a.log_ks_gu) + s][1][l];
      }
      const int col = c0 + (l & 15), tl = blockIdx.x * sets + st;
      if (col >= n_cols || tl >= tiles) continue;
      const int row = p < a.P ? list[col] : a.P + col;
      float h[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = g[e] / (1.f + expf(-g[e])) * u[e];
      // h as two BF16 parts, h to within 2^-17 of itself: the down product
      // takes both, so y keeps fp32's accuracy rather than BF16's
      uint2 hi, lo;
      bf16_split2(h[0], h[1], hi.x, lo.x);
      bf16_split2(h[2], h[3], hi.y, lo.y);
      const int64_t at = (int64_t)row * a.I + 16 * tl + 4 * (l >> 4);
      *reinterpret_cast<uint2*>(a.h_hi + at) = hi;
      *reinterpret_cast<uint2*>(a.h_lo + at) = lo;
    }
  }
}

// ---- down + combine -----------------------------------------------------------
// One workgroup per 16 rows of y for all tokens and experts, so the combine
// needs neither atomics on memory nor a second pass: the column blocks of all
// units' tiles (unit: an expert's pairs, up to 16) go round the 16 waves, each
// adds its gate-weighted results into a y tile of its own in LDS, and the 16
// tiles are summed in wave order.
constexpr int kDnWaves = 16;

template <int G>
__global__ __launch_bounds__(kDnWaves * 64) void q4_down_kernel(Q4Experts a) {
  extern __shared__ float yl[];                       // [wave][T][16]
  __shared__ int s_item[kQ4MaxItems];                 // pair << 16 | first entry
  __shared__ uint8_t s_count[kQ4MaxItems];
  __shared__ int s_slot[kQ4MaxPairs + 1];
  __shared__ int16_t s_ent[kQ4MaxPairs + 64];
  __shared__ int s_wsum[kDnWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane >> 4;
  const int n_units = a.P + (a.shared ? 1 : 0);

  // unit list: items of up to 16 entries, in pair order
  const int i = threadIdx.x;
  int2 u = make_int2(0, -1);
  if (i < n_units) u = a.units[i];
  const int chunks = (u.x + 15) / 16;
  const int packed = chunks << 16 | u.x;
  const int inc = wave_scan_dpp(packed);
  if (lane == 63) s_wsum[wave] = inc;
  for (int j = threadIdx.x; j < kDnWaves * a.T * 16; j += kDnWaves * 64) yl[j] = 0.f;
  __syncthreads();
  int base = inc - packed, total = 0;
#pragma unroll
  for (int v = 0; v < kDnWaves; ++v) {
    if (v < wave) base += s_wsum[v];
    total += s_wsum[v];
  }
  if (i < n_units) {
    s_slot[i] = u.y;
    const int it = base >> 16, en = base & 0xffff;
    for (int c = 0; c < chunks; ++c) {
      s_item[it + c] = i << 16 | (en + 16 * c);
      s_count[it + c] = (uint8_t)min(16, u.x - 16 * c);
    }
    for (int c = 0; c < u.x; ++c)
      s_ent[en + c] = i < a.P ? a.lists[(int64_t)i * a.P + c] : (int16_t)(a.P + c);
  }
  __syncthreads();

  const int items = total >> 16, nkb = (a.I + 127) / 128, jobs = items * nkb;
  const int tile = blockIdx.x;
  float* mine = yl + (int64_t)wave * a.T * 16;

  struct Job {
    Tile<G, false> t;
    u32x4 x[2][4];
    int ent;                                          // this lane's column: an h row, -1 none
  };
  auto load = [&](Job& j, int job) {
    const int it = job / nkb, kb = job - it * nkb;
    const int item = s_item[it], p = item >> 16;
    const uint8_t* block = p < a.P ? a.pool + (int64_t)s_slot[p] * a.expert_bytes : a.shared;
    const Matrix m{block + a.off[4], block + a.off[5], nullptr, nkb};
    load_tile<G, false>(j.t, m, tile, kb);
    const int c = lane & 15;
    j.ent = c < s_count[it] ? s_ent[(item & 0xffff) + c] : -1;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int k = 128 * kb + 32 * s + 8 * q;
      j.x[0][s] = j.x[1][s] = u32x4{0, 0, 0, 0};
      if (j.ent >= 0 && k < a.I) {
        const int64_t at = (int64_t)j.ent * a.I + k;
        j.x[0][s] = *reinterpret_cast<const u32x4*>(a.h_hi + at);
        j.x[1][s] = *reinterpret_cast<const u32x4*>(a.h_lo + at);
      }
    }
  };
  Job cur;
  if (wave < jobs) load(cur, wave);
  for (int job = wave; job < jobs; job += kDnWaves) {
    Job nxt;
    if (job + kDnWaves < jobs) load(nxt, job + kDnWaves);
    bf16x8 x[2][4], w[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      x[0][s] = frag(cur.x[0][s]);
      x[1][s] = frag(cur.x[1][s]);
    }
    v4f cs[128 / G], acc = v4f{0.f, 0.f, 0.f, 0.f};
    group_sums<G, 2>(cs, x);
    tile_weights<G, false>(w, cur.t);
    mul_tile<G, false, 2>(acc, cur.t, w, x, cs);
    if (cur.ent >= 0) {
      const int token = cur.ent < a.P ? cur.ent / a.k : cur.ent - a.P;
      const float wt = cur.ent < a.P ? a.w[cur.ent] : 1.f;
      // LDS adds: a token that names one expert twice has two columns here
#pragma unroll
      for (int e = 0; e < 4; ++e)
        __hip_atomic_fetch_add(&mine[token * 16 + 4 * q + e], wt * acc[e], __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_WORKGROUP);
    }
    cur = nxt;
  }
  __syncthreads();
  for (int j = threadIdx.x; j < a.T * 16; j += kDnWaves * 64) {
    float v = 0.f;
#pragma unroll
    for (int s = 0; s < kDnWaves; ++s) v += yl[(int64_t)s * a.T * 16 + j];
    a.y[(int64_t)(j >> 4) * a.H + 16 * tile + (j & 15)] = v;
  }
}

template <int G>
hipError_t run(const Q4Experts& a, hipStream_t st) {
  const int sets = kGuWaves >> a.log_ks_gu, n_units = a.P + (a.shared ? 1 : 0);
  hipLaunchKernelGGL((q4_gate_up_kernel<G>), dim3((a.I / 16 + sets - 1) / sets, n_units),
                     dim3(kGuWaves * 64), 0, st, a);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL((q4_down_kernel<G>), dim3(a.H / 16), dim3(kDnWaves * 64),
                     (size_t)kDnWaves * a.T * 16 * sizeof(float), st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_q4_experts(Q4Experts a, int group, hipStream_t st) {
  a.P = a.T * a.k;
  if (a.T < 1 || a.P > kQ4MaxPairs || a.T > kQ4MaxTokens) return hipErrorInvalidValue;
  const int nkb = (a.H + 127) / 128;
  a.log_ks_gu = nkb >= 8 ? 3 : nkb >= 4 ? 2 : nkb >= 2 ? 1 : 0;
  if (group == 32) return run<32>(a, st);
  if (group == 64) return run<64>(a, st);
  return run<128>(a, st);
}

}  // namespace moe
