// router_train.hip - the router's product z = x W^T and its gradient:
//   dx = dz W (BF16)         [T][H] = [T][E] [E][H]
//   dW = dz^T x (fp32)       [E][H] = [E][T] [T][H]
//
// All of it runs on the BF16 matrix cores with fp32 accumulation.  Where the
// result is fp32 (z, dW), an fp32 factor enters as three BF16 parts, all its 24
// bits; where it is rounded to BF16 (dx), as two, to within 2^-16, and the
// product of two small parts is left out.
//
// dx is computed transposed, rows h, columns tokens, so that a lane ends up
// with 16 consecutive h of one token: rows r = 4 q + i of the four 16-row
// tiles j of a chunk of 64 are h = 16 q + 4 j + i.
#include "device.hpp"
#include "kernels.hpp"

namespace moe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ bf16x8 frag(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }
__device__ __forceinline__ v4f mfma(u32x4 a, u32x4 b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(a), frag(b), c, 0, 0, 0);
}

__device__ __forceinline__ void split8(const float (&v)[8], u32x4& hi, u32x4& lo) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h, l;
    bf16_split2(v[2 * i], v[2 * i + 1], h, l);
    hi[i] = h;
    lo[i] = l;
  }
}

// three parts: all 24 bits
__device__ __forceinline__ void split8x3(const float (&v)[8], u32x4& hi, u32x4& mid, u32x4& lo) {
  float r[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const v2bf h = {(__bf16)v[2 * i], (__bf16)v[2 * i + 1]};
    hi[i] = __builtin_bit_cast(uint32_t, h);
    r[2 * i] = v[2 * i] - bf16_lo(hi[i]);
    r[2 * i + 1] = v[2 * i + 1] - bf16_hi(hi[i]);
  }
  split8(r, mid, lo);
}

// ---- logits -------------------------------------------------------------------
// z = x W^T, computed transposed: rows are experts (row r = 4 q + i of tile j of
// a block of 16 ET is expert 4 ET q + 4 j + i, so a lane ends up with 4 ET
// consecutive experts of a token), columns tokens.  Both operands have H in
// order, so they go straight from memory into the operand registers.
//
// A workgroup is 8 waves: EW of them side by side over blocks of 16 ET experts,
// all on the same 16 NT tokens (whose x the others find in L1), and 8 / EW
// slices of H, whose sums meet in LDS in slice order.  D - 1 steps of 32 h are
// in flight per wave.  An fp32 W is split into three BF16 parts in registers
// (all 24 bits; BF16 products are exact, so z is an fp32 sum of exact terms).
constexpr int kLgWaves = 8;

template <int NT, int ET, bool RF32, int D>
__global__ __launch_bounds__(kLgWaves * 64, 2) void router_logits_kernel(
    const uint16_t* __restrict__ x, const void* __restrict__ w, int T, int H, int E, int log_ew,
    float* __restrict__ z) {
  extern __shared__ v4f lred[];                       // [slice - 1][e wave][ET * NT][64]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, q = lane >> 4;
  const int EW = 1 << log_ew, ew = wave & (EW - 1), slice = wave >> log_ew;
  const int KW = kLgWaves >> log_ew;
  const int64_t t0 = (int64_t)blockIdx.x * 16 * NT;
  const int e0 = ((int)blockIdx.y * EW + ew) * 16 * ET;
  const int steps = H / 32, n_it = slice < steps ? (steps - slice + KW - 1) / KW : 0;

  // rows past the end read the last one; their results are not stored
  const uint16_t* xp[NT];
  int64_t wo[ET];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int64_t t = t0 + 16 * j + r;
    xp[j] = x + (t < T ? t : T - 1) * H + 8 * q;
  }
#pragma unroll
  for (int j = 0; j < ET; ++j) {
    const int e = e0 + 4 * ET * (r >> 2) + 4 * j + (r & 3);
    wo[j] = (int64_t)(e < E ? e : E - 1) * H + 8 * q;
  }
  struct Step {
    u32x4 x[NT];
    u32x4 w[ET][RF32 ? 2 : 1];
  };
  auto load = [&](Step& s, int it) {
    const int k = 32 * (slice + (it < n_it ? it : n_it - 1) * KW);
#pragma unroll
    for (int j = 0; j < NT; ++j) s.x[j] = *reinterpret_cast<const u32x4*>(xp[j] + k);
#pragma unroll
    for (int j = 0; j < ET; ++j) {
      if (RF32) {
        const u32x4* p =
            reinterpret_cast<const u32x4*>(static_cast<const float*>(w) + wo[j] + k);
        s.w[j][0] = p[0];
        s.w[j][RF32 ? 1 : 0] = p[1];
      } else {
        s.w[j][0] =
            *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(w) + wo[j] + k);
      }
    }
  };
  v4f acc[ET][NT];
#pragma unroll
  for (int e = 0; e < ET; ++e)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[e][j] = v4f{0.f, 0.f, 0.f, 0.f};
  if (n_it > 0) {
    Step s[D];
#pragma unroll
    for (int d = 0; d < D - 1; ++d) load(s[d], d);
    for (int i0 = 0; i0 < n_it; i0 += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (i0 + d >= n_it) break;
        load(s[(d + D - 1) % D], i0 + d + D - 1);     // past the end: the last again
#pragma unroll
        for (int e = 0; e < ET; ++e) {
          if (RF32) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(s[d].w[e][i / 4 * RF32][i % 4]);
            u32x4 hi, mid, lo;
            split8x3(v, hi, mid, lo);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              acc[e][j] = mfma(lo, s[d].x[j], acc[e][j]);
              acc[e][j] = mfma(mid, s[d].x[j], acc[e][j]);
              acc[e][j] = mfma(hi, s[d].x[j], acc[e][j]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[e][j] = mfma(s[d].w[e][0], s[d].x[j], acc[e][j]);
          }
        }
      }
    }
  }
  if (slice > 0) {
#pragma unroll
    for (int e = 0; e < ET; ++e)
#pragma unroll
      for (int j = 0; j < NT; ++j)
        lred[(((slice - 1) * EW + ew) * ET * NT + e * NT + j) * 64 + lane] = acc[e][j];
  }
  __syncthreads();
  if (slice > 0) return;
  for (int k = 0; k < KW - 1; ++k)
#pragma unroll
    for (int e = 0; e < ET; ++e)
#pragma unroll
      for (int j = 0; j < NT; ++j)
        acc[e][j] += lred[((k * EW + ew) * ET * NT + e * NT + j) * 64 + lane];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int64_t t = t0 + 16 * j + r;
    if (t >= T) continue;
#pragma unroll
    for (int e = 0; e < ET; ++e) {
      const int c = e0 + 4 * ET * q + 4 * e;
      float* o = z + t * E + c;
      if (E % 4 == 0) {
        if (c < E) *reinterpret_cast<v4f*>(o) = acc[e][j];
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c + i < E) o[i] = acc[e][j][i];
      }
    }
  }
}

template <int NT, int ET, bool RF32, int D>
hipError_t run_logits(const void* x, const void* w, int T, int H, int E, int log_ew, float* z,
                      hipStream_t st) {
  const int ew = 1 << log_ew;
  const dim3 g((T + 16 * NT - 1) / (16 * NT), (E + 16 * ET * ew - 1) / (16 * ET * ew));
  const size_t lds = (size_t)(kLgWaves - ew) * ET * NT * 64 * sizeof(v4f);
  hipLaunchKernelGGL((router_logits_kernel<NT, ET, RF32, D>), g, dim3(kLgWaves * 64), lds, st,
                     static_cast<const uint16_t*>(x), w, T, H, E, log_ew, z);
  return hipGetLastError();
}

// ---- W in operand order: [chunk of 64 h][32 e][tile j][part][64 lanes] -------
template <bool RF32>
__global__ __launch_bounds__(256) void pack_router_kernel(const void* __restrict__ w, int H, int E,
                                                          u32x4* __restrict__ out) {
  constexpr int PL = RF32 ? 2 : 1;
  const int c = blockIdx.x, ks = blockIdx.y, kq = threadIdx.x >> 6, hh = threadIdx.x & 63;
  const int h = 64 * c + hh;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = 32 * ks + 8 * kq + i;
    v[i] = 0.f;
    if (h < H && e < E) {
      const int64_t at = (int64_t)e * H + h;
      v[i] = RF32 ? static_cast<const float*>(w)[at]
                  : __uint_as_float((uint32_t) static_cast<const uint16_t*>(w)[at] << 16);
    }
  }
  u32x4 hi, lo;
  split8(v, hi, lo);
  const int j = (hh & 15) >> 2, r = 4 * (hh >> 4) + (hh & 3);
  u32x4* o = out + ((((int64_t)c * gridDim.y + ks) * 4 + j) * PL) * 64 + 16 * kq + r;
  o[0] = hi;
  if (RF32) o[64] = lo;
}

// ---- dx -----------------------------------------------------------------------
// A workgroup holds dz of 16 NTL tokens (all experts, both parts, operand
// order) in LDS, and its 8 waves stream chunks of 64 h of W past it.
constexpr int kDxWaves = 8;

template <int NTL, bool RF32>
__global__ __launch_bounds__(kDxWaves * 64) void router_dx_kernel(const float* __restrict__ dz,
                                                                  const u32x4* __restrict__ wf,
                                                                  int T, int H, int E,
                                                                  uint16_t* __restrict__ dx) {
  constexpr int PL = RF32 ? 2 : 1;
  extern __shared__ u32x4 sb[];                       // [e block][token tile][part][64]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 15, q = lane >> 4;
  const int nks = (E + 31) / 32, nc = (H + 63) / 64;
  const int64_t t0 = (int64_t)blockIdx.x * 16 * NTL;
  const bool vec = E % 4 == 0;
  for (int it = wave; it < nks * NTL; it += kDxWaves) {
    const int ks = it / NTL, nt = it % NTL;
    const int64_t t = t0 + 16 * nt + n;
    const int e0 = 32 * ks + 8 * q;
    float v[8] = {};
    if (t < T) {
      const float* src = dz + t * E + e0;
      if (vec) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (e0 + 4 * i < E) {
            const float4 f = *reinterpret_cast<const float4*>(src + 4 * i);
            v[4 * i] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
          }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (e0 + i < E) v[i] = src[i];
      }
    }
    u32x4 hi, lo;
    split8(v, hi, lo);
    sb[(it * 2) * 64 + lane] = hi;
    sb[(it * 2 + 1) * 64 + lane] = lo;
  }
  __syncthreads();
  for (int c = blockIdx.y * kDxWaves + wave; c < nc; c += gridDim.y * kDxWaves) {
    v4f acc[4][NTL];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int t = 0; t < NTL; ++t) acc[j][t] = v4f{0.f, 0.f, 0.f, 0.f};
    const u32x4* src = wf + (int64_t)c * nks * 4 * PL * 64 + lane;
    u32x4 a[4 * PL];
#pragma unroll
    for (int i = 0; i < 4 * PL; ++i) a[i] = src[i * 64];
    for (int ks = 0; ks < nks; ++ks) {
      u32x4 an[4 * PL];
      const u32x4* nsrc = src + (int64_t)(ks + 1 < nks ? ks + 1 : ks) * 4 * PL * 64;
#pragma unroll
      for (int i = 0; i < 4 * PL; ++i) an[i] = nsrc[i * 64];
#pragma unroll
      for (int t = 0; t < NTL; ++t) {
        const u32x4 hi = sb[((ks * NTL + t) * 2) * 64 + lane];
        const u32x4 lo = sb[((ks * NTL + t) * 2 + 1) * 64 + lane];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[j][t] = mfma(a[j * PL], hi, acc[j][t]);
          acc[j][t] = mfma(a[j * PL], lo, acc[j][t]);
          if (RF32) acc[j][t] = mfma(a[j * PL + PL - 1], hi, acc[j][t]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4 * PL; ++i) a[i] = an[i];
    }
    const int h = 64 * c + 16 * q;
    if (h >= H) continue;
#pragma unroll
    for (int t = 0; t < NTL; ++t) {
      const int64_t tok = t0 + 16 * t + n;
      if (tok >= T) continue;
      u32x4 o[2];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const v2bf a0 = {(__bf16)acc[j][t][0], (__bf16)acc[j][t][1]};
        const v2bf a1 = {(__bf16)acc[j][t][2], (__bf16)acc[j][t][3]};
        o[j / 2][2 * (j & 1)] = __builtin_bit_cast(uint32_t, a0);
        o[j / 2][2 * (j & 1) + 1] = __builtin_bit_cast(uint32_t, a1);
      }
      u32x4* d = reinterpret_cast<u32x4*>(dx + tok * H + h);
      d[0] = o[0];
      d[1] = o[1];
    }
  }
}

// ---- dz^T in operand order: [32 tokens][16 e][part][64 lanes] -----------------
// Three parts here: dW is fp32, and with two its error was 2.5e-6 of its norm
// where an fp32 product has 5e-7.
constexpr int kZp = 3;

__global__ __launch_bounds__(256) void pack_dz_kernel(const float* __restrict__ dz, int T, int E,
                                                      int net, u32x4* __restrict__ out) {
  const int64_t kt = blockIdx.x;
  const int Ep = net * 16;
  for (int i = threadIdx.x; i < Ep * 4; i += 256) {
    const int e = i % Ep, kq = i / Ep;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t t = 32 * kt + 8 * kq + j;
      v[j] = t < T && e < E ? dz[t * E + e] : 0.f;
    }
    u32x4 hi, mid, lo;
    split8x3(v, hi, mid, lo);
    u32x4* o = out + ((kt * net + e / 16) * kZp) * 64 + 16 * kq + e % 16;
    o[0] = hi;
    o[64] = mid;
    o[128] = lo;
  }
}

// ---- dW -----------------------------------------------------------------------
// A workgroup: 16 ET experts x 256 h over a slice of the tokens.  dz^T of 32
// tokens goes through LDS (double buffered), shared by the four waves; a wave
// has 64 h of its own, whose x it reads straight from memory (lane (n, q): 8
// tokens x 4 h) and transposes in registers: column n of the f-th operand is
// h = 4 n + f, so a lane ends up with four consecutive h of a row.
constexpr int kDwWaves = 4;

__device__ __forceinline__ uint32_t pack_lo(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x05040100u);
}
__device__ __forceinline__ uint32_t pack_hi(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x07060302u);
}

template <int ET>
__global__ __launch_bounds__(kDwWaves * 64, 2) void router_dw_kernel(
    const uint16_t* __restrict__ x, const u32x4* __restrict__ zf, int T, int H, int E, int net,
    int per_slice, float* __restrict__ out) {
  constexpr int kStage = ET * kZp * 64, kCopies = (kStage + kDwWaves * 64 - 1) / (kDwWaves * 64);
  __shared__ u32x4 sa[2][kStage];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 15, q = lane >> 4;
  const int nkt = (T + 31) / 32;
  const int k0 = blockIdx.z * per_slice, k1 = min(nkt, k0 + per_slice);
  const int h = blockIdx.x * 256 + wave * 64 + 4 * n;
  const bool hin = h < H;
  const u32x4* zsrc = zf + (int64_t)blockIdx.y * ET * kZp * 64;

  u32x4 za[kCopies];
  uint2 xr[8];
  auto load = [&](int kt) {
#pragma unroll
    for (int c = 0; c < kCopies; ++c) {
      const int i = c * kDwWaves * 64 + threadIdx.x;
      if (i < kStage) za[c] = zsrc[(int64_t)kt * net * kZp * 64 + i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t t = 32 * (int64_t)kt + 8 * q + i;
      xr[i] = make_uint2(0, 0);
      if (t < T && hin) xr[i] = *reinterpret_cast<const uint2*>(x + t * H + h);
    }
  };
  auto stage = [&](int b) {
#pragma unroll
    for (int c = 0; c < kCopies; ++c) {
      const int i = c * kDwWaves * 64 + threadIdx.x;
      if (i < kStage) sa[b][i] = za[c];
    }
  };
  v4f acc[ET][4];
#pragma unroll
  for (int e = 0; e < ET; ++e)
#pragma unroll
    for (int f = 0; f < 4; ++f) acc[e][f] = v4f{0.f, 0.f, 0.f, 0.f};
  if (k0 < k1) {
    load(k0);
    stage(0);
  }
  for (int kt = k0; kt < k1; ++kt) {
    u32x4 b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      b[0][i] = pack_lo(xr[2 * i].x, xr[2 * i + 1].x);
      b[1][i] = pack_hi(xr[2 * i].x, xr[2 * i + 1].x);
      b[2][i] = pack_lo(xr[2 * i].y, xr[2 * i + 1].y);
      b[3][i] = pack_hi(xr[2 * i].y, xr[2 * i + 1].y);
    }
    if (kt + 1 < k1) load(kt + 1);
    const int buf = (kt - k0) & 1;
    __syncthreads();                                  // this step's dz is in LDS
#pragma unroll
    for (int e = 0; e < ET; ++e) {
#pragma unroll
      for (int p = kZp - 1; p >= 0; --p) {            // small parts first
        const u32x4 z = sa[buf][(e * kZp + p) * 64 + lane];
#pragma unroll
        for (int f = 0; f < 4; ++f) acc[e][f] = mfma(z, b[f], acc[e][f]);
      }
    }
    // the other buffer was last read a step ago, before this step's barrier
    if (kt + 1 < k1) stage(buf ^ 1);
  }
  if (!hin) return;
  float* o = out + (int64_t)blockIdx.z * E * H;
#pragma unroll
  for (int e = 0; e < ET; ++e)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = (blockIdx.y * ET + e) * 16 + 4 * q + i;
      if (row < E)
        *reinterpret_cast<v4f*>(o + (int64_t)row * H + h) =
            v4f{acc[e][0][i], acc[e][1][i], acc[e][2][i], acc[e][3][i]};
    }
}

// the token slices' partial sums, in slice order
__global__ __launch_bounds__(256) void sum_slices_kernel(const v4f* __restrict__ part, int slices,
                                                         int64_t n4, v4f* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n4) return;
  v4f s = part[i];
  for (int k = 1; k < slices; ++k) s += part[k * n4 + i];
  out[i] = s;
}

// experts per dW workgroup in tiles of 16, the number of those tiles, and the
// token slices: two workgroups per compute unit where a slice has at least 8
// steps of 32 tokens; short batches take fewer experts a workgroup instead
struct DwPlan {
  int et, net, slices, per_slice;
};
DwPlan dw_plan(int T, int H, int E) {
  DwPlan p;
  const int nkt = T > 0 ? (T + 31) / 32 : 1, hx = (H + 255) / 256;
  const int most = nkt / 8 > 1 ? nkt / 8 : 1;
  p.et = E > 64 ? 8 : E > 32 ? 4 : E > 16 ? 2 : 1;
  while (p.et > 1 && hx * ((E + 16 * p.et - 1) / (16 * p.et)) * most < 192) p.et /= 2;
  const int ey = (E + 16 * p.et - 1) / (16 * p.et), tiles = ey * hx;
  p.net = ey * p.et;
  int s = (512 + tiles - 1) / tiles;
  if (s > most) s = most;
  p.per_slice = (nkt + s - 1) / s;
  p.slices = (nkt + p.per_slice - 1) / p.per_slice;
  return p;
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

struct Ws {
  size_t wf, zf, part, total;
};
Ws carve(int T, int H, int E) {
  const DwPlan p = dw_plan(T, H, E);
  Ws w;
  size_t o = 0;
  w.wf = o; o = up256(o + (size_t)((H + 63) / 64) * ((E + 31) / 32) * 4 * 2 * 1024);
  w.zf = o; o = up256(o + (size_t)((T + 31) / 32) * p.net * kZp * 1024);
  w.part = o; o = up256(o + (p.slices > 1 ? (size_t)p.slices * E * H * 4 : 0));
  w.total = o;
  return w;
}

template <bool RF32>
hipError_t run_dx(const RouterBackward& a, const u32x4* wf, hipStream_t st) {
  const int nks = (a.E + 31) / 32, nc = (a.H + 63) / 64;
  // tokens per workgroup: dz of all experts in 128 KB of LDS, and few enough
  // tokens that short batches still spread over the compute units
  int ntl = nks <= 8 ? 8 : nks <= 16 ? 4 : 2;
  while (ntl > 2 && (a.T + 16 * ntl - 1) / (16 * ntl) < 64) ntl /= 2;
  const int gx = (a.T + 16 * ntl - 1) / (16 * ntl);
  int gy = 256 / gx;
  const int most = (nc + kDxWaves - 1) / kDxWaves;
  gy = gy < 1 ? 1 : gy > most ? most : gy;
  const size_t lds = (size_t)nks * ntl * 2 * 1024;
  const dim3 g(gx, gy), b(kDxWaves * 64);
  if (ntl == 8)
    hipLaunchKernelGGL((router_dx_kernel<8, RF32>), g, b, lds, st, a.dz, wf, a.T, a.H, a.E, a.dx);
  else if (ntl == 4)
    hipLaunchKernelGGL((router_dx_kernel<4, RF32>), g, b, lds, st, a.dz, wf, a.T, a.H, a.E, a.dx);
  else
    hipLaunchKernelGGL((router_dx_kernel<2, RF32>), g, b, lds, st, a.dz, wf, a.T, a.H, a.E, a.dx);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_router_logits(const void* x, const void* w, int router_f32, int T, int H, int E,
                                float* z, hipStream_t st) {
  // The widest tile that still gives 192 workgroups (3/4 of the compute units):
  // 64 tokens x 256 experts reads x once and W for every 64 tokens; then fewer
  // experts (more slices of H per workgroup), fewer tokens, last 16 x 16.
  const auto blocks = [&](int tokens, int experts) {
    return (int64_t)((T + tokens - 1) / tokens) * ((E + experts - 1) / experts);
  };
  for (int log_ew = E > 128 ? 2 : E > 64 ? 1 : 0; log_ew >= 0; --log_ew)
    if (blocks(64, 64 << log_ew) >= 192)
      return router_f32 ? run_logits<4, 4, true, 2>(x, w, T, H, E, log_ew, z, st)
                        : run_logits<4, 4, false, 3>(x, w, T, H, E, log_ew, z, st);
  if (blocks(32, 64) >= 192)
    return router_f32 ? run_logits<2, 4, true, 2>(x, w, T, H, E, 0, z, st)
                      : run_logits<2, 4, false, 3>(x, w, T, H, E, 0, z, st);
  if (blocks(16, 64) >= 192)
    return router_f32 ? run_logits<1, 4, true, 2>(x, w, T, H, E, 0, z, st)
                      : run_logits<1, 4, false, 3>(x, w, T, H, E, 0, z, st);
  return router_f32 ? run_logits<1, 1, true, 4>(x, w, T, H, E, 0, z, st)
                    : run_logits<1, 1, false, 4>(x, w, T, H, E, 0, z, st);
}

size_t router_backward_bytes(int T, int H, int E) { return carve(T, H, E).total; }

hipError_t launch_router_backward(const RouterBackward& a, hipStream_t st) {
  const Ws L = carve(a.T, a.H, a.E);
  u32x4* wf = reinterpret_cast<u32x4*>(a.ws + L.wf);
  u32x4* zf = reinterpret_cast<u32x4*>(a.ws + L.zf);
  hipError_t err = hipSuccess;
  if (a.dx) {
    const dim3 g((a.H + 63) / 64, (a.E + 31) / 32);
    if (a.router_f32)
      hipLaunchKernelGGL(pack_router_kernel<true>, g, dim3(256), 0, st, a.w, a.H, a.E, wf);
    else
      hipLaunchKernelGGL(pack_router_kernel<false>, g, dim3(256), 0, st, a.w, a.H, a.E, wf);
    err = hipGetLastError();
    if (err != hipSuccess) return err;
    err = a.router_f32 ? run_dx<true>(a, wf, st) : run_dx<false>(a, wf, st);
    if (err != hipSuccess) return err;
  }
  if (!a.dw) return err;
  const DwPlan p = dw_plan(a.T, a.H, a.E);
  hipLaunchKernelGGL(pack_dz_kernel, dim3((a.T + 31) / 32), dim3(256), 0, st, a.dz, a.T, a.E,
                     p.net, zf);
  err = hipGetLastError();
  if (err != hipSuccess) return err;
  float* out = p.slices > 1 ? reinterpret_cast<float*>(a.ws + L.part) : a.dw;
  const dim3 g((a.H + 255) / 256, p.net / p.et, p.slices), b(kDwWaves * 64);
  const uint16_t* x = static_cast<const uint16_t*>(a.x);
  if (p.et == 8)
    hipLaunchKernelGGL(router_dw_kernel<8>, g, b, 0, st, x, zf, a.T, a.H, a.E, p.net, p.per_slice,
                       out);
  else if (p.et == 4)
    hipLaunchKernelGGL(router_dw_kernel<4>, g, b, 0, st, x, zf, a.T, a.H, a.E, p.net, p.per_slice,
                       out);
  else if (p.et == 2)
    hipLaunchKernelGGL(router_dw_kernel<2>, g, b, 0, st, x, zf, a.T, a.H, a.E, p.net, p.per_slice,
                       out);
  else
    hipLaunchKernelGGL(router_dw_kernel<1>, g, b, 0, st, x, zf, a.T, a.H, a.E, p.net, p.per_slice,
                       out);
  err = hipGetLastError();
  if (err != hipSuccess || p.slices == 1) return err;
  const int64_t n4 = (int64_t)a.E * a.H / 4;
  hipLaunchKernelGGL(sum_slices_kernel, dim3((unsigned)((n4 + 255) / 256)), dim3(256), 0, st,
                     reinterpret_cast<const v4f*>(out), p.slices, n4,
                     reinterpret_cast<v4f*>(a.dw));
  return hipGetLastError();
}

}  // namespace moe
