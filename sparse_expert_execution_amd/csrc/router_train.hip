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
// z = x W^T.  Rows of x and W go through LDS: a copy instruction must take
// consecutive lanes along a row (read straight into operand registers, where
// neighbouring lanes are different rows, every lane costs a cache lookup of its
// own: 131 us where T = 16384, H = 4096, E = 256, whatever the line coverage).
//
// A workgroup is 8 waves on TM tokens x TE experts, 32 KS h per stage, STAGES
// stages in LDS, copied STAGES - 1 ahead (global to LDS, no registers).  Piece
// p (16 bytes) of row i sits at slot p ^ (i / 2) % 8 of a 128-byte row, p ^ i % 16
// of a longer one, so that the 16 rows of an operand read hit distinct banks.  A
// wave takes 16 WT tokens x 16 WE experts of one or more 32-h steps of the
// stage; the sums of the waves along h meet in LDS in order.
//
// The result is transposed, rows experts: row r = 4 q + i of tile j of a wave's
// experts is expert 4 WE q + 4 j + i, so a lane stores 4 WE consecutive ones.
// An fp32 W is split into three BF16 parts in registers (all 24 bits; BF16
// products are exact, so z is an fp32 sum of exact terms).
//
// Bound: for long batches the loads into the compute units (see
// launch_router_logits), twice the time of the matrix instructions; for short
// ones latency.
constexpr int kLgWaves = 8;

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)p;
}

// N operand reads with the wait in the same block: reads the compiler could see
// would also wait for the copies in flight into the other stages
__device__ __forceinline__ void lds_read2(const uint32_t (&a)[2], u32x4 (&v)[2]) {
  asm volatile(
      "ds_read_b128 %0, %2\n\tds_read_b128 %1, %3\n\ts_waitcnt lgkmcnt(0)"
      : "=&v"(v[0]), "=&v"(v[1])
      : "v"(a[0]), "v"(a[1])
      : "memory");
}
__device__ __forceinline__ void lds_read4(const uint32_t (&a)[4], u32x4 (&v)[4]) {
  asm volatile(
      "ds_read_b128 %0, %4\n\tds_read_b128 %1, %5\n\tds_read_b128 %2, %6\n\t"
      "ds_read_b128 %3, %7\n\ts_waitcnt lgkmcnt(0)"
      : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3])
      : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3])
      : "memory");
}
template <int N>
__device__ __forceinline__ void lds_read(const uint32_t (&a)[N], u32x4 (&v)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint32_t b[4] = {a[i], a[i + 1], a[i + 2], a[i + 3]};
      u32x4 t[4];
      lds_read4(b, t);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[i + k] = t[k];
    }
  } else if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const uint32_t b[2] = {a[i], a[i + 1]};
      u32x4 t[2];
      lds_read2(b, t);
      v[i] = t[0];
      v[i + 1] = t[1];
    }
  } else {
    static_assert(N == 1, "one, or an even number of reads");
    asm volatile("ds_read_b128 %0, %1\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(v[0])
                 : "v"(a[0])
                 : "memory");
  }
}

template <int NP>
__device__ __forceinline__ int piece_slot(int row, int p) {
  return NP == 8 ? p ^ ((row >> 1) & 7) : p ^ (row & 15);
}

template <int TM, int TE, int KS, int WT, int WE, bool RF32, int STAGES>
__global__ __launch_bounds__(kLgWaves * 64) void router_logits_kernel(
    const uint16_t* __restrict__ x, const void* __restrict__ w, int T, int H, int E,
    float* __restrict__ z) {
  constexpr int TWN = TM / (16 * WT), EWN = TE / (16 * WE), KWN = kLgWaves / (TWN * EWN);
  constexpr int NPX = 4 * KS, NPW = (RF32 ? 8 : 4) * KS;        // 16-byte pieces of a row
  constexpr int kX = TM * NPX / 64, kW = TE * NPW / 64;         // copies of a stage
  constexpr int kPer = (kX + kW) / kLgWaves;                    // a wave's
  constexpr int kStage = (kX + kW) * 64;                        // u32x4
  static_assert(kX % kLgWaves == 0 && kW % kLgWaves == 0 && KS % KWN == 0, "uneven waves");
  static_assert(KWN * TM * TE * 4 <= STAGES * kStage * 16 + TM * TE * 4, "sums do not fit");
  extern __shared__ u32x4 sl[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, q = lane >> 4;
  const int ew = wave % EWN, tw = wave / EWN % TWN, kw = wave / (EWN * TWN);
  const int64_t t0 = (int64_t)blockIdx.x * TM;
  const int e0 = blockIdx.y * TE;
  const int ns = (H + 32 * KS - 1) / (32 * KS);

  // this wave's copies: source of each at h = 0 and its piece's h; rows past the
  // end copy the last one (their results are not stored)
  const uint8_t* src[kPer];
  int hof[kPer];
#pragma unroll
  for (int c = 0; c < kPer; ++c) {
    const int i = wave * kPer + c;
    // copies 0..kX-1 are x, the rest W, 64 pieces each
    const bool is_x = i < kX;
    const int n = (is_x ? i : i - kX) * 64 + lane, np = is_x ? NPX : NPW;
    const int row = n / np;
    const int p = is_x ? piece_slot<NPX>(row, n % NPX) : piece_slot<NPW>(row, n % NPW);
    if (is_x) {
      const int64_t t = t0 + row < T ? t0 + row : T - 1;
      src[c] = reinterpret_cast<const uint8_t*>(x + t * H);
      hof[c] = 8 * p;
    } else {
      const int e = e0 + row < E ? e0 + row : E - 1;
      src[c] = static_cast<const uint8_t*>(w) + (int64_t)e * H * (RF32 ? 4 : 2);
      hof[c] = (RF32 ? 4 : 8) * p;
    }
  }
  auto issue = [&](int s, int buf) {
#pragma unroll
    for (int c = 0; c < kPer; ++c) {
      const int i = wave * kPer + c;
      int h = 32 * KS * s + hof[c];
      if (h >= H) h = 0;                              // not used
      const uint8_t* g = src[c] + (int64_t)h * (RF32 && i >= kX ? 4 : 2);
      __builtin_amdgcn_global_load_lds(g, &sl[buf * kStage + i * 64], 16, 0, 0);
    }
  };
  v4f acc[WE][WT];
#pragma unroll
  for (int e = 0; e < WE; ++e)
#pragma unroll
    for (int j = 0; j < WT; ++j) acc[e][j] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) issue(s < ns ? s : ns - 1, s);
  for (int s = 0; s < ns; ++s) {
    // this wave's copies of stage s are done once only the later STAGES - 2
    // stages' are outstanding; the barrier shows every wave's, and that the
    // buffer of stage s - 1 is read
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((STAGES - 2) * kPer) : "memory");
    __builtin_amdgcn_s_barrier();
    const int sn = s + STAGES - 1;
    issue(sn < ns ? sn : ns - 1, sn % STAGES);
    const u32x4* bx = &sl[(s % STAGES) * kStage];
    const u32x4* bw = bx + kX * 64;
#pragma unroll
    for (int k = 0; k < KS / KWN; ++k) {
      const int ks = k * KWN + kw;                    // the 32-h step of the stage
      if (32 * (KS * s + ks) >= H) continue;
      uint32_t ax[WT];
      u32x4 vx[WT];
#pragma unroll
      for (int j = 0; j < WT; ++j) {
        const int row = (tw * WT + j) * 16 + r;
        ax[j] = lds_addr(&bx[row * NPX + piece_slot<NPX>(row, 4 * ks + q)]);
      }
      lds_read<WT>(ax, vx);
      constexpr int PW = RF32 ? 2 : 1;
      uint32_t aw[WE * PW];
      u32x4 vw[WE * PW];
#pragma unroll
      for (int j = 0; j < WE; ++j) {
        const int row = ew * WE * 16 + 4 * WE * (r >> 2) + 4 * j + (r & 3);
#pragma unroll
        for (int h = 0; h < PW; ++h)
          aw[j * PW + h] = lds_addr(&bw[row * NPW + piece_slot<NPW>(row, PW * (4 * ks + q) + h)]);
      }
      lds_read<WE * PW>(aw, vw);
#pragma unroll
      for (int e = 0; e < WE; ++e) {
        if (RF32) {
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(vw[e * PW + (i / 4) % PW][i % 4]);
          u32x4 hi, mid, lo;
          split8x3(v, hi, mid, lo);
#pragma unroll
          for (int j = 0; j < WT; ++j) {
            acc[e][j] = mfma(lo, vx[j], acc[e][j]);
            acc[e][j] = mfma(mid, vx[j], acc[e][j]);
            acc[e][j] = mfma(hi, vx[j], acc[e][j]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < WT; ++j) acc[e][j] = mfma(vw[e], vx[j], acc[e][j]);
        }
      }
    }
  }
  if constexpr (KWN > 1) {
    // every copy has landed and every wave has read its operands: the stages
    // become the sums' buffer
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    v4f* red = reinterpret_cast<v4f*>(sl);            // [kw - 1][tw][ew][WE * WT][64]
    if (kw > 0) {
#pragma unroll
      for (int e = 0; e < WE; ++e)
#pragma unroll
        for (int j = 0; j < WT; ++j)
          red[((((kw - 1) * TWN + tw) * EWN + ew) * WE * WT + e * WT + j) * 64 + lane] = acc[e][j];
    }
    __syncthreads();
    if (kw > 0) return;
#pragma unroll
    for (int k = 0; k < KWN - 1; ++k)
#pragma unroll
      for (int e = 0; e < WE; ++e)
#pragma unroll
        for (int j = 0; j < WT; ++j)
          acc[e][j] += red[(((k * TWN + tw) * EWN + ew) * WE * WT + e * WT + j) * 64 + lane];
  }
#pragma unroll
  for (int j = 0; j < WT; ++j) {
    const int64_t t = t0 + (tw * WT + j) * 16 + r;
    if (t >= T) continue;
#pragma unroll
    for (int e = 0; e < WE; ++e) {
      const int c = e0 + ew * WE * 16 + 4 * WE * q + 4 * e;
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

template <int TM, int TE, int KS, int WT, int WE, bool RF32, int STAGES>
hipError_t run_logits(const void* x, const void* w, int T, int H, int E, float* z,
                      hipStream_t st) {
  const dim3 g((T - 1) / TM + 1, (E + TE - 1) / TE);   // T >= 1, up to 2^31 - 1
  constexpr size_t lds = (size_t)STAGES * (TM * 4 + TE * (RF32 ? 8 : 4)) * KS * 16;
  hipLaunchKernelGGL((router_logits_kernel<TM, TE, KS, WT, WE, RF32, STAGES>), g,
                     dim3(kLgWaves * 64), lds, st, static_cast<const uint16_t*>(x), w, T, H, E, z);
  return hipGetLastError();
}

// ---- operand orders -------------------------------------------------------------
// W for dx: [chunk of 64 h][32 e][tile j][part][64 lanes]; dz^T for dW:
// [32 tokens][16 e][part][64 lanes], three parts of it (dW is fp32: with two its
// error was 2.5e-6 of its norm where an fp32 product has 5e-7).  One launch for
// both: workgroups 0 .. nw - 1 take W, the others dz.  Bound: HBM and latency;
// 10 us at T = 16384, H = 4096, E = 256, 3.5 us at 777, 2048, 128 (two launches
// were 3 us more).
constexpr int kZp = 3;

template <bool RF32>
__device__ __forceinline__ void pack_router(const void* __restrict__ w, int H, int E, int c,
                                            int ks, int nks, u32x4* __restrict__ out) {
  constexpr int PL = RF32 ? 2 : 1;
  const int kq = threadIdx.x >> 6, hh = threadIdx.x & 63;
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
  u32x4* o = out + ((((int64_t)c * nks + ks) * 4 + j) * PL) * 64 + 16 * kq + r;
  o[0] = hi;
  if (RF32) o[64] = lo;
}

__device__ __forceinline__ void pack_dz(const float* __restrict__ dz, int T, int E, int net,
                                        int64_t kt, u32x4* __restrict__ out) {
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

template <bool RF32>
__global__ __launch_bounds__(256) void pack_kernel(const void* __restrict__ w,
                                                   const float* __restrict__ dz, int T, int H,
                                                   int E, int nw, int net, u32x4* __restrict__ wf,
                                                   u32x4* __restrict__ zf) {
  const int b = blockIdx.x, nks = (E + 31) / 32;
  if (b < nw) pack_router<RF32>(w, H, E, b / nks, b % nks, nks, wf);
  else pack_dz(dz, T, E, net, b - nw, zf);
}

// ---- dx -----------------------------------------------------------------------
// A workgroup holds dz of 16 NTL tokens (all experts, both parts, operand
// order) in LDS, and its 8 waves stream chunks of 64 h of W past it: W, the
// operand without reuse in a workgroup, comes from the L2 in operand order.
//
// Bound: the matrix cores, 2 T H E operations for each part of dz (three pairs of
// parts where W is fp32).  T = 16384, H = 4096, E = 256: 72 us, 0.95 PFLOP/s.
constexpr int kDxWaves = 8;

template <int NTL, bool RF32>
__device__ __forceinline__ void router_dx(const float* __restrict__ dz,
                                          const u32x4* __restrict__ wf, int T, int H, int E,
                                          uint16_t* __restrict__ dx, int bx, int by, int ny) {
  constexpr int PL = RF32 ? 2 : 1;
  extern __shared__ u32x4 sb[];                       // [e block][token tile][part][64]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 15, q = lane >> 4;
  const int nks = (E + 31) / 32, nc = (H + 63) / 64;
  const int64_t t0 = (int64_t)bx * 16 * NTL;
  const bool vec = E % 4 == 0;
  // W of the first chunk, on its way while dz is staged; from then on always the
  // next 32 experts', into the next chunk
  const int step = ny * kDxWaves;
  int c = by * kDxWaves + wave;
  const u32x4* src = wf + (int64_t)(c < nc ? c : 0) * nks * 4 * PL * 64 + lane;
  u32x4 a[4 * PL];
#pragma unroll
  for (int i = 0; i < 4 * PL; ++i) a[i] = src[i * 64];
  // four pieces' loads in flight before the first is used
  for (int i0 = wave; i0 < nks * NTL; i0 += 4 * kDxWaves) {
    float v[4][8];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int it = i0 + u * kDxWaves, ks = it / NTL, nt = it % NTL;
      const int64_t t = t0 + 16 * nt + n;
      const int e0 = 32 * ks + 8 * q;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = 0.f;
      if (it < nks * NTL && t < T) {
        const float* src = dz + t * E + e0;
        if (vec) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (e0 + 4 * i < E) {
              const float4 f = *reinterpret_cast<const float4*>(src + 4 * i);
              v[u][4 * i] = f.x; v[u][4 * i + 1] = f.y;
              v[u][4 * i + 2] = f.z; v[u][4 * i + 3] = f.w;
            }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (e0 + i < E) v[u][i] = src[i];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int it = i0 + u * kDxWaves;
      if (it < nks * NTL) {
        u32x4 hi, lo;
        split8(v[u], hi, lo);
        sb[(it * 2) * 64 + lane] = hi;
        sb[(it * 2 + 1) * 64 + lane] = lo;
      }
    }
  }
  __syncthreads();
  for (; c < nc; c += step) {
    v4f acc[4][NTL];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int t = 0; t < NTL; ++t) acc[j][t] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int ks = 0; ks < nks; ++ks) {
      u32x4 an[4 * PL];
      if (ks + 1 < nks) src += 4 * PL * 64;
      else if (c + step < nc) src += ((int64_t)(step - 1) * nks + 1) * 4 * PL * 64;
#pragma unroll
      for (int i = 0; i < 4 * PL; ++i) an[i] = src[i * 64];
#pragma unroll
      for (int t = 0; t < NTL; ++t) {
        const u32x4 hi = sb[((ks * NTL + t) * 2) * 64 + lane];
        const u32x4 lo = sb[((ks * NTL + t) * 2 + 1) * 64 + lane];
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j][t] = mfma(a[j * PL], lo, acc[j][t]);
        if (RF32)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[j][t] = mfma(a[j * PL + PL - 1], hi, acc[j][t]);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j][t] = mfma(a[j * PL], hi, acc[j][t]);
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

// ---- dW -----------------------------------------------------------------------
// A workgroup: 16 ET experts x 512 h over a slice of the tokens.  dz^T of 32
// tokens goes through LDS (double buffered), shared by the eight waves; a wave
// has 64 h of its own, whose x it reads straight from memory (lane (n, q): 8
// tokens x 4 h) and transposes in registers: column n of the f-th operand is
// h = 4 n + f, so a lane ends up with four consecutive h of a row.
//
// Bound: the matrix cores, three times 2 T H E operations.  T = 16384, H = 4096, E
// = 256: 92 us, 1.12 PFLOP/s, and 11 us for the sum over 16 slices of tokens.
// The slices run fastest over the workgroups: where their number is a multiple of
// 8, the workgroups of one, which share its dz and x, are on one XCD (160 MB
// fetched; with the chunks of h fastest, every XCD took all of dz: 336 MB, 2 us).
constexpr int kDwWaves = 8, kDwH = 64 * kDwWaves;

__device__ __forceinline__ uint32_t pack_lo(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x05040100u);
}
__device__ __forceinline__ uint32_t pack_hi(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x07060302u);
}

template <int ET>
__device__ __forceinline__ void router_dw(const uint16_t* __restrict__ x,
                                          const u32x4* __restrict__ zf, int T, int H, int E,
                                          int net, int per_slice, float* __restrict__ out, int bx,
                                          int by, int bz) {
  constexpr int kStage = ET * kZp * 64, kCopies = (kStage + kDwWaves * 64 - 1) / (kDwWaves * 64);
  __shared__ u32x4 sa[2][kStage];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 15, q = lane >> 4;
  const int nkt = (T + 31) / 32;
  const int k0 = bz * per_slice, k1 = min(nkt, k0 + per_slice);
  const int h = bx * kDwH + wave * 64 + 4 * n;
  const bool hin = h < H;
  const u32x4* zsrc = zf + (int64_t)by * ET * kZp * 64;

  // The next step's loads, none of them behind a branch: rows past the last token
  // read the last one (dz is packed with zeros there, and what that row does to a
  // sum of its column it does anyway), a step past the slice its last step.  (Two
  // steps ahead in short batches: no change.)
  u32x4 za[kCopies];
  uint2 xr[8];
  const uint16_t* xh = x + (hin ? h : 0);
  auto load = [&](int step) {
    const int kt = min(step, k1 - 1);
#pragma unroll
    for (int c = 0; c < kCopies; ++c) {
      const int i = c * kDwWaves * 64 + threadIdx.x;
      za[c] = zsrc[(int64_t)kt * net * kZp * 64 + min(i, kStage - 1)];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t t = min(32 * kt + 8 * q + i, T - 1);
      xr[i] = *reinterpret_cast<const uint2*>(xh + t * H);
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
    load(kt + 1);
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
    stage(buf ^ 1);
  }
  if (!hin) return;
  float* o = out + (int64_t)bz * E * H;
#pragma unroll
  for (int e = 0; e < ET; ++e)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = (by * ET + e) * 16 + 4 * q + i;
      if (row < E)
        *reinterpret_cast<v4f*>(o + (int64_t)row * H + h) =
            v4f{acc[e][0][i], acc[e][1][i], acc[e][2][i], acc[e][3][i]};
    }
}

template <int NTL, bool RF32>
__global__ __launch_bounds__(kDxWaves * 64) void router_dx_kernel(const float* dz, const u32x4* wf,
                                                                  int T, int H, int E,
                                                                  uint16_t* dx) {
  router_dx<NTL, RF32>(dz, wf, T, H, E, dx, blockIdx.x, blockIdx.y, gridDim.y);
}

template <int ET>
__global__ __launch_bounds__(kDwWaves * 64, 2) void router_dw_kernel(const uint16_t* x,
                                                                     const u32x4* zf, int T,
                                                                     int H, int E, int net,
                                                                     int per_slice, float* out) {
  router_dw<ET>(x, zf, T, H, E, net, per_slice, out, blockIdx.y, blockIdx.z, blockIdx.x);
}

// Both in one launch, where neither fills the chip: workgroups 0 .. ndx - 1 are
// dx's (gx of them side by side), the others dW's.  T = 777, H = 2048, E = 128, W
// fp32: 11.7 us, one after the other 8.1 + 7.8.
template <int ET, bool RF32>
__global__ __launch_bounds__(kDxWaves * 64, 2) void router_both_kernel(
    const uint16_t* x, const float* dz, const u32x4* wf, const u32x4* zf, int T, int H, int E,
    int gx, int gy, int hx, int ey, int net, int per_slice, uint16_t* dx, float* out) {
  static_assert(kDxWaves == kDwWaves, "one block size");
  const int b = blockIdx.x, ndx = gx * gy;
  if (b < ndx) {
    router_dx<2, RF32>(dz, wf, T, H, E, dx, b % gx, b / gx, gy);
  } else {
    const int d = b - ndx;
    router_dw<ET>(x, zf, T, H, E, net, per_slice, out, d % hx, d / hx % ey, d / (hx * ey));
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
// token slices: a workgroup per compute unit where a slice has at least 4
// steps of 32 tokens; short batches take fewer experts a workgroup instead
struct DwPlan {
  int et, net, slices, per_slice;
};
DwPlan dw_plan(int T, int H, int E) {
  DwPlan p;
  const int nkt = T > 0 ? (T + 31) / 32 : 1, hx = (H + kDwH - 1) / kDwH;
  const int most = nkt / 4 > 1 ? nkt / 4 : 1;
  p.et = E > 64 ? 8 : E > 32 ? 4 : E > 16 ? 2 : 1;
  while (p.et > 1 && hx * ((E + 16 * p.et - 1) / (16 * p.et)) * most < 192) p.et /= 2;
  const int ey = (E + 16 * p.et - 1) / (16 * p.et), tiles = ey * hx;
  p.net = ey * p.et;
  int s = (256 + tiles - 1) / tiles;
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

// dx: tokens per workgroup in tiles of 16 (dz of all experts in 128 KB of LDS, and
// few enough that short batches still spread over the compute units) and the
// workgroups side by side over the chunks of 64 h
struct DxPlan {
  int ntl, gx, gy;
  size_t lds;
};
DxPlan dx_plan(int T, int H, int E) {
  DxPlan p;
  const int nks = (E + 31) / 32, nc = (H + 63) / 64;
  p.ntl = nks <= 8 ? 8 : nks <= 16 ? 4 : 2;
  while (p.ntl > 2 && (T + 16 * p.ntl - 1) / (16 * p.ntl) < 64) p.ntl /= 2;
  p.gx = (T + 16 * p.ntl - 1) / (16 * p.ntl);
  const int most = (nc + kDxWaves - 1) / kDxWaves, gy = 256 / p.gx;
  p.gy = gy < 1 ? 1 : gy > most ? most : gy;
  p.lds = (size_t)nks * p.ntl * 2 * 1024;
  return p;
}

template <bool RF32>
hipError_t run_dx(const RouterBackward& a, const DxPlan& p, const u32x4* wf, hipStream_t st) {
  const dim3 g(p.gx, p.gy), b(kDxWaves * 64);
  if (p.ntl == 8)
    hipLaunchKernelGGL((router_dx_kernel<8, RF32>), g, b, p.lds, st, a.dz, wf, a.T, a.H, a.E, a.dx);
  else if (p.ntl == 4)
    hipLaunchKernelGGL((router_dx_kernel<4, RF32>), g, b, p.lds, st, a.dz, wf, a.T, a.H, a.E, a.dx);
  else
    hipLaunchKernelGGL((router_dx_kernel<2, RF32>), g, b, p.lds, st, a.dz, wf, a.T, a.H, a.E, a.dx);
  return hipGetLastError();
}

template <int ET>
hipError_t run_dw(const RouterBackward& a, const DwPlan& p, const u32x4* zf, float* out,
                  hipStream_t st) {
  const dim3 g(p.slices, (a.H + kDwH - 1) / kDwH, p.net / p.et);
  hipLaunchKernelGGL(router_dw_kernel<ET>, g, dim3(kDwWaves * 64), 0, st,
                     static_cast<const uint16_t*>(a.x), zf, a.T, a.H, a.E, p.net, p.per_slice, out);
  return hipGetLastError();
}

template <int ET, bool RF32>
hipError_t run_both(const RouterBackward& a, const DxPlan& d, const DwPlan& p, const u32x4* wf,
                    const u32x4* zf, float* out, hipStream_t st) {
  const int hx = (a.H + kDwH - 1) / kDwH, ey = p.net / p.et;
  hipLaunchKernelGGL((router_both_kernel<ET, RF32>), dim3(d.gx * d.gy + hx * ey * p.slices),
                     dim3(kDxWaves * 64), d.lds, st, static_cast<const uint16_t*>(a.x), a.dz, wf,
                     zf, a.T, a.H, a.E, d.gx, d.gy, hx, ey, p.net, p.per_slice, a.dx, out);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_router_logits(const void* x, const void* w, int router_f32, int T, int H, int E,
                                float* z, hipStream_t st) {
  // A compute unit takes in about 40 GB/s through its L1 here (its misses in
  // flight over the L2's latency), so the tile with the fewest bytes per result
  // that still gives 192 workgroups (3/4 of the compute units) is the fastest:
  // 128 x 128 before 64 x 128 before 64 x 64; last tiles whose waves all split H:
  // 16 x 32, and 32 x 16 where W is fp32 (a row of it is as many bytes as two of
  // x).  T = 16384, H = 4096, E = 256: 128 x 128 tiles 60 us (0.57 PFLOP/s), 64 x
  // 256 63 us; T = 777, H = 2048, E = 128, W fp32: 32 x 16 10.3 us, 16 x 32 11.2.
  const auto blocks = [&](int tokens, int experts) {
    return (int64_t)((T - 1) / tokens + 1) * ((E + experts - 1) / experts);
  };
  if (router_f32) {
    if (E > 64 && blocks(128, 128) >= 192)
      return run_logits<128, 128, 2, 4, 4, true, 3>(x, w, T, H, E, z, st);
    if (E > 64 && blocks(64, 128) >= 192)
      return run_logits<64, 128, 2, 2, 4, true, 3>(x, w, T, H, E, z, st);
    if (blocks(64, 64) >= 192) return run_logits<64, 64, 2, 1, 4, true, 4>(x, w, T, H, E, z, st);
    return run_logits<32, 16, 8, 2, 1, true, 4>(x, w, T, H, E, z, st);
  }
  if (E > 64 && blocks(128, 128) >= 192)
    return run_logits<128, 128, 2, 4, 4, false, 4>(x, w, T, H, E, z, st);
  if (E > 64 && blocks(64, 128) >= 192)
    return run_logits<64, 128, 2, 2, 4, false, 4>(x, w, T, H, E, z, st);
  if (blocks(64, 64) >= 192) return run_logits<64, 64, 2, 1, 4, false, 4>(x, w, T, H, E, z, st);
  return run_logits<16, 32, 8, 1, 2, false, 4>(x, w, T, H, E, z, st);
}

size_t router_backward_bytes(int T, int H, int E) { return carve(T, H, E).total; }

hipError_t launch_router_backward(const RouterBackward& a, hipStream_t st) {
  const Ws L = carve(a.T, a.H, a.E);
  u32x4* wf = reinterpret_cast<u32x4*>(a.ws + L.wf);
  u32x4* zf = reinterpret_cast<u32x4*>(a.ws + L.zf);
  const DwPlan p = dw_plan(a.T, a.H, a.E);
  const int nw = a.dx ? ((a.H + 63) / 64) * ((a.E + 31) / 32) : 0, nz = a.dw ? (a.T + 31) / 32 : 0;
  if (a.router_f32)
    hipLaunchKernelGGL(pack_kernel<true>, dim3(nw + nz), dim3(256), 0, st, a.w, a.dz, a.T, a.H,
                       a.E, nw, p.net, wf, zf);
  else
    hipLaunchKernelGGL(pack_kernel<false>, dim3(nw + nz), dim3(256), 0, st, a.w, a.dz, a.T, a.H,
                       a.E, nw, p.net, wf, zf);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const DxPlan d = dx_plan(a.T, a.H, a.E);
  float* out = p.slices > 1 ? reinterpret_cast<float*>(a.ws + L.part) : a.dw;
  if (a.dx && a.dw && d.ntl == 2 && p.et <= 2) {      // a short batch: both at once
    if (p.et == 1) err = a.router_f32 ? run_both<1, true>(a, d, p, wf, zf, out, st)
                                      : run_both<1, false>(a, d, p, wf, zf, out, st);
    else err = a.router_f32 ? run_both<2, true>(a, d, p, wf, zf, out, st)
                            : run_both<2, false>(a, d, p, wf, zf, out, st);
  } else {
    if (a.dx) {
      err = a.router_f32 ? run_dx<true>(a, d, wf, st) : run_dx<false>(a, d, wf, st);
      if (err != hipSuccess) return err;
    }
    if (!a.dw) return err;
    err = p.et == 8   ? run_dw<8>(a, p, zf, out, st)
          : p.et == 4 ? run_dw<4>(a, p, zf, out, st)
          : p.et == 2 ? run_dw<2>(a, p, zf, out, st)
                      : run_dw<1>(a, p, zf, out, st);
  }
  if (err != hipSuccess || p.slices == 1) return err;
  const int64_t n4 = (int64_t)a.E * a.H / 4;
  hipLaunchKernelGGL(sum_slices_kernel, dim3((unsigned)((n4 + 255) / 256)), dim3(256), 0, st,
                     reinterpret_cast<const v4f*>(out), p.slices, n4,
                     reinterpret_cast<v4f*>(a.dw));
  return hipGetLastError();
}

}  // namespace moe
