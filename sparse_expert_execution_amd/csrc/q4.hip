// q4.hip - matrices of 4-bit integers with a scale per group of columns: the
// dense product y = x W^T, the quantiser and the packer (layout: q4.hpp).
#include "q4.hpp"

namespace moe {
namespace {

using namespace q4;

constexpr int kWaves = 8;

// One workgroup: 8 waves as (8 / KS) sets of RT row tiles x KS slices of the
// columns; a wave walks its slice's column blocks with D - 1 blocks' loads in
// flight, and the KS partial sums of a tile meet in LDS, added in slice order.
// x goes straight into the matrix operand's registers: lane (r, q) reads 16
// bytes of the token in slot r.
// More than four tokens (STAGE): neighbouring lanes of an operand are different
// tokens, and a load of it costs a cache lookup per lane, so x goes through LDS,
// 128 columns at a time and each wave for itself: loads run along the rows (16
// lanes x 16 bytes), piece p of row i is kept at slot p ^ i % 16, from where the
// operand is read without bank conflicts.
//
// Bound: HBM for large matrices, 131072 x 4096 and one token 53 us, 5.2 TB/s; the
// launch for small ones, 768 x 2048 and one token 3.4 us of kernel in 5.4 us a
// call.  With more tokens the operands' way through the L1 and LDS: 8192 x 4096
// (groups of 128) 16 tokens 6.5 us, 32 9.4 us, 64 13.3 us.
template <int NT, int TI, int RT, int G, bool ZERO, bool STAGE>
__global__ __launch_bounds__(kWaves * 64, NT > 1 ? 2 : 4) void
q4_linear_kernel(Q4Linear a) {
  constexpr int D = NT == 1 && RT == 1 ? 3 : NT == 4 ? 1 : 2;
  extern __shared__ float red[];                      // [wave][RT * NT][TI][64]
                                                      // STAGE, before: [wave][16 NT][16] pieces
  const int lane = threadIdx.x & 63, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int KS = 1 << a.log_ks, slice = wave & (KS - 1), set = wave >> a.log_ks;
  const int rt0 = (blockIdx.x * (kWaves >> a.log_ks) + set) * RT;
  const int t0 = blockIdx.y * 16 * NT;
  const Matrix m{a.codes, a.scales, a.zeros, a.nkb};

  float acc[RT][NT][TI];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < TI; ++i) acc[r][j][i] = 0.f;

  int tile[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) tile[r] = rt0 + r < a.tiles ? rt0 + r : a.tiles - 1;

  // a load's row and first column (within 128): operand order, or along the rows.
  // Rows past the last token read the last one: what they give reaches no result
  // of another row.
  constexpr int L = STAGE ? 4 * NT : NT;              // rows of a lane
  int64_t row[L];
  const int col = 8 * (STAGE ? lane & 15 : q);
#pragma unroll
  for (int j = 0; j < L; ++j) {
    const int t = STAGE ? t0 + 4 * j + q : t0 + 16 * j + slot_token(lane & 15);
    row[j] = (int64_t)(t < a.T ? t : a.T - 1) * a.x_ld + col;
  }
  struct Block {
    Tile<G, ZERO> t[RT];
    bf16x8 x[NT][4];
  };
  // whole column blocks, in a pipeline without a branch around any load (the
  // waits count the loads issued after); a last partial one follows
  const int full = a.K / 128;
  const int n_it = slice < full ? (full - slice + KS - 1) >> a.log_ks : 0;
  auto load = [&](Block& b, int it) {
    const bool live = it < n_it;
    const int kb = slice + ((live ? it : 0) << a.log_ks);
#pragma unroll
    for (int r = 0; r < RT; ++r) load_tile<G, ZERO>(b.t[r], m, tile[r], kb, live);
#pragma unroll
    for (int j = 0; j < L; ++j) {
      // a row may start at any element: 16-byte loads of any alignment
      const uint16_t* src = a.x + 128 * kb + (STAGE || live ? row[j] : 0);
#pragma unroll
      for (int s = 0; s < 4 * NT / L; ++s)
        __builtin_memcpy(STAGE ? &b.x[j / 4][j % 4] : &b.x[j % NT][s], src + 32 * s, 16);
    }
  };
  auto load_last = [&](Block& b) {
    const int left = a.K - 128 * full;
#pragma unroll
    for (int r = 0; r < RT; ++r) load_tile<G, ZERO>(b.t[r], m, tile[r], full, true);
#pragma unroll
    for (int j = 0; j < L; ++j)
#pragma unroll
      for (int s = 0; s < 4 * NT / L; ++s) {
        const uint16_t* src = a.x + 128 * full + row[j] + 32 * s;
        const int here = left - 32 * s - col;         // columns from this lane's first on
        u32x4 v = u32x4{0, 0, 0, 0};
        if (here >= 8) __builtin_memcpy(&v, src, 16);
        else
#pragma unroll
          for (int i = 0; i < 7; ++i)
            if (i < here) v[i / 2] |= (uint32_t)src[i] << (16 * (i % 2));
        (STAGE ? b.x[j / 4][j % 4] : b.x[j % NT][s]) = frag(v);
      }
  };

  // STAGE: what the rows' loads brought -> operand order
  u32x4* stage = reinterpret_cast<u32x4*>(red) + wave * 16 * NT * 16;
  auto turn = [&](bf16x8 (&x)[NT][4]) {
    if (!STAGE) return;
#pragma unroll
    for (int j = 0; j < 4 * NT; ++j) {
      const int r = 4 * j + q;
      stage[r * 16 + ((lane & 15) ^ (r & 15))] = __builtin_bit_cast(u32x4, x[j / 4][j % 4]);
    }
    // one wave's LDS accesses are done in order; the compiler must keep them so
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int r = 16 * j + slot_token(lane & 15);
#pragma unroll
      for (int s = 0; s < 4; ++s) x[j][s] = frag(stage[r * 16 + ((4 * s + q) ^ (r & 15))]);
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  };

  if (n_it > 0) {
    Block b[D];
#pragma unroll
    for (int d = 0; d < D - 1; ++d) load(b[d], d);
    for (int i0 = 0; i0 < n_it; i0 += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (i0 + d >= n_it) break;
        load(b[(d + D - 1) % D], i0 + d + D - 1);
        turn(b[d].x);
        mul_tiles<RT, NT, TI, G, ZERO>(acc, b[d].t, b[d].x);
      }
    }
  }
  if (full < a.nkb && slice == (full & (KS - 1))) {
    Block b;
    load_last(b);
    turn(b.x);
    mul_tiles<RT, NT, TI, G, ZERO>(acc, b.t, b.x);
  }
  if (STAGE) __syncthreads();                         // the stages become the sums' buffer

#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < TI; ++i)
        red[((wave * RT * NT + r * NT + j) * TI + i) * 64 + lane] = acc[r][j][i];
  __syncthreads();
  const int items = (kWaves >> a.log_ks) * RT * NT * TI * 64;
  for (int id = threadIdx.x; id < items; id += kWaves * 64) {
    const int l = id & 63, f = id >> 6;               // f: (set, row tile, token tile, result)
    const int st = f / (RT * NT * TI), rji = f % (RT * NT * TI);
    float v = 0.f;
    for (int s = 0; s < KS; ++s) v += red[(((st << a.log_ks) + s) * RT * NT * TI + rji) * 64 + l];
    const int rj = rji / TI, t = t0 + 16 * (rj % NT) + result_token(l, rji % TI);
    const int row = 16 * ((blockIdx.x * (kWaves >> a.log_ks) + st) * RT + rj / NT) + (l & 15);
    if (t >= a.T || row >= a.N) continue;
    const int64_t at = (int64_t)t * a.y_ld + row;
    if (a.y_bf16) static_cast<uint16_t*>(a.y)[at] = __builtin_bit_cast(uint16_t, (__bf16)v);
    else static_cast<float*>(a.y)[at] = v;
  }
}

// ---- quantise / pack --------------------------------------------------------
__device__ __forceinline__ float src_value(const void* src, int bf16, int64_t i) {
  return bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(src)[i] << 16)
              : static_cast<const float*>(src)[i];
}

// One thread per (padded row, group): the group's scale and zero point.
// Symmetric: s = max|v| / 7, z = 8.  With zero points: the range [min(v, 0),
// max(v, 0)] in 15 steps.  s is rounded to BF16 before codes are computed from it.
__global__ __launch_bounds__(256) void q4_scale_kernel(const void* src, int bf16, int N, int K,
                                                       int64_t ld, int G, int Np, int groups,
                                                       uint16_t* scales, uint8_t* zeros) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= (int64_t)Np * groups) return;
  const int row = (int)(id / groups), g = (int)(id % groups);
  float lo = 0.f, hi = 0.f;
  if (row < N)
    for (int k = g * G; k < (g + 1) * G && k < K; ++k) {
      const float v = src_value(src, bf16, (int64_t)row * ld + k);
      lo = fminf(lo, v);
      hi = fmaxf(hi, v);
    }
  const float s = zeros ? (hi - lo) / 15.f : fmaxf(hi, -lo) / 7.f;
  const __bf16 sb = (__bf16)s;
  const float sr = (float)sb;
  const int64_t at = ((int64_t)(row / 16) * groups + g) * 16 + row % 16;
  scales[at] = __builtin_bit_cast(uint16_t, sb);
  if (zeros) zeros[at] = sr > 0.f ? (uint8_t)fminf(fmaxf(rintf(-lo / sr), 0.f), 15.f) : 8;
}

// One thread per (tile, lane): its 32 codes.
__global__ __launch_bounds__(256) void q4_code_kernel(const void* src, int bf16, int N, int K,
                                                      int64_t ld, int G, int nkb, int64_t lanes,
                                                      const uint16_t* scales,
                                                      const uint8_t* zeros, uint4* codes) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= lanes) return;
  const int lane = (int)(id & 63);
  const int64_t at = id >> 6;
  const int kb = (int)(at % nkb), row = (int)(at / nkb) * 16 + (lane & 15);
  uint32_t out[4];
  for (int s = 0; s < 4; ++s) {
    uint32_t w = 0;
    for (int i = 0; i < 8; ++i) {
      const int k = 128 * kb + 32 * s + 8 * (lane >> 4) + i;
      const int64_t gi = ((int64_t)(row / 16) * (nkb * (128 / G)) + k / G) * 16 + row % 16;
      const float sc = __uint_as_float((uint32_t)scales[gi] << 16);
      const float z = zeros ? (float)zeros[gi] : 8.f;
      float q = z;
      if (row < N && k < K && sc > 0.f)
        q = fminf(fmaxf(rintf(src_value(src, bf16, (int64_t)row * ld + k) / sc) + z, 0.f), 15.f);
      w |= ((uint32_t)q & 15u) << (4 * (i / 2 + 4 * (i % 2)));
    }
    out[s] = w;
  }
  codes[id] = make_uint4(out[0], out[1], out[2], out[3]);
}

// One thread per (tile, lane): codes given row-major [N][ceil(K / 2)], low
// nibble first.
__global__ __launch_bounds__(256) void q4_pack_codes_kernel(const uint8_t* src, int N, int K,
                                                            int nkb, int64_t lanes,
                                                            uint4* codes) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= lanes) return;
  const int lane = (int)(id & 63);
  const int64_t at = id >> 6;
  const int kb = (int)(at % nkb), row = (int)(at / nkb) * 16 + (lane & 15);
  uint32_t out[4];
  for (int s = 0; s < 4; ++s) {
    uint32_t w = 0;
    for (int i = 0; i < 8; ++i) {
      const int k = 128 * kb + 32 * s + 8 * (lane >> 4) + i;
      uint32_t q = 8;
      if (row < N && k < K) q = src[(int64_t)row * ((K + 1) / 2) + k / 2] >> (4 * (k % 2)) & 15u;
      w |= q << (4 * (i / 2 + 4 * (i % 2)));
    }
    out[s] = w;
  }
  codes[id] = make_uint4(out[0], out[1], out[2], out[3]);
}

__global__ __launch_bounds__(256) void q4_pack_scales_kernel(const uint16_t* s, const uint8_t* z,
                                                             int N, int given, int Np, int groups,
                                                             uint16_t* scales, uint8_t* zeros) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= (int64_t)Np * groups) return;
  const int row = (int)(id / groups), g = (int)(id % groups);
  const bool in = row < N && g < given;
  const int64_t at = ((int64_t)(row / 16) * groups + g) * 16 + row % 16;
  scales[at] = in ? s[(int64_t)row * given + g] : 0;
  if (zeros) zeros[at] = in ? z[(int64_t)row * given + g] : 8;
}

template <int NT, int TI, int RT, int G, bool ZERO>
hipError_t run_linear(const Q4Linear& a, dim3 grid, hipStream_t st) {
  constexpr bool kStage = TI > 1;
  constexpr size_t sums = (size_t)kWaves * RT * NT * TI * 64 * sizeof(float);
  constexpr size_t stages = kStage ? (size_t)kWaves * NT * 4096 : 0;
  hipLaunchKernelGGL((q4_linear_kernel<NT, TI, RT, G, ZERO, kStage>), grid, dim3(kWaves * 64),
                     sums > stages ? sums : stages, st, a);
  return hipGetLastError();
}

template <int NT, int TI, int RT>
hipError_t pick_group(const Q4Linear& a, int G, dim3 grid, hipStream_t st) {
  if (a.zeros) {
    if (G == 32) return run_linear<NT, TI, RT, 32, true>(a, grid, st);
    if (G == 64) return run_linear<NT, TI, RT, 64, true>(a, grid, st);
    return run_linear<NT, TI, RT, 128, true>(a, grid, st);
  }
  if (G == 32) return run_linear<NT, TI, RT, 32, false>(a, grid, st);
  if (G == 64) return run_linear<NT, TI, RT, 64, false>(a, grid, st);
  return run_linear<NT, TI, RT, 128, false>(a, grid, st);
}

}  // namespace

hipError_t launch_q4_linear(Q4Linear a, int group, hipStream_t st) {
  a.tiles = (a.N + 15) / 16;
  a.nkb = (a.K + 127) / 128;
  a.log_ks = a.nkb >= 8 ? 3 : a.nkb >= 4 ? 2 : a.nkb >= 2 ? 1 : 0;
  const int sets = kWaves >> a.log_ks;
  const int nt = a.T <= 16 ? 1 : a.T <= 32 ? 2 : 4;
  // Row tiles a wave: every workgroup reads all of x, so with more tokens more
  // of them pay, as long as a workgroup per compute unit is left.
  const int rt = a.T <= 4 ? (a.tiles >= 2048 ? 2 : 1)
                          : (nt == 4 && a.tiles >= 2048 ? 4 : a.tiles >= 512 ? 2 : 1);
  const dim3 grid((a.tiles + sets * rt - 1) / (sets * rt), (a.T + 16 * nt - 1) / (16 * nt));
  if (a.T <= 4) return rt == 2 ? pick_group<1, 1, 2>(a, group, grid, st)
                               : pick_group<1, 1, 1>(a, group, grid, st);
  if (a.T <= 8) return rt == 2 ? pick_group<1, 2, 2>(a, group, grid, st)
                               : pick_group<1, 2, 1>(a, group, grid, st);
  if (nt == 1) return rt == 2 ? pick_group<1, 4, 2>(a, group, grid, st)
                              : pick_group<1, 4, 1>(a, group, grid, st);
  if (nt == 2) return rt == 2 ? pick_group<2, 4, 2>(a, group, grid, st)
                              : pick_group<2, 4, 1>(a, group, grid, st);
  if (rt == 4) return pick_group<4, 4, 4>(a, group, grid, st);
  return rt == 2 ? pick_group<4, 4, 2>(a, group, grid, st)
                 : pick_group<4, 4, 1>(a, group, grid, st);
}

hipError_t launch_q4_quantize(const void* src, int bf16, int N, int K, int64_t ld, int group,
                              uint8_t* codes, uint8_t* scales, uint8_t* zeros, hipStream_t st) {
  const int nkb = (K + 127) / 128, tiles = (N + 15) / 16, groups = nkb * (128 / group);
  const int64_t sg = (int64_t)tiles * 16 * groups, lanes = (int64_t)tiles * nkb * 64;
  hipLaunchKernelGGL(q4_scale_kernel, dim3((unsigned)((sg + 255) / 256)), dim3(256), 0, st, src,
                     bf16, N, K, ld, group, tiles * 16, groups,
                     reinterpret_cast<uint16_t*>(scales), zeros);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL(q4_code_kernel, dim3((unsigned)((lanes + 255) / 256)), dim3(256), 0, st, src,
                     bf16, N, K, ld, group, nkb, lanes,
                     reinterpret_cast<const uint16_t*>(scales), zeros,
                     reinterpret_cast<uint4*>(codes));
  return hipGetLastError();
}

hipError_t launch_q4_pack(const uint8_t* q, const uint16_t* s, const uint8_t* z, int N, int K,
                          int group, uint8_t* codes, uint8_t* scales, uint8_t* zeros,
                          hipStream_t st) {
  const int nkb = (K + 127) / 128, tiles = (N + 15) / 16, groups = nkb * (128 / group);
  const int64_t sg = (int64_t)tiles * 16 * groups, lanes = (int64_t)tiles * nkb * 64;
  hipLaunchKernelGGL(q4_pack_scales_kernel, dim3((unsigned)((sg + 255) / 256)), dim3(256), 0, st,
                     s, z, N, (K + group - 1) / group, tiles * 16, groups,
                     reinterpret_cast<uint16_t*>(scales), zeros);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL(q4_pack_codes_kernel, dim3((unsigned)((lanes + 255) / 256)), dim3(256), 0,
                     st, q, N, K, nkb, lanes, reinterpret_cast<uint4*>(codes));
  return hipGetLastError();
}

}  // namespace moe
