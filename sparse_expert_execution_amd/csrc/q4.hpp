// q4.hpp - device side of the 4-bit integer matrices (groups of 32, 64 or 128
// columns sharing a BF16 scale and a zero point), shared by the dense product
// and the routed experts.
//
// Value of an element: s_g (q - z_g), q in 0..15.  A matrix [N][K] is stored
// in tiles of 16 rows x 128 columns, 1 KB each, so that one wave load is 1 KB
// of consecutive memory (on this part 16 rows x 64 bytes of a row-major
// matrix reach about half the rate): lane l = 16 q + r holds 16 bytes of row
// r, and its dword s the columns 32 s + 8 q + (0..7), which is that lane's
// operand of one 16x16x32 BF16 matrix instruction.  Element i of the dword is
// in nibble i / 2 + 4 (i % 2): a shift and an and-or give the BF16 pair
// (2 j, 2 j + 1), both of them 16 + q exactly: 16.0 with the four code bits
// as the upper four mantissa bits.
//
// The products: sum (16 + q) x - (16 + z) sum x, both on the matrix core with
// fp32 accumulation: the second is one more instruction per 32 columns whose
// weight operand is the constant -(16 + z) (an integer BF16 holds exactly),
// which costs no vector instruction and stays below the time of the loads.
// The group's sum is then multiplied by its scale and added in fp32.
//
// The tokens are the instruction's rows and the weights its columns: a lane's
// results all belong to weight row l % 16, so a group has one scale per lane,
// and the multiply-adds with it are only as many as a lane has tokens.  Token
// slot 4 (t % 4) + t / 4 holds token t (result row 4 (l / 16) + i is slot that
// of lane l's i-th result), so up to four tokens cost one multiply-add, eight two.
#pragma once
#include "device.hpp"
#include "kernels.hpp"

namespace moe {
namespace q4 {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ bf16x8 frag(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

__device__ __forceinline__ v4f mfma(bf16x8 a, bf16x8 b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// a dword of eight codes -> eight BF16 values 16 + q
__device__ __forceinline__ bf16x8 codes_plus16(uint32_t w) {
  constexpr uint32_t m = 0x00780078u;
  // in a vector register: an and-or takes one scalar constant, not two
  uint32_t one;
  asm("" : "=v"(one) : "0"(0x41804180u));
  return frag(u32x4{((w << 3) & m) | one, ((w >> 1) & m) | one, ((w >> 5) & m) | one,
                    ((w >> 9) & m) | one});
}

// eight times -(16 + z), exact for z <= 240
__device__ __forceinline__ bf16x8 minus_16_plus(uint32_t z) {
  const uint32_t b = __float_as_uint(-16.f - (float)z);
  const uint32_t p = (b & 0xffff0000u) | (b >> 16);
  return frag(u32x4{p, p, p, p});
}

// token of operand row r, and the other way round: token of lane l's result i
__device__ __forceinline__ int slot_token(int r) { return (r >> 2) + 4 * (r & 3); }
__device__ __forceinline__ int result_token(int lane, int i) { return (lane >> 4) + 4 * i; }

// what a lane holds of one tile: its codes, and of group l / 16 % (128 / G) the
// scale (and zero point) of its row
template <int G, bool ZERO>
struct Tile {
  uint4 codes;
  uint16_t scale;
  uint8_t zero;
};

// v of lane group l / 16 % N -> the N groups' values in every lane.  One load of
// all groups and these exchanges instead of a load per group: a load costs its 64
// addresses whatever it brings.
template <int N>
__device__ __forceinline__ void spread(uint32_t v, uint32_t (&o)[N]) {
  if constexpr (N == 1) {
    o[0] = v;
  } else if constexpr (N == 2) {
    const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    o[0] = p[0];
    o[1] = p[1];
  } else {
    static_assert(N == 4, "groups of 32, 64 or 128");
    const auto h = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    const auto a = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);
    const auto b = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);
    o[0] = a[0];
    o[1] = a[1];
    o[2] = b[0];
    o[3] = b[1];
  }
}

struct Matrix {
  const uint8_t* codes;     // [row tiles][column blocks][64 lanes][16]
  const uint8_t* scales;    // BF16 [row tiles][groups][16 rows]
  const uint8_t* zeros;     // bytes, same order (null: 8)
  int nkb;                  // column blocks of 128
};

// tile, kb and live are the same for the whole wave, so the addresses are a
// scalar base and a lane's constant offset.  live = false: a step past the end,
// whose loads stay so that the waits keep their counts, all lanes on one line.
template <int G, bool ZERO>
__device__ __forceinline__ void load_tile(Tile<G, ZERO>& t, const Matrix& m, int tile, int kb,
                                          bool live) {
  const uint32_t lane = (threadIdx.x & 63) & (live ? 63u : 0u);
  const int64_t at = (int64_t)tile * m.nkb + kb;
  const uint8_t* codes = m.codes + at * 1024;
  t.codes = ldg16(codes + lane * 16);
  const uint8_t* scales = m.scales + at * (128 / G) * 32;
  const uint8_t* zeros = m.zeros + at * (128 / G) * 16;
  const uint32_t i = lane & (16 * 128 / G - 1);
  t.scale = *reinterpret_cast<const uint16_t*>(scales + i * 2);
  if (ZERO) t.zero = zeros[i];
}

// A buffer of `bytes` bytes for loads whose lanes with nothing to read take an
// offset past its end: they read zeros, without a branch.  A branch around a load
// would make every later wait count without it, i.e. wait for loads meant to stay
// in flight (the down product took 60 us with branches where it takes 45).
typedef __amdgpu_buffer_rsrc_t Buffer;
constexpr uint32_t kNowhere = 0x80000000u;            // bytes < 2^31
__device__ __forceinline__ Buffer buffer_of(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00027000);
}

// 128 columns of the operand rows: `row` is the lane's byte offset (or kNowhere),
// `base` (scalar) that of the block's first column, STEP the bytes from one 32
// columns to the next, `left` the columns from there on (a multiple of 32; zeros
// past them).
template <int STEP>
__device__ __forceinline__ void load_rows(bf16x8 (&x)[4], Buffer b, uint32_t row, uint32_t base,
                                          int left) {
#pragma unroll
  for (int s = 0; s < 4; ++s)
    x[s] = __builtin_bit_cast(
        bf16x8, __builtin_amdgcn_raw_buffer_load_b128(b, 32 * s < left ? row : kNowhere,
                                                      base + STEP * s, 0));
}

__device__ __forceinline__ uint32_t dword(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// acc[r][j] += x[j] times tile r, for the first TI results of a lane.  Group by
// group, so that only one group's operands are live.
template <int RT, int NT, int TI, int G, bool ZERO>
__device__ __forceinline__ void mul_tiles(float (&acc)[RT][NT][TI], const Tile<G, ZERO> (&t)[RT],
                                          const bf16x8 (&x)[NT][4]) {
  constexpr int S = G / 32;
  uint32_t sz[RT][128 / G];                           // scale, zero point above it
#pragma unroll
  for (int r = 0; r < RT; ++r)
    spread(ZERO ? t[r].scale | (uint32_t)t[r].zero << 16 : t[r].scale, sz[r]);
#pragma unroll
  for (int g = 0; g < 128 / G; ++g) {
    v4f c[NT];                                        // -24 sum x: for all tiles the same
    if (!ZERO) {
      const bf16x8 k = minus_16_plus(8);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        c[j] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < S; ++s) c[j] = mfma(x[j][g * S + s], k, c[j]);
      }
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      bf16x8 w[S], z;
#pragma unroll
      for (int s = 0; s < S; ++s) w[s] = codes_plus16(dword(t[r].codes, g * S + s));
      if (ZERO) z = minus_16_plus(sz[r][g] >> 16);
      const float sc = __uint_as_float(sz[r][g] << 16);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        v4f d = ZERO ? v4f{0.f, 0.f, 0.f, 0.f} : c[j];
        if (ZERO)
#pragma unroll
          for (int s = 0; s < S; ++s) d = mfma(x[j][g * S + s], z, d);
#pragma unroll
        for (int s = 0; s < S; ++s) d = mfma(x[j][g * S + s], w[s], d);
#pragma unroll
        for (int i = 0; i < TI; ++i) acc[r][j][i] = fmaf(sc, d[i], acc[r][j][i]);
      }
    }
  }
}

}  // namespace q4
}  // namespace moe
