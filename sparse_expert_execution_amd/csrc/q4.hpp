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
  constexpr uint32_t m = 0x00780078u, one = 0x41804180u;
  return frag(u32x4{((w << 3) & m) | one, ((w >> 1) & m) | one, ((w >> 5) & m) | one,
                    ((w >> 9) & m) | one});
}

// eight times -(16 + z), exact for z <= 240
__device__ __forceinline__ bf16x8 minus_16_plus(uint32_t z) {
  const uint32_t b = __float_as_uint(-16.f - (float)z);
  const uint32_t p = (b & 0xffff0000u) | (b >> 16);
  return frag(u32x4{p, p, p, p});
}

// what a lane holds of one tile: its codes, and per group the scales of the
// four result rows 4 (l / 16) + i and (ZERO) the zero point of its own row
template <int G, bool ZERO>
struct Tile {
  uint4 codes;
  uint2 scale[128 / G];
  uint8_t zero[ZERO ? 128 / G : 1];
};

struct Matrix {
  const uint8_t* codes;     // [row tiles][column blocks][64 lanes][16]
  const uint8_t* scales;    // BF16 [row tiles][groups][16 rows]
  const uint8_t* zeros;     // bytes, same order (null: 8)
  int nkb;                  // column blocks of 128
};

template <int G, bool ZERO>
__device__ __forceinline__ void load_tile(Tile<G, ZERO>& t, const Matrix& m, int tile, int kb) {
  const int lane = threadIdx.x & 63;
  const int64_t at = (int64_t)tile * m.nkb + kb;
  t.codes = ldg16(m.codes + (at * 64 + lane) * 16);
#pragma unroll
  for (int g = 0; g < 128 / G; ++g) {
    const int64_t gi = at * (128 / G) + g;
    t.scale[g] = *reinterpret_cast<const uint2*>(m.scales + gi * 32 + (lane >> 4) * 8);
    if (ZERO) t.zero[g] = m.zeros[gi * 16 + (lane & 15)];
  }
}

// -24 sum x of every group (symmetric matrices: the same for all rows)
template <int G, int NP>
__device__ __forceinline__ void group_sums(v4f (&c)[128 / G], const bf16x8 (&x)[NP][4]) {
  const bf16x8 k = minus_16_plus(8);
#pragma unroll
  for (int g = 0; g < 128 / G; ++g) {
    c[g] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = g * (G / 32); s < (g + 1) * (G / 32); ++s)
#pragma unroll
      for (int p = 0; p < NP; ++p) c[g] = mfma(k, x[p][s], c[g]);
  }
}

// acc += this tile times x.  x has NP planes that are summed (a value held as
// BF16 parts), c is group_sums of them (ZERO: unused).
template <int G, bool ZERO, int NP>
__device__ __forceinline__ void mul_tile(v4f& acc, const Tile<G, ZERO>& t,
                                         const bf16x8 (&w)[4], const bf16x8 (&x)[NP][4],
                                         const v4f (&c)[128 / G]) {
#pragma unroll
  for (int g = 0; g < 128 / G; ++g) {
    v4f d = ZERO ? v4f{0.f, 0.f, 0.f, 0.f} : c[g];
    if (ZERO) {
      const bf16x8 z = minus_16_plus(t.zero[g]);
#pragma unroll
      for (int s = g * (G / 32); s < (g + 1) * (G / 32); ++s)
#pragma unroll
        for (int p = 0; p < NP; ++p) d = mfma(z, x[p][s], d);
    }
#pragma unroll
    for (int s = g * (G / 32); s < (g + 1) * (G / 32); ++s)
#pragma unroll
      for (int p = 0; p < NP; ++p) d = mfma(w[s], x[p][s], d);
    const uint2 sc = t.scale[g];
    acc[0] = fmaf(bf16_lo(sc.x), d[0], acc[0]);
    acc[1] = fmaf(bf16_hi(sc.x), d[1], acc[1]);
    acc[2] = fmaf(bf16_lo(sc.y), d[2], acc[2]);
    acc[3] = fmaf(bf16_hi(sc.y), d[3], acc[3]);
  }
}

template <int G, bool ZERO>
__device__ __forceinline__ void tile_weights(bf16x8 (&w)[4], const Tile<G, ZERO>& t) {
  w[0] = codes_plus16(t.codes.x);
  w[1] = codes_plus16(t.codes.y);
  w[2] = codes_plus16(t.codes.z);
  w[3] = codes_plus16(t.codes.w);
}

}  // namespace q4
}  // namespace moe
