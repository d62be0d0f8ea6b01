// q4_experts.hip - decode of experts held as 4-bit integer matrices (q4.hpp):
// gate and up with SwiGLU, then down with the weighted combine.
//
//   h_p  = silu(W_g x_t) * (W_u x_t)        p = (t, j), expert ids[p]
//   y_t  = sum_j w_tj W_d h_tj  (+ the shared expert, weight 1)
//
// Bound: HBM, the bytes of the distinct experts.  The unit of work is a
// distinct expert with the pairs that chose it (the shared expert: all
// tokens).  Up to 64 pairs every workgroup lists the units itself, with one
// wave; more pairs take a launch of their own for the list.
#include "q4.hpp"

namespace moe {
namespace {

using namespace q4;

// ---- units ------------------------------------------------------------------
// One workgroup, thread i is pair i.  An expert's pairs are set in a bit mask
// of its own in LDS, from which each of them reads the expert's first pair, its
// own place and their number.  Units are numbered by first appearance, their
// entries (pair numbers, ascending) stored one after another.  Experts without
// a slot and ids outside [0, E) give no unit.  Bound by latency: 4.8 us for 512
// pairs of 128 experts.
constexpr int kUnitThreads = kQ4MaxPairs, kMaskWords = kQ4MaxPairs / 32;

__global__ __launch_bounds__(kUnitThreads) void q4_units_kernel(Q4Experts a) {
  extern __shared__ uint32_t mask[];                  // [kMaskWords][E]: few bank conflicts
  __shared__ int s_sum[kUnitThreads / 64];
  __shared__ int16_t s_base[kQ4MaxPairs];
  const int i = threadIdx.x, lane = i & 63, wave = i >> 6;
  int id = -1, slot = -1;
  if (i < a.P) {
    id = a.ids[i];
    if (id >= 0 && id < a.E) slot = a.slot_of ? a.slot_of[id] : id;
    if (slot < 0) id = -1;
  }
  for (int w = i; w < kMaskWords * a.E; w += kUnitThreads) mask[w] = 0;
  __syncthreads();
  if (id >= 0) atomicOr(&mask[i / 32 * a.E + id], 1u << (i % 32));
  __syncthreads();
  int first = -1, rank = 0, count = 0;
  if (id >= 0) {
#pragma unroll
    for (int w = kMaskWords - 1; w >= 0; --w) {
      const uint32_t v = mask[w * a.E + id];
      if (v) first = 32 * w + __builtin_ctz(v);
      count += __popc(v);
      rank += w < i / 32 ? __popc(v) : w == i / 32 ? __popc(v & ((1u << (i % 32)) - 1)) : 0;
    }
  }
  const bool lead = id >= 0 && first == i;
  const int packed = lead ? 1 << 16 | count : 0;
  const int inc = wave_scan_dpp(packed);
  if (lane == 63) s_sum[wave] = inc;
  __syncthreads();
  int before = inc - packed, total = 0;
#pragma unroll
  for (int v = 0; v < kUnitThreads / 64; ++v) {
    if (v < wave) before += s_sum[v];
    total += s_sum[v];
  }
  if (lead) {
    s_base[i] = (int16_t)(before & 0xffff);
    a.units[before >> 16] = make_int4(slot, before & 0xffff, count, 0);
  }
  __syncthreads();
  if (id >= 0) a.entries[s_base[first] + rank] = (int16_t)i;
  const int routed = total >> 16, pairs = total & 0xffff;
  if (a.shared) {
    if (i == 0) a.units[routed] = make_int4(-1, pairs, a.T, 0);
    if (i < a.T) a.entries[pairs + i] = (int16_t)(a.P + i);
  }
  if (i == 0) *a.n_units = routed + (a.shared ? 1 : 0);
}

// The same list of at most 64 pairs by one wave, into LDS.  Lane i is pair i.
constexpr int kWavePairs = kQ4WavePairs;

struct UnitList {
  int4 unit[kWavePairs + 1];
  int16_t entry[kWavePairs + kQ4MaxTokens];
  int n;
};

__device__ __forceinline__ void wave_units(const Q4Experts& a, UnitList& u) {
  const int i = threadIdx.x & 63;
  int id = -1, slot = -1;
  if (i < a.P) {
    id = a.ids[i];
    if (id >= 0 && id < a.E) slot = a.slot_of ? a.slot_of[id] : id;
    if (slot < 0) id = -1;
  }
  int first = 64, rank = 0, count = 0;
  for (int j = 0; j < a.P; ++j) {
    const bool same = __builtin_amdgcn_readlane(id, j) == id;
    first = same && j < first ? j : first;
    rank += same && j < i;
    count += same;
  }
  const bool lead = id >= 0 && first == i;
  const int packed = lead ? 1 << 16 | count : 0;
  const int inc = wave_scan_dpp(packed), before = inc - packed;
  const int total = __builtin_amdgcn_readlane(inc, 63);
  const int base = __shfl(before & 0xffff, first & 63, kWave);
  if (lead) u.unit[before >> 16] = make_int4(slot, before & 0xffff, count, 0);
  if (id >= 0) u.entry[base + rank] = (int16_t)i;
  const int routed = total >> 16, pairs = total & 0xffff;
  if (a.shared) {
    if (i == 0) u.unit[routed] = make_int4(-1, pairs, a.T, 0);
    if (i < a.T) u.entry[pairs + i] = (int16_t)(a.P + i);
  }
  if (i == 0) u.n = routed + (a.shared ? 1 : 0);
}

// ---- gate / up --------------------------------------------------------------
// grid (row tiles of I / per, units).  A workgroup's waves are four slices of H for
// `per` row tiles of both matrices, one after the other; the partial sums meet in
// LDS in slice order, while the next tile's loads are in flight.  x comes from the
// L2 straight into the operand's registers.  (Eight waves for one token's few
// workgroups: 7.4 us instead of 7.1.)
//
// Bound: HBM, 4 tokens with 6 experts each and a shared one, H = 4096, I = 2048,
// groups of 32: 50 us, 4.6 TB/s; one token (2048/768, 8 experts) 7 us, latency; 64
// tokens on the 128 experts of 2048/768, groups of 64: 51 us, 4.1 TB/s, the loads
// of x (a cache access per lane) beside those of the experts.
constexpr int kGuWaves = 4;

template <int TI, int G>
__device__ __forceinline__ void gate_up_columns(const Q4Experts& a, const uint8_t* block, int tile0,
                                                int tiles, const int16_t* entries, int n_cols,
                                                float (&red)[2][2][4][kGuWaves][64]) {
  constexpr int D = 2;
  const int lane = threadIdx.x & 63, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nkb = (a.H + 127) / 128;
  const Matrix mg{block + a.off[0], block + a.off[1], nullptr, nkb};
  const Matrix mu{block + a.off[2], block + a.off[3], nullptr, nkb};
  const int c = slot_token(lane & 15);
  const bool live = c < n_cols;
  int token = 0;
  if (live) {
    const int e = entries[c];
    token = e < a.P ? e / a.k : e - a.P;
  }
  const uint32_t xrow = live ? ((uint32_t)token * a.H + 8 * q) * 2 : kNowhere;
  const Buffer xb = buffer_of(a.x, (uint32_t)a.T * a.H * 2);
  struct Block {
    Tile<G, false> t[2];
    bf16x8 x[1][4];
    int valid, flush;                                 // the last block of its row tile
  };
  // where the loads are: row tile `rt`, column block kb; past the last one the
  // first again
  int rt = wave < nkb ? 0 : tiles, kb = wave;
  auto load = [&](Block& b) {
    const bool in = rt < tiles;
    const int k = in ? kb : 0, r = tile0 + (in ? rt : 0);
    load_tile<G, false>(b.t[0], mg, r, k, in);
    load_tile<G, false>(b.t[1], mu, r, k, in);
    load_rows<64>(b.x[0], xb, xrow, 256 * k, in ? a.H - 128 * k : 0);
    b.valid = in;
    kb += kGuWaves;
    b.flush = kb >= nkb;
    if (b.flush) {
      kb = wave;
      ++rt;
    }
  };
  float acc[2][1][TI];
  int done = 0;
  // a row tile's sums: every wave comes here once for each.  Two buffers: a wave
  // writes one of them again only after a barrier behind which all have read it.
  auto finish = [&]() {
    const int buf = done & 1;
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      red[buf][0][i][wave][lane] = acc[0][0][i];
      red[buf][1][i][wave][lane] = acc[1][0][i];
      acc[0][0][i] = acc[1][0][i] = 0.f;
    }
    __syncthreads();
    for (int id = threadIdx.x; id < TI * 64; id += kGuWaves * 64) {
      const int l = id & 63, i = id >> 6;
      float g = 0.f, u = 0.f;
#pragma unroll
      for (int s = 0; s < kGuWaves; ++s) {
        g += red[buf][0][i][s][l];
        u += red[buf][1][i][s][l];
      }
      const int col = result_token(l, i);
      if (col >= n_cols) continue;
      const float h = g / (1.f + expf(-g)) * u;
      // h as three BF16 parts, all 24 bits of it: y keeps fp32's accuracy rather
      // than BF16's.  Laid out [entry][8 of I][part][8], as four neighbouring
      // lanes of the down product read it.
      const int row = 16 * (tile0 + done) + (l & 15);
      const int64_t at = (int64_t)entries[col] * a.I * 3 + (row >> 3) * 24 + (row & 7);
      const __bf16 h0 = (__bf16)h;
      const float r1 = h - (float)h0;
      const __bf16 h1 = (__bf16)r1;
      const __bf16 h2 = (__bf16)(r1 - (float)h1);
      a.h[at] = __builtin_bit_cast(uint16_t, h0);
      a.h[at + 8] = __builtin_bit_cast(uint16_t, h1);
      a.h[at + 16] = __builtin_bit_cast(uint16_t, h2);
    }
    ++done;
  };
#pragma unroll
  for (int i = 0; i < TI; ++i) acc[0][0][i] = acc[1][0][i] = 0.f;
  if (rt == tiles) {                                  // more waves than column blocks
    for (int t = 0; t < tiles; ++t) finish();
  } else {
    Block b[D];
#pragma unroll
    for (int d = 0; d < D - 1; ++d) load(b[d]);
    for (bool more = true; more;) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (!__builtin_amdgcn_readfirstlane(b[d].valid)) {
          more = false;
          break;
        }
        load(b[(d + D - 1) % D]);
        mul_tiles<2, 1, TI, G, false>(acc, b[d].t, b[d].x);
        if (__builtin_amdgcn_readfirstlane(b[d].flush)) finish();
      }
    }
  }
  __syncthreads();                                    // before the next columns' sums
}

template <int G, bool SMALL>
__global__ __launch_bounds__(kGuWaves * 64, 4) void q4_gate_up_kernel(Q4Experts a, int per,
                                                                      bool clear_y) {
  __shared__ float red[2][2][4][kGuWaves][64];
  __shared__ UnitList list;
  if (clear_y) {
    const int64_t all = (int64_t)gridDim.x * gridDim.y * kGuWaves * 64;
    for (int64_t i = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kGuWaves * 64 + threadIdx.x;
         i < (int64_t)a.T * a.H; i += all)
      a.y[i] = 0.f;
  }
  int4 u;
  const int16_t* entries;
  if (SMALL) {
    if (threadIdx.x < 64) wave_units(a, list);
    __syncthreads();
    if ((int)blockIdx.y >= list.n) return;
    u = list.unit[blockIdx.y];
    entries = list.entry + u.y;
  } else {
    if ((int)blockIdx.y >= *a.n_units) return;
    u = a.units[blockIdx.y];
    entries = a.entries + u.y;
  }
  const int slot = __builtin_amdgcn_readfirstlane(u.x);
  const int count = __builtin_amdgcn_readfirstlane(u.z);
  const uint8_t* block = slot < 0 ? a.shared : a.pool + (int64_t)slot * a.expert_bytes;
  const int tile = blockIdx.x * per, tiles = min(per, a.I / 16 - tile);
  for (int c0 = 0; c0 < count; c0 += 16) {
    const int n = min(16, count - c0);
    if (n <= 4) gate_up_columns<1, G>(a, block, tile, tiles, entries + c0, n, red);
    else if (n <= 8) gate_up_columns<2, G>(a, block, tile, tiles, entries + c0, n, red);
    else gate_up_columns<4, G>(a, block, tile, tiles, entries + c0, n, red);
  }
}

// ---- down + combine -----------------------------------------------------------
// One workgroup per 16 RT rows of y, for all tokens and experts, so the combine
// needs no other pass: the units' tiles are cut into jobs (an item, i.e. up to
// four entries of a unit, and a slice of I) that go round the 16 waves; a wave
// adds a job's gate-weighted result into a y tile of its own in LDS, and the 16
// tiles are summed in wave order.  Where that gives too few workgroups for the
// compute units, several share the jobs of a tile: two add into a cleared y (0 + a
// + b has one value whichever comes first), more leave their sums to one more
// launch that adds them in order.
//
// Operand row 4 e + part is part `part` of h of the job's entry e (the fourth row
// of an entry is empty), so one instruction takes four entries, neighbouring lanes
// of a load read 48 bytes of one entry (rows of h apart from each other were a
// cache access per lane), and a lane's results 0, 1, 2 are the parts of entry
// l / 16.
//
// Bound: the loads of h (an item of four entries reads 3 KB of it for each 1 KB of
// codes, half of that with RT = 2) beside the experts' bytes.  The cases of the
// gate / up product: 30 us, 4.0 TB/s (RT = 1: 33); 6 us; 35 us, 3.0 TB/s.
constexpr int kDnWaves = 16;

template <int RT, int G, bool SMALL>
__global__ __launch_bounds__(kDnWaves * 64, 4) void q4_down_kernel(Q4Experts a, int cut) {
  constexpr int D = 3;
  constexpr int kPairs = SMALL ? kWavePairs : kQ4MaxPairs;
  extern __shared__ float yl[];                       // [wave][T][16 RT]
  __shared__ UnitList list;
  __shared__ int4 s_unit[SMALL ? 1 : kPairs + 1];
  __shared__ int16_t s_entry[SMALL ? 1 : kPairs + kQ4MaxTokens];
  __shared__ float s_w[kPairs + kQ4MaxTokens];
  __shared__ int s_item[kPairs + kQ4MaxTokens / 4], s_items;   // a pair each at most
  __shared__ uint8_t s_token[kPairs + kQ4MaxTokens];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane >> 4, n = lane & 15;
  // by pair: the token and the gate weight
  for (int i = threadIdx.x; i < a.P + a.T; i += kDnWaves * 64) {
    s_token[i] = (uint8_t)(i < a.P ? i / a.k : i - a.P);
    s_w[i] = i < a.P ? a.w[i] : 1.f;
  }
  for (int j = threadIdx.x; j < kDnWaves * a.T * 16 * RT; j += kDnWaves * 64) yl[j] = 0.f;
  int n_units;
  const int4* units;
  const int16_t* entries;
  if (SMALL) {
    if (threadIdx.x < 64) wave_units(a, list);
    __syncthreads();
    n_units = list.n;
    units = list.unit;
    entries = list.entry;
  } else {
    n_units = *a.n_units;
    for (int i = threadIdx.x; i < n_units; i += kDnWaves * 64) s_unit[i] = a.units[i];
    for (int i = threadIdx.x; i < a.P + a.T; i += kDnWaves * 64) s_entry[i] = a.entries[i];
    __syncthreads();
    units = s_unit;
    entries = s_entry;
  }
  n_units = __builtin_amdgcn_readfirstlane(n_units);
  // items: unit << 10 | first of its entries' place in the unit.  Whole units as
  // jobs left waves waiting for those that had the units of many entries.
  if (wave == 0) {
    int at = 0;
    for (int i0 = 0; i0 < n_units; i0 += 64) {
      const int i = i0 + lane;
      const int chunks = i < n_units ? (units[i].z + 3) / 4 : 0;
      const int inc = wave_scan_dpp(chunks);
      for (int c = 0; c < chunks; ++c) s_item[at + inc - chunks + c] = i << 10 | 4 * c;
      at += __builtin_amdgcn_readlane(inc, 63);
    }
    if (lane == 0) s_items = at;
  }
  __syncthreads();
  const int n_items = __builtin_amdgcn_readfirstlane(s_items);
  const int nkb = (a.I + 127) / 128, tile = blockIdx.x * RT;
  const int per = (nkb + cut - 1) / cut;              // column blocks of a job
  const int slices = (nkb + per - 1) / per;
  float* mine = yl + (int64_t)wave * a.T * 16 * RT;
  const int e4 = n >> 2, part = n & 3;                // as an operand row

  // Where the loads are: item `ii`, slice `sl` of its columns, column block kb.
  // All of it is the same for the whole wave, and said so to the compiler, which
  // else keeps it in vector registers.
  const auto uni = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
  const int stride = kDnWaves * gridDim.y, item_step = uni(stride / slices);
  const int slice_step = uni(stride - item_step * slices);
  const int job0 = uni(wave) * gridDim.y + blockIdx.y;
  int ii = uni(job0 / slices), sl = uni(job0 - ii * slices);
  int kb = 0, kend = 0, first = 0, count = 0, slot = 0;
  const Buffer hb = buffer_of(a.h, (uint32_t)(a.P + a.T) * a.I * 6);
  uint32_t hrow = kNowhere;                           // bytes
  auto start = [&]() {
    const int item = uni(s_item[ii]), c0 = item & 1023;
    const int4 u = units[item >> 10];
    slot = uni(u.x);
    first = uni(u.y) + c0;
    count = min(4, uni(u.z) - c0);
    kb = sl * per;
    kend = min(kb + per, nkb);
    hrow = part < 3 && e4 < count
               ? (uint32_t)entries[first + e4] * a.I * 6 + q * 48 + part * 16
               : kNowhere;
  };

  // a column block in flight; at the last one of a job: its entries and number
  struct Block {
    Tile<G, false> t[RT];
    bf16x8 x[1][4];
    int valid, flush, at;
  };
  auto load = [&](Block& b) {
    ii = uni(ii);
    kb = uni(kb);
    const bool in = ii < n_items;
    b.valid = in;
    const uint8_t* block = slot < 0 ? a.shared : a.pool + (int64_t)uni(slot) * a.expert_bytes;
    const Matrix m{block + a.off[4], block + a.off[5], nullptr, nkb};
#pragma unroll
    for (int r = 0; r < RT; ++r) load_tile<G, false>(b.t[r], m, tile + r, kb, in);
    load_rows<192>(b.x[0], hb, hrow, 768 * kb, in ? a.I - 128 * kb : 0);
    b.flush = 0;
    b.at = first;
    if (!in) return;
    if (++kb == kend) {
      b.flush = count;
      ii += item_step;
      sl += slice_step;
      if (sl >= slices) {
        sl -= slices;
        ++ii;
      }
      if (ii < n_items) start();
      else kb = 0;        // loads past the last job: a block of this tile, not one past it
    }
  };
  if (ii < n_items) {
    start();
    Block b[D];
#pragma unroll
    for (int d = 0; d < D - 1; ++d) load(b[d]);
    float acc[RT][1][3] = {};
    for (bool more = true; more;) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (!uni(b[d].valid)) {
          more = false;
          break;
        }
        load(b[(d + D - 1) % D]);
        mul_tiles<RT, 1, 3, G, false>(acc, b[d].t, b[d].x);
        const int flush = uni(b[d].flush);
        if (flush == 0) continue;
        if (q < flush) {
          const int e = entries[b[d].at + q];
          // an LDS add: a token that names one expert twice is two entries here
#pragma unroll
          for (int r = 0; r < RT; ++r)
            __hip_atomic_fetch_add(&mine[(s_token[e] * RT + r) * 16 + n],
                                   s_w[e] * (acc[r][0][0] + (acc[r][0][1] + acc[r][0][2])),
                                   __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[r][0][0] = acc[r][0][1] = acc[r][0][2] = 0.f;
      }
    }
  }
  __syncthreads();
  for (int j = threadIdx.x; j < a.T * 16 * RT; j += kDnWaves * 64) {
    float v = 0.f;
#pragma unroll
    for (int s = 0; s < kDnWaves; ++s) v += yl[(int64_t)s * a.T * 16 * RT + j];
    float* y = a.y + (int64_t)(j / (16 * RT)) * a.H + 16 * tile + j % (16 * RT);
    if (a.part) a.part[(int64_t)blockIdx.y * a.T * a.H + (y - a.y)] = v;
    else if (gridDim.y == 1) *y = v;
    else __hip_atomic_fetch_add(y, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
}

// y = the sum of the workgroups' shares, in their order
__global__ __launch_bounds__(256) void q4_sum_kernel(const float* part, int parts, int n,
                                                     float* y) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float s = part[i];
  for (int p = 1; p < parts; ++p) s += part[(int64_t)p * n + i];
  y[i] = s;
}

// Row tiles of a down workgroup: two, with half the loads of h for each, where that
// still gives a workgroup for every second compute unit (H is a multiple of 32), and
// for many pairs, where h is most of what is loaded: 64 tokens of 2048/768 35 us and
// 5 of q4_sum_kernel, the call 92 us; one row tile and no such launch 42, 97.
template <bool SMALL>
int down_tiles(const Q4Experts& a) { return !SMALL || a.H / 32 >= 128 ? 2 : 1; }
// workgroups that share them (two: y is cleared by the gate / up launch)
template <bool SMALL>
int down_split(const Q4Experts& a) {
  return !SMALL ? q4_down_split(a.H) : a.H / (16 * down_tiles<SMALL>(a)) <= 128 ? 2 : 1;
}

template <int RT, int G, bool SMALL>
hipError_t run_down(const Q4Experts& a, int cut, hipStream_t st) {
  hipLaunchKernelGGL((q4_down_kernel<RT, G, SMALL>), dim3(a.H / (16 * RT), down_split<SMALL>(a)),
                     dim3(kDnWaves * 64), (size_t)kDnWaves * a.T * 16 * RT * sizeof(float), st, a,
                     cut);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || !a.part) return err;
  const int n = a.T * a.H;
  hipLaunchKernelGGL(q4_sum_kernel, dim3((n + 255) / 256), dim3(256), 0, st, a.part,
                     down_split<SMALL>(a), n, a.y);
  return hipGetLastError();
}

template <int G, bool SMALL>
hipError_t run_products(const Q4Experts& a, hipStream_t st) {
  const int most = (a.P < a.E ? a.P : a.E) + (a.shared ? 1 : 0);   // units at most
  const int tiles = a.I / 16 * most;
  // The compute units hold 1024 workgroups of gate / up.  Twice that many and more
  // take two row tiles each: 64 tokens of 2048/768, 6144 tiles, 53 -> 51 us; 3200
  // tiles the same; 384 7 -> 9 us.
  const int per = tiles >= 2048 ? 2 : 1;
  hipLaunchKernelGGL((q4_gate_up_kernel<G, SMALL>), dim3((a.I / 16 + per - 1) / per, most),
                     dim3(kGuWaves * 64), 0, st, a, per, down_split<SMALL>(a) > 1 && !a.part);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const int split = down_split<SMALL>(a);
  // enough jobs for four rounds of the waves: an uneven last one costs little
  int cut = (4 * kDnWaves * split + most - 1) / most;
  const int nkb = (a.I + 127) / 128;
  cut = cut < 1 ? 1 : cut > nkb ? nkb : cut;
  if constexpr (SMALL)
    if (down_tiles<SMALL>(a) == 1) return run_down<1, G, SMALL>(a, cut, st);
  return run_down<2, G, SMALL>(a, cut, st);
}

template <int G>
hipError_t run(const Q4Experts& a, hipStream_t st) {
  if (a.P <= kWavePairs) return run_products<G, true>(a, st);
  hipLaunchKernelGGL(q4_units_kernel, dim3(1), dim3(kUnitThreads),
                     (size_t)a.E * kMaskWords * 4, st, a);
  const hipError_t err = hipGetLastError();
  return err != hipSuccess ? err : run_products<G, false>(a, st);
}

}  // namespace

hipError_t launch_q4_experts(Q4Experts a, int group, hipStream_t st) {
  a.P = a.T * a.k;
  if (!q4_down_parts(a.P, a.H)) a.part = nullptr;
  if (a.T < 1 || a.P > kQ4MaxPairs || a.T > kQ4MaxTokens) return hipErrorInvalidValue;
  if (group == 32) return run<32>(a, st);
  if (group == 64) return run<64>(a, st);
  return run<128>(a, st);
}

}  // namespace moe
