// kernels.hpp - host-side launchers of the gfx950 kernels (internal).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

struct DecodeLaunch {
  const void* x;
  const void* w_router;   // null: ids / w are inputs
  int router_f32, renorm;
  int32_t* ids;
  float* w;
  const int32_t* slot_of;
  const void* pool;
  const void* shared;
  unsigned* hdr;          // counter header (zero before first use)
  uint64_t* z;            // kZCopies copies of [T][E] generation-tagged logits
  int64_t zstride;        // uint64 words from one copy to the next
  uint64_t* h;            // [T*k + T][I] generation-tagged h
  unsigned long long* stamps;  // [kMaxWorkgroups][16] phase stamps (timing only)
  float* y;
  int64_t expert_bytes;
  int64_t off[6];
  int64_t goff;           // NVFP4: offset of the three fp32 matrix scales, else 0
  int T, H, I, E, k, wtype;
};

struct PrefillLaunch {
  const void* x;
  const int32_t* ids;
  const float* w;
  const int32_t* slot_of;
  const void* pool;
  const void* shared;
  float* y;
  int64_t expert_bytes;
  int64_t off[6];
  int T, H, I, E, k;
  // workspace carve-up
  uint8_t* xq_codes;     // [T][H/2]
  uint8_t* xq_scales;    // [T][H/32]
  int32_t* chunk_counts; // [n_chunks][E+1]
  int32_t* seg_start;    // [E+2]
  int32_t* tiles;        // [2 * max_tiles + 1]: n_tiles, then (bin, row0) pairs
  int32_t* sorted_pair;  // [n_pairs]
  uint8_t* hq_codes;     // [n_pairs][I/2]   (sorted order); NVFP4: BF16 h [n_pairs][I]
  uint8_t* hq_scales;    // [n_pairs][I/32]; NVFP4: unused
  float* partial;        // [T][k+1][H]
  int nvfp4;             // weights NVFP4 (x not quantised, BF16 GEMMs)
  int64_t goff;          // NVFP4: offset of the three fp32 matrix scales
  int n_chunks, max_tiles;
};

// prefill GEMMs for NVFP4 weights (BF16 matrix cores); the sort is shared
struct NvPrefillArgs {
  const int32_t* slot_of;
  const uint8_t* pool;
  const uint8_t* shared;
  int64_t expert_bytes;
  int64_t off[6];
  int64_t goff;          // offset of the gate, up, down fp32 matrix scales
  int T, H, I, E, k;
  const int32_t* seg_start;
  const int32_t* tiles;
  const int32_t* sorted_pair;
  const uint16_t* x;     // [T][H] bf16
  uint16_t* hb;          // [n_pairs][I] bf16 h, sorted order
  float* partial;        // [T][k+1][H] per-pair outputs
};
hipError_t launch_prefill_nvfp4_gemms(const NvPrefillArgs& a, int max_tiles, hipStream_t st);

// router alone: small T (one wave per expert row, the last workgroup ranks),
// large T (tiled logits + one wave per token)
bool route_small_supported(int router_f32, int H);
hipError_t launch_route_small(const void* x, const void* w_router, int router_f32, int T, int H,
                              int E, int k, int renorm, float* z, unsigned* ticket, int32_t* ids,
                              float* w, hipStream_t st);
hipError_t launch_route_large(const void* x, const void* w_router, int router_f32, int T,
                              int H, int E, int k, int renorm, float* logits, int32_t* ids,
                              float* w, hipStream_t st);

// the gate on given logits, its statistics and its gradient (gate.hip)
struct GateArgs {
  const float* z;          // [T][E]
  const uint8_t* mask;     // [T], zero: not routed; null: all tokens are
  int T, E, k, renorm;
  int32_t* ids;            // [T][k]
  float* w;                // [T][k]
  int32_t* counts;         // [E + 1] or null
  float* loss;             // or null
  // workspace: a row of partial sums per workgroup
  float* part_s;           // [gate_parts(T)][E]
  int32_t* part_c;         // [gate_parts(T)][E]
  int32_t* part_n;         // [gate_parts(T)]
  float* share;            // [64]
  unsigned* ticket;
};
// workgroups (and rows of partial sums) of the gate: 16 tokens each until 256
inline int gate_parts(int T) { return T < 4096 ? (T + 15) / 16 : 256; }
hipError_t launch_gate(const GateArgs& a, hipStream_t st);

struct GateBackward {
  const float* z;
  const int32_t* ids;
  const float* w;
  const float* dw;         // [T][k] or null
  const int32_t* counts;   // [E + 1], with dloss
  const float* dloss;      // one value, or null
  int T, E, k, renorm;
  float* dz;               // [T][E]
};
hipError_t launch_gate_backward(const GateBackward& a, hipStream_t st);

// the router's product alone, and its gradients (router_train.hip)
hipError_t launch_router_logits(const void* x, const void* w, int router_f32, int T, int H, int E,
                                float* z, hipStream_t st);
struct RouterBackward {
  const void* x;           // BF16 [T][H]
  const void* w;           // [E][H]
  const float* dz;         // [T][E]
  int router_f32, T, H, E;
  uint16_t* dx;            // BF16 [T][H] or null
  float* dw;               // [E][H] or null
  uint8_t* ws;             // router_backward_bytes
};
size_t router_backward_bytes(int T, int H, int E);
hipError_t launch_router_backward(const RouterBackward& a, hipStream_t st);

// 4-bit integer matrices (q4.hip; layout in q4.hpp)
struct Q4Linear {
  const uint8_t* codes;
  const uint8_t* scales;
  const uint8_t* zeros;    // null: zero point 8
  const uint16_t* x;       // BF16, rows x_ld apart
  int64_t x_ld;
  int T, N, K;
  void* y;                 // rows y_ld apart
  int64_t y_ld;
  int y_bf16;
  int tiles, nkb, log_ks;  // set by the launcher
};
hipError_t launch_q4_linear(Q4Linear a, int group, hipStream_t st);
hipError_t launch_q4_quantize(const void* src, int src_bf16, int N, int K, int64_t ld, int group,
                              uint8_t* codes, uint8_t* scales, uint8_t* zeros, hipStream_t st);
hipError_t launch_q4_pack(const uint8_t* q, const uint16_t* s, const uint8_t* z, int N, int K,
                          int group, uint8_t* codes, uint8_t* scales, uint8_t* zeros,
                          hipStream_t st);

// decode of experts in that format (q4_experts.hip)
constexpr int kQ4MaxTokens = 64, kQ4MaxPairs = 512;
struct Q4Experts {
  const uint16_t* x;       // BF16 [T][H]
  const int32_t* ids;
  const float* w;
  const int32_t* slot_of;
  const uint8_t* pool;
  const uint8_t* shared;   // or null
  int64_t expert_bytes;
  int64_t off[6];
  int T, H, I, E, k;
  float* y;                // [T][H]
  // workspace
  int32_t* n_units;
  int4* units;             // [P + 1] slot (-1: the shared expert), first entry, entries, 0
  int16_t* entries;        // [P + T] pair numbers, P + t for the shared expert
  uint16_t* h;             // [P + T][I / 8][4][8] h as three BF16 parts (the fourth unused)
  int P;                   // set by the launcher
  float* part;             // [q4_down_parts][T][H], where there are any
};
// Workgroups that share rows of y in the down product of more pairs than one wave
// lists (kQ4WavePairs): 32 rows for each, one workgroup per compute unit, at most 8
// sharing.  More than two of them leave partial sums, added in order by one more
// launch (two add into a cleared y: that has one order).
constexpr int kQ4WavePairs = 64;
inline int q4_down_split(int H) {
  const int s = 256 / (H / 32);
  return s < 1 ? 1 : s > 8 ? 8 : s;
}
inline int q4_down_parts(int pairs, int H) {
  return pairs > kQ4WavePairs && q4_down_split(H) > 2 ? q4_down_split(H) : 0;
}
hipError_t launch_q4_experts(Q4Experts a, int group, hipStream_t st);

// per-workgroup phase stamps at the end of the decode workspace
constexpr size_t kDecodeStampBytes = 1024 * 16 * 8;
// copies of the decode logits (each read by every kZCopies-th workgroup)
constexpr int kZCopies = 64;
// bytes of one copy: [T][E] uint64, rounded to 4 KB, plus 256 B so that the
// copies start at different offsets within a page
inline size_t decode_z_copy_bytes(int T, int E) {
  return (((size_t)T * E * 8 + 4095) & ~(size_t)4095) + 256;
}

// decode: router (optional) + experts + combine in one kernel, at most
// decode_max_tokens(H) tokens per launch
bool decode_shape_supported(int wtype, int H, int I);
int decode_max_tokens(int wtype, int H, int I);
hipError_t launch_decode(const DecodeLaunch& f, hipStream_t st);

// prefill
constexpr int kPrefillChunk = 256;   // pairs per sort chunk
constexpr int kPrefillMT = 128;      // rows per M tile
int prefill_max_tiles(int T, int k, int E);
hipError_t launch_prefill(const PrefillLaunch& p, hipStream_t st);

// formats / merge
hipError_t launch_quantize_mxfp4(const void* src, int src_bf16, int rows, int K, int64_t ld,
                                 uint8_t* codes, uint8_t* scales, hipStream_t st);
// NVFP4: codes [rows][K/2], E4M3 scales [rows][K/16], fp32 matrix scale at g
hipError_t launch_quantize_nvfp4(const void* src, int src_bf16, int rows, int K, uint8_t* codes,
                                 uint8_t* scales, float* g, hipStream_t st);
hipError_t launch_pack_bf16(const void* src, int src_bf16, int rows, int K, uint16_t* dst,
                            hipStream_t st);
hipError_t launch_dequant_mxfp4(const uint8_t* codes, const uint8_t* scales,
                                int64_t n_blocks, float* out, hipStream_t st);
// test hook: per (block, x vector) the decode gate/up block step (MXFP4 or NVFP4)
hipError_t launch_dot_fp4(const uint8_t* codes, const uint8_t* scales, const uint16_t* x,
                          int64_t n_blocks, int n_x, int nvfp4, float* out, hipStream_t st);
// decode header word 32 (a wait expired) to out, optionally cleared
hipError_t launch_decode_status(unsigned* hdr, int32_t* out, int clear, hipStream_t st);
hipError_t launch_merge(const float* a, const float* b, float* y, size_t n,
                        hipStream_t st);
hipError_t launch_mfma_fp4_tile(const uint8_t* a_codes, const uint8_t* a_scales,
                                const uint8_t* b_codes, const uint8_t* b_scales,
                                float* out, hipStream_t st);

hipError_t launch_wave_scan(const int32_t* in, int32_t* out, int n_waves, hipStream_t st);
hipError_t launch_read_probe(const void* src, size_t bytes, int blocks, uint32_t* out,
                             hipStream_t st);

// cache
hipError_t launch_fill_i32(int32_t* dst, int32_t value, int64_t n, hipStream_t st);

}  // namespace moe
