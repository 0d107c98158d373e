// The INT4 mixture-of-experts layer: layouts and launchers shared by the
// kernels (moe.cu) and the entry points (moe_abi.cu).
//
// Blob: a 256-byte header, then for each expert its gate/up section (row blocks
// of 64 gate and 64 up rows) and its down section, in the same 8448-byte units
// of 128 rows x 128 inputs as a block's blob, the eight nibbles u = code + 8 of a
// word placed for f16 operands.  Each 16-bit half of a word holds
//   bits 6-9: u of slot 0    bits 2-5: slot 1    bits 10-13: slot 3
//   bits 14, 15, 0, 1: slot 2, low bit first
// (slots as in the block's units: half 0 holds slots 0..3, half 1 slots 4..7, a
// register pairs slots i and i + 4).  Masked, and with the bytes of each half
// swapped masked again, all of them land in an f16's mantissa without a shift:
// a word takes one byte permutation and four logic operations.  Or-ed with 1.0,
// slots 0 and 2 (rows g of the A fragment) read 1 + u / 16 and slots 1 and 3
// (rows g + 8) 1 + u / 256, one f16 addition away from code/16 and code/256.
//
// Activations are f16 rows, cut into records of 128 inputs (a unit's) and 16
// bytes (which also keep the rows of a tile on different banks).
#pragma once

#include "futr_internal.cuh"
#include "proj.cuh"

namespace futr {

constexpr uint64_t kMoeMagic = 0x3245304d52545546ull;
constexpr uint64_t kMoeWsMagic = 0x5745304d52545546ull;
constexpr int kMoeMaxExperts = 256;
constexpr int kMoeMaxTopK = 16;
constexpr int kMoeMaxPairs = kMaxBatch * kMoeMaxTopK;

// One record of an activation row: 128 f16 values, then room for four floats.  Down
// inputs: each half (inputs 0..63 and 64..127) is divided by the power of two at its
// largest value; the first two floats are these factors.  Gate/up inputs have one a
// token (MoeArgs::rms).
constexpr int kRecHalves = 136;
constexpr int kRecBytes = 2 * kRecHalves;

struct MoeHeader {
  uint64_t magic;
  int32_t version, hidden, inter, n_experts;
};

inline uint64_t moe_gu_bytes(const futr_moe_shape& s) {
  return (uint64_t)(2 * s.inter / kRowsPerBlock) * (s.hidden / kGroup) * kUnitBytes;
}
inline uint64_t moe_down_bytes(const futr_moe_shape& s) {
  return (uint64_t)(s.hidden / kRowsPerBlock) * (s.inter / kGroup) * kUnitBytes;
}

struct MoeArgs {
  int H, I, E, K, T, renorm;
  bool withhold;                       // tests of the failure path: gate/up's CTA 0 issues no copy
  float eps;                           // 0: no normalization
  const __nv_bfloat16* x;              // [T][H]
  const float* gain;                   // [H] or nullptr
  const __nv_bfloat16* router;         // [E][H]
  const uint8_t* blob;
  uint64_t gu_bytes, expert_bytes;
  const __nv_bfloat16* resid;          // [T][H] or nullptr
  __nv_bfloat16* y;                    // [T][H]
  int* ids;                            // [T][K] or nullptr
  float* weights;                      // [T][K] or nullptr
  int* err;
  float* logits;                       // [T][E]
  float* rms;                          // [T] RMSNorm factor times the factor of the token's f16 records
  __half* xh;                          // [T][H / 128][136]: the tokens as f16 records
  __half* act;                         // [I / 128][pairs][136]: the down product's inputs, pairs by expert
  float* rec;                          // split records, two per CTA
  int* choice;                         // [T][K] the router's choices
  float* share;                        // [T][K] and their weights
  int* active;                         // runs of pairs that down streamed (for the sums)
  int down_ctas;                       // the grid of down
  unsigned* cnt;                       // arrival counters: kRouterTiles of the router, then one per CTA
};

constexpr int kRouterT = 8;                                 // tokens of a router CTA
constexpr int kRouterTiles = kMaxBatch / kRouterT;
constexpr int kMoeRecFloats = kMaxBatch * kRowsPerBlock;   // one record: up to 32 columns of 128 rows

int moe_ctas();   // most CTAs any launch uses on the current device
cudaError_t launch_moe(const MoeArgs& a, cudaStream_t st);
// Between a block's nibble order and this one, in place.
cudaError_t launch_moe_place(uint8_t* units, size_t n_units, cudaStream_t st);
cudaError_t launch_moe_unpack(int hidden, int inter, const uint8_t* gu, const uint8_t* down, int which, int8_t* codes,
                              uint16_t* scales, cudaStream_t st);

}  // namespace futr
