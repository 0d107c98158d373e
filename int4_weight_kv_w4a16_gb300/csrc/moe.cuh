// The INT4 mixture-of-experts layer: layouts and launchers shared by the
// kernels (moe.cu) and the entry points (moe_abi.cu).
//
// Blob: a 256-byte header, then for each expert its gate/up section (row blocks
// of 64 gate and 64 up rows) and its down section, in the same 8448-byte units
// of 128 rows x 128 inputs as a block's blob.
#pragma once

#include "futr_internal.cuh"
#include "proj.cuh"

namespace futr {

constexpr uint64_t kMoeMagic = 0x3145304d52545546ull;
constexpr uint64_t kMoeWsMagic = 0x5745304d52545546ull;
constexpr int kMoeMaxExperts = 256;
constexpr int kMoeMaxTopK = 16;
constexpr int kMoeMaxPairs = kMaxBatch * kMoeMaxTopK;

struct MoeHeader {
  uint64_t magic;
  int32_t version, hidden, inter, n_experts;
};

// What the router leaves for the expert kernels.  A pair is one (token, chosen
// expert); pairs are ordered by expert, then token.
struct MoeRoute {
  int n_active;                        // experts that some token chose
  int expert[kMoeMaxExperts];          // their ids, ascending
  int off[kMoeMaxExperts + 1];         // first pair of each
  int token[kMoeMaxPairs];             // token of each pair
  float weight[kMoeMaxPairs];          // its weight
  float rms[kMaxBatch];                // RMSNorm factor of each token
};

inline uint64_t moe_gu_bytes(const futr_moe_shape& s) {
  return (uint64_t)(2 * s.inter / kRowsPerBlock) * (s.hidden / kGroup) * kUnitBytes;
}
inline uint64_t moe_down_bytes(const futr_moe_shape& s) {
  return (uint64_t)(s.hidden / kRowsPerBlock) * (s.inter / kGroup) * kUnitBytes;
}

struct MoeArgs {
  int H, I, E, K, T, renorm;
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
  MoeRoute* route;
  __nv_bfloat16* act;                  // [pairs][I]
  float* rec;                          // split records, two per CTA
  unsigned* cnt;                       // one counter per CTA, then the router's
  int n_cnt;
};

constexpr int kMoeRecFloats = kMaxBatch * kRowsPerBlock;   // one record: up to 32 columns of 128 rows

int moe_ctas();   // most CTAs any launch uses on the current device
cudaError_t launch_moe(const MoeArgs& a, cudaStream_t st);

}  // namespace futr
