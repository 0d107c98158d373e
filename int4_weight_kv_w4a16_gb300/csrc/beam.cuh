// Choice of beams' continuations: workspace layout and launcher, shared by the
// kernels (beam.cu) and the entry points (gen_abi.cu).
#pragma once

#include "futr_internal.cuh"

namespace futr {

constexpr uint64_t kBeamWsMagic = 0x3142575452545546ull;
constexpr int kBeamMaxBeams = 32, kBeamMaxKeep = 64, kBeamMaxRows = 65536;

struct BeamArgs {
  const void* logits;
  long long ld;
  const float* scores;       // [batch][beams]
  const int* done;           // [batch][beams] or nullptr
  int batch, beams, vocab, end, keep, stay;
  float* score_out;
  int *parent, *token, *done_out;
  int* err;                  // the workspace's error words
  uint8_t* rows;             // [rows] row records
  uint8_t* parts;            // [rows][splits] part records
  unsigned* cnt;             // arrival counters: [batch] prompts, [rows] rows
  int splits;                // parts of a row
  uint32_t by_keep, by_beam; // for quotients by keep and by keep * splits
  int by_row;                // a row's parts are made one before the prompt's beams meet
};

// A record of a part or a row: maximum and sum (in two parts), 16 bytes; then `keep` keys.
// (A multiple of 16: the statistics are one access.)
__host__ __device__ inline size_t beam_record(int keep) { return 16 + 16 * (((size_t)keep + 1) / 2); }

int beam_part_ctas(int sms);   // parts of all rows together, where there are fewer rows than that
cudaError_t launch_beam_select(const BeamArgs& a, int dtype, int sms, cudaStream_t st);

}  // namespace futr
