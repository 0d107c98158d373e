// Pages of a paged cache: the pool's layout and the launchers of its calls, shared
// by the kernels (pages.cu) and the entry points (gen_abi.cu).
#pragma once

#include "paged.cuh"

namespace futr {

constexpr uint64_t kPagesMagic = 0x3147504752545546ull;
constexpr int kPagesMaxSeqs = 1024;

// The pool's device memory.
struct PoolView {
  int* refs;            // [n_pages] places that name a page
  unsigned* free;       // [words] bit p % 32 of word p / 32: page p is free
  int* plan;            // what a call decided: see below
  int* err;             // error word; word 2: the number of free pages; word 3: no word of `free` before it has one
  int n_pages, words;
};

// The plan: a header, then lists of n_pages each and one row of four per sequence.
//   header [0] copies, [1] 1: the call goes ahead; [kPlanBad] 1: but the table names a page that
//   is not held, [kPlanMet] CTAs that have read this (both 0 between calls)
//   from, to [n_pages]   pages to copy (to: also the pages that a call takes)
//   slots [n_pages]      slots of a page that are copied; compact: where page p goes
//   seqs [max_seqs][4]   fork: parent's row or -1, its position (0), fresh page for the place of
//                        that position or -1, 1: keeps the parent's places from there on
constexpr int kPlanHeader = 64, kPlanBad = 32, kPlanMet = 33;
inline size_t plan_ints(int n_pages, int max_seqs) {
  // (the sequences' rows are aligned to 16 bytes)
  return kPlanHeader + ((3 * (size_t)n_pages + 3) & ~size_t(3)) + 4 * (size_t)max_seqs; }

struct PagesArgs {
  PoolView p;
  PagedView c;              // layer 0
  int n_layers, d;
  uint64_t layer_codes, layer_scales;   // bytes, floats from a layer to the next
  int batch, table_ld;
  int* table;
  const int* start;         // grow
  const int* parent;        // fork
  int* pos;                 // grow and free only read it
  int window, sinks;        // free
  int lo, hi;               // compact
};

cudaError_t launch_pages_init(const PoolView& p, cudaStream_t st);
cudaError_t launch_pages_hold(const PagesArgs& a, cudaStream_t st);
cudaError_t launch_pages_grow(const PagesArgs& a, cudaStream_t st);
cudaError_t launch_pages_free(const PagesArgs& a, cudaStream_t st);
cudaError_t launch_pages_fork(const PagesArgs& a, int sms, cudaStream_t st);
cudaError_t launch_pages_compact(const PagesArgs& a, int sms, cudaStream_t st);

cudaError_t launch_kv_reorder(const futr_kv& kv, int batch, const int* parent, int* pos, int* err, int sms,
                              cudaStream_t st);

}  // namespace futr
