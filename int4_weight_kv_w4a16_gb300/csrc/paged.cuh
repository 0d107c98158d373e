// The paged 8-bit key/value cache: layout, device view and launchers shared by
// the append kernel (paged.cu) and the attention kernels (paged_attn.cu).
//
// A page holds `page` consecutive positions of one sequence, for every kv-head
//   codes  [layer][page id][kv-head][K, V][slot][d]   e4m3, one byte each
//   scales [layer][page id][kv-head][K, V]            fp32, powers of two where the append wrote them
// value = code * scale.  Powers of two make the scale exact in every use: codes
// are x / s rounded once, a page whose scale grows by 2^n keeps its codes
// exactly (except those that reach e4m3's subnormals, which lose their low
// bits once), so the error of an old token does not build up however often the
// page grows.
#pragma once

#include <cuda.h>

#include "futr_internal.cuh"

namespace futr {

constexpr uint64_t kPagedMagic = 0x3850564b52545546ull;
constexpr uint64_t kPagedWsMagic = 0x3857534b52545546ull;
constexpr int kPagedMinExp = -60;       // smallest page scale 2^-60
constexpr int kPagedMaxPos = 1 << 20;   // positions of the RoPE table

struct PagedView {
  uint8_t* codes;         // layer's first page
  float* scales;          // layer's first page
  const float2* rope;     // [max_pos][d/2] (cos, sin); nullptr: positions are in the rows already
  int n_pages, page, page_log2, n_kv, max_pos;
};

struct PagedRows {          // ragged rows of a call
  const int* pos;           // [batch] tokens cached before the call
  const int* start;         // [batch + 1] first row of each sequence; nullptr: row b is sequence b's only one
  const int* table;         // [batch][table_ld] page ids
  int batch, n_rows, table_ld;
};

// Rows and first position of sequence b; false (and n = 0) when they do not
// fit the call's rows, the table or the positions.
__device__ __forceinline__ bool paged_seq(const PagedRows& r, const PagedView& c, int b, int& row0, int& n, int& p0) {
  row0 = r.start ? r.start[b] : b;
  const int row1 = r.start ? r.start[b + 1] : b + 1;
  p0 = r.pos[b];
  n = row1 - row0;
  if (n == 0) return true;
  const long long cap = (long long)r.table_ld << c.page_log2, end = (long long)p0 + n;
  const bool ok = row0 >= 0 && n > 0 && row1 <= r.n_rows && p0 >= 0 && end <= c.max_pos && end <= cap;
  if (!ok) n = 0;
  return ok;
}

cudaError_t launch_paged_append(const PagedView& c, const PagedRows& r, int d, int dtype, const void* k, long long ld_k,
                                const void* v, long long ld_v, int* err, cudaStream_t st);

struct PagedAttnArgs {
  PagedView c;
  PagedRows r;
  const void* q;
  void* out;
  long long ld_q, ld_out;
  int Hkv, G, window;
  int sinks, sink_tiles, sink_pages;   // first positions that every row sees; tiles and pages that hold them
  int rows_lo, rows_hi;     // sequences of [rows_lo, rows_hi) rows x G are this launch's
  long long block0;         // (layer's first page) * Hkv: outermost coordinate of the tensor map
  float scale_log2;         // softmax scale * log2(e)
  float* rec;               // split records
  unsigned* cnt;            // arrival counters, one per CTA
  int* err;                 // the cache's error word: rows and pages out of range
  int* stop;                // the workspace's error and abort words: a wait ran out
  bool withhold;            // tests of the failure path: the last share's copies are not issued
};

int paged_attn_sms();                        // of the current device
int paged_attn_ctas(int sms);                // most CTAs any launch uses
size_t paged_rec_floats(int d, int sms);     // floats of all their records
size_t paged_tc_rec_floats(int d);           // of one CTA of the many-row kernel
cudaError_t launch_paged_attention_tc(const PagedAttnArgs& a, const CUtensorMap& map, int d, int dtype, int ctas,
                                      cudaStream_t st);
cudaError_t launch_paged_attention(const PagedAttnArgs& a, const CUtensorMap& map, int d, int dtype, cudaStream_t st);
bool make_paged_map(CUtensorMap* m, const void* codes, int d, int page, uint64_t blocks);

}  // namespace futr
