// Reading the caches back into rows (tq_dequantize, tq_kv8_dequantize): arguments shared by their kernels.
#ifndef TQ_READ_H_
#define TQ_READ_H_

#include "tq_kv8.h"

namespace tq {

struct ReadArgs {
  int batch, H, max_len, total_rows;
  const int32_t *start_pos, *lens, *first_row;
  const int32_t* bt;
  int maxp, num_pages;
  int pages;                              // pages of a sequence's run at most
  const uint8_t *kc, *vc;                 // null: not read
  long long k_page_bytes, v_page_bytes;   // 2-4-bit cache
  const float *ks, *vs;                   // 8-bit cache
  void *k_out, *v_out;                    // rows `k_stride`, `v_stride` elements apart
  long long k_stride, v_stride;
  int m;
  KindLayout kl, vl;
  DeviceTables tab;
};

// The run of sequence b: n tokens from position `start` on, to rows `row` and on.  What lies outside the block table, the
// rows or max_len is cut off and flagged.
struct ReadRun {
  int start, n, row;
};
__device__ __forceinline__ ReadRun read_run(const ReadArgs& a, int b) {
  const int start = a.start_pos[b], row = a.first_row[b];
  int n = a.lens[b];
  uint32_t bad = 0;
  if (n < 0 || n > a.max_len || start < 0 || row < 0) {
    bad |= kErrSeqLen;
    n = n < 0 || start < 0 || row < 0 ? 0 : a.max_len;
  }
  const long long room = static_cast<long long>(kPage) * a.maxp - start;
  if (n > 0 && n > room) {                            // (nothing is read of a start beyond the table with a length of 0)
    bad |= kErrBlock;
    n = room > 0 ? static_cast<int>(room) : 0;
  }
  if (n > 0 && n > a.total_rows - row) {
    bad |= kErrSeqLen;
    n = a.total_rows > row ? a.total_rows - row : 0;
  }
  if (bad) atomicOr(a.tab.err, bad);
  return ReadRun{start, n, row};
}
// Page i of the run: its id (-1: none, flagged) and the run's slots [s0, s1) of it; slot s holds token s - off.
struct ReadPage {
  int id, s0, s1, off;
};
__device__ __forceinline__ ReadPage read_page(const ReadArgs& a, int b, const ReadRun& r, int i) {
  ReadPage x{-1, 0, 0, 0};
  if (r.n <= 0 || i > (r.start + r.n - 1) / kPage - r.start / kPage) return x;
  const int page = r.start / kPage + i;
  x.off = r.start - page * kPage;
  x.s0 = max(0, x.off);
  x.s1 = min(kPage, x.off + r.n);
  const int id = a.bt[static_cast<long long>(b) * a.maxp + page];
  if (id < 0 || id >= a.num_pages) atomicOr(a.tab.err, kErrPage);
  else x.id = id;
  return x;
}

cudaError_t launch_read(const ReadArgs& a, int d, bool f32, cudaStream_t s);
bool read_tc_takes(const ReadArgs& a, int d);
cudaError_t launch_read_tc(const ReadArgs& a, bool f32, cudaStream_t s);
cudaError_t launch_kv8_read(const ReadArgs& a, int d, bool f32, cudaStream_t s);

}  // namespace tq

#endif  // TQ_READ_H_
