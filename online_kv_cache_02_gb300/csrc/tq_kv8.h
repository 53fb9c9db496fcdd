// Shared by the translation units of the 8-bit paged KV cache (tq_kv8*.cu).
#ifndef TQ_KV8_H_
#define TQ_KV8_H_

#include "tq_internal.h"

#include <cuda.h>

namespace tq {

constexpr int kE8Min = -100, kE8Max = 119;   // exponents of a block's scale
constexpr uint32_t kErrNonFinite = 32u;      // a rotated input was not finite in fp32
constexpr uint32_t kErrScale = 64u;          // a block's stored scale was no power of two in range

struct Kv8Append {
  const void *k, *v, *q;          // [batch][n_new] tokens, `*_stride` elements apart (null: skipped)
  void* q_out;                    // [batch][n_new][Hq][d]
  int batch, n_new, Hq, H;
  long long k_stride, v_stride, q_stride;
  const int32_t *start_pos, *new_lens;
  uint8_t *kc, *vc;               // [num_pages][H][16][d]
  float *ks, *vs;                 // [num_pages][H]
  const int32_t* bt;
  int maxp, num_pages;
  const float* cs;                // [max_pos][rot]: cosines, then sines (null: no rotation)
  int max_pos, rot, interleaved, axes;
  int sec_end[4];                 // one past each axis' last pair
  const int32_t* pos;             // [axes][batch][n_new] or null
  uint32_t* err;
};

// Attention of T query tokens per sequence.  Query row r = t G + g of a KV
// head; rows are taken in blocks.
struct Kv8Attn {
  const void* q;                  // [B][T][Hq][d]
  void* out;
  int B, T, Hq, H, G;
  const int32_t* lens;            // decode: tokens with the query's own; else the first query's position
  const int32_t* new_lens;        // null: T each
  int decode;
  int max_seq_len;
  const int32_t* bt;
  int maxp, num_pages;
  const uint8_t *kc, *vc;
  const float *ks, *vs;
  int window, sinks;
  float scale_log2;
  float* part;                    // split items: [slot][rows][2 + d]
  uint32_t* err;
};

// A sequence's queries, cut to what its table and max_seq_len hold.
struct Kv8Seq {
  int p0, n;                      // first query's position, queries
};
__device__ __forceinline__ Kv8Seq kv8_seq(const Kv8Attn& a, int b) {
  const int L = a.lens[b];
  long long first = a.decode ? static_cast<long long>(L) - 1 : L;
  int n = a.decode ? (L > 0 ? 1 : 0) : (a.new_lens ? a.new_lens[b] : a.T);
  bool bad = a.decode ? L < 0 : L < 0 || n < 0 || n > a.T;
  n = n < 0 ? 0 : n > a.T ? a.T : n;
  const long long cap = a.max_seq_len < 16LL * a.maxp ? a.max_seq_len : 16LL * a.maxp;
  if (first + n > cap) {
    bad = true;
    if (a.decode) first = cap - 1;
    else n = first >= cap ? 0 : static_cast<int>(cap - first);
    if (first < 0) n = 0;
  }
  if (first < 0) n = 0;
  if (bad) atomicOr(a.err, kErrSeqLen);
  return Kv8Seq{n > 0 ? static_cast<int>(first) : 0, n};
}

// Pages that the queries at positions pmin .. pmax see: pages [0, ns) and [w0, w0 + nw).
struct Kv8Range {
  int ns, w0, nw;
};
__device__ __forceinline__ Kv8Range kv8_range(int window, int sinks, int pmin, int pmax) {
  const int end = pmax / kPage + 1;
  if (!window || window > pmin) return Kv8Range{0, 0, end};
  int ns = static_cast<int>((static_cast<long long>(sinks) + kPage - 1) / kPage);
  const int w0 = (pmin - window + 1) / kPage;
  if (ns >= w0) return Kv8Range{0, 0, end};
  return Kv8Range{ns, w0, end - w0};
}

bool kv8_head_dim(int d);
int kv8_sm_count();                      // of the current device
cudaError_t launch_kv8_append(const Kv8Append& a, int d, bool f32, cudaStream_t s);
size_t kv8_rows_workspace(int T, int G, int d);
cudaError_t launch_kv8_rows(const Kv8Attn& a, int d, bool f32, cudaStream_t s);
// TMA map of a cache's blocks: coordinates (channel, token, block), boxes of one block's 128-channel panel.
bool kv8_block_map(CUtensorMap* map, const void* codes, long long blocks, int d);
// Many query rows on the tensor cores (tq_kv8_tc.cu): whether the call takes
// that form (it has more than kTcRows query rows per KV head, among others),
// whether it then uses a workspace, its size and its launch.
constexpr int kTcRows = 16;
bool kv8_tc_takes(int T, int G, int d, bool f32, float softmax_scale);
bool kv8_tc_splits(int B, int T, int G, int max_seq_len, int d);
size_t kv8_tc_workspace(int B, int T, int G, int H, int max_seq_len, int d);
cudaError_t launch_kv8_tc(const Kv8Attn& a, int d, cudaStream_t s);

}  // namespace tq

#endif  // TQ_KV8_H_
