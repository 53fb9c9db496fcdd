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

// Decode of sequences that share a prefix (tq_kv8_shared_decode_attention): groups of sequences one behind the other,
// whose first pages are the same.  The prefix pass (`tail` 0) takes a group as one sequence of many queries that all see
// the whole prefix, the tail pass (1) each sequence's pages behind it; both leave their sums, which a last kernel joins.
struct Kv8SharedSeq {             // what a pass sees of group (or sequence) b
  int row, n, pages0, pages;      // first query row (of batch) and table, queries, pages [pages0, pages0 + pages)
  int p;                          // the queries' position
};
struct Kv8Share {
  int tail, batch, groups, max_group;
  const int32_t *group_start, *prefix_lens;
  int4* seqs;                     // per sequence, from the prefix pass: prefix pages (0: no prefix), group, the group's first sequence
  int2* items;                    // the pass' items, by block of rows and KV head: the CTAs that hold it (-1: whole, in `state`)
  float* state;                   // per query row: [items per head][maximum, sum, its exponent, 0, channels]
};
// The group of sequence b by bisection of the starts.
__device__ __forceinline__ int kv8_group_of(const Kv8Share& s, int b) {
  int lo = 0, hi = s.groups - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (s.group_start[mid] <= b) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}
// Where starts fall, a sequence can be in two groups.  Bisection leads each sequence to one of them, and never a later sequence
// to an earlier group, whatever the starts are: a group that it finds from its first and from its last sequence it finds from
// all of them, and such groups have no sequence in common.  The others share nothing.  Whether it finds group g from all of
// r0 .. r1 - 1: the places that it looks at follow from g.
__device__ __forceinline__ bool kv8_group_found(const Kv8Share& s, int g, int r0, int r1) {
  bool found = true;
  int lo = 0, hi = s.groups - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2, start = s.group_start[mid];
    found &= mid <= g ? start <= r0 : start >= r1;
    if (mid <= g) lo = mid;
    else hi = mid - 1;
  }
  return found;
}
__device__ __forceinline__ Kv8SharedSeq kv8_group(const Kv8Attn& a, const Kv8Share& s, int g) {
  const int r0 = s.group_start[g], r1 = s.group_start[g + 1], len = s.prefix_lens[g];
  const bool list = r0 >= 0 && r1 >= r0 && r1 <= s.batch && r1 - r0 <= s.max_group &&
                    (r1 == r0 || kv8_group_found(s, g, r0, r1));
  const int cap = min(a.maxp, a.max_seq_len / kPage), pages = len < 0 ? 0 : len / kPage;
  if (!list || len < 0 || pages > cap) atomicOr(a.err, kErrSeqLen);
  if (!list) return Kv8SharedSeq{0, 0, 0, 0, -1};
  const int taken = min(pages, cap);
  return Kv8SharedSeq{r0, taken ? r1 - r0 : 0, 0, taken, kPage * taken - 1};
}
// Sequence b as in Kv8Share::seqs.
__device__ __forceinline__ int4 kv8_share_seq(const Kv8Attn& a, const Kv8Share& s, int b) {
  const int lo = kv8_group_of(s, b);
  const Kv8SharedSeq g = kv8_group(a, s, lo);
  const bool in = g.n > 0 && b >= g.row && b - g.row < g.n;
  if (!in && !(b >= s.group_start[lo] && b < s.group_start[lo + 1])) atomicOr(a.err, kErrSeqLen);   // in no group
  return in ? make_int4(g.pages, lo, g.row, 0) : make_int4(0, 0, 0, 0);
}
// What the join needs of each sequence, by all threads of the prefix pass.
__device__ __forceinline__ void kv8_share_seqs(const Kv8Attn& a, const Kv8Share& s) {
  for (long long b = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; b < s.batch; b += static_cast<long long>(gridDim.x) * blockDim.x)
    s.seqs[b] = kv8_share_seq(a, s, static_cast<int>(b));
}
// The pages of sequence b behind the first ones.
__device__ __forceinline__ Kv8SharedSeq kv8_tail(const Kv8Attn& a, int b, int first) {
  int len = a.lens[b];
  const long long cap = a.max_seq_len < 16LL * a.maxp ? a.max_seq_len : 16LL * a.maxp;
  if (len < 0 || len > cap || (len > 0 && len < kPage * first)) {
    atomicOr(a.err, kErrSeqLen);
    if (len > cap) len = static_cast<int>(cap);
  }
  const int pages = len <= kPage * first ? 0 : (len + kPage - 1) / kPage - first;
  return Kv8SharedSeq{b, pages ? 1 : 0, first, pages, len - 1};
}

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
// Many query rows on the tensor cores (tq_kv8_tc.cuh): whether the call takes
// that form (it has more than kTcRows query rows per KV head, among others),
// whether it then uses a workspace, its size and its launch.
constexpr int kTcRows = 16;
bool kv8_tc_takes(int T, int G, int d, bool f32, float softmax_scale);
bool kv8_tc_splits(int B, int T, int G, int max_seq_len, int d);
size_t kv8_tc_workspace(int B, int T, int G, int H, int max_seq_len, int d);
cudaError_t launch_kv8_tc(const Kv8Attn& a, int d, cudaStream_t s);

// Decode with shared prefixes (tq_kv8_shared.cu).
size_t kv8_shared_workspace(int batch, int Hq, int H, int groups, int max_group, int max_seq_len, int d);
cudaError_t launch_kv8_shared(Kv8Attn a, Kv8Share share, int d, bool f32, float softmax_scale, void* workspace, cudaStream_t s);
// The passes: with `share` the launches below leave sums in share.state.
cudaError_t launch_kv8_rows_shared(const Kv8Attn& a, const Kv8Share& share, int d, bool f32, cudaStream_t s);
cudaError_t launch_kv8_tc_shared(const Kv8Attn& a, const Kv8Share& share, int d, cudaStream_t s);
struct Kv8TcShape {               // of a tcgen05 call: its items per KV head, rows and channels an item, CTAs and blocks
  int per, rows, dv, ctas, nqb;
  size_t records;                 // bytes ahead of the parts
  float lift;                     // of its weights' exponents
};
Kv8TcShape kv8_rows_shape(int T, int G, int d);    // the same of the other form
Kv8TcShape kv8_tc_shape(int B, int T, int G, int H, int max_seq_len, int d);

}  // namespace tq

#endif  // TQ_KV8_H_
