// Attention over packed prompts (tq_prompt_attention): arguments, the sequences' blocks of query rows and the tiles of
// keys that they see, shared by the tensor-core forms (tq_prompt_tc.cu for bf16, tq_prompt_parts.cu to fp32's accuracy) and
// the CUDA-core form (tq_prompt.cu).
#ifndef TQ_PROMPT_H_
#define TQ_PROMPT_H_

#include "tq_internal.h"
#include "tq_prompt_list.h"

namespace tq {

struct PromptArgs {
  const void *q, *k, *v;                  // tokens `*s` elements apart, [heads][d] each
  void* out;                              // [total_q][Hq][d], dense
  long long qs, ks, vs;
  int S, total_q, total_k, Hq, H, G;
  const int32_t *cu_q, *cu_k;             // [S + 1]
  int max_q, max_k;
  int rows;                               // query rows of a block
  int most;                               // blocks that the list takes
  int window, sinks;
  float scale_log2;
  float* part;                            // split items: PSplit per CTA, then [slot][rows][d + 4]
  uint32_t* err;
};

// Sequence s: its first rows of q and k, its queries and keys; none where the lists are no offsets.
struct PromptSeq {
  int q0, k0, n, m;
};
__device__ __forceinline__ PromptSeq prompt_seq(const PromptArgs& a, int s) {
  const int q0 = a.cu_q[s], q1 = a.cu_q[s + 1], k0 = a.cu_k[s], k1 = a.cu_k[s + 1];
  if (!prompt_pair(q0, q1, a.total_q, a.max_q) || !prompt_pair(k0, k1, a.total_k, a.max_k)) {
    atomicOr(a.err, kErrSeqLen);
    return PromptSeq{0, 0, 0, 0};
  }
  return PromptSeq{q0, k0, q1 - q0, k1 - k0};
}

// A block of `rows` query rows r = t G + g from r0 on, of one sequence (and any KV head): the positions of its first and
// last row, and the tiles of TOK keys that it sees: ns from the sequence's start on (the first tokens of a window), then
// nw from key w0 on.
struct PromptBlock {
  PromptSeq seq;
  int r0, rows, pmin, pmax;
  int ns, w0, nw;
  __device__ __forceinline__ int tiles() const { return ns + nw; }
  template <int TOK>
  __device__ __forceinline__ int first_key(int tile) const { return tile < ns ? TOK * tile : w0 + TOK * (tile - ns); }
};
__device__ __forceinline__ int prompt_blocks(const PromptArgs& a, const PromptSeq& s) { return prompt_blocks(s.n, a.G, a.rows); }
template <int TOK>
__device__ __forceinline__ PromptBlock prompt_block(const PromptArgs& a, const PromptSeq& s, int qb) {
  PromptBlock b;
  b.seq = s;
  b.r0 = qb * a.rows;                     // the host keeps total_q Hq below 2^31
  b.rows = min(s.n * a.G - b.r0, a.rows);
  b.pmin = s.m - s.n + b.r0 / a.G;
  b.pmax = s.m - s.n + (b.r0 + b.rows - 1) / a.G;
  b.ns = b.w0 = 0;
  b.nw = b.pmax < 0 ? 0 : b.pmax / TOK + 1;
  if (a.window && a.window <= b.pmin) {
    const int ns = (a.sinks + TOK - 1) / TOK, w0 = b.pmin - a.window + 1;
    if (static_cast<long long>(ns) * TOK < w0) {
      b.ns = ns;
      b.w0 = w0;
      b.nw = (b.pmax - w0) / TOK + 1;
    }
  }
  return b;
}
// Whether the query at position p sees key j.
__device__ __forceinline__ bool prompt_sees(int p, int j, int window, int sinks) {
  return j <= p && (!window || j > p - window || j < sinks);
}

// Those of the 32 keys from j0 on that the query at position p sees.
__device__ __forceinline__ uint32_t prompt_seen32(int p, int j0, int window, int sinks) {
  const int hi = p - j0;                               // up to hi
  uint32_t see = hi < 0 ? 0u : hi >= 31 ? 0xFFFFFFFFu : (2u << hi) - 1u;
  if (window) {
    const int lo = hi - window + 1, sk = sinks - j0;   // from lo on, or below sk
    const uint32_t win = lo <= 0 ? 0xFFFFFFFFu : lo > 31 ? 0u : 0xFFFFFFFFu << lo;
    const uint32_t snk = sk <= 0 ? 0u : sk > 31 ? 0xFFFFFFFFu : (1u << sk) - 1u;
    see &= win | snk;
  }
  return see;
}

// An item (a block and a KV head) that several CTAs share: its first part ends the span of one CTA, the join finds the
// others by it.
struct PSplit {
  int valid, q0, r0, rows, h, last, p0, pad;    // last: the CTA that holds the item's end; p0: position of r = 0
};
// A row's 1 / l.  l = 0 where the row sees nothing (zeros), or where every score is -inf (NaN, as is 0 / 0).
__device__ __forceinline__ float prompt_inverse(float l, int p) {
  return l > 0.0f ? 1.0f / l : l == 0.0f && p < 0 ? 0.0f : __int_as_float(0x7FC00000);
}

// The CTA's place in the list of all items' tiles, cut into spans of equal cost: an item takes COST units, then one per
// tile; the blocks stand sequence by sequence, each for all its `heads`.
struct PromptSpan {
  long long u0, u1, span;                 // this CTA's units; every CTA's length
  int s, qb;                              // the block that holds u0
  long long at;                           // units before it
};
// By all THREADS of a block; `room`: kPromptList * 2 + 64 ints of shared memory.
template <int TOK, int COST, int THREADS>
__device__ PromptSpan prompt_span(const PromptArgs& a, int heads, int min_span, int* room) {
  constexpr int WARPS = THREADS / 32;
  int *firsts = room, *units = room + kPromptList, *sums = units + kPromptList;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto scan = [&](int sum, int& total) {  // sum of the threads before
    int run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, run, o);
      run += lane >= o ? v : 0;
    }
    if (lane == 31) sums[warp] = run;
    __syncthreads();
    int before = run - sum;
    total = 0;
    for (int w = 0; w < WARPS; ++w) {
      before += w < warp ? sums[w] : 0;
      total += sums[w];
    }
    __syncthreads();
    return before;
  };
  // blocks before each sequence
  const int per = (a.S + THREADS - 1) / THREADS;
  int sum = 0, blocks = 0;
  for (int i = 0; i < per && tid * per + i < a.S; ++i) {
    firsts[tid * per + i] = sum;
    sum += prompt_counted(prompt_blocks(a, prompt_seq(a, tid * per + i)), a.most);
  }
  int before = scan(sum, blocks);
  for (int i = 0; i < per && tid * per + i < a.S; ++i) firsts[tid * per + i] += before;
  __syncthreads();
  const int seqs = prompt_taken(firsts, a.S, blocks, a.most);
  if (seqs < a.S) {                       // more blocks than ascending offsets have: the same rows again
    blocks = firsts[seqs];
    if (tid == 0) atomicOr(a.err, kErrSeqLen);
  }
  auto seq_of = [&](int e) {              // the last sequence whose first block is at or before e
    int lo = 0, hi = seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (firsts[mid] <= e) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  };
  // units before each block
  const int perb = (blocks + THREADS - 1) / THREADS;
  int total = 0;
  sum = 0;
  for (int i = 0; i < perb && tid * perb + i < blocks; ++i) {
    const int e = tid * perb + i, s = seq_of(e);
    units[e] = sum;
    const int t = prompt_block<TOK>(a, prompt_seq(a, s), e - firsts[s]).tiles();
    sum += t ? t + COST : 0;
  }
  before = scan(sum, total);
  for (int i = 0; i < perb && tid * perb + i < blocks; ++i) units[tid * perb + i] += before;
  __syncthreads();
  PromptSpan x;
  const long long all = static_cast<long long>(total) * heads;
  x.span = (all + gridDim.x - 1) / gridDim.x;
  x.span = x.span < min_span ? min_span : x.span;
  x.u0 = x.span * blockIdx.x < all ? x.span * blockIdx.x : all;
  x.u1 = x.u0 + x.span < all ? x.u0 + x.span : all;
  x.s = x.qb = 0;
  x.at = 0;
  if (x.u0 < x.u1) {
    int lo = 0, hi = blocks - 1;          // the last block that starts at or before u0 (those without units start there too)
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (static_cast<long long>(units[mid]) * heads <= x.u0) lo = mid;
      else hi = mid - 1;
    }
    x.s = seq_of(lo);
    x.qb = lo - firsts[x.s];
    x.at = static_cast<long long>(units[lo]) * heads;
  }
  __syncthreads();
  return x;
}

// How the items come to the CTAs: listed ones by equal spans, cut where a span ends (a join follows) or whole, by where they
// start; or, where there are more than the list holds, whole items in turn.
enum PromptMode { kPromptCut = 1, kPromptWhole = 2, kPromptTurns = 0 };

// The items of a CTA in order, by whole warps (all of them alike).
template <int TOK, int COST>
struct PromptWalk {
  PromptBlock blk;
  int h, t0, t1, slot;                    // KV head; its tiles [t0, t1); workspace slot, -1 for whole items
  PSplit cut;                             // the record that this CTA leaves
  long long at, whole;
  int s, qb, tiles, heads, nblk, mode;

  __device__ __forceinline__ void start(const PromptArgs& a, PromptSpan& x, int heads_, int mode_) {
    mode = mode_;
    heads = heads_;
    cut = PSplit{};
    at = x.at;
    s = x.s;
    qb = x.qb;
    h = 0;
    whole = blockIdx.x;
    if (mode == kPromptTurns) {
      s = -1;
      at = 0;
      nblk = 0;
      return;
    }
    if (x.u0 >= x.u1) return;
    load(a);
    h = static_cast<int>((x.u0 - at) / (tiles + COST));
    at += static_cast<long long>(h) * (tiles + COST);
    if (mode == kPromptWhole && at < x.u0) pass(a, x);   // it is the CTA's before
  }
  __device__ __forceinline__ void load(const PromptArgs& a) {
    const PromptSeq q = prompt_seq(a, s);
    nblk = prompt_blocks(a, q);
    blk = prompt_block<TOK>(a, q, qb);
    tiles = blk.tiles();
  }
  // The next item with tiles of this CTA; false at the end.
  __device__ __forceinline__ bool next(const PromptArgs& a, PromptSpan& x) {
    slot = -1;
    if (mode == kPromptTurns) {
      const int lane = threadIdx.x & 31;
      for (;; whole += gridDim.x) {
        while (whole >= at + static_cast<long long>(nblk) * heads) {       // at: items before sequence s
          at += static_cast<long long>(nblk) * heads;
          nblk = 0;
          if (s >= a.S - 1) return false;
          // the 32 sequences behind, a lane each: the one that holds the item, or the last
          const int mine = s + 1 + lane < a.S ? prompt_blocks(a, prompt_seq(a, s + 1 + lane)) : 0;
          long long run = mine;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, run, o);
            run += lane >= o ? v : 0;
          }
          const uint32_t there = __ballot_sync(0xffffffffu, whole < at + run * heads);
          const int k = there ? __ffs(there) - 1 : 31;
          at += (__shfl_sync(0xffffffffu, run, k) - __shfl_sync(0xffffffffu, mine, k)) * heads;
          nblk = __shfl_sync(0xffffffffu, mine, k);
          s = min(s + 1 + k, a.S - 1);
        }
        const int i = static_cast<int>(whole - at);
        qb = nblk - 1 - i / heads;        // a sequence's longest rows first
        h = i % heads;
        blk = prompt_block<TOK>(a, prompt_seq(a, s), qb);
        tiles = blk.tiles();
        if (tiles) break;
      }
      whole += gridDim.x;
      t0 = 0;
      t1 = tiles;
      return true;
    }
    if (x.u0 >= x.u1) return false;
    if (mode == kPromptWhole) {
      t0 = 0;
      t1 = tiles;
      return true;
    }
    t0 = max(0, static_cast<int>(x.u0 - at) - COST);
    t1 = static_cast<int>(min(x.u1 - at - COST, static_cast<long long>(tiles)));
    if (t1 <= t0) return false;           // the span ends before the item's first tile
    if (t0 == 0 && t1 < tiles)
      cut = PSplit{1, blk.seq.q0, blk.r0, blk.rows, h, static_cast<int>((at + COST + tiles - 1) / x.span),
                   blk.seq.m - blk.seq.n, 0};
    if (t0 > 0 || t1 < tiles) slot = 2 * static_cast<int>(blockIdx.x) + (t0 ? 0 : 1);
    return true;
  }
  // Behind an item: where the next one starts.
  __device__ __forceinline__ void pass(const PromptArgs& a, PromptSpan& x) {
    if (mode == kPromptTurns) return;
    at += COST + tiles;
    x.u0 = at;
    if (x.u0 >= x.u1) return;
    if (++h < heads) return;
    h = 0;
    do {                                  // (there is one more: units are left, and only listed blocks have units)
      if (++qb >= nblk) {
        qb = 0;
        do nblk = prompt_blocks(a, prompt_seq(a, ++s));
        while (!nblk);
      }
      load(a);
    } while (!tiles);
  }
};

// Rows that see no key (more queries than keys): zeros, by all threads of all CTAs.
template <typename T>
__device__ __forceinline__ void prompt_zero_rows(const PromptArgs& a, int d) {
  for (int s = blockIdx.x; s < a.S; s += gridDim.x) {
    const PromptSeq q = prompt_seq(a, s);
    if (q.n <= q.m) continue;
    T* o = static_cast<T*>(a.out) + static_cast<long long>(q.q0) * a.Hq * d;
    for (long long i = threadIdx.x; i < static_cast<long long>(q.n - q.m) * a.Hq * d; i += blockDim.x) o[i] = T(0.0f);
  }
}

// Blocks that a call can have at most (by its sizes alone), and whether they can be listed.
inline long long prompt_most_blocks(const PromptArgs& a) { return prompt_most_blocks(a.S, a.max_q, a.total_q, a.G, a.rows); }
inline int prompt_list_room(const PromptArgs& a, int tok, int cost) { return prompt_list_room(a.max_k / tok + 2LL + a.sinks / tok + cost); }
inline bool prompt_splits(const PromptArgs& a) { return a.S <= kPromptList && prompt_most_blocks(a) <= a.most; }
// Workspace of either form (whatever the dtype and scale), its CTAs and its launch.
size_t prompt_simt_workspace(int d);
cudaError_t launch_prompt_simt(const PromptArgs& a, int d, bool f32, cudaStream_t s);
int prompt_sms();                         // of the current device
bool prompt_tc_takes(const PromptArgs& a, int d, bool f32);
size_t prompt_tc_workspace(int d);
cudaError_t launch_prompt_tc(const PromptArgs& a, int d, cudaStream_t s);
// Three bf16 parts on the tensor cores: whether the call's sizes are ones of that form.
bool prompt_parts_takes(const PromptArgs& a, int d);
size_t prompt_parts_workspace(int d);
cudaError_t launch_prompt_parts(const PromptArgs& a, int d, bool f32, cudaStream_t s);
// Joins the parts of split items (`rows` of them a slot, d + 4 floats a row: maximum, sum, two zeros, then the channels).
cudaError_t launch_prompt_join(const PromptArgs& a, int d, bool f32, int ctas, int rows, cudaStream_t s);

}  // namespace tq

#endif  // TQ_PROMPT_H_
