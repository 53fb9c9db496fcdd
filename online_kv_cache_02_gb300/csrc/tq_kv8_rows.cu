// Attention over the 8-bit paged cache for few query rows (decode, drafted
// tokens), for fp32 queries and for large softmax scales: mma.sync on e4m3
// codes turned into fp16, which is exact.
//
// An item is (sequence, block of R = 8 NT query rows, KV head); its keys are
// taken a page of 16 tokens at a time:
//   S^T[16 tokens][R] = Kc Q^T        Kc codes, Q scaled per row by a power of two
//                                     (fp16 exact for bf16 input; fp32 input as hi + lo)
//   x = scale log2(e) 2^ek 2^-row S   log2 of the weight, -inf where hidden
//   w = 2^(x + ev - M)                M = running max of x + ev over the keys: the
//                                     page's value scale goes into the weight's exponent,
//                                     so w <= 1 whatever the scales are
//   O^T[d][R] += Vc^T w,  l += w 2^-ev,  out = O / l.
// The transposed product uses all 8 columns of the MMA for 8 query rows.
//
// A CTA's warps take its pages in turn and join their (M, l, O) in shared memory
// at an item's end.  How the pages come to the CTAs:
//   direct  few pages per item, or too many items to list: an item per cluster of 1 to
//           8 CTAs, joined through distributed shared memory, one launch;
//   split   all pages of all items form one list, cut into spans of equal cost, one
//           per CTA (whatever the sequences' lengths); items that cross spans leave partials
//           for a second kernel.
//
// Bound by the memory where contexts are long, by start and end (pages' ids, scales and
// codes are three dependent loads, the join, the second launch: 10 us of one short
// sequence) where they are short.  Measured, bf16, d = 128: 16 sequences of 32,768
// tokens, 32 / 8 heads, 1.08 GB: 177 us, 6.1 TB/s, 89% of a copy's rate (d = 256, 16 / 4
// heads, 1.08 GB: 173, 92%; d = 64, 32 / 8, 539 MB: 113, 70%: half a page's bytes for the
// same steps); 64 of 1,024 to 8,192, 28 / 4 heads: 62 us, 4.9 TB/s (d = 64 45, 256 107;
// fp32 74); a window of 4,096 of 32,768: 35 us; one sequence of 1,000: 10 us.  fp32,
// d = 64, 7 of 3,001 to 9,001: 25 us.  Weights by a new maximum at every page instead of
// the one so far: 1 to 6% more.  fp32 prompts run here too (2,048 tokens: d = 64 385 us,
// 128 560, 256 800 with 16 / 4 heads, 43 to 61 TFLOP/s): eight warps an SM wait on their
// own chains of products.  So do bf16 prompts with |softmax_scale| above 1/sqrt(d)
// (2,048 tokens, d = 128: 409 us, on tcgen05 61).

#include "tq_kv8.h"
#include "tq_kv8_ring.h"
#include "tq_tc.cuh"

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

namespace tq {
namespace {

using tcx::bar_arrive_tx;
using tcx::bar_init;
using tcx::bar_wait;
using tcx::lds128;
using tcx::lds64;
using tcx::su32;

constexpr int kRWarps = 4;
// An item's start and end (its queries, the join) in pages of a CTA's time: spans are equal in pages and items weighed so,
// since short rows of a prompt would otherwise pile up in the first CTAs.  Decode hardly depends on it (64 sequences of
// 1,024 .. 8,192, 32 / 8 heads: 8, 12, 16 within 2% at d = 64, 128 and 256, both types); of an fp32 prompt of 2,048 tokens,
// d = 64, 8 makes 418 us, 12 331, 16 282.
constexpr int kItemCost = 12;
constexpr int kMinSpan = 4 + kItemCost;   // a CTA's share at least (a page per warp)
constexpr int kMaxEntries = 1024;         // (sequence, row block) pairs that the split form lists
// Pages per CTA up to which the direct form is taken: a CTA per item 64, clusters that leave two thirds of the card free
// 48, clusters that fill it 32.  Direct and split form, us, 32 / 8 heads, inputs in L2, at bf16 d = 128, 64, 256 and fp32 d = 128:
//   200 sequences of 100 .. 1,000    55 57   38 44   99 95   66 70
//   64 of 1,024 .. 8,192            125 106 109 73  223 188 155 125
//   1 of 6,000                       16 15   14 14   19 20   18 17
//   2 of 3,000                       12 15   10 14   14 19   14 16
//   16 of 1,000                      13 17   10 15   17 23   16 20
//   7 of 6,000                       33 24   18 21   37 42   41 29
// The rule takes the better one or one within a sixth of it.
constexpr int kDirectOne = 64, kDirectFew = 48, kDirectMany = 32;
// Weights are 2^(kLift + score - M), M kHead above the largest score met (it seldom moves again): the largest weight is
// 2^8, and fp16 keeps 11 bits of them down to 2^-22 of it.  M moves once a weight passes kFull, below the end of fp16:
// that score lies above M + kSlack.
constexpr float kLift = 11.0f, kHead = 3.0f, kSlack = 4.5f, kFull = 61000.0f;
// M adds an exponent to a score, which one fp32 number holds up to some size: at scores of 2^27 a weight was 2^16, past
// fp16, or 0.  A CTA that meets an M beyond kBig does its part of the item once more, without exponents in the weights.
// (M in two numbers instead, in the page loop: 0.3 to 0.9 us more for every call.)
constexpr float kBig = 65536.0f;

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t half2_of(uint32_t two) {     // two e4m3 codes (low 16 bits) -> f16x2
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<unsigned short>(two)));
  return r;
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) {            // relative error about 2^-22; 0 for -inf
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float finite_factor(float f) { return fmaxf(fminf(f, 3.4028234e38f), -3.4028234e38f); }
__device__ __forceinline__ uint32_t pack(__half lo, __half hi) {
  const __half2 h = __halves2half2(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void tma_panel(uint32_t dst, const CUtensorMap* map, int x, int blk, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(0), "r"(blk), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void cluster_sync() {                  // lanes may come to it apart (a loop with a share of the rows)
  asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
}
// Shared-memory address `p` of the cluster's CTA `rank`, and loads from it.
__device__ __forceinline__ uint32_t map_cluster(uint32_t p, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(p), "r"(rank));
  return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t p) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(p));
  return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t p) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(p));
  return v;
}

// CTAs per SM, as shared memory (the rings, the joins and a list of usual length) and registers allow.
__host__ __device__ constexpr int ctas_per_sm(int d, int R) { return R == 16 || d > 128 ? 2 : d == 128 ? 3 : 4; }

// Channels: a lane's K words (four channels each) and V words, in panels of 128.
template <int D> struct Lay {
  static constexpr int KW = D / 16;       // words of one key row per lane (its quarter of the channels)
  static constexpr int VW = D / 32;       // words of one value row per lane (its eighth)
  static constexpr int MT = D / 16;       // 16-channel tiles of the value product
  static constexpr int PAN = D >= 128 ? D / 128 : 1;
  static constexpr int KP = KW / PAN, VP = VW / PAN;   // words per panel
  // a warp's ring of pages: a K and a V block each, in panels of 16 rows x 128 bytes (64 at d = 64), swizzled by TMA
  static constexpr int ROW = D >= 128 ? 128 : 64, PANEL = kPage * ROW, BLOCK = kPage * D, STAGE = 2 * BLOCK;
  static constexpr int ST = D == 64 ? 4 : D == 128 ? 3 : 2;
  __device__ static __forceinline__ uint32_t at(int row, int chunk) {      // 16-byte piece `chunk` of a panel's row
    return static_cast<uint32_t>(row * ROW + ((chunk ^ (ROW == 128 ? row & 7 : (row >> 1) & 3)) << 4));
  }
  __device__ static __forceinline__ int k_ch(int t, int j) { return 128 * (j / KP) + 4 * KP * t + 4 * (j % KP); }
  __device__ static __forceinline__ int v_ch(int g, int w) { return 128 * (w / VP) + 4 * VP * g + 4 * (w % VP); }
};

// An item's first part ends the span of one CTA; the join finds the others by it.
struct RSplit {
  int valid, b, rb, h, n, last, pad[2];   // n: the sequence's queries; last: the CTA that holds the item's end
};

struct Item {
  int b, rb, h;
  int p0, n;                              // the sequence's first query position and queries
  int pmin, pmax;                         // positions of the block's first and last row
  Kv8Range r;
  int pages;
};

__device__ __forceinline__ int block_pages(const Kv8Attn& a, const Kv8Seq& s, int rb, int R, int& pmin, int& pmax,
                                           Kv8Range& r) {
  const long long rows = static_cast<long long>(s.n) * a.G, r0 = static_cast<long long>(rb) * R;
  if (r0 >= rows) return 0;
  const long long r1 = r0 + R < rows ? r0 + R : rows;
  pmin = s.p0 + static_cast<int>(r0 / a.G);
  pmax = s.p0 + static_cast<int>((r1 - 1) / a.G);
  r = kv8_range(a.window, a.sinks, pmin, pmax);
  return r.ns + r.nw;
}

template <int D, int NT, bool F32>
__global__ void __launch_bounds__(32 * kRWarps, ctas_per_sm(D, 8 * NT)) kv8_rows_kernel(const __grid_constant__ Kv8Attn a, const __grid_constant__ CUtensorMap mk,
                                                                const __grid_constant__ CUtensorMap mv, int nrb, int split,
                                                                int cluster) {
  using Y = Lay<D>;
  constexpr int R = 8 * NT, HL = F32 ? 2 : 1;
  // [warps][stages] pages; [warps][R][D] joins; the list's prefix sums
  extern __shared__ __align__(1024) unsigned char sm_raw[];
  unsigned char* ring = sm_raw + ((0u - su32(sm_raw)) & 1023u);
  float* sm = reinterpret_cast<float*>(ring + kRWarps * Y::ST * Y::STAGE);
  __shared__ uint64_t s_bar[kRWarps][Y::ST];
  __shared__ float s_ml[kRWarps][R][2];
  __shared__ int s_scan[2][kRWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const uint32_t my_ring = su32(ring) + warp * Y::ST * Y::STAGE, my_bar = su32(&s_bar[warp][0]);
  if (lane == 0)
    for (int i = 0; i < Y::ST; ++i) bar_init(my_bar + 8 * i, 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  __syncwarp();
  PageRing<Y::ST> pages_in;                                     // this warp's
  pdl_wait();
  if (split) pdl_trigger();                                      // the join's launch, beside the work
  RSplit* records = reinterpret_cast<RSplit*>(a.part);            // one per CTA, then the partials' slots
  float* parts = a.part + static_cast<size_t>(gridDim.x) * (sizeof(RSplit) / sizeof(float));
  RSplit cut{};
  const int entries = a.B * nrb;
  // split form: pages of one head before entry i, the items among those entries, and the entry's sequence
  int* prefix = reinterpret_cast<int*>(sm + kRWarps * R * D);
  int* some = prefix + entries;
  Kv8Seq* seqs = reinterpret_cast<Kv8Seq*>(some + entries);

  long long u0 = 0, u1 = 0, u0_first = 0, span = 1;              // this CTA's span of the list (pages)
  int entry = 0;
  long long item_at = 0;                                         // list position of the current item's first page
  Item it{};
  auto load_entry = [&](int e) {
    it.b = e / nrb;
    it.rb = e % nrb;
    const Kv8Seq s = split ? seqs[e] : kv8_seq(a, it.b);
    it.p0 = s.p0;
    it.n = s.n;
    it.pmin = it.pmax = 0;
    it.pages = block_pages(a, s, it.rb, R, it.pmin, it.pmax, it.r);
  };
  if (split) {
    // pages per entry, scanned: a run of entries per thread, then the threads' sums
    const int per = (entries + 32 * kRWarps - 1) / (32 * kRWarps);
    int sum = 0, cnt = 0;
    for (int i = 0; i < per; ++i) {
      const int e = tid * per + i;
      if (e >= entries) break;
      int x0, x1;
      Kv8Range r;
      const Kv8Seq s = kv8_seq(a, e / nrb);
      const int c = block_pages(a, s, e % nrb, R, x0, x1, r);
      seqs[e] = s;
      prefix[e] = sum;
      some[e] = cnt;
      sum += c;
      cnt += c ? 1 : 0;
    }
    int run = sum, runc = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, run, o), vc = __shfl_up_sync(0xffffffffu, runc, o);
      run += lane >= o ? v : 0;
      runc += lane >= o ? vc : 0;
    }
    if (lane == 31) s_scan[0][warp] = run, s_scan[1][warp] = runc;
    __syncthreads();
    int before = run - sum, beforec = runc - cnt, total = 0, totalc = 0;
#pragma unroll
    for (int w = 0; w < kRWarps; ++w) {
      before += w < warp ? s_scan[0][w] : 0;
      beforec += w < warp ? s_scan[1][w] : 0;
      total += s_scan[0][w];
      totalc += s_scan[1][w];
    }
    for (int i = 0; i < per && tid * per + i < entries; ++i) {
      prefix[tid * per + i] += before;
      some[tid * per + i] += beforec;
    }
    __syncthreads();
    // Spans of equal cost, an item's pages behind its kItemCost: the first page at or behind cost x
    auto cost_before = [&](int e) { return (prefix[e] + static_cast<long long>(kItemCost) * some[e]) * a.H; };
    const long long pages_all = static_cast<long long>(total) * a.H,
                    cost_all = pages_all + static_cast<long long>(kItemCost) * totalc * a.H;
    span = (cost_all + gridDim.x - 1) / gridDim.x;
    span = span < kMinSpan ? kMinSpan : span;
    auto page_at = [&](long long x) {
      if (x >= cost_all) return pages_all;
      int lo = 0, hi = entries - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (cost_before(mid) <= x) lo = mid;
        else hi = mid - 1;
      }
      const int pages = (lo + 1 < entries ? prefix[lo + 1] : total) - prefix[lo];
      const int rem = static_cast<int>(x - cost_before(lo)), h = rem / (pages + kItemCost);
      return static_cast<long long>(prefix[lo]) * a.H + static_cast<long long>(h) * pages +
             max(0, rem - h * (pages + kItemCost) - kItemCost);
    };
    u0 = page_at(span * blockIdx.x);
    u1 = page_at(span * (blockIdx.x + 1LL));
    if (a.decode) {                                              // rows that see nothing: zeros
      for (int e = blockIdx.x; e < entries; e += gridDim.x) {
        if ((e + 1 < entries ? prefix[e + 1] : total) != prefix[e]) continue;
        for (long long i = tid; i < static_cast<long long>(a.H) * R * D; i += 32 * kRWarps) {
          const int row = (e % nrb) * R + static_cast<int>(i / D % R);
          if (row < a.G) {
            const long long o = (static_cast<long long>(e / nrb) * a.Hq + i / (D * R) * a.G + row) * D + i % D;
            if (F32) static_cast<float*>(a.out)[o] = 0.0f;
            else static_cast<unsigned short*>(a.out)[o] = 0;
          }
        }
      }
    }
    if (u0 >= u1) {
      if (tid == 0) records[blockIdx.x].valid = 0;
      return;
    }
    int lo = 0, hi = entries - 1;                                // the entry that holds u0
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (static_cast<long long>(prefix[mid]) * a.H <= u0) lo = mid;
      else hi = mid - 1;
    }
    entry = lo;
    load_entry(entry);
    u0_first = u0;
    const long long base = static_cast<long long>(prefix[entry]) * a.H;
    it.h = static_cast<int>(u0 - base) / it.pages;
    item_at = base + static_cast<long long>(it.h) * it.pages;
  }

  const int step = kRWarps * cluster;
  // The warp's pages: every step-th of the CTA's span (direct form: of an item), counted by k.  A lane looks up one of
  // 32 of them: its block, place in the sequence and scales.
  struct PageInfo {
    int blk, page;
    float ks, vs;
  };
  auto fetch = [&](int k0) {
    PageInfo x{-1, 0, 0.0f, 0.0f};
    const long long u = u0_first + warp + static_cast<long long>(step) * (k0 + lane);
    if (u >= u1) return x;
    int c, h, b;
    Kv8Range r;
    if (split) {
      int lo = 0, hi = entries - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (static_cast<long long>(prefix[mid]) * a.H <= u) lo = mid;
        else hi = mid - 1;
      }
      int x0, x1;
      b = lo / nrb;
      const int pages = block_pages(a, seqs[lo], lo % nrb, R, x0, x1, r);
      const int rem = static_cast<int>(u - static_cast<long long>(prefix[lo]) * a.H);   // below pages H: the host bounds it
      h = rem / pages;
      c = rem - h * pages;
    } else {
      c = static_cast<int>(u);
      h = it.h;
      b = it.b;
      r = it.r;
    }
    x.page = c < r.ns ? c : c - r.ns + r.w0;
    const int pid = a.bt[static_cast<long long>(b) * a.maxp + x.page];
    if (pid < 0 || pid >= a.num_pages) {
      atomicOr(a.err, kErrPage);
      return x;
    }
    x.blk = pid * a.H + h;
    x.ks = a.ks[x.blk];
    x.vs = a.vs[x.blk];
    return x;
  };
  PageInfo cur{-1, 0, 0.0f, 0.0f}, nxt = cur;
  // page k + ahead of the warp into a stage (a page that is not there arrives with no bytes)
  auto send = [&](int ahead, uint32_t st) {
    const int j = (pages_in.k & 31) + ahead;
    const bool far = j >= 32;
    if (lane == (j & 31)) {
      const int blk = far ? nxt.blk : cur.blk;
      const uint32_t bar = my_bar + 8 * st, dst = my_ring + st * Y::STAGE;
      if (blk >= 0) {
        bar_arrive_tx(bar, Y::STAGE);
#pragma unroll
        for (int p = 0; p < Y::PAN; ++p) {
          tma_panel(dst + p * Y::PANEL, &mk, 128 * p, blk, bar);
          tma_panel(dst + Y::BLOCK + p * Y::PANEL, &mv, 128 * p, blk, bar);
        }
      } else {
        tcx::bar_arrive(bar);
      }
    }
    __syncwarp();
  };
  auto start = [&]() {                                           // a new run of pages
    const long long n = u1 - u0_first - warp;
    const int nk = n > 0 ? static_cast<int>((n + step - 1) / step) : 0;
    cur = fetch(0);
    nxt = nk > 32 ? fetch(32) : cur;
    pages_in.start(nk, send);
  };
  auto landed = [&](uint32_t st, uint32_t parity) {
    bool gave_up = false;
    return __all_sync(0xffffffffu, bar_wait(my_bar + 8 * st, parity, gave_up)) != 0;
  };
  // the page's stage is free for the next one
  auto pass = [&]() {
    pages_in.pass(send);
    if ((pages_in.k & 31) == 0) {
      cur = nxt;
      nxt = fetch(pages_in.k + 32);
      __syncwarp();                                              // MMAs are the whole warp's: its lanes meet first, here and below
    }
  };
  if (split) start();

  const int rank = static_cast<int>(blockIdx.x) % cluster;       // in the cluster (split form: 0)
  for (;;) {
    int c0, c1;                                                  // pages of the item that are this CTA's
    bool complete;
    int slot = 0;
    if (split) {
      if (u0 >= u1) break;
      c0 = static_cast<int>(u0 - item_at);
      c1 = static_cast<int>((u1 < item_at + it.pages ? u1 : item_at + it.pages) - item_at);
      complete = c0 == 0 && c1 == it.pages;
      slot = 2 * blockIdx.x + (c0 > 0 ? 0 : 1);
      if (c0 == 0 && !complete)
        cut = RSplit{1, it.b, it.rb, it.h, it.n,                 // the CTA whose span holds the item's last page
                     static_cast<int>(((prefix[entry] + static_cast<long long>(kItemCost) * some[entry]) * a.H +
                                       (it.h + 1LL) * (it.pages + kItemCost) - 1) / span), {0, 0}};
    } else {
      const int item = static_cast<int>(blockIdx.x) / cluster;
      it.h = item % a.H;
      load_entry(entries - 1 - item / a.H);                      // the longest rows of a prompt first
      c0 = 0;
      c1 = it.pages;
      complete = cluster == 1;
      u0_first = kRWarps * rank;
      u1 = it.pages;
      start();
    }
    const int rows = min(R, static_cast<int>(min(static_cast<long long>(R), static_cast<long long>(it.n) * a.G -
                                                                             static_cast<long long>(it.rb) * R)));
    if (rows > 0) {
      // ---- the block's queries as MMA operands ---------------------------------------
      uint32_t qf[NT][HL][Y::KW][2];
      float rf[NT][2];                                           // score factor of columns 2t, 2t + 1
      int pr[NT][2];                                             // their positions
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int row = 8 * nt + g;
        const long long gr = static_cast<long long>(it.rb) * R + row;
        const int tok = static_cast<int>(gr / a.G), hq = it.h * a.G + static_cast<int>(gr % a.G);
        float v[4 * Y::KW];
        float mx = 0.0f;
        const long long base = row < rows ? ((static_cast<long long>(it.b) * a.T + tok) * a.Hq + hq) * D : 0;
#pragma unroll
        for (int j = 0; j < Y::KW; j += 2) {                     // eight channels
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
          if (row < rows) {
            if (F32) {
              const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + base + Y::k_ch(t, j));
              x = q[0];
              y = q[1];
            } else {
              const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const unsigned short*>(a.q) + base + Y::k_ch(t, j));
              x = make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                              __uint_as_float(w.y & 0xFFFF0000u));
              y = make_float4(__uint_as_float(w.z << 16), __uint_as_float(w.z & 0xFFFF0000u), __uint_as_float(w.w << 16),
                              __uint_as_float(w.w & 0xFFFF0000u));
            }
          }
          v[4 * j] = x.x, v[4 * j + 1] = x.y, v[4 * j + 2] = x.z, v[4 * j + 3] = x.w;
          v[4 * j + 4] = y.x, v[4 * j + 5] = y.y, v[4 * j + 6] = y.z, v[4 * j + 7] = y.w;
          mx = fmaxf(fmaxf(fmaxf(mx, fabsf(x.x)), fmaxf(fabsf(x.y), fabsf(x.z))), fabsf(x.w));
          mx = fmaxf(fmaxf(fmaxf(mx, fabsf(y.x)), fmaxf(fabsf(y.y), fabsf(y.z))), fabsf(y.w));
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // the row's largest value into [2^14, 2^15): fp16 then holds bf16 values exactly down to 2^-29 of it
        int e = 14 - (static_cast<int>(__float_as_uint(mx) >> 23) - 127);
        e = mx > 0.0f && mx <= 3.4028234e38f ? (e > 120 ? 120 : e) : 0;
        const float up = __int_as_float((e + 127) << 23), down = __int_as_float((127 - e) << 23);
#pragma unroll
        for (int j = 0; j < Y::KW; ++j) {
          __half hi[4], lo[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = v[4 * j + i] * up;
            hi[i] = __float2half_rn(x);
            lo[i] = __float2half_rn(x - __half2float(hi[i]));
          }
          qf[nt][0][j][0] = pack(hi[0], hi[1]);
          qf[nt][0][j][1] = pack(hi[2], hi[3]);
          if (F32) {
            qf[nt][HL - 1][j][0] = pack(lo[0], lo[1]);
            qf[nt][HL - 1][j][1] = pack(lo[2], lo[3]);
          }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          rf[nt][c] = a.scale_log2 * __shfl_sync(0xffffffffu, down, 4 * (2 * t + c));
          const long long r = static_cast<long long>(it.rb) * R + 8 * nt + 2 * t + c;
          pr[nt][c] = it.p0 + static_cast<int>(r / a.G);
        }
      }
      float o[NT][Y::MT][4], m[NT][2], l[NT][2];
      bool big = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < Y::MT; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.0f;
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.0f;
      }
      // list position of the warp's next page, and of the item's end
      const long long seg_end = split ? item_at + c1 : c1;
      while (pages_in.k < pages_in.n && u0_first + warp + static_cast<long long>(step) * pages_in.k < seg_end) {
        const int from = pages_in.k & 31;
        const int page = __shfl_sync(0xffffffffu, cur.page, from), blk = __shfl_sync(0xffffffffu, cur.blk, from);
        const float kscale = __shfl_sync(0xffffffffu, cur.ks, from), vscale = __shfl_sync(0xffffffffu, cur.vs, from);
        const uint32_t kb = my_ring + pages_in.stage() * Y::STAGE, vb = kb + Y::BLOCK;
        if (!pages_in.land(landed)) break;
        if (blk < 0) {                                           // flagged already: the page's tokens are not there
          pass();
          continue;
        }
        const float evf = static_cast<float>(static_cast<int>((__float_as_uint(vscale) >> 23) & 0xFF) - 127);
        const float vinv = exp2_fast(-evf);

        // ---- scores ----
        float s[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.0f;
        float s_lo[F32 ? NT : 1][4] = {}, s_odd[F32 ? NT : 1][4] = {};   // fp32: the low parts, and every other product
        uint32_t kw[2][Y::KW];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int j = 0; j < Y::KW; j += 4) {
            const uint4 x = lds128(kb + (j / Y::KP) * Y::PANEL + Y::at(g + 8 * r, (Y::KP / 4) * t + (j % Y::KP) / 4));
            kw[r][j] = x.x, kw[r][j + 1] = x.y, kw[r][j + 2] = x.z, kw[r][j + 3] = x.w;
          }
#pragma unroll
        for (int j = 0; j < Y::KW; ++j) {
          const uint32_t a0 = half2_of(kw[0][j]), a2 = half2_of(kw[0][j] >> 16);
          const uint32_t a1 = half2_of(kw[1][j]), a3 = half2_of(kw[1][j] >> 16);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16816(F32 && (j & 1) ? s_odd[F32 ? nt : 0] : s[nt], a0, a1, a2, a3, qf[nt][0][j][0], qf[nt][0][j][1]);
            if (F32) mma16816(s_lo[F32 ? nt : 0], a0, a1, a2, a3, qf[nt][HL - 1][j][0], qf[nt][HL - 1][j][1]);
          }
        }
        if constexpr (F32) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[nt][i] += s_odd[nt][i] + s_lo[nt][i];
        }
        const int j0 = 16 * page;
        // does every row see the whole page?
        const bool full = j0 + 15 <= it.pmin && (!a.window || j0 > it.pmax - a.window || j0 + 15 < a.sinks);
        uint32_t live = 0xFFFFu;                                 // tokens that some row sees
        // The factors first: they cancel where small queries meet large keys, and the sum times one of them could pass fp32.
        // One that is too large for fp32 leaves zeros zero.
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float f0 = finite_factor(kscale * rf[nt][0]), f1 = finite_factor(kscale * rf[nt][1]);
          s[nt][0] *= f0, s[nt][2] *= f0;
          s[nt][1] *= f1, s[nt][3] *= f1;
        }
        if (!full) {
          live = 0u;
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const int j = j0 + k;
            if (j <= it.pmax && (!a.window || j > it.pmin - a.window || j < a.sinks)) live |= 1u << k;
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int j = j0 + g + 8 * (i >> 1), p = pr[nt][i & 1];
              if (!(j <= p && (!a.window || j > p - a.window || j < a.sinks))) s[nt][i] = -INFINITY;
            }
        }
        // ---- weights ----
        // By the maximum so far, while none passes fp16 (a new maximum costs six shuffles); else the maximum anew.
        uint32_t pf[NT][HL][2];
        float w[NT][4];
        bool over = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            w[nt][i] = exp2_fast(s[nt][i] - (m[nt][i & 1] - evf - kLift));
            over |= w[nt][i] > kFull || m[nt][i & 1] == -INFINITY;
          }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float mx = fmaxf(s[nt][c], s[nt][2 + c]) + evf;
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
              if (mx > m[nt][c] + kSlack) {
                const float mn = mx + kHead, al = exp2_fast(m[nt][c] - mn);
                big |= fabsf(mn) > kBig;
                l[nt][c] *= al;
#pragma unroll
                for (int i = 0; i < Y::MT; ++i) {
                  o[nt][i][c] *= al;
                  o[nt][i][2 + c] *= al;
                }
                m[nt][c] = mn;
              }
              const float base = m[nt][c] == -INFINITY ? 0.0f : m[nt][c] - evf - kLift;
              w[nt][c] = exp2_fast(s[nt][c] - base);
              w[nt][2 + c] = exp2_fast(s[nt][2 + c] - base);
            }
          __syncwarp();
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          l[nt][0] += (w[nt][0] + w[nt][2]) * vinv;
          l[nt][1] += (w[nt][1] + w[nt][3]) * vinv;
          __half hh[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) hh[i] = __float2half_rn(w[nt][i]);
          pf[nt][0][0] = transpose8(pack(hh[0], hh[1]));
          pf[nt][0][1] = transpose8(pack(hh[2], hh[3]));
          if (F32) {
            __half ll[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) ll[i] = __float2half_rn(w[nt][i] - __half2float(hh[i]));
            pf[nt][HL - 1][0] = transpose8(pack(ll[0], ll[1]));
            pf[nt][HL - 1][1] = transpose8(pack(ll[2], ll[3]));
          }
        }
        // ---- values ----
        uint32_t vw[4][Y::VW];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 2 * t + (r & 1) + 8 * (r >> 1);
          if (Y::VP == 2) {
            const uint2 x = lds64(vb + Y::at(row, g >> 1) + 8 * (g & 1));
            vw[r][0] = x.x, vw[r][1] = x.y;
          } else {
#pragma unroll
            for (int w = 0; w < Y::VW; w += 4) {
              const uint4 x = lds128(vb + (w / Y::VP) * Y::PANEL + Y::at(row, g));
              vw[r][w] = x.x, vw[r][w + 1] = x.y, vw[r][(w + 2) % Y::VW] = x.z, vw[r][(w + 3) % Y::VW] = x.w;
            }
          }
        }
        // The slot has been read: the next page into it.  The fence orders the reads before the copy, which is another
        // proxy's: without it they may sink behind it (fp32, 16 rows: now and then a run had a page wrong).
        tcx::fence_async_smem();
        __syncwarp();
        pass();
        if (live != 0xFFFFu) {                                   // what no row sees may hold anything
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (!((live >> (2 * t + (r & 1) + 8 * (r >> 1))) & 1u))
#pragma unroll
              for (int w = 0; w < Y::VW; ++w) vw[r][w] = 0u;
          __syncwarp();
        }
#pragma unroll
        for (int w = 0; w < Y::VW; ++w) {
          const uint32_t x0 = __byte_perm(vw[0][w], vw[1][w], 0x5140), x1 = __byte_perm(vw[0][w], vw[1][w], 0x7362);
          const uint32_t y0 = __byte_perm(vw[2][w], vw[3][w], 0x5140), y1 = __byte_perm(vw[2][w], vw[3][w], 0x7362);
          const uint32_t a0 = half2_of(x0), a1 = half2_of(x0 >> 16), a2 = half2_of(y0), a3 = half2_of(y0 >> 16);
          const uint32_t b0 = half2_of(x1), b1 = half2_of(x1 >> 16), b2 = half2_of(y1), b3 = half2_of(y1 >> 16);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if constexpr (F32) {                                 // a page's sum by itself, added in fp32: the tensor cores' sums are cut, not rounded
              float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int hl = HL - 1; hl >= 0; --hl) {
                mma16816(x, a0, a1, a2, a3, pf[nt][hl][0], pf[nt][hl][1]);
                mma16816(y, b0, b1, b2, b3, pf[nt][hl][0], pf[nt][hl][1]);
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                o[nt][2 * w][i] += x[i];
                o[nt][2 * w + 1][i] += y[i];
              }
            } else {
              mma16816(o[nt][2 * w], a0, a1, a2, a3, pf[nt][0][0], pf[nt][0][1]);
              mma16816(o[nt][2 * w + 1], b0, b1, b2, b3, pf[nt][0][0], pf[nt][0][1]);
            }
          }
        }
      }

      // ---- join the warps ----------------------------------------------------------------
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float sum = l[nt][c];
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
          const int row = 8 * nt + 2 * t + c;
          if (g == 0) {
            s_ml[warp][row][0] = m[nt][c];
            s_ml[warp][row][1] = sum;
          }
#pragma unroll
          for (int w = 0; w < Y::VW; ++w)
            *reinterpret_cast<float4*>(sm + (warp * R + row) * D + Y::v_ch(g, w)) =
                make_float4(o[nt][2 * w][c], o[nt][2 * w][2 + c], o[nt][2 * w + 1][c], o[nt][2 * w + 1][2 + c]);
        }
      if (__builtin_expect(__syncthreads_or(big), 0)) {
        // ---- scores beyond kBig: this part again, a row per warp, the weights by the plain maximum -----------
        // (as M = maximum + kLift + 8 of the join: the weights are at most 2^-8, the values have their scales)
        constexpr int kC = D / 32;                               // channels per lane
        for (int row = warp; row < rows; row += kRWarps) {
          const int gr = it.rb * R + row, tok = gr / a.G;
          const long long at = ((static_cast<long long>(it.b) * a.T + tok) * a.Hq + it.h * a.G + (gr - tok * a.G)) * D + kC * lane;
          float x[kC], mx = 0.0f, top = -INFINITY, sum = 0.0f, acc[kC] = {};
#pragma unroll
          for (int i = 0; i < kC; ++i) {
            x[i] = F32 ? static_cast<const float*>(a.q)[at + i] : __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[at + i]);
            mx = fmaxf(mx, fabsf(x[i]));
          }
          // the row by a power of two, so that no product passes fp32 that the score does not
          mx = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mx)));
          int e = 14 - (static_cast<int>(__float_as_uint(mx) >> 23) - 127);
          e = mx > 0.0f && mx <= 3.4028234e38f ? (e > 120 ? 120 : e) : 0;
#pragma unroll
          for (int i = 0; i < kC; ++i) x[i] *= __int_as_float((e + 127) << 23);
          const float rowf = a.scale_log2 * __int_as_float((127 - e) << 23);
          const int p = it.p0 + tok;
#pragma unroll 1
          for (int c = c0; c < c1; ++c) {
            if (!split && c / kRWarps % cluster != rank) continue;
            const int page = c < it.r.ns ? c : c - it.r.ns + it.r.w0, pid = a.bt[static_cast<long long>(it.b) * a.maxp + page];
            if (pid < 0 || pid >= a.num_pages) continue;         // flagged already
            const long long blk = static_cast<long long>(pid) * a.H + it.h;
            const float f = finite_factor(a.ks[blk] * rowf), vs = a.vs[blk];
#pragma unroll 1
            for (int i = 0; i < kPage; ++i) {
              const int j = kPage * page + i;
              if (!(j <= p && (!a.window || j > p - a.window || j < a.sinks))) continue;
              const long long from = (blk * kPage + i) * D + kC * lane;
              float kv[2][kC];                                   // the token's codes, of keys and of values
#pragma unroll
              for (int n = 0; n < kC; n += 2) {
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                  const uint32_t h2 = half2_of(*reinterpret_cast<const unsigned short*>((w ? a.vc : a.kc) + from + n));
                  const float2 two = __half22float2(*reinterpret_cast<const __half2*>(&h2));
                  kv[w][n] = two.x, kv[w][n + 1] = two.y;
                }
              }
              float dot = 0.0f;
#pragma unroll
              for (int n = 0; n < kC; ++n) dot = fmaf(x[n], kv[0][n], dot);
#pragma unroll
              for (int n = 16; n > 0; n >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, n);
              const float score = __fmul_rn(dot, f);
              if (score > top) {
                const float al = exp2_fast(top - score);
                sum *= al;
#pragma unroll
                for (int n = 0; n < kC; ++n) acc[n] *= al;
                top = score;
              }
              const float w = score == -INFINITY ? 0.0f : exp2_fast(__fsub_rn(score, top) - 8.0f);
              sum += w;
#pragma unroll
              for (int n = 0; n < kC; ++n) acc[n] = fmaf(w, kv[1][n] * vs, acc[n]);
            }
          }
          if (lane < kRWarps) {
            s_ml[lane][row][0] = lane ? -INFINITY : top + (kLift + 8.0f);
            s_ml[lane][row][1] = lane ? 0.0f : sum;
          }
#pragma unroll
          for (int w = 0; w < kRWarps; ++w)
#pragma unroll
            for (int n = 0; n < kC; ++n) sm[(w * R + row) * D + kC * lane + n] = w ? 0.0f : acc[n];
        }
        __syncthreads();
      }
      // four channels of one row's result
      auto store_row = [&](int row, int ch, float4 acc, float L) {
        const float inv = L > 0.0f ? 1.0f / L : L == L ? 0.0f : L;
        const int gr = it.rb * R + row, tok = gr / a.G;
        const long long at = ((static_cast<long long>(it.b) * a.T + tok) * a.Hq + it.h * a.G + (gr - tok * a.G)) * D + ch;
        if (F32) {
          *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) =
              make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        } else {
          const __nv_bfloat162 x = __floats2bfloat162_rn(acc.x * inv, acc.y * inv),
                               y = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
          *reinterpret_cast<uint2*>(static_cast<unsigned short*>(a.out) + at) =
              make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
        }
      };
      for (int i = tid; i < R * D / 4; i += 32 * kRWarps) {
        const int row = i / (D / 4), ch = 4 * (i % (D / 4));
        if (row >= rows) continue;
        float M = -INFINITY, L = 0.0f;
#pragma unroll
        for (int w = 0; w < kRWarps; ++w) M = fmaxf(M, s_ml[w][row][0]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (M == -INFINITY) {                                    // no key, or scores that are all NaN: L is 0 or NaN
#pragma unroll
          for (int w = 0; w < kRWarps; ++w) L += s_ml[w][row][1];
        } else {
#pragma unroll
          for (int w = 0; w < kRWarps; ++w) {
            const float f = exp2_fast(s_ml[w][row][0] - M);
            L += f * s_ml[w][row][1];
            const float4 x = *reinterpret_cast<const float4*>(sm + (w * R + row) * D + ch);
            acc.x += f * x.x, acc.y += f * x.y, acc.z += f * x.z, acc.w += f * x.w;
          }
        }
        if (complete) {
          store_row(row, ch, acc, L);
        } else {
          // the pages' room serves the direct form (its pages have been read), the workspace the split one
          float* p = split ? parts + (static_cast<long long>(slot) * R + row) * (D + 4)
                           : reinterpret_cast<float*>(ring) + row * (D + 4);
          *reinterpret_cast<float4*>(p + 4 + ch) = acc;
          if (ch == 0) {
            p[0] = M;
            p[1] = L;
          }
        }
      }
      __syncthreads();
      if (!complete && !split) {
        // ---- join the cluster's CTAs: each takes a share of the rows' channels ------------
        cluster_sync();
        for (int i = rank * 32 * kRWarps + tid; i < rows * D / 4; i += 32 * kRWarps * cluster) {
          const int row = i / (D / 4), ch = 4 * (i % (D / 4));
          const uint32_t p = su32(ring) + row * (D + 4) * 4;
          float M = -INFINITY, L = 0.0f;
          for (int r = 0; r < cluster; ++r) M = fmaxf(M, ld_cluster(map_cluster(p, r)));
          const float ref = M == -INFINITY ? 0.0f : M;           // no key, or scores that are all NaN: sums of 0 or NaN
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int r = 0; r < cluster; ++r) {
            const uint32_t q = map_cluster(p, r);
            const float f = M == -INFINITY ? 1.0f : exp2_fast(ld_cluster(q) - ref);
            L += f * ld_cluster(q + 4);
            const float4 x = ld_cluster4(q + 16 + 4 * ch);
            acc.x += f * x.x, acc.y += f * x.y, acc.z += f * x.z, acc.w += f * x.w;
          }
          store_row(row, ch, acc, L);
        }
        cluster_sync();                                          // nobody leaves before its sums were read
      }
    } else if (a.decode && !split && rank == 0 && tid < 32) {    // an empty sequence: zeros
      const int dr = min(R, a.G - it.rb * R);
      for (int i = lane; i < dr * D; i += 32) {
        const long long at = (static_cast<long long>(it.b) * a.Hq + it.h * a.G + it.rb * R + i / D) * D + i % D;
        if (F32) static_cast<float*>(a.out)[at] = 0.0f;
        else static_cast<unsigned short*>(a.out)[at] = 0;
      }
    }
    if (!split) break;
    u0 = item_at + c1;
    if (u0 >= u1) break;
    item_at += it.pages;
    if (++it.h == a.H) {
      it.h = 0;
      do load_entry(++entry);
      while (it.pages == 0);
    }
  }
  if (split && tid == 0) records[blockIdx.x] = cut;
  if (pages_in.failed && lane == 0) atomicOr(a.err, kErrTimeout);
}

// Joins the parts of the items that cross spans: a block per CTA of the first kernel, 16 / R warps per row.
template <int D, int R, bool F32>
__global__ void __launch_bounds__(512) kv8_join_kernel(const __grid_constant__ Kv8Attn a, int ctas) {
  constexpr int kPer = 16 / R, kV = D >= 128 ? D / 128 : 1;      // warps per row, float4 per lane
  __shared__ float4 s_acc[16][D / 4];
  __shared__ float s_l[16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = warp / kPer, part_of = warp % kPer, c = blockIdx.x;
  pdl_wait();
  const RSplit cut = reinterpret_cast<const RSplit*>(a.part)[c];
  if (!cut.valid) return;
  const float* parts = a.part + static_cast<size_t>(ctas) * (sizeof(RSplit) / sizeof(float));
  const int gr = cut.rb * R + row;
  const bool live = gr < cut.n * a.G;
  // the first part is in its CTA's second slot, the others in their CTAs' first
  auto part = [&](int k) { return parts + ((2LL * k + (k == c ? 1 : 0)) * R + row) * (D + 4); };
  float M = -INFINITY, L = 0.0f;
  float4 acc[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (live) {
    for (int k = c + lane; k <= cut.last; k += 32) M = fmaxf(M, part(k)[0]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float ref = M == -INFINITY ? 0.0f : M;                 // no key, or scores that are all NaN: sums of 0 or NaN
#pragma unroll 8
    for (int k = c + part_of; k <= cut.last; k += kPer) {
      const float* p = part(k);
      const float f = exp2_fast(p[0] - ref);
      L += M == -INFINITY ? p[1] : f * p[1];
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        if (128 * i + 4 * lane >= D) continue;
        const float4 x = *reinterpret_cast<const float4*>(p + 4 + 128 * i + 4 * lane);
        acc[i].x += f * x.x, acc[i].y += f * x.y, acc[i].z += f * x.z, acc[i].w += f * x.w;
      }
    }
  }
  if (kPer > 1) {
#pragma unroll
    for (int i = 0; i < kV; ++i)
      if (128 * i + 4 * lane < D) s_acc[warp][32 * i + lane] = acc[i];
    if (lane == 0) s_l[warp] = L;
    __syncthreads();
    if (part_of != 0) return;
    for (int w = 1; w < kPer; ++w) {
      L += s_l[warp + w];
#pragma unroll
      for (int i = 0; i < kV; ++i)
        if (128 * i + 4 * lane < D) {
          const float4 x = s_acc[warp + w][32 * i + lane];
          acc[i].x += x.x, acc[i].y += x.y, acc[i].z += x.z, acc[i].w += x.w;
        }
    }
  }
  if (!live) return;
  const float inv = L > 0.0f ? 1.0f / L : L == L ? 0.0f : L;
  const long long o = ((static_cast<long long>(cut.b) * a.T + gr / a.G) * a.Hq + cut.h * a.G + gr % a.G) * D;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    if (128 * i + 4 * lane >= D) continue;
    const float4 y = make_float4(acc[i].x * inv, acc[i].y * inv, acc[i].z * inv, acc[i].w * inv);
    const long long at = o + 128 * i + 4 * lane;
    if (F32) {
      *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = y;
    } else {
      const __nv_bfloat162 p0 = __floats2bfloat162_rn(y.x, y.y), p1 = __floats2bfloat162_rn(y.z, y.w);
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&p0), *reinterpret_cast<const uint32_t*>(&p1));
    }
  }
}

// Query rows per block: 16 where a KV head has more than 8 (d = 256: its accumulators fill the registers at 8).
int rows_per_block(int T, int G, int d) { return static_cast<long long>(T) * G > 8 && d <= 128 ? 16 : 8; }
int row_blocks(int T, int G, int R) { return static_cast<int>((static_cast<long long>(T) * G + R - 1) / R); }

// launch_pdl with thread-block clusters.
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, int cluster,
                           Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

template <int D, int NT, bool F32>
cudaError_t launch_t(const Kv8Attn& a, cudaStream_t s) {
  constexpr int R = 8 * NT;
  const long long nrb = row_blocks(a.T, a.G, R);
  const long long entries = a.B * nrb, items = entries * a.H;
  if (items > 0x7FFFFFFFLL || items * R > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
  using Y = Lay<D>;
  const int slots = ctas_per_sm(D, R) * kv8_sm_count();
  // Pages that an item can have, and the CTAs per item that fill the card.
  const long long span = a.window ? static_cast<long long>(a.window) + a.T + a.sinks + 2 * kPage : a.max_seq_len;
  const long long pages = (std::min<long long>(span, a.max_seq_len) + kPage - 1) / kPage;
  int cluster = 8;
  while (cluster > 1 && (items * cluster > slots || pages <= cluster / 2 * kRWarps)) cluster /= 2;
  const int most = cluster == 1 ? kDirectOne : 3 * items * cluster <= slots ? kDirectFew : kDirectMany;
  // the list counts pages in 32 bits
  const bool split = pages > static_cast<long long>(most) * cluster && entries <= kMaxEntries && entries * pages <= 0x7FFFFFFFLL;
  const size_t fixed = 1024 + kRWarps * (Y::ST * Y::STAGE + sizeof(float) * R * D);
  const size_t list = sizeof(Kv8Seq) + 2 * sizeof(int);
  const size_t smem = fixed + (split ? list * entries : 0);
  static std::atomic<unsigned long long> configured{0};
  cudaError_t e = smem_attr_once(kv8_rows_kernel<D, NT, F32>, static_cast<int>(fixed + list * kMaxEntries), configured);
  if (e != cudaSuccess) return e;
  CUtensorMap mk, mv;
  const long long blocks = static_cast<long long>(a.num_pages) * a.H;
  if (!kv8_block_map(&mk, a.kc, blocks, D) || !kv8_block_map(&mv, a.vc, blocks, D)) return cudaErrorInvalidValue;
  if (!split)
    return launch_cluster(kv8_rows_kernel<D, NT, F32>, dim3(static_cast<unsigned>(items * cluster)), dim3(32 * kRWarps), smem, s,
                          cluster, a, mk, mv, static_cast<int>(nrb), 0, cluster);
  e = launch_pdl(kv8_rows_kernel<D, NT, F32>, dim3(slots), dim3(32 * kRWarps), smem, s, a, mk, mv, static_cast<int>(nrb), 1, 1);
  if (e != cudaSuccess) return e;
  return launch_pdl(kv8_join_kernel<D, R, F32>, dim3(slots), dim3(512), 0, s, a, slots);
}

template <int D>
cudaError_t launch_d(const Kv8Attn& a, bool f32, cudaStream_t s) {
  if constexpr (D <= 128) {
    if (rows_per_block(a.T, a.G, D) == 16) return f32 ? launch_t<D, 2, true>(a, s) : launch_t<D, 2, false>(a, s);
  }
  return f32 ? launch_t<D, 1, true>(a, s) : launch_t<D, 1, false>(a, s);
}

}  // namespace

bool kv8_head_dim(int d) { return d == 64 || d == 128 || d == 256; }

size_t kv8_rows_workspace(int T, int G, int d) {
  const int R = rows_per_block(T, G, d);
  return static_cast<size_t>(ctas_per_sm(d, R)) * kv8_sm_count() * (sizeof(RSplit) + 2 * sizeof(float) * R * (d + 4));
}

cudaError_t launch_kv8_rows(const Kv8Attn& a, int d, bool f32, cudaStream_t s) {
  switch (d) {
    case 64: return launch_d<64>(a, f32, s);
    case 128: return launch_d<128>(a, f32, s);
    case 256: return launch_d<256>(a, f32, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace tq
