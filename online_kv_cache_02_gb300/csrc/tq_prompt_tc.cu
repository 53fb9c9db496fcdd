// Attention over packed prompts on the tensor cores (tcgen05), bf16, d = 64, 128 or 256.
//
// An item is (sequence, KV head, block of query rows r = t G + g): whole tokens, two halves A and B of at most 128 rows
// (TMA brings a half's rows as one box of tokens and heads); keys go by in tiles of 128.  All items' tiles form one list
// that is cut into equal spans, one per CTA; the parts of an item that crosses spans are joined by a second kernel.  Per
// tile, with x = scale log2(e) <q, k>:
//   S = Q K^T              bf16, from tiles that TMA puts in place
//   w = 2^(x - M)          bf16 and fp32 hold the weights whatever M is, within 2^126: M starts as 0, and only a tile whose
//                          weights sum to more than 2^24, or that leaves a row that sees something with a sum below
//                          2^-24, looks for a maximum
//   O += w V, l += sum w   w as bf16 (off by 2^-8 at most) in tensor memory, V's token rows read MN-major;
//   out = O / l.
// The halves take turns: while the softmax of one runs, the tensor cores work on the other.  An item follows the one
// before like a tile does: its queries are there ahead of time (a ring of halves), and its results are left to warps of
// their own.  Tensor memory: S of A and B (each overlaid by its weights), O of A and B, 512 columns; at d = 64, where O takes
// half of that, S has three rooms in turn and the scores run a half's tile further ahead.  An item that fits one
// half is in both: A takes the even tiles, B the odd ones, and their sums are added at the end.  At d = 256 every item is
// one half of rows, in the same turns, and tensor memory has one O of 256 columns, to which both add: M is the row's in
// both, and a half that moves it does so between the other's products.
//
// A key that a row does not see has weight zero, but zero times an infinity is NaN: the values of tiles that some row does
// not see in full are looked through before they are multiplied, what is not finite there is taken out, and added to the
// rows that see it at the end.
//
// Warps 0-3 and 4-7: the softmax of A and B (thread = row); 8-11: the results; 12: items, the copies of queries and keys;
// 13: MMA issue; 14: a look at the values of edge tiles; 15: the values' copies.  Every wait is bounded; a wait that gives
// up sets the device error word.
//
// What bounds it: a key tile's 2 x 128 rows take 1,024 cycles of the tensor cores at d = 128 (512 at 64) and 1,024 of the
// exponentials (32 lanes a cycle and SM), which two halves overlap as far as a half's own chain lets them: scores, softmax,
// weights, values, one behind the other.  A prompt of 8,192 tokens, 32 / 8 heads: d = 128 330 us in a burst (1,670 TFLOP/s,
// tensor pipe 78% of the cycles by its counter) and 363 in a long series, where power lowers the clock (1,515), d = 64 256 us
// (tensor pipe and exponentials 48% each, issue slots 48%), d = 256 (16 / 4 heads) 355 us.  Two dozen prompts of up to 2,500
// tokens 329 to 343 us, of which the ends of 3,408 items and the join.
// Slower were an O of its own for each half at d = 256 (every score twice: 552 us) and the softmax in two parts of 64 keys
// (less code, d = 128: 397 us).

#include "tq_prompt.h"
#include "tq_tc.cuh"
#include "tq_tc_attn.cuh"

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

namespace tq {
namespace {

using namespace tcx;

constexpr int kTok = 128;                 // keys per tile
constexpr int kThreads = 512;
constexpr int kItems = 4;                 // items announced ahead
// An item's start and end, in tiles' time.  1, 2, 3, 4: windows of 1,024 at d = 64 133, 129, 128, 130 us, chunks at d = 256 275,
// 276, 277, 279, two dozen prompts at d = 128 334, 333, 342, 341.
constexpr int kItemCost = 3;
constexpr int kMinSpan = 2 + kItemCost;   // a CTA's share of the list at least
constexpr float kFull = 16777216.0f, kTiny = 5.9604645e-8f;       // 2^24 and 2^-24: bounds of a row's sum
// x - M in one rounding is off by half a step of M against the other tiles' M: beyond 2^16 scores are rounded first, so that
// small differences of large ones are exact.
constexpr float kBig = 65536.0f;
constexpr int kCheckRing = 8;

// Registers: 16 warps start with 128 a thread, and the eight of the softmax take what the others give back.
constexpr int kRegsSoftmax = 176, kRegsResults = 80, kRegsOthers = 80;
static_assert(8 * kRegsSoftmax + 4 * kRegsResults + 4 * kRegsOthers <= 16 * 128, "more registers than the block starts with");

template <int D>
struct PG {
  static constexpr bool WIDE = D == 256;
  static constexpr int HALVES = WIDE ? 1 : 2;          // of query rows per item
  static constexpr int ROWS = 128 * HALVES;
  static constexpr int SB = D == 64 ? 3 : 2;           // rooms of S, 128 columns each
  static constexpr int VCH = WIDE ? 2 : 1, VTOK = kTok / VCH;      // pieces of a tile's values, and their tokens
  static constexpr int KCH = D > 128 ? D / 128 : 1;    // pieces of a tile's keys, 128 channels each
  static constexpr int PIECE = kTok * 2 * (D < 128 ? D : 128);      // bytes of a piece
  static constexpr int QX = 128 * 2 * D;               // a half's queries
  static constexpr int QST = D == 64 ? 4 : D == 128 ? 3 : 1, KST = D == 64 ? 5 : 2, VST = D == 64 ? 5 : D == 128 ? 2 : 3;
  static constexpr int PART = D + 4;                   // floats of a row's partial
  static constexpr int Q = 0;                          // [stage][64-channel panels][128 rows][128 B]
  static constexpr int K = Q + QST * QX;               // [stage][64-channel panels][128 tokens][128 B]
  static constexpr int V = K + KST * PIECE;            // [stage][64-channel panels][VTOK tokens][128 B]
  static constexpr int ITEM = V + VST * PIECE;
  static constexpr int BAR = ITEM + kItems * 64;
};
enum Bar {
  bQFull = 0, bQFree = bQFull + 4, bKFull = bQFree + 4, bKFree = bKFull + 5, bVFull = bKFree + 5, bVFree = bVFull + 5, bVOk = bVFree + 5,
  bSFull = bVOk + 5, bPFull = bSFull + 6, bProducts = bPFull + 3, bTold = bProducts + 2, bSums = bTold + 4, bODone = bSums + 2, bOFree = bODone + 2, bItem = bOFree + 2,
  bItemFree = bItem + kItems, bChecked = bItemFree + kItems, bDrain = bChecked + kCheckRing, bCount
};
template <int D>
struct PS {                                            // behind the barriers
  static constexpr int SUMS = PG<D>::BAR + 8 * ((bCount + 1) & ~1);      // (M, l) of the halves' rows; d = 256: [l of A, l of B, M of the half
                                                                         // that ends first, M] of 128 rows
  static constexpr int ODD = SUMS + 2 * 128 * 8;   // per item: values that are not finite in edge tiles
  static constexpr int MOVES = ODD + 4 * kCheckRing;   // d = 256: how often M has moved, by 32 rows: item + 1, times
  static constexpr int QUEUE = MOVES + 32;             // of the MMA warp, four words
  static constexpr int TMEM = QUEUE + 16;
  static constexpr int BYTES = TMEM + 16;
};
static_assert(PS<64>::BYTES <= 232448 && PS<128>::BYTES <= 232448 && PS<256>::BYTES <= 232448, "shared memory per block");
static_assert(PG<64>::ITEM >= 4 * (2 * kPromptList + 64), "the list's room");
template <int D>
__device__ __forceinline__ constexpr uint32_t col_o(uint32_t X) { return D == 64 ? 384u + 64u * X : D == 128 ? 256u + 128u * X : 256u; }

// A place in a ring of N and its phase: counted where N divides without effort, else kept.
template <int N>
struct Ring {
  static constexpr bool COUNTS = (N & (N - 1)) == 0;
  int at = 0, turn = 0;
  __device__ __forceinline__ int place() const { return COUNTS ? at & (N - 1) : at; }
  __device__ __forceinline__ int phase() const { return COUNTS ? at / N : turn; }
  __device__ __forceinline__ void next() {
    ++at;
    if (!COUNTS && at == N) {
      at = 0;
      turn ^= 1;
    }
  }
};
// What the load warp tells the others of an item.
struct alignas(16) ItemMsg {
  int valid, h, q0, r0;                   // h: KV head
  int rows, p0, pmin, pmax;               // p0: position of the sequence's first query
  int ntile, t0, slot, k0;                // slot: of the workspace for a part of the tiles; -1 for all of them
  int ns, w0, pad[2];
  __device__ __forceinline__ int first_key(int i) const {          // of its i-th tile
    const int t = t0 + i;
    return t < ns ? kTok * t : w0 + kTok * (t - ns);
  }
  // every row sees every key of the tile from j0 on
  __device__ __forceinline__ bool full(int j0, int window, int sinks) const {
    return j0 + kTok - 1 <= pmin && (!window || j0 > pmax - window || j0 + kTok - 1 < sinks);
  }
};
static_assert(sizeof(ItemMsg) == 64, "items in shared memory");

// S = Q K^T, 128 channels (64 at d = 64): steps of 16 channels (32 B, 2 descriptor units), panels of 64 channels 16 KB
// apart; one statement, one elected lane.
template <int ACC>
__device__ __forceinline__ void mma8_scores(uint32_t d, uint64_t q, uint64_t k, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred e, t, f;\n .reg .b64 q1, q2, q3, q4, q5, q6, q7, k1, k2, k3, k4, k5, k6, k7;\n"
      " add.u64 q1, %1, 2;\n add.u64 q2, %1, 4;\n add.u64 q3, %1, 6;\n add.u64 q4, %1, 1024;\n add.u64 q5, %1, 1026;\n"
      " add.u64 q6, %1, 1028;\n add.u64 q7, %1, 1030;\n"
      " add.u64 k1, %2, 2;\n add.u64 k2, %2, 4;\n add.u64 k3, %2, 6;\n add.u64 k4, %2, 1024;\n add.u64 k5, %2, 1026;\n"
      " add.u64 k6, %2, 1028;\n add.u64 k7, %2, 1030;\n"
      " setp.ne.b32 t, 1, 0;\n setp.ne.b32 f, %4, 0;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], q1, k1, %3, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], q2, k2, %3, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], q3, k3, %3, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], q4, k4, %3, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], q5, k5, %3, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], q6, k6, %3, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], q7, k7, %3, t;\n}\n" ::"r"(d),
      "l"(q), "l"(k), "r"(idesc), "n"(ACC)
      : "memory");
}
__device__ __forceinline__ void mma4_scores(uint32_t d, uint64_t q, uint64_t k, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred e, t, f;\n .reg .b64 q1, q2, q3, k1, k2, k3;\n"
      " add.u64 q1, %1, 2;\n add.u64 q2, %1, 4;\n add.u64 q3, %1, 6;\n add.u64 k1, %2, 2;\n add.u64 k2, %2, 4;\n add.u64 k3, %2, 6;\n"
      " setp.ne.b32 t, 1, 0;\n setp.ne.b32 f, 0, 0;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], q1, k1, %3, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], q2, k2, %3, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], q3, k3, %3, t;\n}\n" ::"r"(d),
      "l"(q), "l"(k), "r"(idesc)
      : "memory");
}
// O (+)= w V for 64 keys: four steps of 16 (8 columns of weights, 2048 B or 128 descriptor units of values).
__device__ __forceinline__ void mma4_values(uint32_t d, uint32_t w, uint64_t v, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred e, t, p;\n .reg .b32 w1, w2, w3;\n .reg .b64 v1, v2, v3;\n"
      " add.u32 w1, %1, 8;\n add.u32 w2, %1, 16;\n add.u32 w3, %1, 24;\n"
      " add.u64 v1, %2, 128;\n add.u64 v2, %2, 256;\n add.u64 v3, %2, 384;\n"
      " setp.ne.b32 p, %4, 0;\n setp.ne.b32 t, 1, 0;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [w1], v1, %3, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [w2], v2, %3, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [w3], v3, %3, t;\n}\n" ::"r"(d),
      "r"(w), "l"(v), "r"(idesc), "r"(acc)
      : "memory");
}
// kind::f16 with bf16 A and B, fp32 accumulate, M = 128, N = n
__host__ __device__ constexpr uint32_t idesc_bf16(int n) { return idesc_f16(n) | (1u << 7) | (1u << 10); }
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int x, int head, int row, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(head), "r"(row), "r"(bar)
      : "memory");
}
__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Whether one of two bf16 values is not finite.
__device__ __forceinline__ bool odd_pair(uint32_t w) { return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u; }
__device__ __forceinline__ bool odd_piece(uint4 w) { return odd_pair(w.x) || odd_pair(w.y) || odd_pair(w.z) || odd_pair(w.w); }

// One tile's weights of a thread's row with a new M, the largest score met; scores are rounded before they are compared.
// accumulated: O holds tiles before, of which the row has seen something (had): M is then the row's reference, only raised
// where O has another half's sums in it (shared).  Returns M and l.
template <int DV>
__device__ __noinline__ float2 careful_tile(uint32_t ts, uint32_t to, int j0, int p, int window, int sinks, float f, bool accumulated,
                                            float m, float l, bool had, bool shared) {
  auto scores = [&](int c, float (&y)[32]) {
    tld32(ts + 32u * c, y);
    const uint32_t see = prompt_seen32(p, j0 + 32 * c, window, sinks);
#pragma unroll
    for (int k = 0; k < 32; ++k) y[k] = (see >> k) & 1u ? __fmul_rn(y[k], f) : -INFINITY;
    __syncwarp();
  };
  // of the sum so far: l 2^m, about 2^(m + log2 l), so that alpha l is about 1 at most
  float y[32], mn = had ? (shared ? m : m + log2f(l)) : -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    scores(c, y);
#pragma unroll
    for (int k = 0; k < 32; ++k) mn = fmaxf(mn, y[k]);
  }
  if (mn == -INFINITY) mn = 0.0f;                      // nothing seen
  const float alpha = had ? ex2(m - mn) : 1.0f;
  __syncwarp();
  if (accumulated) rescale_o<DV>(to, alpha);
  l *= alpha;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {                        // (the weights overlay scores that were read)
    uint32_t w[16];
    scores(c, y);
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float y0 = ex2(__fsub_rn(y[2 * k], mn)), y1 = ex2(__fsub_rn(y[2 * k + 1], mn));
      sum += y0 + y1;
      w[k] = bf16x2_bits(y0, y1);
    }
    l += sum;
    tst16(ts + 16u * c, w);
  }
  return make_float2(mn, l);
}

// What is not finite among the values that a row sees of an item's edge tiles, added to its O.  `v`: the item's first value
// channel of the sequence's key 0.
template <int DV>
__device__ __noinline__ void add_odd_values(uint32_t to, const __nv_bfloat16* v, long long stride, int t0, int ntile, int ns, int w0, int pmin,
                                            int pmax, int p, int window, int sinks) {
  ItemMsg it;
  it.t0 = t0, it.ns = ns, it.w0 = w0, it.pmin = pmin, it.pmax = pmax;
#pragma unroll 1
  for (int c = 0; c < DV / 16; ++c) {
    float o[16];
    uint32_t x[16];
    tld16(to + 16u * c, o);
#pragma unroll 1
    for (int t = 0; t < ntile; ++t) {
      const int j0 = it.first_key(t);
      if (it.full(j0, window, sinks)) continue;
#pragma unroll 1
      for (int j = j0; j < j0 + kTok && j <= pmax; ++j) {
        const uint4* from = reinterpret_cast<const uint4*>(v + j * stride + 16 * c);
        const uint4 w[2] = {from[0], from[1]};         // the same for the whole warp
        if (!odd_piece(w[0]) && !odd_piece(w[1])) continue;
        const bool see = prompt_sees(p, j, window, sinks);
        const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float lo = __uint_as_float(u[k] << 16), hi = __uint_as_float(u[k] & 0xFFFF0000u);
          o[2 * k] += see && !(fabsf(lo) <= 3.4028234e38f) ? lo : 0.0f;
          o[2 * k + 1] += see && !(fabsf(hi) <= 3.4028234e38f) ? hi : 0.0f;
        }
      }
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] = __float_as_uint(o[k]);
    tst16(to + 16u * c, x);
  }
  tst_wait();
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_tc_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                     const __grid_constant__ CUtensorMap mv, int mode) {
  using L = PG<D>;
  using P = PS<D>;
  extern __shared__ __align__(1024) unsigned char sm_raw[];
  unsigned char* sm = sm_raw;
  const uint32_t sb = su32(sm);
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const int half = a.rows / L::HALVES;                 // rows of a half: whole tokens
  auto bar = [&](int i) { return sb + L::BAR + 8u * static_cast<uint32_t>(i); };
  ItemMsg* item_ring = reinterpret_cast<ItemMsg*>(sm + L::ITEM);
  float2* sums = reinterpret_cast<float2*>(sm + P::SUMS);
  volatile int* odd_of = reinterpret_cast<volatile int*>(sm + P::ODD);
  PSplit* splits = reinterpret_cast<PSplit*>(a.part);              // one per CTA, then the partials' slots
  if (sb & 1023u) {                                    // the swizzles' period: the kernel's only shared memory starts on one
    pdl_wait();
    if (tid == 0) {
      atomicOr(a.err, kErrLayout);
      if (mode == kPromptCut) splits[blockIdx.x].valid = 0;
    }
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < L::QST; ++i) {
      bar_init(bar(bQFull + i), 1);
      bar_init(bar(bQFree + i), 1);
    }
    for (int i = 0; i < L::KST; ++i) {
      bar_init(bar(bKFull + i), 1);
      bar_init(bar(bKFree + i), 1);
    }
    for (int i = 0; i < L::VST; ++i) {
      bar_init(bar(bVFull + i), 1);
      bar_init(bar(bVFree + i), 1);
      bar_init(bar(bVOk + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(bar(bProducts + i), 1);
      bar_init(bar(bTold + 2 * i), 4);
      bar_init(bar(bTold + 2 * i + 1), 4);
      bar_init(bar(bSums + i), 4);
      bar_init(bar(bODone + i), 1);
      bar_init(bar(bOFree + i), 4);
    }
    for (int i = 0; i < L::SB; ++i) bar_init(bar(bPFull + i), 4);
    // S of a half's tiles: as many barriers as rooms, in turn.  One that both halves waited on would pass B by while items
    // have one tile, and one per half would pass A by, whose scores may be three tiles ahead there.
    for (int i = 0; i < 2 * L::SB; ++i) bar_init(bar(bSFull + i), 1);
    for (int i = 0; i < kItems; ++i) {
      bar_init(bar(bItem + i), 1);
      bar_init(bar(bItemFree + i), 15);                // every warp but the one that announces
    }
    for (int i = 0; i < kCheckRing; ++i) {
      bar_init(bar(bChecked + i), 1);
      odd_of[i] = 0;
    }
    for (int i = 0; i < 4; ++i) reinterpret_cast<long long*>(sm + P::MOVES)[i] = 0;
    bar_init(bar(bDrain), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 13) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sb + P::TMEM), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  if (mode == kPromptCut) pdl_trigger();                            // the join's launch
  prompt_zero_rows<__nv_bfloat16>(a, D);
  PromptSpan span{};
  if (mode != kPromptTurns) span = prompt_span<kTok, kItemCost, kThreads>(a, a.H, kMinSpan, reinterpret_cast<int*>(sm));
  fence_async_smem();
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = *reinterpret_cast<const uint32_t*>(sm + P::TMEM);
  float* parts = a.part + static_cast<size_t>(gridDim.x) * (sizeof(PSplit) / sizeof(float));
  bool failed = false;
  // a warp's wait for phase `phase` of a barrier; once one gave up, every later one returns at once
  auto wait = [&](int i, int phase) {
    if (!failed && __all_sync(0xffffffffu, wait_short(bar(i), phase & 1))) return true;
    failed = true;
    return false;
  };
  // the n-th item of this CTA, from the ring
  auto next_item = [&](int n) {
    ItemMsg x{};
    if (wait(bItem + n % kItems, n / kItems)) x = item_ring[n % kItems];
    __syncwarp();
    if (lane == 0) bar_arrive(bar(bItemFree + n % kItems));
    return x;
  };

  // a piece of keys or of values, in panels of 64 channels
  auto copy = [&](const CUtensorMap* map, uint32_t dst, int panel, int ch, int head, int row, uint32_t full) {
    if (lane == 0) {
      bar_arrive_tx(full, L::PIECE);
      for (int i = 0; i < L::PIECE / panel; ++i) tma_rows(dst + panel * i, map, ch + 64 * i, head, row, full);
    }
    __syncwarp();
  };

  if (warp < 8) {
    // ---- softmax of half X (thread = row) --------------------------------------------------
    // Accesses to tensor memory are the whole warp's: behind a branch that only some lanes take they meet again first.
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int X = warp >> 2, wq = warp & 3, r = 32 * wq + lane;
    const uint32_t trow = tmem + (static_cast<uint32_t>(32 * wq) << 16);
    const uint32_t to = trow + col_o<D>(X);
    const float f = a.scale_log2;
    int unit = 0, items = 0, tiles = 0, other = 0;     // halves' tiles before the item; items of this half, tiles of it and of the other half
    volatile float* wide_sums = reinterpret_cast<volatile float*>(sm + P::SUMS);
    volatile float* moved = wide_sums + 384;
    volatile long long* moves = reinterpret_cast<volatile long long*>(sm + P::MOVES);
    int seen_moves = 0;
    for (int n = 0;; ++n) {
      const ItemMsg it = next_item(n);
      if (!it.valid) break;
      const bool turns = it.rows <= half;              // the halves take the tiles in turn
      const int ntile = it.ntile;
      const int rx = turns ? r : half * X + r;
      const bool live = r < half && rx < it.rows;      // what the other lanes hold is no row, and nobody looks at it
      const int p = it.p0 + (it.r0 + rx) / a.G;
      const int first = turns ? X : 0, step = turns ? 2 : 1;
      float m = 0.0f, l = 0.0f;
      bool bigs = false;                               // a row of the warp has had an M beyond kBig
      const int before = other;
      if (L::WIDE) seen_moves = 0;
      // d = 256: the other half's tile before has its weights.  Two barriers in turn: that half may be one tile further on, at
      // the next item's first.
      auto told = [&]() { return wait(bTold + 2 * (X ^ 1) + ((other - 1) & 1), (other - 1) / 2); };
      // d = 256: to the M that the other half has moved to; false if it has not.
      auto follow = [&]() {
        const long long at = moves[wq];
        const int now = static_cast<int>(at >> 32) == n + 1 ? static_cast<int>(at) : 0;
        __syncwarp();
        if (now == seen_moves) return false;
        seen_moves = now;
        const float to_m = moved[r];
        l = l > 0.0f ? l * ex2(m - to_m) : l;
        m = to_m;
        bigs = __any_sync(0xffffffffu, live && fabsf(m) > kBig);
        return true;
      };
      for (int t = first; t < ntile; t += step) {
        const int u = unit + (turns ? t : 2 * t + X), room = u % L::SB;
        const uint32_t ts = trow + 128u * static_cast<uint32_t>(room);
        if (!wait(bSFull + X * L::SB + tiles % L::SB, tiles / L::SB)) break;
        tc_after();
        const int j0 = it.first_key(t);
        if (L::WIDE) other = before + (t + X) / 2;     // the other half's tiles up to this one
        bool done = false;
        for (bool again = true; again;) {              // (twice where the other half has moved M meanwhile)
          again = false;
          if (bigs) break;
          float x[kTok];
          uint32_t w[kTok / 2];
          tld32x4(ts, x);
          bool sees = live;                            // the row sees something of the tile
          if (!it.full(j0, a.window, a.sinks)) {
            uint32_t all = 0u;
#pragma unroll
            for (int c = 0; c < kTok; c += 32) {
              const uint32_t see = prompt_seen32(p, j0 + c, a.window, a.sinks);
              all |= see;
              if (__any_sync(0xffffffffu, see != 0xFFFFFFFFu)) {
#pragma unroll
                for (int k = 0; k < 32; ++k) x[c + k] = (see >> k) & 1u ? x[c + k] : -INFINITY;
              }
            }
            sees = live && all != 0u;
          }
          const uint64_t f2 = pack2(f, f), b2 = pack2(-m, -m);
          uint64_t s2 = 0ull, s3 = 0ull;
#pragma unroll
          for (int c = 0; c < kTok; c += 4) {
            float y0, y1, y2, y3;
            unpack2(fma2(pack2(x[c], x[c + 1]), f2, b2), y0, y1);
            unpack2(fma2(pack2(x[c + 2], x[c + 3]), f2, b2), y2, y3);
            y0 = ex2(y0);
            y1 = ex2(y1);
            y2 = ex2(y2);
            y3 = ex2(y3);
            s2 = add2(s2, pack2(y0, y1));
            s3 = add2(s3, pack2(y2, y3));
            w[c / 2] = bf16x2_bits(y0, y1);
            w[c / 2 + 1] = bf16x2_bits(y2, y3);
          }
          float s0, s1;
          unpack2(add2(s2, s3), s0, s1);
          s0 += s1;
          if (L::WIDE && t > 0) {
            // The tile before is the other half's: its weights are there, and M is what they were made with.
            if (!told()) break;
            if (follow()) {
              again = true;
              continue;
            }
          }
          if (!__any_sync(0xffffffffu, sees && (s0 > kFull || l + s0 < kTiny))) {
            l += s0;
            tst32(ts, *reinterpret_cast<uint32_t(*)[32]>(w));
            tst32(ts + 32u, *reinterpret_cast<uint32_t(*)[32]>(w + 32));
            done = true;
          }
        }
        if (failed) break;
        if (!done) {
          if (L::WIDE && t > 0) {                      // O is at rest behind the products of the tile before
            if (!told() || !wait(bProducts + (X ^ 1), other - 1)) break;
            tc_after();
            (void)follow();
          } else if (L::WIDE && items > 0 && !wait(bOFree, items - 1)) {     // (the item before has M in its results)
            break;
          } else if (L::SB > 2 && t > first) {         // (with two rooms the scores come behind them)
            if (!wait(bProducts + X, tiles - 1)) break;
            tc_after();
          }
          bool had = l > 0.0f;                         // has the row seen anything?
          if (L::WIDE)
            for (int i = 0; i < t && !had; ++i)
              for (int c = 0; c < kTok; c += 32) had |= prompt_seen32(p, it.first_key(i) + c, a.window, a.sinks) != 0u;
          __syncwarp();
          const float2 next = careful_tile<D>(ts, to, j0, p, a.window, a.sinks, f, L::WIDE ? t > 0 : t > first, m, l, had, L::WIDE);
          m = next.x;
          l = next.y;
          bigs = __any_sync(0xffffffffu, live && fabsf(m) > kBig);
          if (L::WIDE) {
            moved[r] = m;
            ++seen_moves;
            __syncwarp();
            if (lane == 0) moves[wq] = (static_cast<long long>(n + 1) << 32) | seen_moves;
            __syncwarp();
          }
        }
        tst_wait();
        tc_before();
        __syncwarp();
        if (lane == 0) {
          bar_arrive(bar(bPFull + room));
          if (L::WIDE) bar_arrive(bar(bTold + 2 * X + (tiles & 1)));
        }
        ++tiles;
      }
      if (failed) break;
      unit += turns ? ntile : 2 * ntile;
      if (L::WIDE) other = before + (X ? (ntile + 1) / 2 : ntile / 2);
      if (first >= ntile) continue;                    // one tile in one half: nothing for B
      if (items > 0 && !wait(bOFree + X, items - 1)) break;      // the sums before were taken
      ++items;
      if (L::WIDE) {
        wide_sums[128 * X + r] = l;
        wide_sums[(((ntile - 1) & 1) == X ? 384 : 256) + r] = m;
      } else {
        sums[128 * X + r] = make_float2(l == 0.0f ? -INFINITY : m, l);       // M of nothing counts below every other
      }
      __syncwarp();
      if (lane == 0) bar_arrive(bar(bSums + X));
    }
  } else if (warp < 12) {
    // ---- results (or partials) of both halves, thread = row ---------------------------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsResults));
    const int wq = warp & 3, r = 32 * wq + lane;
    const uint32_t trow = tmem + (static_cast<uint32_t>(32 * wq) << 16);
    const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;   // whole sectors per store
    int nO0 = 0, nO1 = 0;                              // items of the halves
    for (int n = 0; !failed; ++n) {
      const ItemMsg it = next_item(n);
      if (!it.valid) break;
      const bool turns = it.rows <= half, joins = turns && it.ntile > 1;
#pragma unroll 1
      for (int X = 0; X < (turns ? 1 : 2); ++X) {
        const int rx = half * X + r, gr = it.r0 + rx, tok = gr / a.G, p = it.p0 + tok;
        const bool live = r < half && rx < it.rows;
        const uint32_t to = trow + col_o<D>(X);
        if (!wait(bSums + X, X ? nO1 : nO0) || !wait(bODone + X, X ? nO1 : nO0)) break;
        if (X) ++nO1;
        else ++nO0;
        if (joins) {
          if (!wait(bSums + 1, nO1) || (!L::WIDE && !wait(bODone + 1, nO1))) break;
          ++nO1;
        }
        tc_after();
        float2 mine = sums[128 * X + r];
        if (L::WIDE) {                                 // one O, by the M of the half that ends last
          const float* w = reinterpret_cast<const float*>(sm + P::SUMS);
          const int last = (it.ntile - 1) & 1;
          mine = make_float2(w[384 + r], w[128 * last + r]);
          const float l2 = joins ? w[128 * (last ^ 1) + r] : 0.0f;
          mine.y += l2 > 0.0f ? l2 * ex2(w[256 + r] - mine.x) : l2;
        }
        float m = mine.x, l = mine.y, fa = 1.0f, fb = 0.0f;
        if (joins && !L::WIDE) {
          const float2 other = sums[128 + r];
          m = fmaxf(mine.x, other.x);
          fa = m == -INFINITY ? 1.0f : ex2(mine.x - m);
          fb = m == -INFINITY ? 1.0f : ex2(other.x - m);
          l = fa * l + fb * other.y;
        }
        if (X == 0 && !wait(bChecked + n % kCheckRing, n / kCheckRing)) break;
        const bool odd = __any_sync(0xffffffffu, odd_of[n % kCheckRing] == n + 1);
        if (__builtin_expect(odd, 0)) {
          if (joins && !L::WIDE) {                     // (the sums first)
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              float o[16], o2[16];
              uint32_t u[16];
              tld16(to + 16u * c, o);
              tld16(trow + col_o<D>(1) + 16u * c, o2);
#pragma unroll
              for (int k = 0; k < 16; ++k) u[k] = __float_as_uint(fa * o[k] + fb * o2[k]);
              tst16(to + 16u * c, u);
            }
            tst_wait();
            fa = 1.0f;
          }
          add_odd_values<D>(to, static_cast<const __nv_bfloat16*>(a.v) + it.k0 * a.vs + static_cast<long long>(it.h) * D, a.vs, it.t0, it.ntile,
                            it.ns, it.w0, it.pmin, it.pmax, p, a.window, a.sinks);
        }
        const bool both = joins && !odd && !L::WIDE;
        const float inv = it.slot < 0 ? prompt_inverse(l, p) : 1.0f;
        fa *= inv;
        fb *= inv;
        const long long at = ((static_cast<long long>(it.q0) + tok) * a.Hq + it.h * a.G + (gr - tok * a.G)) * D;
        float* part = parts + (static_cast<long long>(it.slot) * L::ROWS + rx) * L::PART;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          tld32(to + 32u * c, o);
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] *= fa;
          if (both) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              float o2[16];
              tld16(trow + col_o<D>(1) + 32u * c + 16u * q, o2);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[16 * q + k] = fmaf(fb, o2[k], o[16 * q + k]);
            }
          }
          if (live && it.slot < 0) {
            uint32_t w[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) w[k] = bf16x2_bits(o[2 * k], o[2 * k + 1]);
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + at + 32 * c;
            if (wide) {
              stg256(dst, w);
              stg256(dst + 16, w + 8);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k) reinterpret_cast<uint4*>(dst)[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
            }
          } else if (live) {
            float4* dst = reinterpret_cast<float4*>(part + 4 + 32 * c);
#pragma unroll
            for (int k = 0; k < 8; ++k) dst[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
            if (c == 0) *reinterpret_cast<float4*>(part) = make_float4(l == 0.0f ? -INFINITY : m, l, 0.0f, 0.0f);
          }
          __syncwarp();                                // lanes with no row wait: the loads are the whole warp's
        }
        tc_before();                                   // the next item's products may overwrite what was read
        __syncwarp();
        if (lane == 0) {
          bar_arrive(bar(bOFree + X));
          if (joins) bar_arrive(bar(bOFree + 1));
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOthers));
    if (warp == 12) {
      // ---- items, queries, keys ---------------------------------------------------------------
      int n = 0, cq = 0, ck = 0;                       // items, and halves of queries and pieces of keys asked for
      int q_left = 0, q_head = 0, q_row = 0;           // halves of queries that are still to come, and where they stand
      auto publish = [&](const ItemMsg& x) {
        // Every warp has taken the one before.  If one has not within the limit, its room stays as it is, and the others'
        // waits for this one give up too.
        if (n >= kItems && !__all_sync(0xffffffffu, wait_short(bar(bItemFree + n % kItems), (n / kItems - 1) & 1))) {
          failed = true;
          return;
        }
        if (lane == 0) {
          item_ring[n % kItems] = x;
          bar_arrive(bar(bItem + n % kItems));
        }
        ++n;
      };
      PromptWalk<kTok, kItemCost> w;
      auto announce = [&]() {
        const PromptBlock& b = w.blk;
        publish(ItemMsg{1, w.h, b.seq.q0, b.r0, b.rows, b.seq.m - b.seq.n, b.pmin, b.pmax, w.t1 - w.t0, w.t0, w.slot, b.seq.k0, b.ns, b.w0, {0, 0}});
        q_left = b.rows <= half ? 1 : 2;
        q_head = w.h * a.G;
        q_row = b.seq.q0 + b.r0 / a.G;
      };
      // The halves of queries of the item that was announced last: ahead of time, as soon as a room is free (wait: all of
      // them now).
      auto queries = [&](bool now) {
        for (; q_left > 0 && !failed; --q_left, ++cq, q_row += half / a.G) {
          const int st = cq % L::QST;
          if (cq >= L::QST) {
            if (!now && !__all_sync(0xffffffffu, bar_poll(bar(bQFree + st), (cq / L::QST - 1) & 1))) return;
            if (now && !wait(bQFree + st, cq / L::QST - 1)) return;
          }
          if (lane == 0) {
            bar_arrive_tx(bar(bQFull + st), static_cast<uint32_t>(half) * 2 * D);
#pragma unroll
            for (int i = 0; i < D / 64; ++i) tma_rows(sb + L::Q + st * L::QX + 16384 * i, &mq, 64 * i, q_head, q_row, bar(bQFull + st));
          }
          __syncwarp();
        }
      };
      w.start(a, span, a.H, mode);
      bool more = w.next(a, span);
      while (!failed && more) {
        // The item's copies from what is kept of it here: the next one is looked up (and announced) behind the first of them.
        const PromptBlock b = w.blk;
        const int head = w.h, t0 = w.t0, t1 = w.t1;
        if (n == 0) announce();
        const int ahead = b.rows <= half ? 2 : 1;      // a tile's scores are issued so many steps before its values
        auto keys = [&](int t) {
          for (int i = 0; i < L::KCH; ++i, ++ck) {
            if (ck >= L::KST && !wait(bKFree + ck % L::KST, ck / L::KST - 1)) return;
            copy(&mk, sb + L::K + (ck % L::KST) * L::PIECE, 16384, 128 * i, head, b.seq.k0 + b.first_key<kTok>(t), bar(bKFull + ck % L::KST));
          }
        };
        // (the queries ahead of the second tile's keys, whose room may come free by the first one's scores)
        queries(false);
        keys(t0);
        if (!failed) queries(true);
        if (!failed && ahead == 2 && t0 + 1 < t1) keys(t0 + 1);
        if (failed) break;
        w.pass(a, span);
        more = w.next(a, span);
        if (more) announce();
        else publish(ItemMsg{});
        for (int t = t0 + ahead; t < t1 && !failed; ++t) {
          queries(false);
          keys(t);
        }
      }
      if (n == 0 && !failed) publish(ItemMsg{});       // no item at all
      if (mode == kPromptCut && lane == 0) splits[blockIdx.x] = w.cut;
      // copies still in flight land before the CTA ends
      bool f2 = false;
      for (int s = cq >= L::QST ? cq - L::QST : 0; s < cq; ++s) (void)bar_wait(bar(bQFull + s % L::QST), (s / L::QST) & 1, f2);
      for (int s = ck >= L::KST ? ck - L::KST : 0; s < ck; ++s) (void)bar_wait(bar(bKFull + s % L::KST), (s / L::KST) & 1, f2);
    } else if (warp == 13) {
      // ---- MMA issue, the warp converged: O += w V of a half's tile, then the scores of a later one, in strict order of the
      // halves (left to mix, both halves' MMAs would end together and neither softmax overlap the other).  Between a
      // softmax's end and its next scores stands what this warp executes in between, so that few instructions count: with
      // a loop per kind of item, a queue in registers and rings by division a d = 64 prompt of 8,192 took 279 us, not 256,
      // and two dozen d = 128 prompts 341, not 309 (in a burst) -------------------------------------------------------------------------
      auto ready = [&](int i, int phase) {             // wait() in few instructions
        if (__all_sync(0xffffffffu, wait_short(bar(i), phase & 1))) return true;
        failed = true;
        return false;
      };
      // A unit is a half's tile; units have the rooms of S in turn.  The scores are SB units ahead of the values, over items.
      int n = 0, no0 = 0, no1 = 0;                     // items taken; items of the halves (their O)
      Ring<L::QST> queries;                            // halves of queries
      Ring<L::KST> keys_at;                            // pieces of keys and of values
      Ring<L::VST> values_at;
      Ring<L::SB> scores_a, scores_b, weights_at;      // tiles of A, of B; units
      // items between the scores and the values: 2 * units + two, 0 for the end
      volatile int* queue = reinterpret_cast<volatile int*>(sm + P::QUEUE);
      // the scores' item: its units, the next of them, its first half of queries
      int units = 0, su = 0;
      Ring<L::QST> qa;
      bool two = false;                                // rows in half B
      auto take = [&]() {
        const ItemMsg x = next_item(n);
        const bool open = __all_sync(0xffffffffu, x.valid) && !failed;
        two = open && __all_sync(0xffffffffu, x.rows > half);
        units = uniform(open ? (two ? 2 * x.ntile : x.ntile) : 0);
        su = 0;
        qa = queries;
        if (open) queries.next();
        if (two) queries.next();
        queue[n % 4] = 2 * units + (two ? 1 : 0);      // (every lane the same)
        __syncwarp();
        ++n;
      };
      take();
      // The scores of the next unit, if there is one.
      auto scores = [&](uint32_t to) {
        if (!units) return true;
        const bool b = su & 1, second = two && b;
        Ring<L::QST> qi = qa;
        if (second) qi.next();
        if (!second)                                   // (a tile's pieces have one phase)
          for (int i = 0; i < L::KCH; ++i)
            if (!ready(bKFull + keys_at.place() + i, keys_at.phase())) return false;
        if (su <= (two ? 1 : 0) && !ready(bQFull + qi.place(), qi.phase())) return false;
        tc_after();
        const uint64_t q = sdesc(sb + L::Q + qi.place() * L::QX);
        auto keys = [&](int i) { return sdesc(sb + L::K + (keys_at.place() + i) * L::PIECE); };
        if (D == 64) {
          mma4_scores(to, q, keys(0), idesc_bf16(128));
        } else {
          mma8_scores<0>(to, q, keys(0), idesc_bf16(128));
          if (L::WIDE) mma8_scores<1>(to, q + (32768 >> 4), keys(1), idesc_bf16(128));
        }
        mma_commit_warp(bar(bSFull + (b ? L::SB + scores_b.place() : scores_a.place())));
        if (b) scores_b.next();
        else scores_a.next();
        if (!two || b)
          for (int i = 0; i < L::KCH; ++i, keys_at.next()) mma_commit_warp(bar(bKFree + keys_at.place()));
        su += 1;
        if (su + (two ? 1 : 0) >= units) mma_commit_warp(bar(bQFree + qi.place()));
        if (su == units) take();
        return !failed;
      };
      auto values_done = [&]() {
        mma_commit_warp(bar(bVFree + values_at.place()));
        values_at.next();
      };
      auto values_there = [&]() { return ready(bVOk + values_at.place(), values_at.phase()); };
      bool ok = !failed;
      for (int i = 0; i < L::SB && ok; ++i) ok = scores(tmem + 128u * i);
      for (int vn = 0; ok; ++vn) {
        const int word = uniform(queue[vn % 4]), vunits = word >> 1;
        const bool vtwo = word & 1;
        if (!word) break;
        for (int vu = 0; vu < vunits; ++vu, weights_at.next()) {
          const uint32_t X = vu & 1;
          const uint32_t w = tmem + 128u * static_cast<uint32_t>(weights_at.place());
          if (!(vtwo && X)) ok = values_there();
          if (ok && vu < (L::WIDE ? 1 : 2)) {          // O of the half is free: the item before it was taken from there
            const int k = X ? no1++ : no0++;
            ok = k == 0 || ready(bOFree + X, k - 1);
          }
          const uint32_t first = vu < (L::WIDE ? 1 : 2) ? 0u : 1u;
          const uint64_t v = vdesc(sb + L::V + values_at.place() * L::PIECE);
          ok = ok && ready(bPFull + weights_at.place(), weights_at.phase());
          if (!ok) break;
          tc_after();
          if (!L::WIDE) {
            mma8_values(tmem + col_o<D>(X), w, v, idesc_bf16(D) | (1u << 16), first);
            if (L::SB > 2) mma_commit_warp(bar(bProducts + X));
          } else {                                     // 64 tokens a piece: panels 8 KB apart
            auto desc = [&]() { return vdesc(sb + L::V + values_at.place() * L::PIECE) - (static_cast<uint64_t>((16384 - 8192) >> 4) << 16); };
            mma4_values(tmem + col_o<D>(0), w, desc(), idesc_bf16(D) | (1u << 16), first);
            values_done();
            ok = values_there();
            if (!ok) break;
            tc_after();
            mma4_values(tmem + col_o<D>(0), w + 32u, desc(), idesc_bf16(D) | (1u << 16), 1u);
            mma_commit_warp(bar(bProducts + X));
          }
          if (!vtwo || X) values_done();
          if (L::WIDE ? vu == vunits - 1 : vu + 2 >= vunits) mma_commit_warp(bar(bODone + (L::WIDE ? 0 : X)));
          ok = scores(w);
          if (!ok) break;
        }
      }
      mma_commit_warp(bar(bDrain));                    // every MMA issued completes before the CTA ends
      bool f2 = false;
      (void)bar_wait(bar(bDrain), 0, f2);
      __syncwarp();
    } else if (warp == 14) {
      // ---- the values of tiles that some row does not see in full: what is not finite is taken out ----------------------
      int cv = 0;
      for (int n = 0;; ++n) {
        const ItemMsg it = next_item(n);
        if (!it.valid) break;
        const int ntile = it.ntile;
        bool any = false;
        for (int i = 0; i < ntile * L::VCH; ++i, ++cv) {
          if (!wait(bVFull + cv % L::VST, cv / L::VST)) break;
          if (!it.full(it.first_key(i / L::VCH), a.window, a.sinks)) {
            const uint32_t at = sb + L::V + (cv % L::VST) * L::PIECE + lane * 16;
            uint32_t most = 0u;                        // largest magnitudes: bf16 bits order as integers
#pragma unroll 1
            for (int k0 = 0; k0 < L::PIECE; k0 += 512 * 8) {
              uint4 v[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) v[k] = lds128(at + k0 + 512 * k);
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                most = __vmaxu2(__vmaxu2(most, v[k].x & 0x7FFF7FFFu), v[k].y & 0x7FFF7FFFu);
                most = __vmaxu2(__vmaxu2(most, v[k].z & 0x7FFF7FFFu), v[k].w & 0x7FFF7FFFu);
              }
            }
            if (__any_sync(0xffffffffu, odd_pair(most))) {
              any = true;
#pragma unroll 1
              for (int k0 = 0; k0 < L::PIECE; k0 += 512) {
                const uint4 v = lds128(at + k0);
                uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  if ((u[q] & 0x7F80u) == 0x7F80u) u[q] &= 0xFFFF0000u;
                  if ((u[q] & 0x7F800000u) == 0x7F800000u) u[q] &= 0xFFFFu;
                }
                sts128(at + k0, u[0], u[1], u[2], u[3]);
              }
              fence_async_smem();
            }
          }
          __syncwarp();
          if (lane == 0) bar_arrive(bar(bVOk + cv % L::VST));
        }
        if (failed) break;
        if (lane == 0) {
          if (any) odd_of[n % kCheckRing] = n + 1;
          bar_arrive(bar(bChecked + n % kCheckRing));
        }
        __syncwarp();
      }
    } else {
      // ---- values ---------------------------------------------------------------------------
      int cv = 0;
      for (int n = 0; !failed; ++n) {
        const ItemMsg it = next_item(n);
        if (!it.valid) break;
        const int ntile = it.ntile;
        for (int t = 0; t < ntile && !failed; ++t)
          for (int i = 0; i < L::VCH; ++i, ++cv) {
            if (cv >= L::VST && !wait(bVFree + cv % L::VST, cv / L::VST - 1)) break;
            copy(&mv, sb + L::V + (cv % L::VST) * L::PIECE, 128 * L::VTOK, 0, it.h, it.k0 + it.first_key(t) + i * L::VTOK, bar(bVFull + cv % L::VST));
          }
      }
      // copies still in flight land before the CTA ends
      bool f2 = false;
      for (int s = cv >= L::VST ? cv - L::VST : 0; s < cv; ++s) (void)bar_wait(bar(bVFull + s % L::VST), (s / L::VST) & 1, f2);
    }
  }
  if (failed && lane == 0) atomicOr(a.err, kErrTimeout);
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 13) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {        // from the driver, looked up once
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}
// Rows of queries, keys or values: coordinates (channel, head, row), boxes of 64 channels of some heads and rows.
bool rows_map(CUtensorMap* map, const void* p, int d, int heads, long long rows, long long stride, int box_heads, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_t(const PromptArgs& args, cudaStream_t s) {
  using L = PG<D>;
  PromptArgs a = args;
  const int tokens = 128 / a.G;                        // of a half
  a.rows = L::HALVES * tokens * a.G;
  a.most = prompt_list_room(a, kTok, kItemCost);
  CUtensorMap mq, mk, mv;
  if (!rows_map(&mq, a.q, D, a.Hq, a.total_q, a.qs, a.G, tokens) || !rows_map(&mk, a.k, D, a.H, a.total_k, a.ks, 1, kTok) ||
      !rows_map(&mv, a.v, D, a.H, a.total_k, a.vs, 1, L::VTOK))
    return cudaErrorInvalidValue;
  static std::atomic<unsigned long long> configured{0};
  cudaError_t e = smem_attr_once(prompt_tc_kernel<D>, PS<D>::BYTES, configured);
  if (e != cudaSuccess) return e;
  const long long items = prompt_most_blocks(a) * a.H, tiles = a.max_k / kTok + 2 + a.sinks / kTok;
  // items of few tiles are not cut (and need no join)
  // (nor are few of them listed: the list takes 4 us)
  const int sms = prompt_sms();
  const int mode = !prompt_splits(a) || (tiles <= 4 && items <= sms) ? kPromptTurns : tiles > 4 ? kPromptCut : kPromptWhole;
  const long long most = mode == kPromptCut ? (items * (tiles + kItemCost) + kMinSpan - 1) / kMinSpan : items;
  const int ctas = static_cast<int>(most < sms ? (most < 1 ? 1 : most) : sms);
  e = launch_pdl(prompt_tc_kernel<D>, dim3(ctas), dim3(kThreads), PS<D>::BYTES, s, a, mq, mk, mv, mode);
  if (e != cudaSuccess || mode != kPromptCut) return e;
  return launch_prompt_join(a, D, false, ctas, L::ROWS, s);
}

}  // namespace

bool prompt_tc_takes(const PromptArgs& a, int d, bool f32) {
  return !f32 && (d == 64 || d == 128 || d == 256) && a.G <= 128 && a.scale_log2 > 0.0f && a.total_k > 0;
}

size_t prompt_tc_workspace(int d) {
  const int rows = d == 256 ? 128 : 256;
  return static_cast<size_t>(prompt_sms()) * (sizeof(PSplit) + 2 * sizeof(float) * rows * (d + 4));
}

cudaError_t launch_prompt_tc(const PromptArgs& a, int d, cudaStream_t s) {
  switch (d) {
    case 64: return launch_t<64>(a, s);
    case 128: return launch_t<128>(a, s);
    case 256: return launch_t<256>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace tq
