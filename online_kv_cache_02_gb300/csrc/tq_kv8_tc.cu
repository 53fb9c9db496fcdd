// Attention of many query rows per KV head over the 8-bit paged cache on the tensor
// cores (tcgen05), bf16 queries, d = 64, 128 or 256.
//
// An item is (sequence, KV head, block of 256 query rows r = t G + g); keys go by in
// tiles of 128 tokens (8 pages).  All items' tiles form one list that is cut into
// equal spans, one per CTA; the parts of an item that crosses spans are joined by a
// second kernel.  Per tile:
//   S = (Qh + Ql) Kc^T    kind::f8f6f4 straight from the cache's codes, which TMA
//                         puts in place: no conversion of K.  A query row, scaled
//                         by a power of two, is the sum of two e4m3 parts: exact
//                         for bf16 down to 2^-10 of the row's largest value, off
//                         by at most 2^-17 of it below;
//   w = 2^(f S + ev - M)  f = scale log2(e) 2^ek 2^-row per page, ev the page's
//                         value exponent, M the row's running maximum (moved only
//                         when passed by 2^8): block scales cost no instruction
//                         beyond the softmax's own multiply-add;
//   O += w Vc             w as fp16 in tensor memory, Vc as fp16 (exact), turned
//                         from codes by four warps, token rows read MN-major;
//   l += w 2^-ev,  out = O / l.
//
// Two 128-row halves A and B of the block take turns: while the softmax of one
// runs, the tensor cores work on the other.  Tensor memory: S of A and B (each
// overlaid by its weights), O of A and B, 512 columns.  Warps 0-3 and 4-7: the
// softmax of A and B (thread = row), which also split the queries and write the
// results; 8-11: values to fp16; 12: items, pages and the keys' copies; 13: MMA issue;
// 14: the values' copies (a copy per page costs its warp about 100 cycles, a tile of
// keys and values more than the MMAs of twenty rows); 15: queries to L2.
// An item of at most 128 rows (drafted tokens, decode with many heads per KV head) has
// its rows in both halves: A takes the even tiles, B the odd ones, and A adds B's sums
// to its own at the item's end, from B's columns of the same lanes.
// Every wait is bounded; a wait that gives up sets the device error word.
//
// Bound by the tensor cores and the halves' turns behind them: the MMAs of a tile of 256
// rows take 2,048 cycles (two e4m3 products at the rate of one fp16 product, then one
// fp16 product), and over a whole call a tile takes 2,920 in a chunk behind a long cache
// and 3,180 in a prompt of 8,192 tokens (the tensor pipe is active 70% and 64% of the
// time), items' starts and ends among them.  Measured, bf16, d = 128, 32 / 8 heads: a
// prompt of 8,192 tokens 402 us, 1.37 PFLOP/s, 71% of a large bf16 library product's
// rate; 2 x 1,024 tokens behind 15,000 to 30,000, 482 us, 76%; three prompts of up to
// 4,000 in a window of 1,024 (28 / 4 heads) 167 us, 43%, where an item of nine tiles pays
// for its queries and its result with the time of four; five drafted tokens of 16
// sequences of 2,000 to 8,000, 54 us, 45% of a copy's rate (MMAs of 128 rows of which 20
// are there).  d = 64, 32 / 8 heads, a prompt of 4,096 tokens 119 us, of 8,192 350 (41%:
// as many weights for half the products).  d = 256, 16 / 4 heads, 2,048 tokens 81 us
// (mma.sync: 618), 8,192 615 (46%).
// Slower, each by itself: 64-token tiles in two buffers, sixteen softmax warps, two
// issuing warps, the queries' copies beside the last tile (from the softmax warps or
// a warp of their own: code in the tile loop, or a copy slower than four warps').

#include "tq_kv8.h"
#include "tq_tc.cuh"

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>

namespace tq {
namespace {

using namespace tcx;

constexpr int kTTok = 128;                // tokens per tile
constexpr int kTPg = kTTok / kPage;       // pages per tile
constexpr int kTThreads = 512;
constexpr int kItems = 4;                 // items announced ahead
constexpr float kMNone = -3.0e38f;         // a maximum before any score: finite, and below the scores of fp32
// Weights are 2^(kLift + score - M).  M is set kHead above the largest score met, so that it seldom moves again: the
// largest weight is then 2^3, and fp16 keeps 11 bits down to 2^-17 of it.  M moves when a page's 16 weights sum to more
// than kFull, below the end of fp16: the largest of them is then 2^11.9 at least, a score above M + kSlack.
constexpr float kSlack = 4.5f, kLift = 7.0f, kHead = 4.0f, kFull = 61000.0f;
// M adds an exponent to a score, which one fp32 number holds up to some size (at scores of 2^27 the weights were past fp16
// or 0).  Beyond kBig a row's M is a score, and an exponent, a whole number in [-96, 123], beside it.
constexpr float kBig = 65536.0f;
constexpr int kMaxBlocks = 2048;          // (sequence, query block) pairs that the split form lists
constexpr int kItemCost = 5;              // an item's start and end, in tiles' time
constexpr int kMinSpan = 2 + kItemCost;   // a CTA's share of the list at least
constexpr int kNoPage = 1 << 30;          // first position of a page that is not there: no query sees it

struct TileDesc {                         // one tile of the stream, by page
  float fac[kTPg];                        // scale log2(e) 2^ek
  float ev[kTPg];                         // value exponent
  float vinv[kTPg];                       // 2^-ev
  int j0[kTPg];                           // first position
  int blk[kTPg];                          // block of the cache; -1: not there
  int full, pad[3];                       // every row of the block sees every token
};

constexpr int kDoneRing = 8;
enum Bar {                                // room for the most stages that a head dimension has
  bKFull = 0, bKFree = bKFull + 3, bVFull = bKFree + 2, bVEmpty = bVFull + 3, bReady = bVEmpty + 3, bSFull = bReady + 2,
  bPFull = bSFull + 2, bODone = bPFull + 2, bQReady = bODone + 2, bQFree = bQReady + 2, bItem = bQFree + 1,
  bItemFree = bItem + kItems, bDesc = bItemFree + kItems, bDone = bDesc + 8, bJoin = bDone + kDoneRing, bOFree, bDrain, bCount
};

// Shared memory by head dimension.  It has no room to be moved up to a 1024-byte boundary (the swizzles' period): the
// kernel's only shared memory starts on one, and the kernel checks that.
// d = 256 (WIDE): an item is 128 rows and one half of the values' channels, the scores of both halves are the same work
// twice (of 3,072 cycles a tile a third, but queries, keys and values of 256 rows and channels would not fit); the
// halves A and B share the queries.
template <int D>
struct TG {
  static constexpr bool WIDE = D == 256;
  static constexpr int ROWS = WIDE ? 128 : 256;        // query rows per item
  static constexpr int DV = WIDE ? 128 : D;            // value channels per item
  static constexpr int PER = D / DV;                   // items per KV head and block of rows
  static constexpr int KST = WIDE ? 2 : 3, VST = KST;  // stages of keys and of raw values
  static constexpr int DESCS = WIDE ? 4 : 8;           // tiles announced ahead
  static constexpr int KT = kTTok * D, VRT = kTTok * DV, VT = 2 * VRT;   // a tile's keys, values, and values as fp16
  static constexpr int QX = 128 * 2 * D;               // 128 rows' queries, both parts
  static constexpr int QB = WIDE ? 0 : QX;             // from half A's queries to half B's
  static constexpr int PART = DV + 4;                  // floats of a row's partial
  static constexpr int Q = 0;                          // [A, B] halves, see qpos
  static constexpr int K = Q + QX + QB;                // [stage][128-channel panels][128 tokens][128 B] (64 at d = 64)
  static constexpr int VR = K + KST * KT;              // [stage][128 tokens][DV B]
  static constexpr int V = VR + VST * VRT;             // [buffer][64-channel blocks][128 tokens][128 B]
  static constexpr int DESC = V + 2 * VT;
  static constexpr int ITEM = DESC + DESCS * static_cast<int>(sizeof(TileDesc));
  static constexpr int BAR = ITEM + kItems * 48;
  static constexpr int JOIN = BAR + 8 * ((bCount + 1) & ~1);     // half B's (M, l) of 128 rows
  static constexpr int ROWF = JOIN + 1024;             // WIDE: the rows' scales, from half A to half B
  static constexpr int END = ROWF + (WIDE ? 512 : 0);
  // Piece c (sixteen channels) of part hi (0) or lo (1) of a row, in rows of 128 bytes with the 128-byte swizzle: the
  // parts have a tile per 128 channels each, at d = 64 a row holds both.
  __device__ static __forceinline__ uint32_t qpos(int row, int c, int part) {
    return D == 64 ? static_cast<uint32_t>(row * 128 + (((c + 4 * part) ^ (row & 7)) << 4))
                   : static_cast<uint32_t>(part * (QX / 2) + (c >> 3) * 16384 + row * 128 + (((c & 7) ^ (row & 7)) << 4));
  }
  // 16-byte piece c of a token's value codes as TMA swizzled them.
  __device__ static __forceinline__ uint32_t vpos(int t, int c) {
    return static_cast<uint32_t>(t * DV + ((c ^ (DV == 128 ? t & 7 : (t >> 1) & 3)) << 4));
  }
};
template <int D>
constexpr int tmem_at() { return TG<D>::END; }
template <int D>
constexpr int smem_bytes() { return tmem_at<D>() + 16; }
static_assert(smem_bytes<128>() <= 232448 && smem_bytes<256>() <= 232448, "shared memory per block");
static_assert(sizeof(TileDesc) % 16 == 0, "items behind the descriptors");
// tensor-memory columns of half X
__device__ __forceinline__ constexpr uint32_t col_s(uint32_t X) { return 128u * X; }
__device__ __forceinline__ constexpr uint32_t col_o(uint32_t X) { return 256u + 128u * X; }

// Eight MMAs in one statement, one elected lane: the issuing warps share their schedulers with the softmax, so that
// every instruction between two MMAs counts.  S = Qh Kc^T + Ql Kc^T: four steps of 32 channels (32 B, 2 descriptor
// units) each; ACC: on top of what is there.
template <int ACC>
__device__ __forceinline__ void mma8_scores(uint32_t d, uint64_t qh, uint64_t ql, uint64_t k, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred e, t, f;\n .reg .b64 h1, h2, h3, l1, l2, l3, k1, k2, k3;\n"
      " add.u64 h1, %1, 2;\n add.u64 h2, %1, 4;\n add.u64 h3, %1, 6;\n"
      " add.u64 l1, %2, 2;\n add.u64 l2, %2, 4;\n add.u64 l3, %2, 6;\n"
      " add.u64 k1, %3, 2;\n add.u64 k2, %3, 4;\n add.u64 k3, %3, 6;\n"
      " setp.ne.b32 t, 1, 0;\n setp.ne.b32 f, %5, 0;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %3, %4, f;\n"
      " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], h1, k1, %4, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], h2, k2, %4, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], h3, k3, %4, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %2, %3, %4, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], l1, k1, %4, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], l2, k2, %4, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], l3, k3, %4, t;\n}\n" ::"r"(d),
      "l"(qh), "l"(ql), "l"(k), "r"(idesc), "n"(ACC)
      : "memory");
}
// The same at d = 64: two steps each, the query's parts side by side in a row.
__device__ __forceinline__ void mma4_scores(uint32_t d, uint64_t q, uint64_t k, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred e, t, f;\n .reg .b64 q1, q2, q3, k1;\n"
      " add.u64 q1, %1, 2;\n add.u64 q2, %1, 4;\n add.u64 q3, %1, 6;\n add.u64 k1, %2, 2;\n"
      " setp.ne.b32 t, 1, 0;\n setp.ne.b32 f, 0, 0;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, f;\n"
      " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], q1, k1, %3, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], q2, %2, %3, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], q3, k1, %3, t;\n}\n" ::"r"(d),
      "l"(q), "l"(k), "r"(idesc)
      : "memory");
}
// O (+)= w V: eight steps of 16 tokens (8 columns of weights, 2048 B or 128 descriptor units of values).
__device__ __forceinline__ void mma8_values(uint32_t d, uint32_t w, uint64_t v, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred e, t, p;\n .reg .b32 w1, w2, w3, w4, w5, w6, w7;\n .reg .b64 v1, v2, v3, v4, v5, v6, v7;\n"
      " add.u32 w1, %1, 8;\n add.u32 w2, %1, 16;\n add.u32 w3, %1, 24;\n add.u32 w4, %1, 32;\n add.u32 w5, %1, 40;\n"
      " add.u32 w6, %1, 48;\n add.u32 w7, %1, 56;\n"
      " add.u64 v1, %2, 128;\n add.u64 v2, %2, 256;\n add.u64 v3, %2, 384;\n add.u64 v4, %2, 512;\n"
      " add.u64 v5, %2, 640;\n add.u64 v6, %2, 768;\n add.u64 v7, %2, 896;\n"
      " setp.ne.b32 p, %4, 0;\n setp.ne.b32 t, 1, 0;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [w1], v1, %3, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [w2], v2, %3, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [w3], v3, %3, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [w4], v4, %3, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [w5], v5, %3, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [w6], v6, %3, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [w7], v7, %3, t;\n}\n" ::"r"(d),
      "r"(w), "l"(v), "r"(idesc), "r"(acc)
      : "memory");
}
// kind::f8f6f4, fp32 accumulate, e4m3 A and B, K-major, M = 128, N = 128
constexpr uint32_t kIdF8 = (1u << 4) | (static_cast<uint32_t>(kTTok >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
// e4m3 rows of D bytes, K-major with a swizzle of their length, in groups of eight
template <int D>
__device__ __forceinline__ uint64_t kdesc8(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (1ull << 16) | (static_cast<uint64_t>(8 * D >> 4) << 32) |
         (1ull << 46) | ((D == 128 ? 2ull : 4ull) << 61);
}
// MN-major operand, 128-byte swizzle: token rows of 64 channels, 8-row groups 1024 B apart, channel halves 16 KB apart
__device__ __forceinline__ uint64_t vdesc(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(16384 >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// One block's panel of (at most) 128 channels from channel x on.
__device__ __forceinline__ void tma_block(uint32_t dst, const CUtensorMap* map, int x, int blk, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(0), "r"(blk), "r"(bar)
      : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t codes_to_half2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<unsigned short>(two)));
  return r;
}
__device__ __forceinline__ uint32_t half2_to_codes(uint32_t h2) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h2));
  return r;
}
__device__ __forceinline__ uint32_t sub_half2(uint32_t x, uint32_t y) {
  const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// Pairs of fp32 in one 64-bit register (Blackwell's packed fp32 arithmetic).
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// 128 columns of this thread's lane: four loads in flight, one wait.  The values pass through an empty statement
// behind the wait, so that nothing uses them before it.
__device__ __forceinline__ void tld32_start(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr));
}
__device__ __forceinline__ void pin8(float* v) {
  asm volatile("" : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]));
}
__device__ __forceinline__ void tld32x4(uint32_t taddr, float (&v)[128]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) tld32_start(taddr + 32u * i, v + 32 * i);
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) pin8(v + 8 * i);
}
// A bounded wait in few instructions, for the issuing warp: the tensor pipe's queue is short, and between two batches
// of MMAs every instruction of the wait is a gap in it.
__device__ __forceinline__ uint32_t wait_short(uint32_t b, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .u32 n;\n mov.u32 n, %3;\n"
      "W%=:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra D%=;\n"
      " sub.u32 n, n, 1;\n setp.ne.u32 q, n, 0;\n @q bra W%=;\nD%=:\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(b), "r"(parity), "n"(kWaitS)
      : "memory");
  return done;
}

// A value that is the same in the whole warp, by a reduction: its result is a uniform register, and so is what follows
// from it (the MMAs' operands, so that no issue waits for moves).
__device__ __forceinline__ int uniform(int v) {       // v >= 0
  return static_cast<int>(__reduce_max_sync(0xffffffffu, static_cast<unsigned>(v)));
}

__device__ __forceinline__ void stg256(void* p, const uint32_t* v) {   // 32-byte aligned
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
               "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// A block of query rows of one sequence, and the pages that it sees.
struct TBlock {
  int b, qb, p0, rows;                    // sequence, block, the sequence's first query position, rows of the block
  int pmin, pmax;
  Kv8Range r;
  int pages;
};
// Block `e` of the list (sequence by sequence); its tiles, 0 if there is nothing to do.  In the list an item takes
// kItemCost units, then one per tile.
template <int ROWS>
__device__ __forceinline__ int tc_block(const Kv8Attn& a, int e, int nqb, TBlock& k) {
  k.b = e / nqb;
  k.qb = e - k.b * nqb;
  const Kv8Seq s = kv8_seq(a, k.b);
  const int rows = s.n * a.G, r0 = k.qb * ROWS;      // the host keeps batch T Hq below 2^27
  k.p0 = s.p0;
  k.rows = min(rows - r0, ROWS);
  k.pages = 0;
  if (k.rows <= 0) return 0;
  k.pmin = s.p0 + r0 / a.G;
  k.pmax = s.p0 + (r0 + k.rows - 1) / a.G;
  k.r = kv8_range(a.window, a.sinks, k.pmin, k.pmax);
  k.pages = k.r.ns + k.r.nw;
  return (k.pages + kTPg - 1) / kTPg;
}
// What the load warp tells the others of an item: a block, a KV head, and a run of its tiles.
struct alignas(16) ItemMsg {
  int valid, b, h, qb;                    // h: item of the block (KV head, at d = 256 with a half of the values' channels)
  int p0, rows, pmin, pmax;
  int ntile, slot, pad[2];                // slot: of the workspace for a part of the tiles; -1 for all of them
};
// A split item's first part ends the span of one CTA; the join finds the others by it.
struct TSplit {
  int valid, b, h, qb, p0, rows, last, pad;            // last: the CTA that holds the item's end
};

// A score's factor: never zero (a hidden score stays -inf) nor infinite (a score of zero stays zero), and NaN stays NaN.
__device__ __forceinline__ float score_factor(float fac, float rowf) {
  return fminf(fmaxf(fac * rowf, 1.2e-38f), 3.4028234e38f) + (rowf - rowf);
}
// Slots of the page at position j0 that a query at p sees.
__device__ __forceinline__ uint32_t page_seen(int p, int j0, int window, int sinks) {
  const int hi = p - j0;                               // up to hi
  uint32_t see = hi < 0 ? 0u : hi >= 15 ? 0xFFFFu : (2u << hi) - 1u;
  if (window) {
    const int lo = hi - window + 1, sk = sinks - j0;   // from lo on, or below sk
    const uint32_t win = lo <= 0 ? 0xFFFFu : lo > 15 ? 0u : 0xFFFFu << lo;
    const uint32_t snk = sk <= 0 ? 0u : sk > 15 ? 0xFFFFu : (1u << sk) - 1u;
    see &= win | snk;
  }
  return see;
}
template <int DV>
__device__ __forceinline__ void rescale_o(uint32_t to, float alpha) {
#pragma unroll 1
  for (int c = 0; c < DV / 16; ++c) {
    float o[16];
    uint32_t u[16];
    tld16(to + 16u * c, o);
#pragma unroll
    for (int k = 0; k < 16; ++k) u[k] = __float_as_uint(o[k] * alpha);
    tst16(to + 16u * c, u);
  }
}
// One tile's weights of a thread's row with M in two parts (m and me), by differences from it: the scores are rounded
// before they are compared, so that small differences are exact.  full: the row sees every token; accumulated: O holds
// tiles before.  Returns the two parts and l.  A function of its own: in the tile loop it cost five drafted tokens 54.4 us
// instead of 53.5, a prompt of 2,048 tokens at d = 256 82.8 instead of 78.6.
template <int DV>
__device__ __noinline__ float3 large_scores(uint32_t ts, uint32_t to, const TileDesc& d, bool full, int p, int window, int sinks,
                                            float rowf, bool accumulated, float m, float me, float l) {
  auto scores = [&](int c, float (&y)[32]) {           // of pages 2c and 2c + 1
    tld32(ts + 32u * c, y);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int pg = 2 * c + q;
      const uint32_t see = full ? 0xFFFFu : page_seen(p, d.j0[pg], window, sinks);
      const float f = score_factor(d.fac[pg], rowf);
#pragma unroll
      for (int k = 0; k < 16; ++k) y[16 * q + k] = (see >> k) & 1u ? __fmul_rn(y[16 * q + k], f) : -INFINITY;
    }
    __syncwarp();
  };
  float y[32], ref = m, top = -INFINITY, alpha = 1.0f;
#pragma unroll 1
  for (int c = 0; c < kTPg / 2; ++c) {
    scores(c, y);
#pragma unroll
    for (int k = 0; k < 32; ++k) ref = fmaxf(ref, y[k]);
  }
#pragma unroll 1
  for (int c = 0; c < kTPg / 2; ++c) {
    scores(c, y);
#pragma unroll
    for (int k = 0; k < 32; ++k) top = fmaxf(top, y[k] - ref + d.ev[2 * c + (k >> 4)]);
  }
  if (top > m - ref + me + kSlack) {
    const bool two = fabsf(ref) > kBig;
    const float mn = two ? ref : ref + (top + kHead), en = two ? ceilf(top + kHead) : 0.0f;
    alpha = ex2((m - mn) + (me - en));
    m = mn;
    me = en;
  }
  __syncwarp();
  l *= alpha;
  if (accumulated) rescale_o<DV>(to, alpha);
#pragma unroll 1
  for (int c = 0; c < kTPg / 2; ++c) {                 // (the weights overlay scores that were read)
    uint32_t w[16];
    scores(c, y);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float more = d.ev[2 * c + q] - me + kLift;
      float sum = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float y0 = ex2(__fsub_rn(y[16 * q + 2 * k], m) + more), y1 = ex2(__fsub_rn(y[16 * q + 2 * k + 1], m) + more);
        sum += y0 + y1;
        w[8 * q + k] = half2_bits(y0, y1);
      }
      l = fmaf(sum, d.vinv[2 * c + q], l);
    }
    tst16(ts + 16u * c, w);
  }
  return make_float3(m, me, l);
}

template <int D>
__global__ void __launch_bounds__(kTThreads, 1)
    kv8_tc_kernel(const __grid_constant__ Kv8Attn a, const __grid_constant__ CUtensorMap mk,
                  const __grid_constant__ CUtensorMap mv, int nqb, int split) {
  using L = TG<D>;
  extern __shared__ __align__(1024) unsigned char sm_raw[];
  unsigned char* sm = sm_raw;
  const uint32_t sb = su32(sm);
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  auto bar = [&](int i) { return sb + L::BAR + 8u * static_cast<uint32_t>(i); };
  TileDesc* descs = reinterpret_cast<TileDesc*>(sm + L::DESC);
  ItemMsg* item_ring = reinterpret_cast<ItemMsg*>(sm + L::ITEM);
  TSplit* splits = reinterpret_cast<TSplit*>(a.part);              // one per CTA, then the partials' slots
  if (sb & 1023u) {
    pdl_wait();
    if (tid == 0) {
      atomicOr(a.err, kErrLayout);
      if (split) splits[blockIdx.x].valid = 0;
    }
    return;
  }

  if (tid == 0) {
    for (int i = 0; i < L::KST; ++i) bar_init(bar(bKFull + i), 1);
    for (int i = 0; i < 2; ++i) bar_init(bar(bKFree + i), 1);
    bar_init(bar(bQFree), 4);
    for (int i = 0; i < L::VST; ++i) {
      bar_init(bar(bVFull + i), 1);
      bar_init(bar(bVEmpty + i), 4);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(bar(bReady + i), 4);
      bar_init(bar(bSFull + i), 1);
      bar_init(bar(bPFull + i), 4);
      bar_init(bar(bODone + i), 1);
      bar_init(bar(bQReady + i), 4);
    }
    for (int i = 0; i < kDoneRing; ++i) bar_init(bar(bDone + i), 1);
    bar_init(bar(bJoin), 4);
    bar_init(bar(bOFree), 4);
    for (int i = 0; i < L::DESCS; ++i) bar_init(bar(bDesc + i), 1);
    for (int i = 0; i < kItems; ++i) {
      bar_init(bar(bItem + i), 1);
      bar_init(bar(bItemFree + i), 15);                // every warp but the one that announces
    }
    bar_init(bar(bDrain), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 13) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sb + tmem_at<D>()), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  if (split) pdl_trigger();                            // the join's launch
  if (a.decode) {                                      // a sequence that is empty: zeros
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
      if (kv8_seq(a, b).n > 0) continue;
      uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + static_cast<long long>(b) * a.Hq * D);
      for (long long i = tid; i < static_cast<long long>(a.Hq) * (D / 8); i += kTThreads) o[i] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  // the list, cut into equal spans: units before each block (of one head), by a scan in the queries' room
  const int entries = a.B * nqb, heads = a.H * L::PER;
  long long u0 = 0, u1 = 0, span = 1;
  int entry0 = 0, before0 = 0;
  if (split) {
    int* prefix = reinterpret_cast<int*>(sm + L::Q);
    int* warp_sum = prefix + kMaxBlocks;
    const int per = (entries + kTThreads - 1) / kTThreads;
    TBlock k;
    int sum = 0;
    for (int i = 0; i < per && tid * per + i < entries; ++i) {
      prefix[tid * per + i] = sum;
      const int tiles = tc_block<L::ROWS>(a, tid * per + i, nqb, k);
      sum += tiles ? tiles + kItemCost : 0;
    }
    int run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, run, o);
      run += lane >= o ? v : 0;
    }
    if (lane == 31) warp_sum[tid >> 5] = run;
    __syncthreads();
    int base = run - sum, total = 0;
    for (int w = 0; w < kTThreads / 32; ++w) {
      base += w < (tid >> 5) ? warp_sum[w] : 0;
      total += warp_sum[w];
    }
    for (int i = 0; i < per && tid * per + i < entries; ++i) prefix[tid * per + i] += base;
    __syncthreads();
    const long long units = static_cast<long long>(total) * heads;
    span = (units + gridDim.x - 1) / gridDim.x;
    span = span < kMinSpan ? kMinSpan : span;
    u0 = span * blockIdx.x < units ? span * blockIdx.x : units;
    u1 = u0 + span < units ? u0 + span : units;
    int lo = 0, hi = entries - 1;                      // the block that holds u0
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (static_cast<long long>(prefix[mid]) * heads <= u0) lo = mid;
      else hi = mid - 1;
    }
    entry0 = lo;
    before0 = prefix[lo];
  }
  fence_async_smem();
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = *reinterpret_cast<const uint32_t*>(sm + tmem_at<D>());
  float* parts = a.part + static_cast<size_t>(gridDim.x) * (sizeof(TSplit) / sizeof(float));
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

  if (warp < 8) {
    // ---- softmax of half X (thread = row), the queries' split, the results ----------------
    // Accesses to tensor memory are the whole warp's: behind a branch that only some lanes take they meet again first.
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    const int X = warp >> 2, wq = warp & 3, r = 32 * wq + lane;
    const uint32_t trow = tmem + (static_cast<uint32_t>(32 * wq) << 16);
    const uint32_t ts = trow + col_s(X), to = trow + col_o(X);
    const float sgn = a.scale_log2 < 0.0f ? -1.0f : 1.0f;
    const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;   // whole sectors per store
    int seq = 0, nS = 0, nO = 0, nJ = 0;               // tiles seen, phases of S, of the final O and of the halves' join
    float2* join = reinterpret_cast<float2*>(sm + L::JOIN);
    float* rowf_sm = reinterpret_cast<float*>(sm + L::ROWF);
    int nF = 0;                                        // phases of the queries' release by half B
    // The row of an item that is this thread's.
    struct Row {
      bool live;
      int p;                                           // position; -1: an absent row sees nothing
      long long at;                                    // its element of q and out
      float rowf;
    };
    auto mine = [&](const ItemMsg& x) { return x.valid && (X == 0 || x.rows > 128 || x.ntile > 1); };
    // Loads the row and leaves it in shared memory as two e4m3 parts, scaled so that its largest value lies in
    // [128, 256).  The item before has no score MMA left: its last scores were read.
    auto queries = [&](const ItemMsg& x) {
      Row w;
      const int rx = x.rows > 128 ? 128 * X + r : r;
      const unsigned gr = static_cast<unsigned>(x.qb * L::ROWS + rx), tok = gr / static_cast<unsigned>(a.G);
      w.live = rx < x.rows;
      w.p = w.live ? x.p0 + static_cast<int>(tok) : -1;
      w.at = ((static_cast<long long>(x.b) * a.T + tok) * a.Hq + x.h / L::PER * a.G + (gr - tok * a.G)) * D;
      w.rowf = 0.0f;
      if (L::WIDE && X) return w;                      // half A does the work for both
      // The warp's 32 rows, D / 8 lanes per row (a lane per row would ask for 32 lines with each load); the raw 16-byte
      // pieces 2c and 2c + 1 of a row wait where the parts of its channels 16c .. 16c + 15 will stand.
      const uint32_t qx = sb + L::Q + X * L::QB;
      {
        constexpr int kP = D / 8, kR = 32 / kP;        // pieces per row, rows per load
        const long long where = w.live ? w.at : -1;
        const int piece = lane % kP;
        constexpr int kB = kP < 16 ? kP : 16;          // loads in flight
#pragma unroll 1
        for (int i0 = 0; i0 < kP; i0 += kB) {
          uint4 v4[kB];
#pragma unroll
          for (int i = 0; i < kB; ++i) {
            const long long at = __shfl_sync(0xffffffffu, where, kR * (i0 + i) + lane / kP);
            v4[i] = at >= 0 ? reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + at)[piece]
                            : make_uint4(0u, 0u, 0u, 0u);
          }
#pragma unroll
          for (int i = 0; i < kB; ++i)
            sts128(qx + L::qpos(32 * wq + kR * (i0 + i) + lane / kP, piece >> 1, piece & 1), v4[i].x, v4[i].y, v4[i].z, v4[i].w);
        }
      }
      __syncwarp();
      uint32_t mx2 = 0u;                               // largest magnitudes: bf16 bits order as integers
#pragma unroll 8
      for (int i = 0; i < D / 8; ++i) {
        const uint4 v = lds128(qx + L::qpos(r, i >> 1, i & 1));
        mx2 = __vmaxu2(__vmaxu2(mx2, v.x & 0x7FFF7FFFu), v.y & 0x7FFF7FFFu);
        mx2 = __vmaxu2(__vmaxu2(mx2, v.z & 0x7FFF7FFFu), v.w & 0x7FFF7FFFu);
      }
      const uint32_t mx = max(mx2 & 0xFFFFu, mx2 >> 16);
      int e = 7 - (static_cast<int>(mx >> 7) - 127);
      e = mx && mx < 0x7F80u ? min(e, 120) : 0;
      const float up = __int_as_float((e + 127) << 23) * sgn;
      w.rowf = __int_as_float((127 - e) << 23);
      // rolled: a loop that runs once an item, out of the instruction cache otherwise (3.6 us unrolled)
#pragma unroll 1
      for (int c = 0; c < D / 16; ++c) {
        const uint32_t ph = qx + L::qpos(r, c, 0), pl = qx + L::qpos(r, c, 1);
        const uint4 ua = lds128(ph), ub = lds128(pl);
        const uint32_t u[8] = {ua.x, ua.y, ua.z, ua.w, ub.x, ub.y, ub.z, ub.w};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {                  // fp16 holds the scaled bf16 values and their remainders exactly
          const uint32_t a0 = u[2 * k], a1 = u[2 * k + 1];
          const uint32_t f0 = half2_bits(__uint_as_float(a0 << 16) * up, __uint_as_float(a0 & 0xFFFF0000u) * up);
          const uint32_t f1 = half2_bits(__uint_as_float(a1 << 16) * up, __uint_as_float(a1 & 0xFFFF0000u) * up);
          const uint32_t h0 = half2_to_codes(f0), h1 = half2_to_codes(f1);
          hi[k] = h0 | (h1 << 16);
          lo[k] = half2_to_codes(sub_half2(f0, codes_to_half2(h0))) | (half2_to_codes(sub_half2(f1, codes_to_half2(h1))) << 16);
        }
        sts128(ph, hi[0], hi[1], hi[2], hi[3]);
        sts128(pl, lo[0], lo[1], lo[2], lo[3]);
      }
      // a row that is not finite: every score NaN, and so the result
      if (mx >= 0x7F80u) w.rowf = __int_as_float(0x7FC00000);
      if (L::WIDE) rowf_sm[r] = w.rowf;
      fence_async_smem();
      __syncwarp();
      if (lane == 0) bar_arrive(bar(bQReady + X));
      return w;
    };
    ItemMsg it = next_item(0);
    Row row{};
    if (mine(it)) row = queries(it);
    for (int n = 0; it.valid; ++n) {
      const int ntile = it.ntile;
      if (!mine(it)) {                                 // one tile of at most 128 rows: nothing for B
        seq += ntile;
        it = next_item(n + 1);
        if (mine(it)) row = queries(it);
        continue;
      }
      float rowf = row.rowf;
      const int p = row.p;
      const bool turns = it.rows <= 128;               // the halves take the tiles in turn
      const int t0 = turns ? X : 0, dt = turns ? 2 : 1, seq0 = seq;
      float m = kMNone, me = 0.0f, l = 0.0f;           // me: M's exponent where m is beyond kBig, else 0
      bool bigs = false;                               // a row of the warp has had such an M
      seq += t0;
      for (int t = t0; t < ntile; t += dt, seq += dt) {
        if (!wait(bDesc + seq % L::DESCS, seq / L::DESCS) || !wait(bSFull + X, nS)) break;
        ++nS;
        tc_after();
        if (L::WIDE && X) {                            // the row's scale is there with the first scores
          if (t == t0) rowf = rowf_sm[r];
          __syncwarp();
          if (lane == 0 && t + dt >= ntile) bar_arrive(bar(bQFree));
          __syncwarp();
        }
        const TileDesc& d = descs[seq % L::DESCS];
        auto factor = [&](int pg) { return score_factor(d.fac[pg], rowf); };
        // The tile as it mostly is: every token seen and no score far above the maximum so far.  The weights by the
        // old maximum tell by themselves: a page's sum below kFull means that each fits fp16.  No maximum is taken.
        bool done = false;
        if (d.full && t > t0 && !bigs) {
          float x[kTTok];
          uint32_t w[kTTok / 2];
          tld32x4(ts, x);
          float most = 0.0f, lt = l;
#pragma unroll
          for (int pg = 0; pg < kTPg; ++pg) {
            const float f = factor(pg), base = d.ev[pg] - m + kLift;
            const uint64_t f2 = pack2(f, f), b2 = pack2(base, base);
            uint64_t s2 = 0ull;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              float y0, y1;
              unpack2(fma2(pack2(x[16 * pg + 2 * k], x[16 * pg + 2 * k + 1]), f2, b2), y0, y1);
              y0 = ex2(y0);
              y1 = ex2(y1);
              s2 = add2(s2, pack2(y0, y1));
              w[8 * pg + k] = half2_bits(y0, y1);
            }
            float s0, s1;
            unpack2(s2, s0, s1);
            s0 += s1;
            most = fmaxf(most, s0);
            lt = fmaf(s0, d.vinv[pg], lt);
          }
          if (!__any_sync(0xffffffffu, most > kFull)) {
            l = lt;
            tst32(ts, *reinterpret_cast<uint32_t(*)[32]>(w));
            tst32(ts + 32u, *reinterpret_cast<uint32_t(*)[32]>(w + 32));
            done = true;
          }
        }
        if (!done) {                                   // an edge, an item's first tile, or a maximum that moves
          float x[kTTok];
          tld32x4(ts, x);
          if (!d.full) {
#pragma unroll
            for (int pg = 0; pg < kTPg; ++pg) {
              const uint32_t see = page_seen(p, d.j0[pg], a.window, a.sinks);
#pragma unroll
              for (int k = 0; k < 16; ++k) x[16 * pg + k] = (see >> k) & 1u ? x[16 * pg + k] : -INFINITY;
            }
          }
          float mx = -INFINITY;
#pragma unroll
          for (int pg = 0; pg < kTPg; ++pg) {
            float m0 = x[16 * pg], m1 = x[16 * pg + 1];
#pragma unroll
            for (int k = 2; k < 16; k += 2) {
              m0 = fmaxf(m0, x[16 * pg + k]);
              m1 = fmaxf(m1, x[16 * pg + k + 1]);
            }
            mx = fmaxf(mx, fmaf(fmaxf(m0, m1), factor(pg), d.ev[pg]));
          }
          const bool moved = mx > m + kSlack;
          if (__any_sync(0xffffffffu, moved)) {
            if (__any_sync(0xffffffffu, moved && fabsf(mx) > kBig)) bigs = true;
            if (!bigs) {
              const float alpha = moved ? ex2(m - (mx + kHead)) : 1.0f;
              if (moved) {
                m = mx + kHead;
                l *= alpha;
              }
              __syncwarp();
              if (t > t0) rescale_o<L::DV>(to, alpha); // O of the tiles before (their MMAs have run: S came after)
            }
          }
          if (__builtin_expect(!bigs, 1)) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {                // the weights overlay the scores
              uint32_t w[16];
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const int pg = 2 * c + q;
                const float f = factor(pg), base = d.ev[pg] - m + kLift;
                const uint64_t f2 = pack2(f, f), b2 = pack2(base, base);
                uint64_t s2 = 0ull;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  float y0, y1;
                  unpack2(fma2(pack2(x[16 * pg + 2 * k], x[16 * pg + 2 * k + 1]), f2, b2), y0, y1);
                  y0 = ex2(y0);
                  y1 = ex2(y1);
                  s2 = add2(s2, pack2(y0, y1));
                  w[8 * q + k] = half2_bits(y0, y1);
                }
                float s0, s1;
                unpack2(s2, s0, s1);
                l = fmaf(s0 + s1, d.vinv[pg], l);
              }
              tst16(ts + 16u * c, w);
            }
          } else {
            const float3 next = large_scores<L::DV>(ts, to, d, d.full, p, a.window, a.sinks, rowf, t > t0, m, me, l);
            m = next.x;
            me = next.y;
            l = next.z;
          }
        }
        tst_wait();
        tc_before();
        __syncwarp();
        if (lane == 0) bar_arrive(bar(bPFull + X));
      }
      if (failed) break;
      seq = seq0 + ntile;
      // the next item's queries first: its scores then run beside what is left of this one
      const ItemMsg done_item = it;
      const Row done_row = row;
      it = next_item(n + 1);
      if (L::WIDE && X == 0 && ntile > 1 && !wait(bQFree, nF++)) break;     // half B has its last scores too
      if (mine(it)) row = queries(it);
      // ---- the row's result (or partial) ----
      if (!wait(bODone + X, nO)) break;
      ++nO;
      tc_after();
      const bool joins = turns && ntile > 1;
      if (joins) {
        if (X) {
          // (m, l); beyond kBig with M's exponent in the last bits of l, which has 15 left
          join[r] = make_float2(m, fabsf(m) > kBig ? __uint_as_float((__float_as_uint(l) & ~0xFFu) | static_cast<uint32_t>(static_cast<int>(me) + 128)) : l);
          tc_before();
          __syncwarp();
          if (lane == 0) bar_arrive(bar(bJoin));
          if (!wait(bOFree, nJ++)) break;              // A has read this half's sums: the next item may overwrite them
          tc_after();
          continue;
        }
        if (!wait(bJoin, nJ++)) break;
        tc_after();
        const float2 other = join[r];
        const bool two = fabsf(other.x) > kBig;
        const float lb = two ? __uint_as_float(__float_as_uint(other.y) & ~0xFFu) : other.y;
        const float eb = two ? static_cast<float>(static_cast<int>(__float_as_uint(other.y) & 0xFFu) - 128) : 0.0f;
        const float ref = fmaxf(m, other.x), da = m - ref + me, db = other.x - ref + eb;
        m = ref;
        me = fmaxf(da, db);
        const float fa = ex2(da - me), fb = ex2(db - me);
        l = fa * l + fb * lb;
#pragma unroll 1
        for (int c = 0; c < L::DV / 16; ++c) {
          float o[16], o2[16];
          uint32_t u[16];
          tld16(to + 16u * c, o);
          tld16(trow + col_o(1) + 16u * c, o2);
#pragma unroll
          for (int k = 0; k < 16; ++k) u[k] = __float_as_uint(fa * o[k] + fb * o2[k]);
          tst16(to + 16u * c, u);
        }
        tst_wait();
        tc_before();
        __syncwarp();
        if (lane == 0) bar_arrive(bar(bOFree));
        __syncwarp();
      }
      const float inv = l > 0.0f ? 1.0f / l : l == l ? 0.0f : l;
      float* part = parts + (static_cast<long long>(done_item.slot) * L::ROWS + (turns ? 0 : 128 * X) + r) * L::PART;
#pragma unroll 1
      for (int c = 0; c < L::DV / 32; ++c) {
        float o[32];
        tld32(to + 32u * c, o);
        if (done_row.live && done_item.slot < 0) {
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const __nv_bfloat162 y = __floats2bfloat162_rn(o[2 * k] * inv, o[2 * k + 1] * inv);
            w[k] = *reinterpret_cast<const uint32_t*>(&y);
          }
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + done_row.at + done_item.h % L::PER * L::DV + 32 * c;
          if (wide) {
            stg256(dst, w);
            stg256(dst + 16, w + 8);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              reinterpret_cast<uint4*>(dst)[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
          }
        } else if (done_row.live) {
          float4* dst = reinterpret_cast<float4*>(part + 4 + 32 * c);
#pragma unroll
          for (int k = 0; k < 8; ++k) dst[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          if (c == 0) *reinterpret_cast<float4*>(part) = make_float4(m, l, me, 0.0f);
        }
        __syncwarp();                                  // lanes with no row wait: the loads are the whole warp's
      }
      tc_before();                                     // O is read before the next item's first P is announced
    }
  } else if (warp < 12) {
    // ---- values to fp16: thread = token of the tile ----------------------------------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    const int t = tid - 256, pg = t >> 4;
    int seq = 0, keys = 0;                             // tiles, and how many tiles' keys are there
    for (int n = 0;; ++n) {
      const ItemMsg it = next_item(n);
      if (!it.valid) break;
      const int ntile = it.ntile, ahead = it.rows <= 128 ? 2 : 1, end = seq + ntile;
      for (int i = 0; i < ntile; ++i, ++seq) {
        if (!wait(bVFull + seq % L::VST, seq / L::VST)) break;
        if (seq >= 2 && !wait(bDone + (seq - 2) % kDoneRing, (seq - 2) / kDoneRing)) break;
        const int j = descs[seq % L::DESCS].j0[pg] + (t & 15);
        // what no row sees may hold anything: zeros instead
        const bool see = j <= it.pmax && (!a.window || j > it.pmin - a.window || j < a.sinks);
        const uint32_t src = sb + L::VR + (seq % L::VST) * L::VRT;
        const uint32_t dst = sb + L::V + (seq & 1) * L::VT + t * 128;
        uint4 w[L::DV / 16];                             // every load ahead of the stores
#pragma unroll
        for (int c = 0; c < L::DV / 16; ++c) w[c] = lds128(src + L::vpos(t, c));
#pragma unroll
        for (int c = 0; c < L::DV / 16; ++c) {
          if (!see) w[c] = make_uint4(0u, 0u, 0u, 0u);
          const uint32_t o0 = static_cast<uint32_t>((((2 * c) & 7) ^ (t & 7)) << 4),
                         o1 = static_cast<uint32_t>((((2 * c + 1) & 7) ^ (t & 7)) << 4);
          const uint32_t half = dst + (c >> 2) * 16384;
          sts128(half + o0, codes_to_half2(w[c].x), codes_to_half2(w[c].x >> 16), codes_to_half2(w[c].y),
                 codes_to_half2(w[c].y >> 16));
          sts128(half + o1, codes_to_half2(w[c].z), codes_to_half2(w[c].z >> 16), codes_to_half2(w[c].w),
                 codes_to_half2(w[c].w >> 16));
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) bar_arrive(bar(bVEmpty + seq % L::VST));
        // the issuing warp's one wait for a tile covers the keys of the scores that it issues behind the tile
        for (; keys <= seq + ahead && keys < end && !failed; ++keys) (void)wait(bKFull + keys % L::KST, keys / L::KST);
        if (failed) break;
        if (lane == 0) bar_arrive(bar(bReady + (seq & 1)));
      }
      if (failed) break;
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 12) {
      // ---- items, pages, keys -----------------------------------------------------------------
      int seq = 0, n = 0, nk = 0;                      // tiles, items, and tiles whose copies were issued
      int free0 = 0, free1 = 0, free2 = 0;             // the steps after which the keys of the last three tiles are read
      auto publish = [&](const ItemMsg& x) {
        // Every warp has taken the one before.  If one has not within the limit, its room stays as it is (a message read
        // half old, half new would send rows anywhere), and the others' waits for this one give up too.
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
      TBlock it;
      TSplit cut{};
      int e = entry0, h = 0, tiles = split && u0 < u1 ? tc_block<L::ROWS>(a, e, nqb, it) : 0;
      long long at = static_cast<long long>(before0) * heads;         // the item's first unit in the list
      if (tiles) {
        h = static_cast<int>((u0 - at) / (tiles + kItemCost));
        at += static_cast<long long>(h) * (tiles + kItemCost);
      }
      long long whole = blockIdx.x;                    // not split: whole items in turn, the longest rows first
      const long long items = static_cast<long long>(entries) * heads;
      for (;;) {
        int t0 = 0, t1 = 0;                            // the item's tiles that are this CTA's
        if (split) {
          if (u0 >= u1) break;
          t0 = max(0, static_cast<int>(u0 - at) - kItemCost);
          t1 = static_cast<int>(min(u1 - at - kItemCost, static_cast<long long>(tiles)));
          if (t1 <= t0) break;                         // the span ends before the item's first tile
          if (t0 == 0 && t1 < tiles) {
            cut = TSplit{1, it.b, h, it.qb, it.p0, it.rows, static_cast<int>((at + kItemCost + tiles - 1) / span), 0};
          }
        } else {
          if (whole >= items) break;
          h = static_cast<int>(whole % heads);
          t1 = tiles = tc_block<L::ROWS>(a, entries - 1 - static_cast<int>(whole / heads), nqb, it);
          whole += gridDim.x;
          if (!tiles) continue;
        }
        const int slot = t0 == 0 && t1 == tiles ? -1 : 2 * static_cast<int>(blockIdx.x) + (t0 ? 0 : 1);
        publish(ItemMsg{1, it.b, h, it.qb, it.p0, it.rows, it.pmin, it.pmax, t1 - t0, slot, {0, 0}});
        const int ahead = it.rows <= 128 ? 2 : 1;      // a tile's scores are issued so many steps before its values
        const int c0 = t0 * kTPg, c1 = min(it.pages, t1 * kTPg);
        const int* table = a.bt + static_cast<long long>(it.b) * a.maxp;
        // lane i holds page i of four tiles (lanes 8k .. 8k + 7: tile k); the next four tiles' ids and scales are on
        // their way meanwhile (two dependent loads are as long as a tile)
        struct PageInfo {
          int blk, j0, ev;
          float ks;
        };
        auto fetch = [&](int ci) {
          PageInfo x{-1, kNoPage, 0, 1.0f};
          if (ci < c1) {
            const int page = ci < it.r.ns ? ci : ci - it.r.ns + it.r.w0;
            const int pid = table[page];
            if (pid >= 0 && pid < a.num_pages) {
              x.blk = pid * a.H + h / L::PER;
              x.j0 = kPage * page;
              x.ks = a.ks[x.blk];
              x.ev = static_cast<int>((__float_as_uint(a.vs[x.blk]) >> 23) & 0xFF) - 127;
            } else {
              atomicOr(a.err, kErrPage);
            }
          }
          return x;
        };
        PageInfo cur = fetch(c0 + lane);
        for (int c4 = c0; c4 < c1 && !failed; c4 += 4 * kTPg) {
          const PageInfo nxt = fetch(c4 + 4 * kTPg + lane);
          const bool seen = cur.j0 + 15 <= it.pmin && (!a.window || cur.j0 > it.pmax - a.window || cur.j0 + 15 < a.sinks);
          const uint32_t seen4 = __ballot_sync(0xffffffffu, seen), there4 = __ballot_sync(0xffffffffu, cur.blk >= 0);
          for (int k = 0; k < 4 && c4 + k * kTPg < c1; ++k, ++seq) {
            const bool on = (lane >> 3) == k;
            const int pg = lane & 7;
            const uint32_t bytes = static_cast<uint32_t>(__popc((there4 >> (8 * k)) & 0xFFu)) * kPage * D;
            if (L::WIDE) {
              if (seq >= 2 && !wait(bKFree + (seq & 1), seq / 2 - 1)) break;
            } else {
              if (seq >= 3 && !wait(bDone + free0 % kDoneRing, free0 / kDoneRing)) break;
              free0 = free1, free1 = free2;
              free2 = c4 + k * kTPg >= c0 + ahead * kTPg ? seq - ahead : seq;
            }
            TileDesc& d = descs[seq % L::DESCS];
            if (on) {
              d.fac[pg] = fabsf(a.scale_log2) * cur.ks;
              d.ev[pg] = static_cast<float>(cur.ev);
              d.vinv[pg] = exp2f(static_cast<float>(-cur.ev));
              d.j0[pg] = cur.j0;
              d.blk[pg] = cur.blk;
              if (pg == 0) d.full = ((seen4 >> (8 * k)) & 0xFFu) == 0xFFu ? 1 : 0;
            }
            __syncwarp();
            if (lane == 0) {
              bar_arrive(bar(bDesc + seq % L::DESCS));
              if (bytes) bar_arrive_tx(bar(bKFull + seq % L::KST), bytes);
              else bar_arrive(bar(bKFull + seq % L::KST));
            }
            __syncwarp();
            ++nk;
            if (on && cur.blk >= 0)
              tma_block(sb + L::K + (seq % L::KST) * L::KT + pg * kPage * L::DV, &mk, 0, cur.blk, bar(bKFull + seq % L::KST));
          }
          cur = nxt;
        }
        if (failed) break;
        if (split) {
          at += kItemCost + tiles;
          u0 = at;
          if (u0 >= u1) break;
          if (++h == heads) {
            h = 0;
            do tiles = tc_block<L::ROWS>(a, ++e, nqb, it);
            while (!tiles);
          }
        }
      }
      publish(ItemMsg{});
      if (split && lane == 0) splits[blockIdx.x] = cut;
      // copies still in flight land before the CTA ends
      bool f2 = false;
      for (int s = nk >= L::KST ? nk - L::KST : 0; s < nk; ++s) (void)bar_wait(bar(bKFull + s % L::KST), (s / L::KST) & 1, f2);
    } else if (warp == 13) {
      // ---- MMA issue, the warp converged: O += w V of a tile and the next tile's scores, half A, then half B.  The
      // order is strict: left to mix, both halves' MMAs end together, both softmaxes run together and neither overlaps
      // the other (4,370 cycles a tile). ---------------------------------------------------------------------------
      auto ready = [&](int i, int phase) {             // wait() in few instructions
        if (__all_sync(0xffffffffu, wait_short(bar(i), phase & 1))) return true;
        failed = true;
        return false;
      };
      int seq = 0, n = 0;
      ItemMsg it = next_item(0);
      int nq0 = 0, nq1 = 0, np0 = 0, np1 = 0;          // phases of the queries and of the weights
      int tiles = 0;
      bool two = false;                                // rows in half B
      auto open_item = [&]() {
        tiles = uniform(it.ntile);
        two = __all_sync(0xffffffffu, it.rows > 128);
      };
      auto scores = [&](uint32_t X, int s) {
        const uint32_t q = sb + L::Q + X * L::QB, k = sb + L::K + (s % L::KST) * L::KT;
        if (D == 64) {
          mma4_scores(tmem + col_s(X), sdesc(q), kdesc8<64>(k), kIdF8);
        } else {
          mma8_scores<0>(tmem + col_s(X), sdesc(q), sdesc(q + L::QX / 2), kdesc8<128>(k), kIdF8);
          if (L::WIDE) mma8_scores<1>(tmem + col_s(X), sdesc(q + 16384), sdesc(q + L::QX / 2 + 16384), kdesc8<128>(k + 16384), kIdF8);
        }
        mma_commit_warp(bar(bSFull + X));
        if (L::WIDE) mma_commit_warp(bar(bKFree + (s & 1)));
      };
      auto values = [&](uint32_t X, int s, bool first) {
        mma8_values(tmem + col_o(X), tmem + col_s(X), vdesc(sb + L::V + (s & 1) * L::VT), idesc_f16(L::DV) | (1u << 16), first ? 0u : 1u);
      };
      // the first tile of an item: its keys and its queries
      auto first_scores = [&](int s) {
        if (!ready(bKFull + s % L::KST, s / L::KST) || !ready(bQReady, nq0++)) return false;
        tc_after();
        scores(0, s);
        if (two || tiles > 1) {
          const int s1 = two ? s : s + 1;
          if (!two && !ready(bKFull + s1 % L::KST, s1 / L::KST)) return false;
          if (!L::WIDE && !ready(bQReady + 1, nq1++)) return false;
          tc_after();
          scores(1, s1);
        }
        return true;
      };
      bool ok = __all_sync(0xffffffffu, it.valid);
      bool open = ok;
      if (ok) {
        open_item();
        ok = first_scores(0);
      }
      while (ok && open) {
        const int my_tiles = tiles;
        const bool my_two = two;
        for (int t = 0; t < my_tiles && !my_two; ++t, ++seq) {   // the halves' tiles in turn
          const uint32_t X = t & 1;
          ok = ready(bReady + (seq & 1), seq >> 1) && ready(bPFull + X, X ? np1++ : np0++);
          if (!ok) break;
          tc_after();
          values(X, seq, t < 2);
          if (t + 2 < my_tiles) scores(X, seq + 2);
          else mma_commit_warp(bar(bODone + X));
          mma_commit_warp(bar(bDone + seq % kDoneRing));
        }
        for (int t = 0; t < my_tiles && my_two; ++t, ++seq) {
          const bool last = t == my_tiles - 1;
          ok = ready(bReady + (seq & 1), seq >> 1) && ready(bPFull, np0++);
          if (!ok) break;
          tc_after();
          values(0, seq, t == 0);
          if (last) mma_commit_warp(bar(bODone));
          else scores(0, seq + 1);
          ok = ready(bPFull + 1, np1++);
          if (!ok) break;
          tc_after();
          values(1, seq, t == 0);
          if (last) mma_commit_warp(bar(bODone + 1));
          else scores(1, seq + 1);
          mma_commit_warp(bar(bDone + seq % kDoneRing));   // the tile's keys and values have been read
        }
        if (!ok) break;
        it = next_item(++n);
        open = __all_sync(0xffffffffu, it.valid);
        if (failed) ok = false;
        if (ok && open) {
          open_item();
          ok = first_scores(seq);
        }
      }
      mma_commit_warp(bar(bDrain));                    // every MMA issued completes before the CTA ends
      bool f2 = false;
      (void)bar_wait(bar(bDrain), 0, f2);
      __syncwarp();
    } else if (warp == 14) {
      // ---- values ---------------------------------------------------------------------------
      int seq = 0;
      for (int n = 0;; ++n) {
        const ItemMsg it = next_item(n);
        if (!it.valid) break;
        const int ntile = it.ntile;
        for (int i = 0; i < ntile; ++i, ++seq) {
          if (!wait(bDesc + seq % L::DESCS, seq / L::DESCS)) break;
          const int blk = lane < kTPg ? descs[seq % L::DESCS].blk[lane] : -1;
          if (seq >= L::VST && !wait(bVEmpty + seq % L::VST, seq / L::VST - 1)) break;
          const uint32_t bytes = static_cast<uint32_t>(__popc(__ballot_sync(0xffffffffu, blk >= 0))) * kPage * L::DV;
          if (lane == 0) {
            if (bytes) bar_arrive_tx(bar(bVFull + seq % L::VST), bytes);
            else bar_arrive(bar(bVFull + seq % L::VST));
          }
          __syncwarp();
          if (blk >= 0)
            tma_block(sb + L::VR + (seq % L::VST) * L::VRT + lane * kPage * L::DV, &mv, it.h % L::PER * L::DV, blk,
                      bar(bVFull + seq % L::VST));
        }
        if (failed) break;
      }
      // copies still in flight land before the CTA ends
      bool f2 = false;
      for (int s = seq >= L::VST ? seq - L::VST : 0; s < seq; ++s) (void)bar_wait(bar(bVFull + s % L::VST), (s / L::VST) & 1, f2);
    } else {
      // ---- an item's queries on their way to L2 as soon as it is known ------------------------
      int seq = 0;
      for (int n = 0;; ++n) {
        const ItemMsg it = next_item(n);
        if (!it.valid) break;
        constexpr int kLines = D / 64;                 // 128-byte lines of a row
        for (int i = lane; i < it.rows * kLines; i += 32) {
          const unsigned gr = static_cast<unsigned>(it.qb * L::ROWS + i / kLines), tok = gr / static_cast<unsigned>(a.G);
          const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) +
                                   ((static_cast<long long>(it.b) * a.T + tok) * a.Hq + it.h / L::PER * a.G + (gr - tok * a.G)) * D;
          asm volatile("prefetch.global.L2 [%0];" ::"l"(q + 64 * (i % kLines)));
        }
        if (L::WIDE) {                                 // the keys' upper channels
          const int ntile = it.ntile;
          for (int i = 0; i < ntile; ++i, ++seq) {
            if (!wait(bDesc + seq % L::DESCS, seq / L::DESCS)) break;
            const int blk = lane < kTPg ? descs[seq % L::DESCS].blk[lane] : -1;
            if (blk >= 0) tma_block(sb + L::K + (seq & 1) * L::KT + 16384 + lane * kPage * 128, &mk, 128, blk, bar(bKFull + (seq & 1)));
          }
          if (failed) break;
        }
      }
    }
  }
  if (failed && lane == 0) atomicOr(a.err, kErrTimeout);
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 13) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

// Joins the parts of the items that cross spans: 32 rows a block, a warp per row.
template <int D>
__global__ void __launch_bounds__(256) kv8_tc_join_kernel(const __grid_constant__ Kv8Attn a, int ctas) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x;
  pdl_wait();
  const TSplit cut = reinterpret_cast<const TSplit*>(a.part)[c];
  if (!cut.valid) return;
  const float* parts = a.part + static_cast<size_t>(ctas) * (sizeof(TSplit) / sizeof(float));
  using L = TG<D>;
  constexpr int kPart = L::PART, DV = L::DV;
  const long long step = static_cast<long long>(L::ROWS) * kPart;
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    const int rr = 32 * blockIdx.y + 8 * i + warp;
    if (rr >= cut.rows) return;
    // the first part is in its CTA's second slot, the others in their CTAs' first
    auto part = [&](int k) { return parts + (2LL * k + (k == c ? 1 : 0)) * step + static_cast<long long>(rr) * kPart; };
    float M = kMNone, E = 0.0f;                        // the joined M, in its two parts
    bool two = false;
    for (int k = c + lane; k <= cut.last; k += 32) {
      const float4 h = *reinterpret_cast<const float4*>(part(k));
      M = fmaxf(M, h.x);
      two |= h.z != 0.0f;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (__any_sync(0xffffffffu, two)) {
      E = -INFINITY;
      for (int k = c + lane; k <= cut.last; k += 32) E = fmaxf(E, part(k)[0] - M + part(k)[2]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) E = fmaxf(E, __shfl_xor_sync(0xffffffffu, E, o));
    }
    float L = 0.0f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = c; k <= cut.last; ++k) {
      const float* p = part(k);
      const float f = ex2(p[0] - M + p[2] - E);
      L = fmaf(f, p[1], L);
      if (4 * lane >= DV) continue;
      const float4 x = *reinterpret_cast<const float4*>(p + 4 + 4 * lane);
      acc.x = fmaf(f, x.x, acc.x), acc.y = fmaf(f, x.y, acc.y), acc.z = fmaf(f, x.z, acc.z), acc.w = fmaf(f, x.w, acc.w);
    }
    if (4 * lane >= DV) continue;
    const float inv = L > 0.0f ? 1.0f / L : L == L ? 0.0f : L;
    const __nv_bfloat162 y0 = __floats2bfloat162_rn(acc.x * inv, acc.y * inv),
                         y1 = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
    const unsigned gr = static_cast<unsigned>(cut.qb * L::ROWS + rr), tok = gr / static_cast<unsigned>(a.G);
    const long long at = ((static_cast<long long>(cut.b) * a.T + tok) * a.Hq + cut.h / L::PER * a.G + (gr - tok * a.G)) * D +
                         cut.h % L::PER * DV + 4 * lane;
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&y0), *reinterpret_cast<const uint32_t*>(&y1));
  }
}

int rows_of(int d) { return d == 256 ? TG<256>::ROWS : TG<128>::ROWS; }
int items_per_head(int d) { return d == 256 ? TG<256>::PER : 1; }
int query_blocks(int T, int G, int d) { return static_cast<int>((static_cast<long long>(T) * G + rows_of(d) - 1) / rows_of(d)); }

// CTAs of a call: one per SM, fewer where the list of tiles cannot be that long.
long long tiles_of(int max_seq_len) { return (static_cast<long long>(max_seq_len) + kTTok - 1) / kTTok + 1; }
int ctas_for(int B, int H, int nqb, int max_seq_len) {
  const long long most = static_cast<long long>(B) * H * nqb * tiles_of(max_seq_len);
  const long long n = (most * (1 + kItemCost) + kMinSpan - 1) / kMinSpan;
  const int sms = kv8_sm_count();
  return static_cast<int>(n < sms ? (n < 1 ? 1 : n) : sms);
}
// The list holds so many blocks, and counts units in 32 bits.
bool splits(int B, int nqb, int max_seq_len) {
  const long long blocks = static_cast<long long>(B) * nqb;
  return blocks <= kMaxBlocks && blocks * (tiles_of(max_seq_len) + kItemCost) <= 0x7FFFFFFFLL;
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

}  // namespace

int kv8_sm_count() {
  static std::atomic<int> known[64];                   // per device: the query costs as much as a launch
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 152;
  int sms = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
  if (sms > 0) return sms;
  sms = 152;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && dev < 64)
    known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

bool kv8_block_map(CUtensorMap* map, const void* codes, long long blocks, int d) {
  auto fn = encode_fn();
  if (!fn) return false;
  const int row = d < 128 ? d : 128;                   // 128-byte panels
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), kPage, static_cast<cuuint64_t>(blocks)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(d) * kPage};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(row), kPage, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(codes), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, row == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// More rows than a block of the mma.sync form has.  32 / 8 heads, 64 sequences of 2,000 to 8,000 tokens: 16 rows 157 us
// there and 158 here (d = 64: 134 and 134), 20 rows 292 and 161 (248 and 137).  16 sequences, d = 256: 16 rows 101 and
// 104, 20 rows 138 and 106, 64 rows 348 and 113.  A larger scale would make the query's rounding to two e4m3 parts count
// (and costs: prompts of 2,048 to 4,096 tokens at scale 1, d = 128, 64, 256: 409, 1,048, 618 us on mma.sync, 61, 116, 81 here).
bool kv8_tc_takes(int T, int G, int d, bool f32, float softmax_scale) {
  return !f32 && static_cast<long long>(T) * G > kTcRows && softmax_scale != 0.0f &&
         std::fabs(static_cast<double>(softmax_scale)) <= (1.0 + 1e-6) / std::sqrt(static_cast<double>(d));
}

bool kv8_tc_splits(int B, int T, int G, int max_seq_len, int d) { return splits(B, query_blocks(T, G, d), max_seq_len); }

size_t kv8_tc_workspace(int B, int T, int G, int H, int max_seq_len, int d) {
  const int nqb = query_blocks(T, G, d);
  return static_cast<size_t>(ctas_for(B, H * items_per_head(d), nqb, max_seq_len)) *
         (sizeof(TSplit) + 2 * sizeof(float) * static_cast<size_t>(rows_of(d)) * (d / items_per_head(d) + 4));
}

namespace {
template <int D>
cudaError_t launch_t(const Kv8Attn& a, cudaStream_t s) {
  const int nqb = query_blocks(a.T, a.G, D);
  CUtensorMap mk, mv;
  const long long blocks = static_cast<long long>(a.num_pages) * a.H;
  if (!kv8_block_map(&mk, a.kc, blocks, D) || !kv8_block_map(&mv, a.vc, blocks, D)) return cudaErrorInvalidValue;
  static std::atomic<unsigned long long> configured{0};
  cudaError_t e = smem_attr_once(kv8_tc_kernel<D>, smem_bytes<D>(), configured);
  if (e != cudaSuccess) return e;
  const int ctas = ctas_for(a.B, a.H * TG<D>::PER, nqb, a.max_seq_len);
  const bool split = splits(a.B, nqb, a.max_seq_len);
  e = launch_pdl(kv8_tc_kernel<D>, dim3(ctas), dim3(kTThreads), smem_bytes<D>(), s, a, mk, mv, nqb, split ? 1 : 0);
  if (e != cudaSuccess || !split) return e;
  return launch_pdl(kv8_tc_join_kernel<D>, dim3(ctas, TG<D>::ROWS / 32), dim3(256), 0, s, a, ctas);
}
}  // namespace

cudaError_t launch_kv8_tc(const Kv8Attn& a, int d, cudaStream_t s) {
  switch (d) {
    case 64: return launch_t<64>(a, s);
    case 128: return launch_t<128>(a, s);
    case 256: return launch_t<256>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace tq
