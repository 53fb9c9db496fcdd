// Reading the 2-4-bit cache back on the tensor cores (tcgen05), d = m = 128.
//
//   k = n16/sqrt(d) (c[code] Pi) + sqrt(pi/2)/m rho16 (s (S Pi)),   v = n16/sqrt(d) (c[code] Pi)
// for 128 vectors (eight (page, KV head) blocks) at a time: M = 128 vectors, N = 128 channels, K = 128 codes or signs.  Pi
// and S Pi stand in shared memory in fp16 (the quantize kernels' table read the other way round, MN-major, and one of its
// own); the left operands are made from the records in registers, a code picking the two bytes of its centroid by prmt, four
// codes at a time, for any bit width, and go to tensor memory (in shared memory they would take half of its bandwidth).
// bf16 rows take the fp16 tables (2^-11 of each factor, half a step of bf16 being 2^-8), and both products one sum: a row's
// larger factor is applied at the end, the other operand is scaled by their ratio.  fp32 rows take centroids and tables in
// two fp16 parts each; the two products are summed apart, the small parts ahead of the large ones, since the tensor cores
// cut a sum instead of rounding it: by up to 2^-23 of what it is at each of the large product's eight steps, 2^-20 of an element
// (2-bit values whose elements are four times the root of their terms' squares are off by 1.3 times 2^-19 of that root, all toward
// zero).  Rows leave through shared memory, so that a store takes whole lines.
//
// Warps 0-15: the operands, in two groups that take the tiles in turn (thread = vector and half of its channels); 16-19: the
// rows (thread = vector); 20: blocks of records by bulk copies; 21: MMA issue.  Every wait is bounded; a wait that gives up
// sets the device error word.
//
// Bound by the operands' making, then by the rows' stores.  Eight sequences of 16,384 tokens, 8 heads, 3.5-bit keys and
// values into bf16 rows: 150 us (4.5 TB/s of rows and records; on CUDA cores 4,340), 8,192 tokens each into fp32 rows 150.  By
// counters: integer pipe 63% and issue slots 64% of the cycles (the operands), shared memory 52%, DRAM 51%, tensor pipe 29%.
// Left operands through shared memory took its bandwidth from the tables; rows by bulk copies of a lane each took 2,600
// cycles to issue.  Some dozen pages a sequence: 17 us (on CUDA cores 72): the tables' way into shared memory and the list of pages
// (5.5 stalls an issue at barriers), ahead of a tile or two a CTA.

#include "tq_read.h"
#include "tq_tc.cuh"
#include "tq_tc_attn.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

namespace tq {
namespace {

using namespace tcx;

constexpr int kMakers = 16, kGroup = 8;                // warps that make operands, and of one group
constexpr int kThreads = 32 * (kMakers + 6);
constexpr int kVec = 128, kBlocks = kVec / kPage;      // vectors and blocks a tile
constexpr int kTable = 128 * 256;                      // bytes of a table
constexpr int kRecord = kBlocks * 1344;                // room for a tile's blocks: 16 x (64 code bytes, 16 of signs, two norms)
constexpr int kInfos = 4;
constexpr int kList = 512;                             // sequences whose pages are listed without gaps

// Shared memory: tables (bf16 rows: Pi, S Pi; fp32: both parts of each), records, rows on their way out.  Tensor memory:
// STAGES of accumulators, then four left operands.
template <bool F32>
struct RG {
  static constexpr int TABLES = F32 ? 4 : 2, SLOTS = 4, STAGES = F32 ? 1 : 2, ACC = F32 ? 256 : 128;
  static constexpr int RECORDS = F32 ? 2 : 7;
  static constexpr int ROW = (F32 ? 512 : 256) + 16;               // bytes from row to row: the banks in turn
  static constexpr int REC = TABLES * kTable;
  static constexpr int OUT = REC + RECORDS * kRecord;              // [128]
  static constexpr int INFO = OUT + kVec * ROW;             // [kInfos][128] {row factors, row}
  static constexpr int BLK = INFO + kInfos * kVec * 16;            // [RECORDS][8] blocks
  static constexpr int BAR = BLK + RECORDS * kBlocks * 16;
  static constexpr int BOOK = BAR + 8 * 32;                        // [kind][part of the centroid][group] bytes for prmt
  static constexpr int LIST = BOOK + 8 * 16;                       // pages before each sequence, sums of warps
  static constexpr int TMEM = LIST + 4 * (kList + 32);
  static constexpr int BYTES = TMEM + 16;
  static constexpr uint32_t A = 256;                               // first column of the left operands
};
static_assert(RG<false>::BYTES <= 232448 && RG<true>::BYTES <= 232448, "shared memory per block");
enum Bar {
  bRec = 0, bRecFree = bRec + 7, bFull = bRecFree + 7, bFree = bFull + 4, bDone = bFree + 4, bTaken = bDone + 2,
  bInfo = bTaken + 2, bTab = bInfo + kInfos, bDrain, bCount
};
static_assert(bCount <= 32, "barriers");

struct alignas(16) BlockInfo {
  int head, slots, row0, pad;             // slots: first | end << 8 (0: nothing); row0: output row of slot 0
};
struct alignas(16) RowInfo {
  float fa, fb;
  int row, head;                          // row -1: none
};

// The two bytes of eight centroids (those of the magnitudes for four bits), as prmt takes them.
struct Bytes {
  uint32_t lo0, lo1, hi0, hi1;
};
__device__ __forceinline__ Bytes table_bytes(const GroupBook& g, bool low) {
  uint32_t lo[2] = {0u, 0u}, hi[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int code = g.bits == 4 ? 8 + i : i;
    float x = 0.0f;
    if (i < (1 << g.bits)) {
      const __half h = __float2half_rn(g.c[code]);
      x = low ? g.c[code] - __half2float(h) : g.c[code];
    }
    const uint32_t u = __half_as_ushort(__float2half_rn(x));
    lo[i >> 2] |= (u & 0xFFu) << (8 * (i & 3));
    hi[i >> 2] |= (u >> 8) << (8 * (i & 3));
  }
  return Bytes{lo[0], lo[1], hi[0], hi[1]};
}
// Four codes (nibbles of sel, below 8) as two words of fp16 pairs; sign: their signs in bit 3 of the nibbles of raw.
template <bool SIGN>
__device__ __forceinline__ void four_codes(const Bytes& t, uint32_t sel, uint32_t raw, uint32_t& a, uint32_t& b) {
  const uint32_t lo = prmt(t.lo0, t.lo1, sel);
  uint32_t hi = prmt(t.hi0, t.hi1, sel);
  if (SIGN) {
    uint32_t s = raw & 0x8888u;           // to bit 7 of the bytes
    s = (s | (s << 8)) & 0x00FF00FFu;
    s = (s << 4 | s << 8) & 0x80808080u;
    hi ^= s;
  }
  a = prmt(lo, hi, 0x5140);
  b = prmt(lo, hi, 0x7362);
}
// Nibbles of the eight codes (BITS below 4) from their stored bits at the low end of x.
template <int BITS>
__device__ __forceinline__ uint32_t nibbles(uint32_t x) {
  if (BITS == 3) {                        // channels 0-5 in nibbles, 6 and 7 in the spare top bits
    const uint32_t c6 = ((x >> 3) & 1u) | ((x >> 10) & 2u) | ((x >> 17) & 4u), c7 = ((x >> 7) & 1u) | ((x >> 14) & 2u) | ((x >> 21) & 4u);
    return (x & 0x00777777u) | (c6 << 24) | (c7 << 28);
  }
  if (BITS == 2) {
    x &= 0xFFFFu;
    x = (x | (x << 8)) & 0x00FF00FFu;
    x = (x | (x << 4)) & 0x0F0F0F0Fu;
    return (x | (x << 2)) & 0x33333333u;
  }
  x &= 0xFFu;
  x = (x | (x << 12)) & 0x000F000Fu;
  x = (x | (x << 6)) & 0x03030303u;
  return (x | (x << 3)) & 0x11111111u;
}
// 32 channels of a row from its stored words at `src`, as fp16 pairs.
template <int BITS>
__device__ __forceinline__ void block32(const Bytes& t, uint32_t src, uint32_t* v) {
  uint32_t w[BITS];
#pragma unroll
  for (int i = 0; i < BITS; ++i) w[i] = lds32(src + 4u * i);
#pragma unroll
  for (int o = 0; o < 4; ++o) {           // eight channels
    constexpr int kB = 8 * BITS;
    const int at = kB * o / 32, sh = kB * o % 32;
    uint32_t x = w[at] >> sh;
    if (sh + kB > 32 && at + 1 < BITS) x |= w[at + 1] << (32 - sh);
    if (BITS == 4) {
      const uint32_t m = x & 0x77777777u;
      four_codes<true>(t, m & 0xFFFFu, x & 0xFFFFu, v[4 * o], v[4 * o + 1]);
      four_codes<true>(t, m >> 16, x >> 16, v[4 * o + 2], v[4 * o + 3]);
    } else {
      const uint32_t n = nibbles<BITS>(x);
      four_codes<false>(t, n & 0xFFFFu, 0u, v[4 * o], v[4 * o + 1]);
      four_codes<false>(t, n >> 16, 0u, v[4 * o + 2], v[4 * o + 3]);
    }
  }
}
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, __half2 b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), b);
  return *reinterpret_cast<const uint32_t*>(&r);
}
// Eight MMAs of one table: rows of 16 codes (2048 B, 128 descriptor units) against 8 columns of the left operand.
__device__ __forceinline__ void mma8_table(uint32_t d, uint32_t a, uint32_t table, bool first) {
  mma8_values(d, a, vdesc(table), idesc_f16(kVec) | (1u << 16), first ? 0u : 1u);
}
template <bool F32>
__global__ void __launch_bounds__(kThreads, 1) read_tc_kernel(const __grid_constant__ ReadArgs a) {
  using L = RG<F32>;
  extern __shared__ __align__(1024) unsigned char sm_raw[];
  unsigned char* sm = sm_raw;
  const uint32_t sb = su32(sm);
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  auto bar = [&](int i) { return sb + L::BAR + 8u * static_cast<uint32_t>(i); };
  BlockInfo* blocks = reinterpret_cast<BlockInfo*>(sm + L::BLK);
  RowInfo* infos = reinterpret_cast<RowInfo*>(sm + L::INFO);
  if (sb & 1023u) {                                    // the swizzle's period: the kernel's only shared memory starts on one
    pdl_wait();
    if (tid == 0) atomicOr(a.tab.err, kErrLayout);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < L::RECORDS; ++i) {
      bar_init(bar(bRec + i), 1);
      bar_init(bar(bRecFree + i), kGroup);
    }
    for (int i = 0; i < L::SLOTS; ++i) {
      bar_init(bar(bFull + i), kGroup);
      bar_init(bar(bFree + i), 1);
    }
    for (int i = 0; i < L::STAGES; ++i) {
      bar_init(bar(bDone + i), 1);
      bar_init(bar(bTaken + i), 4);
    }
    for (int i = 0; i < kInfos; ++i) bar_init(bar(bInfo + i), 4);
    bar_init(bar(bTab), 1);
    bar_init(bar(bDrain), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMakers + 5) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sb + L::TMEM), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  __syncthreads();
  if (warp == kMakers + 4 && lane == 0) {                       // the tables (no kernel writes them)
    bar_arrive_tx(bar(bTab), static_cast<uint32_t>(L::TABLES * kTable));
    g2s(sb, a.tab.pih_sw, kTable, bar(bTab));
    g2s(sb + kTable, a.tab.ah_sw, kTable, bar(bTab));
    if (F32) {
      g2s(sb + 2 * kTable, a.tab.pil_sw, kTable, bar(bTab));
      g2s(sb + 3 * kTable, a.tab.al_sw, kTable, bar(bTab));
    }
  }
  if (tid < 8) {
    const Bytes t = table_bytes((tid & 4 ? a.vl : a.kl).g[tid & 1], (tid & 2) != 0);
    reinterpret_cast<uint4*>(sm + L::BOOK)[tid] = make_uint4(t.lo0, t.lo1, t.hi0, t.hi1);
  }
  pdl_wait();
  // pages before each sequence, where there are not too many of them; else `pages` for each
  const bool listed = a.batch <= kList;
  int *s_firsts = reinterpret_cast<int*>(sm + L::LIST), *s_sum = s_firsts + kList;
  int total = 0;
  if (listed) {
    constexpr int kPer = (kList + kThreads - 1) / kThreads;
    int n[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = tid * kPer + i;
      n[i] = 0;
      if (b < a.batch) {
        const ReadRun r = read_run(a, b);
        if (r.n > 0) n[i] = (r.start + r.n - 1) / kPage - r.start / kPage + 1;
      }
      sum += n[i];
    }
    int run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, run, o);
      run += lane >= o ? v : 0;
    }
    if (lane == 31) s_sum[tid >> 5] = run;
    __syncthreads();
    run -= sum;
    for (int w = 0; w < kThreads / 32; ++w) {
      run += w < (tid >> 5) ? s_sum[w] : 0;
      total += s_sum[w];
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (tid * kPer + i < a.batch) s_firsts[tid * kPer + i] = run;
      run += n[i];
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = *reinterpret_cast<const uint32_t*>(sm + L::TMEM);
  // The CTA's tiles, two of keys and two of values in turn (a pair for the two groups).
  const long long pages = listed ? total : static_cast<long long>(a.batch) * a.pages;
  const long long per_kind = (pages * a.H + kBlocks - 1) / kBlocks;
  const int kinds = (a.kc ? 1 : 0) + (a.vc ? 1 : 0);
  auto is_key = [&](int n) { return kinds == 2 ? (n & 2) == 0 : a.kc != nullptr; };
  auto tile_of = [&](int n) {                          // of its kind; per_kind or beyond: nothing
    const int k = kinds == 2 ? (n >> 2) * 2 + (n & 1) : n;
    return blockIdx.x + static_cast<long long>(k) * gridDim.x;
  };
  const int mine_of_kind = per_kind > blockIdx.x ? static_cast<int>((per_kind - blockIdx.x + gridDim.x - 1) / gridDim.x) : 0;
  const int count = kinds == 2 ? 2 * (mine_of_kind + (mine_of_kind & 1)) : mine_of_kind;     // (a last one may hold nothing)
  bool failed = false;
  auto wait = [&](int i, int phase) {
    if (!failed && __all_sync(0xffffffffu, wait_short(bar(i), phase & 1))) return true;
    failed = true;
    return false;
  };

  if (warp < kMakers) {
    // ---- left operands: row r of the tile, half of its channels --------------------------------------
    const int group = warp / kGroup, part = (warp >> 2) & 1, r = 32 * (warp & 3) + lane;
    const uint32_t ta = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + L::A + 32u * part;
    int slot = 0;                                      // operands, of both groups
    auto operands = [&](int n) { return (F32 ? 2 : 1) + (is_key(n) && a.kl.qjl ? 1 : 0); };
    if (group) slot = count ? operands(0) : 0;
    for (int n = group; n < count && !failed; n += 2) {
      const bool key = is_key(n);
      const KindLayout& K = key ? a.kl : a.vl;
      const int st = n % L::RECORDS;
      if (!wait(bRec + st, n / L::RECORDS)) break;
      const uint32_t rec = sb + L::REC + st * kRecord + (r >> 4) * K.block_bytes;
      const int s = r & 15;
      if (n >= kInfos && !wait(bInfo + n % kInfos, n / kInfos - 1)) break;
      const float n16 = __half2float(__ushort_as_half(static_cast<unsigned short>(lds16(rec + K.off_norm + 2 * s))));
      const float r16 = K.qjl ? __half2float(__ushort_as_half(static_cast<unsigned short>(lds16(rec + K.off_rnorm + 2 * s)))) : 0.0f;
      const float fa = n16 * (0.08838834764831845f / kPiScale), fb = r16 * (1.2533141373155003f / 128.0f);
      const float f = F32 ? fa : fmaxf(fabsf(fa), fabsf(fb)), inv = f > 0.0f ? 1.0f / f : 0.0f;
      if (part == 0) {
        const BlockInfo b = blocks[st * kBlocks + (r >> 4)];
        const bool live = s >= (b.slots & 0xFF) && s < (b.slots >> 8);
        // (a norm that is not finite spoils its row)
        infos[(n % kInfos) * kVec + r] = RowInfo{f + (fa - fa) + (fb - fb), fb, live ? b.row0 + s : -1, b.head};
      }
      auto open = [&]() {                              // the next operand's room
        if (slot >= L::SLOTS && !wait(bFree + slot % L::SLOTS, slot / L::SLOTS - 1)) return false;
        tc_after();
        return true;
      };
      auto close = [&](const uint32_t (&v)[32]) {
        tst32(ta + 64u * static_cast<uint32_t>(slot % L::SLOTS), v);
        tst_wait();
        tc_before();
        __syncwarp();
        if (lane == 0) bar_arrive(bar(bFull + slot % L::SLOTS));
        ++slot;
      };
#pragma unroll 1
      for (int low = F32 ? 1 : 0; low >= 0; --low) {   // (the small products first)
        uint32_t v[32];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int ch = 64 * part + 32 * q, g = ch < K.split ? 0 : 1, bits = K.g[g].bits;
          const uint32_t src = rec + s * K.code_bytes + (g ? (K.split * K.g[0].bits + (ch - K.split) * bits) / 8 : ch * bits / 8);
          const uint4 u = lds128(sb + L::BOOK + 16 * ((key ? 0 : 4) + 2 * low + g));
          const Bytes tb{u.x, u.y, u.z, u.w};
          if (bits == 4) block32<4>(tb, src, v + 16 * q);
          else if (bits == 3) block32<3>(tb, src, v + 16 * q);
          else if (bits == 2) block32<2>(tb, src, v + 16 * q);
          else block32<1>(tb, src, v + 16 * q);
        }
        if (!F32 && key && K.qjl) {
          const __half2 ra = __float2half2_rn(fa * inv);
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = mul_half2(v[k], ra);
        }
        __syncwarp();
        if (!open()) break;
        close(v);
      }
      if (failed) break;
      if (key && K.qjl) {
        const uint2 two = lds64(rec + K.off_signs + 16 * s + 8 * part);
        const __half2 rb = __float2half2_rn(F32 ? 1.0f : fb * inv);
        const uint32_t one = *reinterpret_cast<const uint32_t*>(&rb);
        uint32_t v[32];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint32_t w = ~(q ? two.y : two.x);     // a set bit is +1
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const uint32_t x = w >> (2 * k);
            v[16 * q + k] = one ^ ((x << 15) & 0x8000u) ^ ((x << 30) & 0x80000000u);
          }
        }
        __syncwarp();
        if (!open()) break;
        close(v);
      }
      fence_async_smem();                              // the next copy into the room comes behind these reads
      __syncwarp();
      if (lane == 0) bar_arrive(bar(bRecFree + st));
      if (n + 1 < count) slot += operands(n + 1);      // the other group's
    }
  } else if (warp < kMakers + 4) {
    // ---- rows: through shared memory, whole lines a store (32 bytes a lane's row: 1,000 cycles of the store pipe a tile; a
    // bulk copy a row: 2,600 to issue) -----------------------------------------------------------------
    const int r = 32 * (warp & 3) + lane;
    const uint32_t trow = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    for (int n = 0; n < count; ++n) {
      const bool key = is_key(n), two = F32 && key && a.kl.qjl;
      const int st = n % L::STAGES;
      if (!wait(bDone + st, n / L::STAGES)) break;
      tc_after();
      const RowInfo x = infos[(n % kInfos) * kVec + r];
      __syncwarp();
      if (lane == 0) bar_arrive(bar(bInfo + n % kInfos));
      const uint32_t acc = trow + static_cast<uint32_t>(L::ACC * st);
      const uint32_t room = sb + L::OUT + 32 * (warp & 3) * L::ROW, to = room + lane * L::ROW;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        float o[32];
        tld32(acc + 32u * c, o);
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] *= x.fa;
        if (two) {
          float p[32];
          tld32(acc + 128u + 32u * c, p);
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = fmaf(p[k], x.fb, o[k]);
        }
        if (F32) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            sts128(to + 128u * c + 16u * k, __float_as_uint(o[4 * k]), __float_as_uint(o[4 * k + 1]), __float_as_uint(o[4 * k + 2]), __float_as_uint(o[4 * k + 3]));
        } else {
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const __nv_bfloat162 y = __floats2bfloat162_rn(o[2 * k], o[2 * k + 1]);
            w[k] = *reinterpret_cast<const uint32_t*>(&y);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) sts128(to + 64u * c + 16u * k, w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
        }
      }
      tc_before();
      __syncwarp();
      if (lane == 0) bar_arrive(bar(bTaken + st));
      constexpr int kE = F32 ? 4 : 2, kLanes = 8 * kE, kRows = 32 / kLanes;      // lanes a row, rows at once
      const long long at = x.row < 0 ? -1 : (static_cast<long long>(x.row) * (key ? a.k_stride : a.v_stride) + static_cast<long long>(x.head) * 128) * kE;
      char* out = static_cast<char*>(key ? a.k_out : a.v_out) + 16 * (lane % kLanes);
#pragma unroll 1
      for (int i = 0; i < 32; i += 8 * kRows) {
        uint4 v[8];
        long long where[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int row = i + kRows * k + lane / kLanes;
          v[k] = lds128(room + row * L::ROW + 16 * (lane % kLanes));
          where[k] = __shfl_sync(0xffffffffu, at, row);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (where[k] >= 0) *reinterpret_cast<uint4*>(out + where[k]) = v[k];
      }
      __syncwarp();                                    // the room has been read
    }
  } else if (warp == kMakers + 4) {
    // ---- records: a lane per block, four tiles looked up at once and ahead of time --------------------
    struct Found {
      BlockInfo info;
      const uint8_t* src;
    };
    auto look_up = [&](int m) {                        // block lane % 8 of the CTA's tile m
      Found x{BlockInfo{0, 0, 0, 0}, nullptr};
      const long long g = tile_of(m) * kBlocks + (lane & 7), page = g / a.H;
      if (m >= count || page >= pages) return x;
      const bool key = is_key(m);
      int b = 0;
      if (listed) {                                    // the last sequence whose pages start at or before it
        int lo = 0, hi = a.batch - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) / 2;
          if (s_firsts[mid] <= page) lo = mid;
          else hi = mid - 1;
        }
        b = lo;
      } else {
        b = static_cast<int>(page / a.pages);
      }
      const int i = static_cast<int>(page - (listed ? s_firsts[b] : static_cast<long long>(b) * a.pages));
      x.info.head = static_cast<int>(g - page * a.H);
      const ReadRun run = read_run(a, b);
      const ReadPage p = read_page(a, b, run, i);
      if (p.id >= 0) {
        x.info.slots = p.s0 | (p.s1 << 8);
        x.info.row0 = run.row - p.off;
        x.src = (key ? a.kc : a.vc) + p.id * (key ? a.k_page_bytes : a.v_page_bytes) +
                static_cast<long long>(x.info.head) * (key ? a.kl : a.vl).block_bytes;
      }
      return x;
    };
    int n = 0;
    Found next = look_up(lane >> 3);
    while (n < count && !failed) {
      const Found cur = next;
      next = look_up(n + 4 + (lane >> 3));
      __syncwarp();
      for (int k = 0; k < 4 && n < count; ++k, ++n) {
        const KindLayout& K = is_key(n) ? a.kl : a.vl;
        const int st = n % L::RECORDS;
        const bool mine = (lane >> 3) == k;
        if (n >= L::RECORDS && !wait(bRecFree + st, n / L::RECORDS - 1)) break;
        if (mine) blocks[st * kBlocks + (lane & 7)] = cur.info;
        const uint32_t there = __ballot_sync(0xffffffffu, mine && cur.src != nullptr);
        __syncwarp();
        if (lane == 0) {
          if (there) bar_arrive_tx(bar(bRec + st), static_cast<uint32_t>(__popc(there) * K.block_bytes));
          else bar_arrive(bar(bRec + st));
        }
        __syncwarp();
        if (mine && cur.src) g2s(sb + L::REC + st * kRecord + (lane & 7) * K.block_bytes, cur.src, K.block_bytes, bar(bRec + st));
      }
    }
    // copies still in flight land before the CTA ends
    bool f2 = false;
    for (int s = n >= L::RECORDS ? n - L::RECORDS : 0; s < n; ++s) (void)bar_wait(bar(bRec + s % L::RECORDS), (s / L::RECORDS) & 1, f2);
    (void)bar_wait(bar(bTab), 0, f2);
    __syncwarp();
  } else {
    // ---- MMA issue, the warp converged ------------------------------------------------------------
    int slot = 0;
    bool ok = count ? wait(bTab, 0) : false;
    for (int n = 0; ok && n < count; ++n) {
      const bool two = is_key(n) && a.kl.qjl;
      const int st = n % L::STAGES;
      const uint32_t acc = tmem + static_cast<uint32_t>(L::ACC * st);
      ok = n < L::STAGES || wait(bTaken + st, n / L::STAGES - 1);
      if (!ok) break;
      auto operand = [&]() {                           // the next left operand
        const int s = slot % L::SLOTS;
        ok = wait(bFull + s, slot / L::SLOTS);
        tc_after();
        return tmem + L::A + 64u * static_cast<uint32_t>(s);
      };
      auto done = [&]() {
        mma_commit_warp(bar(bFree + slot % L::SLOTS));
        ++slot;
      };
      uint32_t x = operand();
      if (!ok) break;
      mma8_table(acc, x, sb, true);
      done();
      if (F32) {                                       // (that was the centroids' low part)
        x = operand();
        if (!ok) break;
        mma8_table(acc, x, sb + 2 * kTable, false);
        mma8_table(acc, x, sb, false);
        done();
      }
      if (two) {
        x = operand();
        if (!ok) break;
        if (F32) mma8_table(acc + 128u, x, sb + 3 * kTable, true);
        mma8_table(F32 ? acc + 128u : acc, x, sb + kTable, false);
        done();
      }
      mma_commit_warp(bar(bDone + st));
    }
    mma_commit_warp(bar(bDrain));                      // every MMA issued completes before the CTA ends
    bool f2 = false;
    (void)bar_wait(bar(bDrain), 0, f2);
    __syncwarp();
  }
  if (failed && lane == 0) atomicOr(a.tab.err, kErrTimeout);
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == kMakers + 5) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

template <bool F32>
cudaError_t launch_t(const ReadArgs& a, cudaStream_t s) {
  static std::atomic<unsigned long long> configured{0};
  const cudaError_t e = smem_attr_once(read_tc_kernel<F32>, RG<F32>::BYTES, configured);
  if (e != cudaSuccess) return e;
  const long long tiles = (static_cast<long long>(a.batch) * a.pages * a.H + kBlocks - 1) / kBlocks * ((a.kc ? 1 : 0) + (a.vc ? 1 : 0));
  const dim3 grid(static_cast<unsigned>(std::min<long long>(tiles, kv8_sm_count())));
  return launch_pdl(read_tc_kernel<F32>, grid, dim3(kThreads), RG<F32>::BYTES, s, a);
}

}  // namespace

bool read_tc_takes(const ReadArgs& a, int d) {
  const auto fits = [](const KindLayout& L) { return L.block_bytes * kBlocks <= kRecord; };
  return d == kD && a.m == kMaxM && fits(a.kl) && fits(a.vl);
}
cudaError_t launch_read_tc(const ReadArgs& a, bool f32, cudaStream_t s) { return f32 ? launch_t<true>(a, s) : launch_t<false>(a, s); }

}  // namespace tq
