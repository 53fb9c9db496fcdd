// Attention over packed prompts on the tensor cores (tcgen05) to fp32's accuracy, d = 64 or 128: fp32 inputs, and bf16 ones
// that the bf16 form does not take.
//
// An fp32 number is the sum of three bf16 ones, each the nearest to what the ones before leave (the first no larger than the
// largest), so that the remainders are exact.  The second and third are at most 2^-8 and 2^-17 of the number's power of two:
// of the products of two such sums the six largest count, and what is left out is 2^-24 of the product at most, to either side
// (parts cut off instead of rounded leave out up to 2^-21, always toward zero).  Per block of 128 query rows (row r = t G + g)
// of a KV head and 64 keys:
//   S = Q K^T                 six products (bf16 inputs: one), the small ones first: the tensor cores cut a sum instead of
//                             rounding it, and the large product's few steps are the ones that count
//   w = 2^(x - M)             fp32, M the running maximum
//   O = alpha O + w V         the tile's product by itself, six products again (bf16: three), added in rounded fp32 in registers
// What is not finite among keys and values is not multiplied in parts (infinity times a part that is zero would be NaN): it
// is taken out; a key's scores are then formed by the rows themselves, a value is added to the rows that see it.
//
// Warps 0-3: softmax (thread = row); 4-7: O and results; 8-11: keys, from memory to parts in shared memory; 12-15: values;
// both: queries; 16: MMA issue, a tile's scores ahead of the values before.  Every warp walks the list of items by itself.
// Every wait is bounded; a wait that gives up sets the device error word.
//
// Bound by the chain from rows in memory to parts, scores, weights and products: 3.9 us a tile, of which the MMAs take 1.7 and
// their operands 2.1 of shared memory by arithmetic (480 KB, the queries being read 48 times, at 128 B a cycle).  By counters
// (three prompts of up to 1,111 tokens) no unit is busy for more than a third of the time: issue slots 37%, integer pipe 34%,
// tensor pipe 27%; 6.6 stalls an issue wait for loads.
// Two thousand tokens, 32 / 8 heads, fp32: d = 128 256 us (134 TFLOP/s; CUDA cores 1,076), d = 64 172; three prompts of up to
// 1,111 tokens 96 (293); eight single tokens behind 4,000 keys 126 (their bytes take 38).  Slower were 16 warps for keys and
// values (274) and both at once by eight (356), fewer pieces in flight (279).

#include "tq_kv8.h"
#include "tq_prompt.h"
#include "tq_tc.cuh"
#include "tq_tc_attn.cuh"

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

namespace tq {
namespace {

using namespace tcx;

constexpr int kTok = 64, kRows = 128, kThreads = 640;
constexpr int kItemCost = 3;              // an item's start and end, in tiles' time
constexpr int kMinSpan = 1 + kItemCost;
constexpr int kSlots = 4;

// Registers: five groups of four warps start with 96 a thread.
constexpr int kRegsSoftmax = 120, kRegsSums = 168, kRegsLoad = 72, kRegsMma = 48;
static_assert(kRegsSoftmax + kRegsSums + 2 * kRegsLoad + kRegsMma <= 5 * 96, "more registers than the block starts with");

template <int D, bool F32>
struct PL {
  static constexpr int PARTS = F32 ? 3 : 1;
  static constexpr int QB = 2 * kRows * D, KB = 2 * kTok * D;       // bytes of a part
  static constexpr int Q = 0, K = Q + PARTS * QB, V = K + PARTS * KB;            // [part][64-channel panels][rows][128 B], swizzled
  static constexpr int ALPHA = V + PARTS * KB;         // [slot][row]: O's factor of a tile
  static constexpr int SUMS = ALPHA + kSlots * kRows * 4;           // [slot][row]: (M, l) of an item
  static constexpr int ODD = SUMS + kSlots * kRows * 8;             // [slot][warp]: keys (64 bits) with what is not finite; values
  static constexpr int BAR = ODD + kSlots * 4 * 8 + kSlots * 4 * 8;
};
enum Bar {
  bQFull = 0, bKFull, bKFree, bVFull, bPFull, bPDone, bSFull, bOFull = bSFull + 2, bOFree = bOFull + 2, bAlpha = bOFree + 2, bDrain = bAlpha + kSlots, bCount
};
template <int D, bool F32>
struct PB {
  static constexpr int TMEM = PL<D, F32>::BAR + 8 * ((bCount + 1) & ~1);
  static constexpr int BYTES = TMEM + 16;
};
static_assert(PB<128, true>::BYTES <= 232448, "shared memory per block");
static_assert(PL<64, false>::ALPHA >= 4 * (2 * kPromptList + 64), "the list's room");
// Tensor memory: two S of 64 columns, the weights' three parts of 32, two O of D.
constexpr uint32_t kColP = 128, kColO = 256;

__host__ __device__ constexpr uint32_t idesc_bf16(int n) { return idesc_f16(n) | (1u << 7) | (1u << 10); }
// 64 tokens a tile: panels 8 KB apart.
__device__ __forceinline__ uint64_t vdesc64(uint32_t at) { return vdesc(at) - (static_cast<uint64_t>((16384 - 8192) >> 4) << 16); }

template <bool F32>
__device__ __forceinline__ void load8(const void* p, long long at, float (&x)[8]) {
  if (F32) {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    const float4 a = f[0], b = f[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + at);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(u[i] << 16), x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ bool is_odd(float x) { return (__float_as_uint(x) & 0x7F800000u) == 0x7F800000u; }
// The next parts of a and b as a pair of bf16, and what they leave.  FIRST: of numbers that may be beyond the largest bf16
// (infinity is one in the second part then).
template <bool FIRST>
__device__ __forceinline__ uint32_t part_pair(float& a, float& b) {
  uint32_t w;
  if (FIRST) asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
  a = __fsub_rn(a, __uint_as_float(w << 16));
  b = __fsub_rn(b, __uint_as_float(w & 0xFFFF0000u));
  return w;
}
// 16 bytes of each part at `at`.
template <int PARTS>
__device__ __forceinline__ void put_parts(uint32_t at, int bytes, float (&x)[8]) {
#pragma unroll
  for (int p = 0; p < PARTS; ++p) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = p == 0 ? part_pair<PARTS == 3>(x[2 * i], x[2 * i + 1]) : part_pair<false>(x[2 * i], x[2 * i + 1]);
    sts128(at + p * bytes, w[0], w[1], w[2], w[3]);
  }
}
// <q, k> of one row, for keys that are not finite.
template <int D, bool F32>
__device__ __noinline__ float row_dot(const void* q, long long qa, const void* k, long long ka) {
  float s = 0.0f;
#pragma unroll 1
  for (int c = 0; c < D; c += 8) {
    float x[8], y[8];
    load8<F32>(q, qa + c, x);
    load8<F32>(k, ka + c, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(x[i], y[i], s);
  }
  return s;
}

template <int D, bool F32>
__global__ void __launch_bounds__(kThreads, 1) prompt_parts_kernel(const __grid_constant__ PromptArgs a, int mode) {
  using L = PL<D, F32>;
  using B = PB<D, F32>;
  constexpr int CH = D / 8;                            // 16-byte pieces of a row's part
  extern __shared__ __align__(1024) unsigned char sm_raw[];
  unsigned char* sm = sm_raw;
  const uint32_t sb = su32(sm);
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31, group = warp >> 2;
  auto bar = [&](int i) { return sb + L::BAR + 8u * static_cast<uint32_t>(i); };
  float* alphas = reinterpret_cast<float*>(sm + L::ALPHA);
  float2* sums = reinterpret_cast<float2*>(sm + L::SUMS);
  volatile unsigned long long* odd_keys = reinterpret_cast<volatile unsigned long long*>(sm + L::ODD);
  volatile unsigned long long* odd_values = odd_keys + kSlots * 4;
  PSplit* splits = reinterpret_cast<PSplit*>(a.part);              // one per CTA, then the partials' slots
  if (sb & 1023u) {                                    // the swizzles' period
    pdl_wait();
    if (tid == 0) {
      atomicOr(a.err, kErrLayout);
      if (mode == kPromptCut) splits[blockIdx.x].valid = 0;
    }
    return;
  }
  if (tid == 0) {
    bar_init(bar(bQFull), 8);
    bar_init(bar(bKFull), 4);
    bar_init(bar(bKFree), 1);
    bar_init(bar(bVFull), 4);
    bar_init(bar(bPFull), 4);
    bar_init(bar(bPDone), 1);
    for (int i = 0; i < 2; ++i) {
      bar_init(bar(bSFull + i), 1);
      bar_init(bar(bOFull + i), 1);
      bar_init(bar(bOFree + i), 4);
    }
    for (int i = 0; i < kSlots; ++i) bar_init(bar(bAlpha + i), 4);
    bar_init(bar(bDrain), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 16) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sb + B::TMEM), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  if (mode == kPromptCut) pdl_trigger();               // the join's launch
  if (F32) prompt_zero_rows<float>(a, D);
  else prompt_zero_rows<__nv_bfloat16>(a, D);
  PromptSpan span{};
  if (mode != kPromptTurns) span = prompt_span<kTok, kItemCost, kThreads>(a, a.H, kMinSpan, reinterpret_cast<int*>(sm));
  fence_async_smem();
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = *reinterpret_cast<const uint32_t*>(sm + B::TMEM);
  float* parts = a.part + static_cast<size_t>(gridDim.x) * (sizeof(PSplit) / sizeof(float));
  bool failed = false;
  // a warp's wait for phase `phase` of a barrier; once one gave up, every later one returns at once
  auto wait = [&](int i, int phase) {
    if (!failed && __all_sync(0xffffffffu, wait_short(bar(i), phase & 1))) return true;
    failed = true;
    return false;
  };
  auto arrive = [&](int i) {
    __syncwarp();
    if (lane == 0) bar_arrive(bar(i));
  };
  PromptWalk<kTok, kItemCost> w;
  w.start(a, span, a.H, mode);
  int T = 0;                                           // tiles so far

  if (group == 0) {
    // ---- softmax -----------------------------------------------------------------------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const uint32_t trow = tmem + (static_cast<uint32_t>(32 * warp) << 16);
    const float f = a.scale_log2;
    for (int n = 0; !failed && w.next(a, span); ++n) {
      const PromptBlock& b = w.blk;
      const bool live = tid < b.rows;
      const int gr = b.r0 + tid, p = live ? b.seq.m - b.seq.n + gr / a.G : -1;
      float m = -INFINITY, l = 0.0f;
      for (int t = w.t0; t < w.t1; ++t, ++T) {
        if (!wait(bSFull + (T & 1), T >> 1)) break;
        tc_after();
        const uint32_t ts = trow + 64u * static_cast<uint32_t>(T & 1);
        const int j0 = b.first_key<kTok>(t);
        unsigned long long odd = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) odd |= odd_keys[4 * (T % kSlots) + i];
        if (__builtin_expect(__any_sync(0xffffffffu, odd != 0), 0)) {
#pragma unroll 1
          for (; odd; odd &= odd - 1) {
            const int k = __ffsll(static_cast<long long>(odd)) - 1;
            float s = 0.0f;
            if (live)
              s = row_dot<D, F32>(a.q, (static_cast<long long>(b.seq.q0) + gr / a.G) * a.qs + static_cast<long long>(w.h * a.G + gr % a.G) * D, a.k,
                                  (static_cast<long long>(b.seq.k0) + j0 + k) * a.ks + static_cast<long long>(w.h) * D);
            __syncwarp();
            tst1(ts + k, __float_as_uint(s));
          }
          tst_wait();
        }
        float y[kTok], top = -INFINITY;
        tld32(ts, *reinterpret_cast<float(*)[32]>(y));
        tld32(ts + 32u, *reinterpret_cast<float(*)[32]>(y + 32));
#pragma unroll
        for (int c = 0; c < kTok; c += 32) {
          const uint32_t see = prompt_seen32(p, j0 + c, a.window, a.sinks);
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            y[c + k] = (see >> k) & 1u ? __fmul_rn(y[c + k], f) : -INFINITY;
            top = fmaxf(top, y[c + k]);
          }
        }
        const float mn = fmaxf(m, top), ref = mn == -INFINITY ? 0.0f : mn, al = ex2(m - ref);
        m = mn;
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int k = 0; k < kTok; k += 2) {
          y[k] = ex2(__fsub_rn(y[k], ref));
          y[k + 1] = ex2(__fsub_rn(y[k + 1], ref));
          s0 += y[k];
          s1 += y[k + 1];
        }
        l = fmaf(l, al, s0 + s1);
        __syncwarp();
        if (T > 0 && !wait(bPDone, T - 1)) break;      // the weights' room
        tc_after();
#pragma unroll
        for (int c = 0; c < kTok; c += 32)
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            uint32_t u[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) u[k] = part_pair<false>(y[c + 2 * k], y[c + 2 * k + 1]);
            tst16(trow + kColP + 32u * i + c / 2, u);
          }
        alphas[kRows * (T % kSlots) + tid] = al;
        if (t == w.t1 - 1) sums[kRows * (n % kSlots) + tid] = make_float2(m, l);
        tst_wait();
        tc_before();
        arrive(bPFull);
        if (lane == 0) bar_arrive(bar(bAlpha + T % kSlots));
      }
      w.pass(a, span);
    }
  } else if (group == 1) {
    // ---- O, results (or the part's sums) -----------------------------------------------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSums));
    const int r = tid - 128;
    const uint32_t trow = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    for (int n = 0; !failed && w.next(a, span); ++n) {
      const PromptBlock& b = w.blk;
      const bool live = r < b.rows;
      const int gr = b.r0 + r, tok = gr / a.G, g = gr - tok * a.G, p = live ? b.seq.m - b.seq.n + tok : -1;
      float o[D];
#pragma unroll
      for (int c = 0; c < D; ++c) o[c] = 0.0f;
      for (int t = w.t0; t < w.t1; ++t, ++T) {
        if (!wait(bAlpha + T % kSlots, T / kSlots) || !wait(bOFull + (T & 1), T >> 1)) break;
        tc_after();
        const float al = alphas[kRows * (T % kSlots) + r];
        const uint32_t to = trow + kColO + 128u * static_cast<uint32_t>(T & 1);
#pragma unroll
        for (int c = 0; c < D; c += 16) {
          float x[16];
          tld16(to + c, x);
#pragma unroll
          for (int k = 0; k < 16; ++k) o[c + k] = fmaf(o[c + k], al, x[k]);
        }
        unsigned long long odd = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) odd |= odd_values[4 * (T % kSlots) + i];
        if (__builtin_expect(__any_sync(0xffffffffu, odd != 0), 0)) {
          const int j0 = b.first_key<kTok>(t);
#pragma unroll 1
          for (; odd; odd &= odd - 1) {
            const int j = j0 + __ffsll(static_cast<long long>(odd)) - 1;
            const bool see = prompt_sees(p, j, a.window, a.sinks);
            const long long at = (static_cast<long long>(b.seq.k0) + j) * a.vs + static_cast<long long>(w.h) * D;
#pragma unroll
            for (int c = 0; c < D; c += 8) {
              float x[8];
              load8<F32>(a.v, at + c, x);
#pragma unroll
              for (int k = 0; k < 8; ++k) o[c + k] += see && is_odd(x[k]) ? x[k] : 0.0f;
            }
          }
          __syncwarp();
        }
        tc_before();
        const float2 ml = t == w.t1 - 1 ? sums[kRows * (n % kSlots) + r] : make_float2(0.0f, 0.0f);
        arrive(bOFree + (T & 1));
        if (t < w.t1 - 1 || !live) continue;
        float4* to4;
        float inv = 1.0f;
        if (w.slot < 0) {
          inv = prompt_inverse(ml.y, p);
          const long long at = ((static_cast<long long>(b.seq.q0) + tok) * a.Hq + w.h * a.G + g) * D;
          if (!F32) {
            uint4* to16 = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + at);
#pragma unroll
            for (int c = 0; c < D; c += 8) {
              uint32_t u[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const __nv_bfloat162 v = __floats2bfloat162_rn(o[c + 2 * k] * inv, o[c + 2 * k + 1] * inv);
                u[k] = *reinterpret_cast<const uint32_t*>(&v);
              }
              to16[c / 8] = make_uint4(u[0], u[1], u[2], u[3]);
            }
            continue;
          }
          to4 = reinterpret_cast<float4*>(static_cast<float*>(a.out) + at);
        } else {
          float* part = parts + (static_cast<long long>(w.slot) * kRows + r) * (D + 4);
          *reinterpret_cast<float4*>(part) = make_float4(ml.x, ml.y, 0.0f, 0.0f);
          to4 = reinterpret_cast<float4*>(part + 4);
        }
#pragma unroll
        for (int c = 0; c < D; c += 4) to4[c / 4] = make_float4(o[c] * inv, o[c + 1] * inv, o[c + 2] * inv, o[c + 3] * inv);
      }
      __syncwarp();
      w.pass(a, span);
    }
    if (mode == kPromptCut && tid == 128) splits[blockIdx.x] = w.cut;
  } else if (group < 4) {
    // ---- keys (group 2), values (group 3), queries (both): to parts ---------------------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLoad));
    const bool keys = group == 2;
    const int i0 = tid & 127;
    for (int n = 0; !failed && w.next(a, span); ++n) {
      const PromptBlock& b = w.blk;
      if (T > 0 && !wait(bKFree, T - 1)) break;        // the scores of the item before have read its queries
#pragma unroll 1
      for (int i = i0 + (keys ? 0 : 128); i < kRows * CH; i += 1024) {
        float x[4][8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int at = i + 256 * k, r = at / CH, c = at % CH, gr = b.r0 + r, tok = gr / a.G;
#pragma unroll
          for (int e = 0; e < 8; ++e) x[k][e] = 0.0f;
          if (at < kRows * CH && r < b.rows)
            load8<F32>(a.q, (static_cast<long long>(b.seq.q0) + tok) * a.qs + static_cast<long long>(w.h * a.G + gr - tok * a.G) * D + 8 * c, x[k]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int at = i + 256 * k;
          if (at < kRows * CH) put_parts<L::PARTS>(sb + L::Q + chunk_off(at / CH, at % CH, kRows), L::QB, x[k]);
        }
      }
      fence_async_smem();
      arrive(bQFull);
      const void* from = keys ? a.k : a.v;
      const long long stride = keys ? a.ks : a.vs;
      const uint32_t dst = sb + (keys ? L::K : L::V);
      for (int t = w.t0; t < w.t1; ++t, ++T) {
        const int j0 = b.first_key<kTok>(t);
        unsigned long long odd = 0;
        bool free = false;
#pragma unroll 1
        for (int i = i0; i < kTok * CH; i += 512) {
          float x[4][8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = (i + 128 * k) / CH, c = (i + 128 * k) % CH, j = j0 + r;
#pragma unroll
            for (int e = 0; e < 8; ++e) x[k][e] = 0.0f;
            // what no row sees may hold anything
            if (j <= b.pmax && (!a.window || j > b.pmin - a.window || j < a.sinks))
              load8<F32>(from, (static_cast<long long>(b.seq.k0) + j) * stride + static_cast<long long>(w.h) * D + 8 * c, x[k]);
          }
          __syncwarp();
          if (!free && T > 0 && !wait(keys ? bKFree : bPDone, T - 1)) break;
          free = true;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = (i + 128 * k) / CH, c = (i + 128 * k) % CH;
            bool bad = false;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const bool o = is_odd(x[k][e]);
              bad |= o;
              x[k][e] = o ? 0.0f : x[k][e];
            }
            odd |= static_cast<unsigned long long>(bad) << r;
            put_parts<L::PARTS>(dst + chunk_off(r, c, kTok), L::KB, x[k]);
          }
        }
        if (failed) break;
        const unsigned lo = __reduce_or_sync(0xffffffffu, static_cast<unsigned>(odd)), hi = __reduce_or_sync(0xffffffffu, static_cast<unsigned>(odd >> 32));
        if (lane == 0) (keys ? odd_keys : odd_values)[4 * (T % kSlots) + (warp & 3)] = (static_cast<unsigned long long>(hi) << 32) | lo;
        fence_async_smem();
        arrive(keys ? bKFull : bVFull);
      }
      w.pass(a, span);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsMma));
    if (warp == 16) {
      // ---- MMA issue, the warp converged -------------------------------------------------------
      auto values = [&](int x) {
        if (!wait(bVFull, x) || (x >= 2 && !wait(bOFree + (x & 1), (x >> 1) - 1)) || !wait(bPFull, x)) return;
        tc_after();
        const uint32_t to = tmem + kColO + 128u * static_cast<uint32_t>(x & 1), id = idesc_bf16(D) | (1u << 16);
#pragma unroll 1
        for (int i = F32 ? 0 : 3; i < 6; ++i) {
          // parts of the weights and of the values: (2,0) (1,1) (0,2) (1,0) (0,1) (0,0); one of the values: (2,0) (1,0) (0,0)
          const int pa = F32 ? (0x001012 >> (4 * i)) & 3 : 5 - i, pb = F32 ? (0x010210 >> (4 * i)) & 3 : 0;
          const uint64_t v = vdesc64(sb + L::V + pb * L::KB);
          const uint32_t u = tmem + kColP + 32u * pa;
#pragma unroll
          for (int s = 0; s < kTok / 16; ++s) mma_ts_warp(to, u + 8u * s, v + 128u * s, id, i > (F32 ? 0 : 3) || s > 0 ? 1u : 0u);
        }
        mma_commit_warp(bar(bPDone));
        mma_commit_warp(bar(bOFull + (x & 1)));
      };
      for (int n = 0; !failed && w.next(a, span); ++n) {
        if (!wait(bQFull, n)) break;
        for (int t = w.t0; t < w.t1 && !failed; ++t, ++T) {
          if (!wait(bKFull, T)) break;
          tc_after();
          const uint32_t to = tmem + 64u * static_cast<uint32_t>(T & 1);
#pragma unroll 1
          for (int i = F32 ? 0 : 5; i < 6; ++i) {
            const int pa = F32 ? (0x001012 >> (4 * i)) & 3 : 0, pb = F32 ? (0x010210 >> (4 * i)) & 3 : 0;
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
              mma_ss_warp(to, kdesc(sb + L::Q + pa * L::QB, kRows, s), kdesc(sb + L::K + pb * L::KB, kTok, s), idesc_bf16(kTok),
                          i > (F32 ? 0 : 5) || s > 0 ? 1u : 0u);
          }
          mma_commit_warp(bar(bSFull + (T & 1)));
          mma_commit_warp(bar(bKFree));
          if (t > w.t0) values(T - 1);
        }
        if (!failed) values(T - 1);
        w.pass(a, span);
      }
      mma_commit_warp(bar(bDrain));                    // every MMA issued completes before the CTA ends
      bool f2 = false;
      (void)bar_wait(bar(bDrain), 0, f2);
      __syncwarp();
    }
  }
  if (failed && lane == 0) atomicOr(a.err, kErrTimeout);
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 16) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

template <int D, bool F32>
cudaError_t launch_t(const PromptArgs& args, cudaStream_t s) {
  PromptArgs a = args;
  a.rows = kRows;
  a.most = prompt_list_room(a, kTok, kItemCost);
  static std::atomic<unsigned long long> configured{0};
  cudaError_t e = smem_attr_once(prompt_parts_kernel<D, F32>, PB<D, F32>::BYTES, configured);
  if (e != cudaSuccess) return e;
  const long long items = prompt_most_blocks(a) * a.H, tiles = a.max_k / kTok + 2 + a.sinks / kTok;
  const int sms = prompt_sms();
  // items of few tiles are not cut (and need no join)
  const int mode = !prompt_splits(a) ? kPromptTurns : tiles > 4 ? kPromptCut : kPromptWhole;
  const long long most = mode == kPromptCut ? (items * (tiles + kItemCost) + kMinSpan - 1) / kMinSpan : items;
  const int ctas = static_cast<int>(most < sms ? (most < 1 ? 1 : most) : sms);
  e = launch_pdl(prompt_parts_kernel<D, F32>, dim3(ctas), dim3(kThreads), PB<D, F32>::BYTES, s, a, mode);
  if (e != cudaSuccess || mode != kPromptCut) return e;
  return launch_prompt_join(a, D, F32, ctas, kRows, s);
}

}  // namespace

// All sizes but a tile of keys for a few rows, which is latency alone (4 tokens, 4 heads per KV head: 14 us, CUDA cores 11);
// from there on this form is ahead (5 tokens 14 us against 17; eight single tokens behind 4,000 keys 126 against 230, fp32).
bool prompt_parts_takes(const PromptArgs& a, int d) {
  return (d == 64 || d == 128) && (a.max_k > kTok || static_cast<long long>(a.max_q) * a.G > 16);
}
size_t prompt_parts_workspace(int d) {
  return static_cast<size_t>(prompt_sms()) * (sizeof(PSplit) + 2 * sizeof(float) * kRows * (d + 4));
}
cudaError_t launch_prompt_parts(const PromptArgs& a, int d, bool f32, cudaStream_t s) {
  switch (d) {
    case 64: return f32 ? launch_t<64, true>(a, s) : launch_t<64, false>(a, s);
    case 128: return f32 ? launch_t<128, true>(a, s) : launch_t<128, false>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace tq
