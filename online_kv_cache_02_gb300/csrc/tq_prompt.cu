// Attention over packed prompts on CUDA cores: the head dimensions that neither tensor-core form takes, and fp32 calls of
// few rows and keys.
//
//   s_j = scale <q, k_j>,  out = sum_j 2^(s_j log2 e - M) v_j / sum_j 2^(s_j log2 e - M),  M the running maximum,
// over the keys j that the query's position sees.  A CTA takes 64 query rows of a KV head, or 16 where no sequence has more
// (row r = t G + g, so that a key that is read serves every query head of its group) and 64 keys at a time; keys and queries stand transposed in
// shared memory, so that a thread's 4 x 4 scores take two 16-byte loads per channel; sums are fp32 throughout.
// Bound by the FMA pipes and the shared-memory loads that feed them (27 to 32 TFLOP/s; 2,048 tokens, 16 / 4 heads, d = 256,
// fp32: 1,253 us).  Two blocks an SM up to d = 128, the weights where the keys were: by a quarter faster than one.

#include "tq_kv8.h"
#include "tq_prompt.h"

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

namespace tq {
namespace {

constexpr int kTok = 64, kThreads = 256;
constexpr int kItemCost = 2;              // an item's start and end, in tiles' time
constexpr int kMinSpan = 1 + kItemCost;
constexpr int kLd = 68;                   // floats from channel to channel of the transposed tiles

// RM: query rows a thread (16 threads side by side hold them all)
template <int D, int RM>
struct SG {
  static constexpr int ROWS = 16 * RM, LQ = ROWS + 4;              // LQ: floats from channel to channel of the queries, key to key of the weights
  // floats; the weights stand where the keys were (with a barrier between), for two blocks an SM up to d = 128
  static constexpr int Q = 0, K = Q + D * LQ, P = K, V = K + (D > kTok ? D : kTok) * kLd, END = V + kTok * D;
  static constexpr int BYTES = 4 * (END > 2 * kPromptList + 64 ? END : 2 * kPromptList + 64);
};

__device__ __forceinline__ float exp2_fast(float x) {            // relative error about 2^-22; 0 for -inf
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Four channels of a row in fp32.
template <bool F32>
__device__ __forceinline__ float4 load4(const void* p, long long at) {
  if (F32) return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
  const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const unsigned short*>(p) + at);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xFFFF0000u));
}
__device__ __forceinline__ bool finite4(float4 x) {
  return fabsf(x.x) <= 3.4028234e38f && fabsf(x.y) <= 3.4028234e38f && fabsf(x.z) <= 3.4028234e38f && fabsf(x.w) <= 3.4028234e38f;
}

// RM floats of shared memory.
template <int RM>
__device__ __forceinline__ void load_rows(const float* p, float (&x)[RM]) {
  if constexpr (RM == 4) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else {
    x[0] = *p;
  }
}

template <int D, bool F32, int RM>
__global__ void __launch_bounds__(kThreads, D <= 128 ? 2 : 1) prompt_simt_kernel(const __grid_constant__ PromptArgs a, int mode) {
  using L = SG<D, RM>;
  constexpr int kRows = L::ROWS, LQ = L::LQ;
  extern __shared__ __align__(16) float sm[];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  pdl_wait();
  if (mode == kPromptCut) pdl_trigger();
  if (F32) prompt_zero_rows<float>(a, D);
  else prompt_zero_rows<__nv_bfloat16>(a, D);
  PromptSpan span{};
  if (mode != kPromptTurns) span = prompt_span<kTok, kItemCost, kThreads>(a, a.H, kMinSpan, reinterpret_cast<int*>(sm));
  PSplit* splits = reinterpret_cast<PSplit*>(a.part);
  float* parts = a.part + static_cast<size_t>(gridDim.x) * (sizeof(PSplit) / sizeof(float));
  PromptWalk<kTok, kItemCost> w;
  w.start(a, span, a.H, mode);
  while (w.next(a, span)) {
    const PromptBlock& b = w.blk;
    // ---- queries, transposed: a warp's lanes take 32 rows of the same channels ------------------
    __syncthreads();                                   // the last item's shared memory has been read
    for (int i = tid; i < kRows * (D / 4); i += kThreads) {
      const int r = i % kRows, c = 4 * (i / kRows);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < b.rows) {
        const int gr = b.r0 + r, tok = gr / a.G, g = gr - tok * a.G;
        x = load4<F32>(a.q, (static_cast<long long>(b.seq.q0) + tok) * a.qs + static_cast<long long>(w.h * a.G + g) * D + c);
      }
      float* q = sm + L::Q + c * LQ + r;
      q[0] = x.x, q[LQ] = x.y, q[2 * LQ] = x.z, q[3 * LQ] = x.w;
    }
    int p[RM];
    float m[RM], l[RM], o[RM][D / 16];
#pragma unroll
    for (int i = 0; i < RM; ++i) {
      const int r = RM * ty + i;
      p[i] = r < b.rows ? b.seq.m - b.seq.n + (b.r0 + r) / a.G : -1;
      m[i] = -INFINITY;
      l[i] = 0.0f;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) o[i][c] = 0.0f;
    }
    for (int t = w.t0; t < w.t1; ++t) {
      const int j0 = b.first_key<kTok>(t);
      __syncthreads();                                 // the last tile's keys, values and weights have been read
      bool odd = false;                                // a value that is not finite
      for (int i = tid; i < kTok * (D / 4); i += kThreads) {
        const int r = i % kTok, c = 4 * (i / kTok), j = j0 + r;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j <= b.pmax) x = load4<F32>(a.k, (static_cast<long long>(b.seq.k0) + j) * a.ks + static_cast<long long>(w.h) * D + c);
        float* k = sm + L::K + c * kLd + r;
        k[0] = x.x, k[kLd] = x.y, k[2 * kLd] = x.z, k[3 * kLd] = x.w;
      }
      for (int i = tid; i < kTok * (D / 4); i += kThreads) {
        const int r = i / (D / 4), c = 4 * (i % (D / 4)), j = j0 + r;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);    // what no row sees may hold anything
        if (j <= b.pmax && (!a.window || j > b.pmin - a.window || j < a.sinks))
          x = load4<F32>(a.v, (static_cast<long long>(b.seq.k0) + j) * a.vs + static_cast<long long>(w.h) * D + c);
        odd |= !finite4(x);
        *reinterpret_cast<float4*>(sm + L::V + r * D + c) = x;
      }
      odd = __syncthreads_or(odd);
      // ---- scores: rows RM ty + i, keys 4 tx + k -------------------------------------------------
      float s[RM][4] = {};
#pragma unroll 8
      for (int c = 0; c < D; ++c) {
        float qa[RM];
        load_rows<RM>(sm + L::Q + c * LQ + RM * ty, qa);
        const float4 k = *reinterpret_cast<const float4*>(sm + L::K + c * kLd + 4 * tx);
        const float ka[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
        for (int i = 0; i < RM; ++i)
#pragma unroll
          for (int n = 0; n < 4; ++n) s[i][n] = fmaf(qa[i], ka[n], s[i][n]);
      }
#pragma unroll
      for (int i = 0; i < RM; ++i) {
        float top = -INFINITY;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          s[i][n] = prompt_sees(p[i], j0 + 4 * tx + n, a.window, a.sinks) ? __fmul_rn(s[i][n], a.scale_log2) : -INFINITY;
          top = fmaxf(top, s[i][n]);
        }
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float mn = fmaxf(m[i], top), ref = mn == -INFINITY ? 0.0f : mn, al = exp2_fast(m[i] - ref);
        m[i] = mn;
        float sum = 0.0f;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          s[i][n] = exp2_fast(__fsub_rn(s[i][n], ref));
          sum += s[i][n];
        }
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        l[i] = fmaf(l[i], al, sum);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) o[i][c] *= al;
      }
      __syncthreads();                                 // the keys have been read
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        float* w = sm + L::P + (4 * tx + n) * LQ + RM * ty;
        if constexpr (RM == 4) *reinterpret_cast<float4*>(w) = make_float4(s[0][n], s[1][n], s[2][n], s[3][n]);
        else *w = s[0][n];
      }
      __syncthreads();
      // ---- values: channels 2 tx + 32 c, + 1 -----------------------------------------------------
      auto values = [&](bool masked) {
#pragma unroll 4
        for (int k = 0; k < kTok; ++k) {
          float pa[RM];
          load_rows<RM>(sm + L::P + k * LQ + RM * ty, pa);
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            const float2 v = *reinterpret_cast<const float2*>(sm + L::V + k * D + 2 * tx + 32 * c);
#pragma unroll
            for (int i = 0; i < RM; ++i) {
              if (masked && !prompt_sees(p[i], j0 + k, a.window, a.sinks)) continue;
              o[i][2 * c] = fmaf(pa[i], v.x, o[i][2 * c]);
              o[i][2 * c + 1] = fmaf(pa[i], v.y, o[i][2 * c + 1]);
            }
          }
        }
      };
      if (__builtin_expect(odd, 0)) values(true);      // a hidden infinity times a weight of zero would be NaN
      else values(false);
    }
    // ---- results, or the part's sums ------------------------------------------------------------
#pragma unroll
    for (int i = 0; i < RM; ++i) {
      const int r = RM * ty + i;
      if (r >= b.rows) continue;
      const int gr = b.r0 + r, tok = gr / a.G, g = gr - tok * a.G;
      if (w.slot < 0) {
        const float inv = prompt_inverse(l[i], p[i]);
        const long long at = ((static_cast<long long>(b.seq.q0) + tok) * a.Hq + w.h * a.G + g) * D;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          if (F32)
            *reinterpret_cast<float2*>(static_cast<float*>(a.out) + at + 2 * tx + 32 * c) = make_float2(o[i][2 * c] * inv, o[i][2 * c + 1] * inv);
          else
            *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(a.out) + at + 2 * tx + 32 * c) =
                __floats2bfloat162_rn(o[i][2 * c] * inv, o[i][2 * c + 1] * inv);
        }
      } else {
        float* x = parts + (static_cast<long long>(w.slot) * kRows + r) * (D + 4);
        if (tx == 0) *reinterpret_cast<float4*>(x) = make_float4(m[i], l[i], 0.0f, 0.0f);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) *reinterpret_cast<float2*>(x + 4 + 2 * tx + 32 * c) = make_float2(o[i][2 * c], o[i][2 * c + 1]);
      }
    }
    w.pass(a, span);
  }
  if (mode == kPromptCut && tid == 0) splits[blockIdx.x] = w.cut;
}

// Joins the parts of the items that cross spans: a warp per row.
template <int D, bool F32>
__global__ void __launch_bounds__(256) prompt_join_kernel(const __grid_constant__ PromptArgs a, int ctas, int rows) {
  constexpr int PART = D + 4, V4 = (D + 127) / 128;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x;
  pdl_wait();
  const PSplit cut = reinterpret_cast<const PSplit*>(a.part)[c];
  const int rr = 8 * blockIdx.y + warp;
  if (!cut.valid || rr >= cut.rows) return;
  const float* parts = a.part + static_cast<size_t>(ctas) * (sizeof(PSplit) / sizeof(float));
  const long long step = static_cast<long long>(rows) * PART;
  // the first part is in its CTA's second slot, the others in their CTAs' first
  auto part = [&](int k) { return parts + (2LL * k + (k == c ? 1 : 0)) * step + static_cast<long long>(rr) * PART; };
  float M = -INFINITY;
  for (int k = c + lane; k <= cut.last; k += 32) M = fmaxf(M, part(k)[0]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float ref = M == -INFINITY ? 0.0f : M;         // no key, or scores that are all NaN: sums of 0 or NaN
  float L = 0.0f;
  float4 acc[V4];
#pragma unroll
  for (int i = 0; i < V4; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = c; k <= cut.last; ++k) {
    const float* p = part(k);
    const float f = exp2_fast(p[0] - ref);
    L = fmaf(f, p[1], L);
#pragma unroll
    for (int i = 0; i < V4; ++i) {
      if (128 * i + 4 * lane >= D) continue;
      const float4 x = *reinterpret_cast<const float4*>(p + 4 + 128 * i + 4 * lane);
      acc[i].x = fmaf(f, x.x, acc[i].x), acc[i].y = fmaf(f, x.y, acc[i].y), acc[i].z = fmaf(f, x.z, acc[i].z), acc[i].w = fmaf(f, x.w, acc[i].w);
    }
  }
  const int gr = cut.r0 + rr, tok = gr / a.G, g = gr - tok * a.G;
  const float inv = prompt_inverse(L, cut.p0 + tok);
  const long long at = ((static_cast<long long>(cut.q0) + tok) * a.Hq + cut.h * a.G + g) * D;
#pragma unroll
  for (int i = 0; i < V4; ++i) {
    const int ch = 128 * i + 4 * lane;
    if (ch >= D) continue;
    const float4 y = make_float4(acc[i].x * inv, acc[i].y * inv, acc[i].z * inv, acc[i].w * inv);
    if (F32) {
      *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at + ch) = y;
    } else {
      const __nv_bfloat162 y0 = __floats2bfloat162_rn(y.x, y.y), y1 = __floats2bfloat162_rn(y.z, y.w);
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at + ch) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&y0), *reinterpret_cast<const uint32_t*>(&y1));
    }
  }
}

int simt_ctas(int d) { return prompt_sms() * (d > 128 ? 1 : 2); }

template <int D, int RM>
cudaError_t launch_t(const PromptArgs& args, bool f32, cudaStream_t s) {
  using L = SG<D, RM>;
  PromptArgs a = args;
  a.rows = L::ROWS;
  a.most = prompt_list_room(a, kTok, kItemCost);
  static std::atomic<unsigned long long> done16{0}, done32{0};
  cudaError_t e = f32 ? smem_attr_once(prompt_simt_kernel<D, true, RM>, L::BYTES, done32)
                      : smem_attr_once(prompt_simt_kernel<D, false, RM>, L::BYTES, done16);
  if (e != cudaSuccess) return e;
  const long long tiles = a.max_k / kTok + 2 + a.sinks / kTok;
  // items of few tiles are not cut (and need no join)
  const int mode = !prompt_splits(a) ? kPromptTurns : tiles > 4 ? kPromptCut : kPromptWhole;
  const int ctas = simt_ctas(D);
  e = f32 ? launch_pdl(prompt_simt_kernel<D, true, RM>, dim3(ctas), dim3(kThreads), L::BYTES, s, a, mode)
          : launch_pdl(prompt_simt_kernel<D, false, RM>, dim3(ctas), dim3(kThreads), L::BYTES, s, a, mode);
  if (e != cudaSuccess || mode != kPromptCut) return e;
  return launch_prompt_join(a, D, f32, ctas, L::ROWS, s);
}
template <int D>
cudaError_t launch_d(const PromptArgs& a, bool f32, cudaStream_t s) {
  if constexpr (D != 64 && D != 128) {                 // (there only a few rows come here)
    if (static_cast<long long>(a.max_q) * a.G > 16) return launch_t<D, 4>(a, f32, s);
  }
  return launch_t<D, 1>(a, f32, s);
}
}  // namespace

int prompt_sms() { return kv8_sm_count(); }

cudaError_t launch_prompt_join(const PromptArgs& a, int d, bool f32, int ctas, int rows, cudaStream_t s) {
  const dim3 grid(ctas, rows / 8), block(256);
  auto go = [&](auto k16, auto k32) { return f32 ? launch_pdl(k32, grid, block, 0, s, a, ctas, rows) : launch_pdl(k16, grid, block, 0, s, a, ctas, rows); };
  switch (d) {
    case 32: return go(prompt_join_kernel<32, false>, prompt_join_kernel<32, true>);
    case 64: return go(prompt_join_kernel<64, false>, prompt_join_kernel<64, true>);
    case 96: return go(prompt_join_kernel<96, false>, prompt_join_kernel<96, true>);
    case 128: return go(prompt_join_kernel<128, false>, prompt_join_kernel<128, true>);
    case 160: return go(prompt_join_kernel<160, false>, prompt_join_kernel<160, true>);
    case 192: return go(prompt_join_kernel<192, false>, prompt_join_kernel<192, true>);
    case 224: return go(prompt_join_kernel<224, false>, prompt_join_kernel<224, true>);
    case 256: return go(prompt_join_kernel<256, false>, prompt_join_kernel<256, true>);
    default: return cudaErrorInvalidValue;
  }
}

size_t prompt_simt_workspace(int d) {
  return static_cast<size_t>(simt_ctas(d)) * (sizeof(PSplit) + 2 * sizeof(float) * 64 * (d + 4));
}

cudaError_t launch_prompt_simt(const PromptArgs& a, int d, bool f32, cudaStream_t s) {
  switch (d) {
    case 32: return launch_d<32>(a, f32, s);
    case 64: return launch_d<64>(a, f32, s);
    case 96: return launch_d<96>(a, f32, s);
    case 128: return launch_d<128>(a, f32, s);
    case 160: return launch_d<160>(a, f32, s);
    case 192: return launch_d<192>(a, f32, s);
    case 224: return launch_d<224>(a, f32, s);
    case 256: return launch_d<256>(a, f32, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace tq
