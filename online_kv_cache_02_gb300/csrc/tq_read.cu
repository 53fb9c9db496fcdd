// Reading the caches back into rows.
//
// 2-4-bit cache (tq_dequantize), per vector of a KV head:
//   k = Pi^T (n16/sqrt(d) c[code] + sqrt(pi/2)/m rho16 S^T s)      s the signs, +-1
//   v = Pi^T (n16/sqrt(d) c[code])
// so that <q, k> is the score that the decode forms and the v are the values that it sums.
// 8-bit cache (tq_kv8_dequantize): code * scale, exact in bf16 and fp32.
//
// [P4] riverfrot.github.io "TurboQuant란 무엇이며…", §4.1-§4.3: the reconstruction of rotation, codebook and residual;
// §3.1 pages and tables.

#include "tq_read.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

namespace tq {
namespace {

constexpr float kSqrtHalfPi = 1.2533141373155003f;

// Code of channel j from a record's bytes (any format, see tq.h).
__device__ __forceinline__ int code_at(const uint8_t* rec, const KindLayout& L, int j) {
  const int grp = j < L.split ? 0 : 1, b = L.g[grp].bits, c = grp ? j - L.split : j, base = grp ? L.split * L.g[0].bits : 0;
  auto bit = [&](int p) { return (rec[p >> 3] >> (p & 7)) & 1; };
  if (b == 3) {
    const int ob = base + 24 * (c >> 3), i = c & 7;
    const int s0 = i < 6 ? ob + 4 * i : ob + 3 + 4 * (i - 6), step = i < 6 ? 1 : 8;
    return bit(s0) | (bit(s0 + step) << 1) | (bit(s0 + 2 * step) << 2);
  }
  int v = 0;
  for (int q = 0; q < b; ++q) v |= bit(base + b * c + q) << q;
  return b == 4 ? ((v & 8) ? 7 - (v & 7) : 8 + v) : v;
}

template <bool F32>
__device__ __forceinline__ void put(void* out, long long at, float x) {
  if (F32) static_cast<float*>(out)[at] = x;
  else static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(x);
}

// Any configuration, on CUDA cores: a block of 128 threads per (page, KV head) block of K or V; its 16 vectors stand in
// shared memory in the rotated domain, a thread forms one output channel of all of them.  Bound by the FMA pipe and the
// tables' reads from L2 (d = 128, eight sequences of 16,384 tokens, 8 heads: 4,340 us, where the tensor cores take 150).
template <bool F32>
__global__ void __launch_bounds__(128) read_generic_kernel(const __grid_constant__ ReadArgs a, int d) {
  __shared__ __align__(16) float y[kDMax + kMaxM][kPage];
  __shared__ float scale[2][kPage];
  const int tid = threadIdx.x;
  pdl_wait();
  const long long blocks = 2LL * a.batch * a.pages * a.H;
  for (long long at = blockIdx.x; at < blocks; at += gridDim.x) {
    const bool key = at % 2 == 0;
    const long long x = at / 2;
    const int h = static_cast<int>(x % a.H), i = static_cast<int>(x / a.H % a.pages), b = static_cast<int>(x / a.H / a.pages);
    const uint8_t* cache = key ? a.kc : a.vc;
    if (!cache) continue;
    const ReadRun run = read_run(a, b);
    const ReadPage pg = read_page(a, b, run, i);
    if (pg.id < 0) continue;
    const KindLayout& L = key ? a.kl : a.vl;
    const uint8_t* blk = cache + pg.id * (key ? a.k_page_bytes : a.v_page_bytes) + static_cast<long long>(h) * L.block_bytes;
    const int m = L.qjl ? a.m : 0;
    __syncthreads();                                   // the last block's vectors have been read
    if (tid < kPage) {
      scale[0][tid] = __half2float(*reinterpret_cast<const __half*>(blk + L.off_norm + 2 * tid)) * __frsqrt_rn(static_cast<float>(d));
      scale[1][tid] = L.qjl ? __half2float(*reinterpret_cast<const __half*>(blk + L.off_rnorm + 2 * tid)) * (kSqrtHalfPi / m) : 0.0f;
    }
    __syncthreads();
    for (int e = tid; e < kPage * d; e += 128) {
      const int t = e / d, j = e % d;
      y[j][t] = L.g[j < L.split ? 0 : 1].c[code_at(blk + t * L.code_bytes, L, j)] * scale[0][t];
    }
    for (int e = tid; e < kPage * m; e += 128) {
      const int t = e / m, p = e % m;
      y[d + p][t] = (blk[L.off_signs + t * (m / 8) + p / 8] >> (p & 7)) & 1 ? scale[1][t] : -scale[1][t];
    }
    __syncthreads();
    for (int c = tid; c < d; c += 128) {
      // sums of 32 terms at a time, which rounds less
      float acc[kPage] = {}, total[kPage] = {};
      auto fold = [&]() {
#pragma unroll
        for (int t = 0; t < kPage; ++t) total[t] += acc[t], acc[t] = 0.0f;
      };
      auto add = [&](int row, float w) {
#pragma unroll
        for (int q = 0; q < kPage / 4; ++q) {
          const float4 v = *reinterpret_cast<const float4*>(&y[row][4 * q]);
          acc[4 * q] = fmaf(w, v.x, acc[4 * q]);
          acc[4 * q + 1] = fmaf(w, v.y, acc[4 * q + 1]);
          acc[4 * q + 2] = fmaf(w, v.z, acc[4 * q + 2]);
          acc[4 * q + 3] = fmaf(w, v.w, acc[4 * q + 3]);
        }
      };
      for (int k0 = 0; k0 < d; k0 += 32, fold())
#pragma unroll 4
        for (int k = k0; k < k0 + 32; ++k) add(k, a.tab.pi[k * d + c]);
      for (int p0 = 0; p0 < m; p0 += 32, fold())
#pragma unroll 4
        for (int p = p0; p < p0 + 32; ++p) add(d + p, a.tab.a_df[2 * (p * d + c)]);
      void* out = key ? a.k_out : a.v_out;
      const long long stride = key ? a.k_stride : a.v_stride;
#pragma unroll
      for (int s = 0; s < kPage; ++s)
        if (s >= pg.s0 && s < pg.s1) put<F32>(out, (static_cast<long long>(run.row) + s - pg.off) * stride + h * d + c, total[s]);
    }
  }
}

// Four e4m3 codes as fp32.
__device__ __forceinline__ float4 codes4(uint32_t w) {
  uint32_t lo, hi;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"(static_cast<unsigned short>(w)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"(static_cast<unsigned short>(w >> 16)));
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo)), y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return make_float4(x.x, x.y, y.x, y.y);
}

// 8-bit cache: a warp per (page, KV head), keys and values at once (one look at the tables for both); a lane takes as many
// codes as make 16 bytes of a row, so that stores are whole lines.  Bound by the stores: eight sequences of 16,384 tokens,
// 8 heads, d = 128, into bf16 rows 121 us (6.7 TB/s, 0.98 of a copy's; with a block per
// page 150).
template <int D, bool F32>
__global__ void __launch_bounds__(256) kv8_read_kernel(const __grid_constant__ ReadArgs a) {
  constexpr int C = F32 ? 4 : 8, STEPS = kPage * D / (32 * C);     // codes a lane at a time, and times
  using Word = std::conditional_t<F32, uint32_t, uint2>;
  const int lane = threadIdx.x & 31;
  pdl_wait();
  const long long blocks = static_cast<long long>(a.batch) * a.pages * a.H;
  for (long long at = blockIdx.x * 8LL + (threadIdx.x >> 5); at < blocks; at += 8LL * gridDim.x) {
    const long long page = at / a.H;
    const int h = static_cast<int>(at - page * a.H), b = static_cast<int>(page / a.pages), i = static_cast<int>(page - static_cast<long long>(b) * a.pages);
    const ReadRun run = read_run(a, b);
    const ReadPage pg = read_page(a, b, run, i);
    if (pg.id < 0) continue;
    const long long blk = static_cast<long long>(pg.id) * a.H + h;
    Word w[2][STEPS];
    float scale[2];
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      const uint8_t* codes = kind ? a.vc : a.kc;
      scale[kind] = codes ? (kind ? a.vs : a.ks)[blk] : 0.0f;
#pragma unroll
      for (int n = 0; n < STEPS; ++n)
        if (codes) w[kind][n] = reinterpret_cast<const Word*>(codes + blk * kPage * D)[32 * n + lane];
    }
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      if (!(kind ? a.vc : a.kc)) continue;
      void* out = kind ? a.v_out : a.k_out;
      const long long stride = kind ? a.v_stride : a.k_stride;
#pragma unroll
      for (int n = 0; n < STEPS; ++n) {
        const int e = C * (32 * n + lane), s = e / D;
        if (s < pg.s0 || s >= pg.s1) continue;
        const long long to = (static_cast<long long>(run.row) + s - pg.off) * stride + static_cast<long long>(h) * D + e % D;
        if constexpr (F32) {
          float4 f = codes4(w[kind][n]);
          f.x *= scale[kind], f.y *= scale[kind], f.z *= scale[kind], f.w *= scale[kind];
          *reinterpret_cast<float4*>(static_cast<float*>(out) + to) = f;
        } else {
          const float4 f = codes4(w[kind][n].x), g = codes4(w[kind][n].y);
          const float c = scale[kind];
          const __nv_bfloat162 y0 = __floats2bfloat162_rn(f.x * c, f.y * c), y1 = __floats2bfloat162_rn(f.z * c, f.w * c),
                               y2 = __floats2bfloat162_rn(g.x * c, g.y * c), y3 = __floats2bfloat162_rn(g.z * c, g.w * c);
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + to) =
              make_uint4(*reinterpret_cast<const uint32_t*>(&y0), *reinterpret_cast<const uint32_t*>(&y1),
                         *reinterpret_cast<const uint32_t*>(&y2), *reinterpret_cast<const uint32_t*>(&y3));
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_read(const ReadArgs& a, int d, bool f32, cudaStream_t s) {
  const long long blocks = 2LL * a.batch * a.pages * a.H;
  const dim3 grid(static_cast<unsigned>(std::min<long long>(blocks, 1 << 20)));
  return f32 ? launch_pdl(read_generic_kernel<true>, grid, dim3(128), 0, s, a, d)
             : launch_pdl(read_generic_kernel<false>, grid, dim3(128), 0, s, a, d);
}

cudaError_t launch_kv8_read(const ReadArgs& a, int d, bool f32, cudaStream_t s) {
  const long long blocks = static_cast<long long>(a.batch) * a.pages * a.H;
  // a (page, head) a warp: handed out by the hardware they end closer together than strides of a resident grid (8 x 16,384
  // tokens: 122 us, 129 with 8 blocks an SM)
  const dim3 grid(static_cast<unsigned>(std::min<long long>((blocks + 7) / 8, 1 << 24)));
  auto go = [&](auto k16, auto k32) { return f32 ? launch_pdl(k32, grid, dim3(256), 0, s, a) : launch_pdl(k16, grid, dim3(256), 0, s, a); };
  switch (d) {
    case 64: return go(kv8_read_kernel<64, false>, kv8_read_kernel<64, true>);
    case 128: return go(kv8_read_kernel<128, false>, kv8_read_kernel<128, true>);
    case 256: return go(kv8_read_kernel<256, false>, kv8_read_kernel<256, true>);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace tq
