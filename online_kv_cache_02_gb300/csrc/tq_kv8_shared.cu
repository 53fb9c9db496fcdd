// Decode attention of sequences that share a prefix (tq_kv8_shared_decode_attention).
//
// A group's sequences have the same pages at their head.  With s_j the scores of one query,
//   out = (sum_{j in prefix} 2^s_j v_j + sum_{j behind} 2^s_j v_j) / (sum_prefix 2^s_j + sum_behind 2^s_j),
// so that the two sums can be formed apart and joined by their maxima:
//   prefix pass   the queries of a group are rows of one block per KV head (n G of them), all of which see the whole
//                 prefix: its pages are read once for the group, by the tcgen05 kernel from 17 rows on;
//   tail pass     each sequence's pages behind the prefix, by the decode kernel;
//   join          this file: a warp per query row, over the prefix's parts (an item may be cut into several) and the tail.

#include "tq_kv8.h"

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

namespace tq {
namespace {

struct ShareJoin {
  const float* tail_state;                // (Kv8Share::state is the prefix's)
  const float* parts;                     // of the prefix's cut items
  int tc, rows, nqb, heads;               // prefix pass: tcgen05 or not, its blocks and items
  float prefix_lift, tail_lift;
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The sums of one query row: their maximum M (a score, and an exponent beside it), l and O = sum of weights
// 2^(lift + score - M) and of those times the values.
template <int D, bool F32>
__global__ void __launch_bounds__(256) kv8_share_join_kernel(const __grid_constant__ Kv8Attn a, const __grid_constant__ Kv8Share share,
                                                             const __grid_constant__ ShareJoin j) {
  constexpr int DV = D == 256 ? 128 : D, PER = D / DV, PART = DV + 4;
  const int lane = threadIdx.x & 31;
  const long long task = blockIdx.x * 8LL + (threadIdx.x >> 5);
  if (task >= static_cast<long long>(share.batch) * a.Hq * PER) return;
  const long long row = task / PER;
  const int half = static_cast<int>(task % PER), b = static_cast<int>(row / a.Hq), hq = static_cast<int>(row - static_cast<long long>(b) * a.Hq);
  pdl_wait();
  const int len = a.lens[b];
  const int4 seq = share.seqs[b];
  const Kv8SharedSeq tail = kv8_tail(a, share, b);
  const long long at = (row * PER + half) * PART;
  // the parts: the tail's, then the prefix's
  const int nt = tail.n > 0 ? 1 : 0;
  int first = -1, np = 0, rr = 0;
  if (seq.x > 0) {
    np = 1;
    if (j.tc) {
      const int r = (b - seq.z) * a.G + hq % a.G;
      rr = r % j.rows;
      const int2 who = share.items[(static_cast<long long>(seq.y) * j.nqb + r / j.rows) * j.heads + hq / a.G * PER + half];
      if (who.x >= 0) {
        first = who.x;
        np = who.y - who.x + 1;
      }
    }
  }
  auto part = [&](int i) {
    if (i < nt) return j.tail_state + at;
    if (first < 0) return static_cast<const float*>(share.state) + at;
    const int k = first + i - nt;         // the first part is in its CTA's second slot, the others in their CTAs' first
    return j.parts + ((2LL * k + (k == first ? 1 : 0)) * j.rows + rr) * PART;
  };
  const int n = len > 0 ? nt + np : 0;
  float M = -INFINITY, E = -INFINITY;
  for (int i = lane; i < n; i += 32) M = fmaxf(M, part(i)[0]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float ref = M == -INFINITY ? 0.0f : M;         // no key, or scores that are all NaN: sums of 0 or NaN
  auto power = [&](int i, const float* p) { return p[0] - ref + (p[2] - (i < nt ? j.tail_lift : j.prefix_lift)); };
  for (int i = lane; i < n; i += 32) E = fmaxf(E, power(i, part(i)));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) E = fmaxf(E, __shfl_xor_sync(0xffffffffu, E, o));
  if (E == -INFINITY) E = 0.0f;
  float L = 0.0f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float* p = part(i);
    const float f = exp2_fast(power(i, p) - E);
    L = fmaf(f, p[1], L);
    if (4 * lane >= DV) continue;
    const float4 x = *reinterpret_cast<const float4*>(p + 4 + 4 * lane);
    acc.x = fmaf(f, x.x, acc.x), acc.y = fmaf(f, x.y, acc.y), acc.z = fmaf(f, x.z, acc.z), acc.w = fmaf(f, x.w, acc.w);
  }
  if (4 * lane >= DV) return;
  const float inv = L > 0.0f ? 1.0f / L : L == L ? 0.0f : L;
  const float4 y = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  const long long to = row * D + half * DV + 4 * lane;
  if (F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + to) = y;
  } else {
    const __nv_bfloat162 y0 = __floats2bfloat162_rn(y.x, y.y), y1 = __floats2bfloat162_rn(y.z, y.w);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + to) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&y0), *reinterpret_cast<const uint32_t*>(&y1));
  }
}

// The workspace: sequences, items, the two passes' sums, then each pass' parts (the join reads the prefix's).
struct Room {
  size_t items, prefix, tail, pass, rest, total;
};
size_t align16(size_t x) { return (x + 15) & ~static_cast<size_t>(15); }
Room room(int batch, int Hq, int H, int groups, int max_group, int max_seq_len, int d) {
  const Kv8TcShape t = kv8_tc_shape(groups, max_group, Hq / H, H, max_seq_len, d);
  const size_t sums = static_cast<size_t>(batch) * Hq * t.per * (t.dv + 4) * sizeof(float);
  Room r;
  r.items = static_cast<size_t>(batch) * sizeof(int4);
  r.prefix = r.items + align16(static_cast<size_t>(groups) * t.nqb * H * t.per * sizeof(int2));
  r.tail = r.prefix + align16(sums);
  r.pass = r.tail + align16(sums);
  // no less than for smaller sizes: the blocks of 8 rows can take more than those of 16
  const size_t least = kv8_rows_workspace(1, 1, d), rows = std::max(least, kv8_rows_workspace(max_group, Hq / H, d));
  r.rest = r.pass + align16(std::max(rows, kv8_tc_workspace(groups, max_group, Hq / H, H, max_seq_len, d)));
  r.total = r.rest + std::max(least, kv8_rows_workspace(1, Hq / H, d));
  return r;
}

template <int D>
cudaError_t launch_join(const Kv8Attn& a, const Kv8Share& share, const ShareJoin& j, bool f32, cudaStream_t s) {
  const long long tasks = static_cast<long long>(share.batch) * a.Hq * (D == 256 ? 2 : 1);
  const dim3 grid(static_cast<unsigned>((tasks + 7) / 8));
  return f32 ? launch_pdl(kv8_share_join_kernel<D, true>, grid, dim3(256), 0, s, a, share, j)
             : launch_pdl(kv8_share_join_kernel<D, false>, grid, dim3(256), 0, s, a, share, j);
}

}  // namespace

size_t kv8_shared_workspace(int batch, int Hq, int H, int groups, int max_group, int max_seq_len, int d) {
  return room(batch, Hq, H, groups, max_group, max_seq_len, d).total;
}

cudaError_t launch_kv8_shared(Kv8Attn a, Kv8Share share, int d, bool f32, float softmax_scale, void* workspace, cudaStream_t s) {
  const Room r = room(share.batch, a.Hq, a.H, share.groups, share.max_group, a.max_seq_len, d);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  share.seqs = reinterpret_cast<int4*>(ws);
  share.items = reinterpret_cast<int2*>(ws + r.items);
  share.state = reinterpret_cast<float*>(ws + r.prefix);
  a.part = reinterpret_cast<float*>(ws + r.pass);
  // the prefix: groups as sequences of max_group queries
  Kv8Attn p = a;
  p.B = share.groups;
  p.T = share.max_group;
  share.tail = 0;
  const bool tc = kv8_tc_takes(p.T, a.G, d, f32, softmax_scale);
  cudaError_t e = tc ? launch_kv8_tc_shared(p, share, d, s) : launch_kv8_rows_shared(p, share, d, f32, s);
  if (e != cudaSuccess) return e;
  const Kv8TcShape t = kv8_tc_shape(p.B, p.T, a.G, a.H, a.max_seq_len, d);
  ShareJoin j{reinterpret_cast<const float*>(ws + r.tail), a.part + t.records / sizeof(float), tc ? 1 : 0, t.rows, t.nqb, a.H * t.per,
              tc ? t.lift : kv8_rows_lift(), kv8_rows_lift()};
  // the tails
  Kv8Share rest = share;
  rest.tail = 1;
  rest.state = reinterpret_cast<float*>(ws + r.tail);
  Kv8Attn b = a;
  b.B = share.batch;
  b.T = 1;
  b.part = reinterpret_cast<float*>(ws + r.rest);
  e = launch_kv8_rows_shared(b, rest, d, f32, s);
  if (e != cudaSuccess) return e;
  switch (d) {
    case 64: return launch_join<64>(a, share, j, f32, s);
    case 128: return launch_join<128>(a, share, j, f32, s);
    case 256: return launch_join<256>(a, share, j, f32, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace tq
