// Decode attention of sequences that share a prefix (tq_kv8_shared_decode_attention).
//
// A group's sequences have the same pages at their head.  With s_j the scores of one query,
//   out = (sum_{j in prefix} 2^s_j v_j + sum_{j behind} 2^s_j v_j) / (sum_prefix 2^s_j + sum_behind 2^s_j),
// so that the two sums can be formed apart and joined by their maxima:
//   prefix pass   the queries of a group are rows of one block per KV head (n G of them), all of which see the whole
//                 prefix: its pages are read once for the group, by the tcgen05 kernel from 17 rows on;
//   tail pass     each sequence's pages behind the prefix, by the decode kernel;
//   join          this file: a warp per query row, over the prefix's parts (an item may be cut into several) and the tail.
// The tail pass runs beside the prefix pass' last blocks (it waits for none of them but at its end).  64 sequences behind
// 32,768 tokens, 32 / 8 heads, d = 128: 66 us (one after the other 75, with a join per pass 81; the decode kernel over every
// sequence by itself reads the prefix 64 times); three groups of 3 to 17 behind 1,000 to 6,000 tokens 37.5 us.  Each kernel by
// itself: prefix 42, tails 21, join 10 us (groups: 24, 16, 7.5).  In the prefix pass the tensor pipe is active for 38% of the
// cycles (groups 9%) and 5.9 stalls an issue (9.2) wait for loads; DRAM gives a fifth to a fourth of its rate in all three.

#include "tq_kv8.h"
#include "tq_kv8_parts.h"

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

namespace tq {
namespace {

// One pass, as the join finds it.
struct Pass {
  const float* state;                     // whole items' sums, by query row
  const float* parts;                     // of the cut ones
  const int2* items;
  int rows, nqb, heads, per, part;        // rows a block, blocks, items and items per head; floats of a part's row
  int ctas;                               // that can hold parts
  float lift;
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A query row's parts in one pass: n of them, their rows `step` floats apart (the first by itself).
struct Parts {
  const float *first, *rest;
  long long step;
  int n;
  __device__ __forceinline__ const float* at(int i) const { return i ? rest + i * step : first; }
};
// Row `r` of group (or sequence) b in the pass; `whole`: where its sums stand if its item is whole.  An item that the pass did
// not come to has no parts.
template <int DV>
__device__ __forceinline__ Parts parts_of(const Pass& p, int b, int r, int kv_head, int half, const float* whole) {
  const int2 who = p.items[(static_cast<long long>(b) * p.nqb + r / p.rows) * p.heads + kv_head * p.per + (p.per > 1 ? half : 0)];
  if (who.x < 0) return Parts{whole, whole, 0, 1};
  const long long slot = static_cast<long long>(p.rows) * p.part, row = static_cast<long long>(r % p.rows) * p.part;
  // the first part is in its CTA's second slot, the others in their CTAs' first
  return Parts{p.parts + (2LL * who.x + 1) * slot + row, p.parts + 2LL * who.x * slot + row, 2 * slot, kv8_item_parts(who.x, who.y, p.ctas)};
}

// The sums of one query row: their maximum M (a score, and an exponent beside it), l and O = sum of weights
// 2^(lift + score - M) and of those times the values.  A warp per row (at d = 256 per half of its channels); a lane per part
// works out the part's weight, then all lanes take a part's channels.
template <int D, bool F32>
__global__ void __launch_bounds__(128) kv8_share_join_kernel(const __grid_constant__ Kv8Attn a, const __grid_constant__ Kv8Share share,
                                                             const __grid_constant__ Pass prefix, const __grid_constant__ Pass tails) {
  constexpr int DV = D == 256 ? 128 : D, PER = D / DV, PART = DV + 4;
  const int lane = threadIdx.x & 31;
  const long long task = blockIdx.x * 4LL + (threadIdx.x >> 5);
  if (task >= static_cast<long long>(share.batch) * a.Hq * PER) return;
  const long long row = task / PER;
  const int half = static_cast<int>(task % PER), b = static_cast<int>(row / a.Hq), hq = static_cast<int>(row - static_cast<long long>(b) * a.Hq);
  pdl_wait();
  const int len = a.lens[b];
  const int4 seq = share.seqs[b];
  const Kv8SharedSeq tail = kv8_tail(a, b, seq.x);
  const long long at = (row * PER + half) * PART;
  Parts pt{nullptr, nullptr, 0, 0}, pp = pt;
  if (len > 0 && tail.n > 0) pt = parts_of<DV>(tails, b, hq % a.G, hq / a.G, half, tails.state + at);
  if (len > 0 && seq.x > 0) pp = parts_of<DV>(prefix, seq.y, (b - seq.z) * a.G + hq % a.G, hq / a.G, half, prefix.state + at);
  const int n = pt.n + pp.n;
  auto part = [&](int i) { return i < pt.n ? pt.at(i) : pp.at(i - pt.n); };
  // a part's row holds all channels where the pass has one item a head: this half's stand behind the others
  auto channels = [&](int i) {
    const Pass& p = i < pt.n ? tails : prefix;
    const bool whole = i < pt.n ? pt.step == 0 : pp.step == 0;
    return part(i) + 4 + (p.per == 1 && !whole ? half * DV : 0) + 4 * lane;
  };
  auto number = [&](int i) {                           // M, l and M's exponent less the lift
    if (i >= n) return make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
    float4 x = *reinterpret_cast<const float4*>(part(i));
    x.z -= i < pt.n ? tails.lift : prefix.lift;
    return x;
  };
  // the first parts' numbers and channels at once: what they weigh is worked out while the channels come
  constexpr int kAhead = 8;
  const float4 mine = number(lane);
  float4 y[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    y[i] = i < n && 4 * lane < DV ? *reinterpret_cast<const float4*>(channels(i)) : make_float4(0.f, 0.f, 0.f, 0.f);
  float M = mine.x, E = -INFINITY, L = 0.0f;
  for (int i = lane + 32; i < n; i += 32) M = fmaxf(M, number(i).x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float ref = M == -INFINITY ? 0.0f : M;         // no key, or scores that are all NaN: sums of 0 or NaN
  E = mine.x - ref + mine.z;
  for (int i = lane + 32; i < n; i += 32) {
    const float4 x = number(i);
    E = fmaxf(E, x.x - ref + x.z);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) E = fmaxf(E, __shfl_xor_sync(0xffffffffu, E, o));
  if (E == -INFINITY) E = 0.0f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float f, float4 v) {
    acc.x = fmaf(f, v.x, acc.x), acc.y = fmaf(f, v.y, acc.y), acc.z = fmaf(f, v.z, acc.z), acc.w = fmaf(f, v.w, acc.w);
  };
  for (int i0 = 0; i0 < n; i0 += 32) {
    const float4 x = i0 ? number(i0 + lane) : mine;
    const float f = exp2_fast(x.x - ref + x.z - E);
    float sum = f * x.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    L += sum;
    for (int i = 0; i < min(32, n - i0); i += kAhead) {
      float4 z[kAhead];                                // the next ones on their way
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int next = i0 + i + kAhead + k;
        z[k] = next < n && 4 * lane < DV ? *reinterpret_cast<const float4*>(channels(next)) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const float fk = __shfl_sync(0xffffffffu, f, i + k);
        if (i0 + i + k < n) add(fk, y[k]);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) y[k] = z[k];
    }
  }
  if (4 * lane >= DV) return;
  const float inv = L > 0.0f ? 1.0f / L : L == L ? 0.0f : L;
  const float4 o = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  const long long to = row * D + half * DV + 4 * lane;
  if (F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + to) = o;
  } else {
    const __nv_bfloat162 y0 = __floats2bfloat162_rn(o.x, o.y), y1 = __floats2bfloat162_rn(o.z, o.w);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + to) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&y0), *reinterpret_cast<const uint32_t*>(&y1));
  }
}

// The workspace: sequences, items, the two passes' sums, then each pass' parts (the join reads the prefix's).
struct Room {
  size_t items, rest_items, prefix, tail, pass, rest, total;
};
size_t align16(size_t x) { return (x + 15) & ~static_cast<size_t>(15); }
Room room(int batch, int Hq, int H, int groups, int max_group, int max_seq_len, int d) {
  const int G = Hq / H;
  const Kv8TcShape t = kv8_tc_shape(groups, max_group, G, H, max_seq_len, d);
  const size_t sums = static_cast<size_t>(batch) * Hq * t.per * (t.dv + 4) * sizeof(float);
  // blocks of the fewest rows that a pass can have, which never fall with larger sizes
  const auto blocks = [&](int seqs, int T) { return static_cast<size_t>(seqs) * ((static_cast<long long>(T) * G + 7) / 8) * H * t.per * sizeof(int2); };
  Room r;
  r.items = static_cast<size_t>(batch) * sizeof(int4);
  r.rest_items = r.items + align16(blocks(groups, max_group));
  r.prefix = r.rest_items + align16(blocks(batch, 1));
  r.tail = r.prefix + align16(sums);
  r.pass = r.tail + align16(sums);
  // no less than for smaller sizes: the blocks of 8 rows can take more than those of 16
  const size_t least = kv8_rows_workspace(1, 1, d), rows = std::max(least, kv8_rows_workspace(max_group, G, d));
  r.rest = r.pass + align16(std::max(rows, kv8_tc_workspace(groups, max_group, G, H, max_seq_len, d)));
  r.total = r.rest + std::max(least, kv8_rows_workspace(1, G, d));
  return r;
}

template <int D>
cudaError_t launch_join(const Kv8Attn& a, const Kv8Share& share, const Pass& prefix, const Pass& tails, bool f32, cudaStream_t s) {
  const long long tasks = static_cast<long long>(share.batch) * a.Hq * (D == 256 ? 2 : 1);
  const dim3 grid(static_cast<unsigned>((tasks + 3) / 4));
  return f32 ? launch_pdl(kv8_share_join_kernel<D, true>, grid, dim3(128), 0, s, a, share, prefix, tails)
             : launch_pdl(kv8_share_join_kernel<D, false>, grid, dim3(128), 0, s, a, share, prefix, tails);
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
  const auto pass = [&](const Kv8TcShape& x, const Kv8Share& sh, const float* work) {
    return Pass{sh.state, work + x.records / sizeof(float), sh.items, x.rows, x.nqb, a.H * x.per, x.per, x.dv + 4, x.ctas, x.lift};
  };
  const Pass prefix = pass(tc ? kv8_tc_shape(p.B, p.T, a.G, a.H, a.max_seq_len, d) : kv8_rows_shape(p.T, a.G, d), share, p.part);
  // the tails
  Kv8Share rest = share;
  rest.tail = 1;
  rest.state = reinterpret_cast<float*>(ws + r.tail);
  rest.items = reinterpret_cast<int2*>(ws + r.rest_items);
  Kv8Attn b = a;
  b.B = share.batch;
  b.T = 1;
  b.part = reinterpret_cast<float*>(ws + r.rest);
  e = launch_kv8_rows_shared(b, rest, d, f32, s);
  if (e != cudaSuccess) return e;
  const Pass tails = pass(kv8_rows_shape(1, a.G, d), rest, b.part);
  switch (d) {
    case 64: return launch_join<64>(a, share, prefix, tails, f32, s);
    case 128: return launch_join<128>(a, share, prefix, tails, f32, s);
    case 256: return launch_join<256>(a, share, prefix, tails, f32, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace tq
