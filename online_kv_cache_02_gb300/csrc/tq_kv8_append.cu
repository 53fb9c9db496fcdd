// Append to the 8-bit paged KV cache with the position rotation on the way.
//
// A block is one KV head of one 16-token page: e4m3 codes and one scale 2^e, e
// the smallest exponent with amax <= 448 2^e over the tokens written so far.  A
// power of two costs no precision (codes are floating point) and lets a growing
// block be rescaled by an exponent shift: a code is rounded again only where it
// falls into the subnormals.  A pair (x1, x2) of keys and queries becomes
// (x1 c - x2 s, x2 c + x1 s).
//
// Codes are those of exact arithmetic: the fp32 rotation carries a bound, a
// code that the bound leaves open (about one in 10^5) is taken again in fp64,
// and so is the block's maximum next to a power-of-two border.
//
// A CTA takes one page of one sequence and a group of its heads: the page's
// cosines and sines go to shared memory once, with every pair's axis resolved,
// and each warp takes whole (page, head) blocks: its 16 tokens by asynchronous
// copies into shared memory, the next block's while this one is worked on, then
// one pass for the maximum and one for the codes.  (Held in registers instead, a
// block left room for eight warps an SM.)
//
// Bound by the memory and, close behind it, by the instructions of the two passes:
// 8 x 4,096 tokens of 32 + 8 + 8 heads, bf16, d = 128, 755 MB: 142 us, 5.3 TB/s, 79%
// of a copy's rate (held in registers 367 us; two CTAs an SM 170 us); d = 64, 378 MB:
// 83 us, 67%; d = 256, 4 x 4,096 tokens of 16 + 4 + 4, 386 MB: 99 us, 57% (two CTAs an
// SM, one block in flight a warp).  fp32 with three axes, 3 x 777 tokens of 28 + 4 + 4,
// 67 MB: 19 us (15 with the inputs in L2), half of it the launch and the last wave; the
// same in bf16 13.  A single token of 16 sequences: 5 us on the GPU, the latency of
// three dependent loads.

#include "tq_kv8.h"
#include "tq_tc.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <type_traits>

namespace tq {
namespace {

constexpr int kAWarps = 8;

__device__ __forceinline__ uint32_t cvt_e4m3x2(float hi, float lo) {   // byte 0 = lo
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void e4m3x2_to_float(uint32_t two, float& lo, float& hi) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<unsigned short>(two)));
  const __half2 h = *reinterpret_cast<const __half2*>(&h2);
  lo = __low2float(h);
  hi = __high2float(h);
}
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }   // e in [-126, 127]

// Smallest e in [kE8Min, kE8Max] with amax <= 448 2^e (448 = 1.75 2^8); amax >= 0 and finite.
__device__ __forceinline__ int block_exp(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return e < kE8Min ? kE8Min : e > kE8Max ? kE8Max : e;
}
__device__ __forceinline__ int block_exp64(double amax) {
  const unsigned long long b = static_cast<unsigned long long>(__double_as_longlong(amax));
  const int e = static_cast<int>(b >> 52) - 1023 - 8 + ((b & 0xFFFFFFFFFFFFFull) > 0xC000000000000ull ? 1 : 0);
  return e < kE8Min ? kE8Min : e > kE8Max ? kE8Max : e;
}

// Sixteen channels of one token: chunks A and B of eight.
template <bool F32>
struct Chunk2 {
  uint4 w[F32 ? 4 : 2];
  __device__ __forceinline__ void load(uint32_t row, int ca, int cb) {   // from the token's row in shared memory
    constexpr int kB = F32 ? 32 : 16;
#pragma unroll
    for (int i = 0; i < kB / 16; ++i) {
      w[i] = tcx::lds128(row + kB * ca + 16 * i);
      w[kB / 16 + i] = tcx::lds128(row + kB * cb + 16 * i);
    }
  }
  // channel i (0 .. 15: chunk A, then chunk B)
  __device__ __forceinline__ float get(int i) const {
    const uint32_t* o = reinterpret_cast<const uint32_t*>(w);
    if (F32) return __uint_as_float(o[i]);
    const uint32_t x = o[i >> 1];
    return __uint_as_float((i & 1) ? (x & 0xFFFF0000u) : (x << 16));
  }
};

struct Turned {
  float r1, r2, b1, b2;         // values and bounds on their errors
};
__device__ __forceinline__ Turned turn(float x1, float x2, float c, float s) {
  Turned t;
  const float u = x2 * s, v = x1 * s;
  t.r1 = fmaf(x1, c, -u);
  t.r2 = fmaf(x2, c, v);
  // each product and each result is off by at most half a step, 2^-24; twice that covers the bounds' own rounding
  t.b1 = fmaf(fabsf(u), 0x1p-23f, fabsf(t.r1) * 0x1p-23f);
  t.b2 = fmaf(fabsf(v), 0x1p-23f, fabsf(t.r2) * 0x1p-23f);
  return t;
}
__device__ __forceinline__ bool finite32(float x) { return fabsf(x) <= 3.4028234e38f; }
// What a code is made of: NaN counts as zero, an infinity as the largest value.
__device__ __forceinline__ void tame(float& r, float& b) {
  if (!finite32(r)) {
    r = r == r ? copysignf(3.4028234e38f, r) : 0.0f;
    b = 0.0f;
  }
}

// Bytes of a block's input, and blocks in flight per warp.
template <int D, bool F32>
struct Stage {
  static constexpr int ROW = D * (F32 ? 4 : 2), BYTES = kPage * ROW, N = BYTES <= 4096 ? 2 : 1;
};

template <int D, bool F32, bool INTER>
__global__ void __launch_bounds__(32 * kAWarps, D == 256 ? (F32 ? 1 : 2) : 3) kv8_append_kernel(const __grid_constant__ Kv8Append a, int tasks_per_cta) {
  using S = Stage<D, F32>;
  constexpr int kLanes = D / 16;                 // lanes per token, sixteen channels each
  constexpr int kTok = 32 / kLanes;              // tokens per step of a warp
  extern __shared__ __align__(16) unsigned char sm_raw[];
  float* cs_sm = reinterpret_cast<float*>(sm_raw + kAWarps * S::N * S::BYTES);   // [16][rot]
  __shared__ int tok_ok[kPage];                  // the token is there and its position in the table
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t stages = tcx::su32(sm_raw) + warp * S::N * S::BYTES;
  const int npg = (a.n_new + 2 * kPage - 2) / kPage;
  const int b = blockIdx.x / npg, ip = blockIdx.x % npg;
  pdl_wait();
  const int start = a.start_pos[b];
  int n = a.new_lens ? a.new_lens[b] : a.n_new;
  if (start < 0 || n < 0 || n > a.n_new) {
    if (tid == 0) atomicOr(a.err, kErrSeqLen);
    n = n > a.n_new ? a.n_new : n;
    if (start < 0) return;
  }
  const int slot0 = ip == 0 ? start % kPage : 0;           // first slot of this page that the call writes
  const int t0 = ip == 0 ? 0 : ip * kPage - start % kPage; // its token
  const int nt = min(kPage - slot0, n - t0);               // tokens of this page
  if (nt <= 0) return;
  const int half = a.rot / 2;
  const int nk = a.k ? a.H : 0, nv = a.v ? a.H : 0, nq = a.q ? a.Hq : 0;
  const int task0 = blockIdx.y * tasks_per_cta, task1 = min(nk + nv + nq, task0 + tasks_per_cta);

  // a block's tokens into the warp's stage
  auto fetch = [&](int task, uint32_t dst) {
    const int kind = task < nk ? 0 : task < nk + nv ? 1 : 2;
    const int h = kind == 0 ? task : kind == 1 ? task - nk : task - nk - nv;
    const long long stride = (kind == 0 ? a.k_stride : kind == 1 ? a.v_stride : a.q_stride) * (F32 ? 4 : 2);
    const char* src = static_cast<const char*>(kind == 0 ? a.k : kind == 1 ? a.v : a.q) +
                      (static_cast<long long>(b) * a.n_new + t0) * stride + static_cast<long long>(h) * S::ROW;
    if (((reinterpret_cast<uintptr_t>(src) | static_cast<uintptr_t>(stride)) & 15) == 0) {
      for (int i = lane; i < nt * (S::ROW / 16); i += 32)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + 16 * i),
                     "l"(src + (i / (S::ROW / 16)) * stride + 16 * (i % (S::ROW / 16))));
    } else {                                     // rows off the 16-byte grid, element by element
      for (int i = lane; i < nt * D; i += 32) {
        const char* p = src + (i / D) * stride + (i % D) * (F32 ? 4 : 2);
        if (F32) asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst + 4 * i), "r"(*reinterpret_cast<const uint32_t*>(p)) : "memory");
        else asm volatile("st.shared.b16 [%0], %1;" ::"r"(dst + 2 * i), "h"(*reinterpret_cast<const unsigned short*>(p)) : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (task0 + warp < task1) fetch(task0 + warp, stages);

  // ---- the page's cosines and sines, one row per token -------------------------------
  if (tid < kPage) tok_ok[tid] = 1;
  __syncthreads();
  if (a.rot > 0) {
    for (int i = tid; i < nt * half; i += 32 * kAWarps) {
      const int t = i / half, pr = i % half;
      int ax = 0;
      while (ax < a.axes - 1 && pr >= a.sec_end[ax]) ++ax;
      const long long p = a.pos ? a.pos[(static_cast<long long>(ax) * a.batch + b) * a.n_new + t0 + t]
                                : static_cast<long long>(start) + t0 + t;
      float c = 1.0f, s = 0.0f;
      if (p < 0 || p >= a.max_pos) {
        tok_ok[t] = 0;
        atomicOr(a.err, kErrBlock);
      } else {
        c = a.cs[p * a.rot + pr];
        s = a.cs[p * a.rot + half + pr];
      }
      cs_sm[t * a.rot + pr] = c;
      cs_sm[t * a.rot + half + pr] = s;
    }
  }
  __syncthreads();

  // ---- the lane's place: sixteen channels of token `sub` of each step ----------------
  const int sub = lane / kLanes, li = lane % kLanes;
  const int rch = a.rot / 16;                    // chunk pairs that turn
  const bool turns = li < rch;
  // rotated chunks pair up `rot / 2` channels apart (interleaved pairs lie inside a chunk: any pairing does)
  const int ca = turns ? li : 2 * rch + 2 * (li - rch);
  const int cb = turns ? li + rch : ca + 1;
  // the lane's pairs: eight in a row, or four of chunk A and four of chunk B
  const int pa = INTER ? 4 * ca : 8 * li, pb = INTER ? 4 * cb : 8 * li + 4;
  const long long page_pos = (static_cast<long long>(start) + t0) / kPage;
  const int steps = (nt + kTok - 1) / kTok;

  int buf = 0;
  for (int task = task0 + warp; task < task1; task += kAWarps) {
    const int kind = task < nk ? 0 : task < nk + nv ? 1 : 2;
    const int h = kind == 0 ? task : kind == 1 ? task - nk : task - nk - nv;
    const bool rot = turns && kind != 1;
    const uint32_t in = stages + buf * S::BYTES;
    if (S::N == 2 && task + kAWarps < task1) {
      __syncwarp();                              // the stage's last block has been read
      fetch(task + kAWarps, stages + (buf ^ 1) * S::BYTES);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    __syncwarp();
    // the eight pairs of a step's token, turned: f(first, second channel of the sixteen, Turned, x1, x2, cos, sin).
    // INTER is a template argument so that register indices stay static.
    auto pairs = [&](int t, auto&& f) {
      Chunk2<F32> x;
      x.load(in + t * S::ROW, ca, cb);
      if (rot) {
        float c[8], s[8];
        const float* row = cs_sm + t * a.rot;
        *reinterpret_cast<float4*>(c) = *reinterpret_cast<const float4*>(row + pa);
        *reinterpret_cast<float4*>(c + 4) = *reinterpret_cast<const float4*>(row + pb);
        *reinterpret_cast<float4*>(s) = *reinterpret_cast<const float4*>(row + half + pa);
        *reinterpret_cast<float4*>(s + 4) = *reinterpret_cast<const float4*>(row + half + pb);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i1 = INTER ? 2 * j : j, i2 = INTER ? 2 * j + 1 : 8 + j;
          const float x1 = x.get(i1), x2 = x.get(i2);
          f(i1, i2, turn(x1, x2, c[j], s[j]), x1, x2, c[j], s[j]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i1 = INTER ? 2 * j : j, i2 = INTER ? 2 * j + 1 : 8 + j;
          const float x1 = x.get(i1), x2 = x.get(i2);
          f(i1, i2, Turned{x1, x2, 0.0f, 0.0f}, x1, x2, 1.0f, 0.0f);
        }
      }
    };
    auto there = [&](int t) { return t < nt && tok_ok[t]; };

    if (kind == 2) {                             // queries: turned and rounded once
#pragma unroll 1
      for (int st = 0; st < steps; ++st) {
        const int t = st * kTok + sub;
        if (!there(t)) continue;
        float y[16];
        pairs(t, [&](int i1, int i2, const Turned& r, float, float, float, float) {
          y[i1] = r.r1;
          y[i2] = r.r2;
        });
        const long long at = ((static_cast<long long>(b) * a.n_new + t0 + t) * a.Hq + h) * D;
        if (F32) {
          float* o = static_cast<float*>(a.q_out) + at;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            *reinterpret_cast<float4*>(o + 8 * ca + 4 * i) = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
            *reinterpret_cast<float4*>(o + 8 * cb + 4 * i) =
                make_float4(y[8 + 4 * i], y[9 + 4 * i], y[10 + 4 * i], y[11 + 4 * i]);
          }
        } else {
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&p);
          }
          unsigned short* o = static_cast<unsigned short*>(a.q_out) + at;
          *reinterpret_cast<uint4*>(o + 8 * ca) = make_uint4(w[0], w[1], w[2], w[3]);
          *reinterpret_cast<uint4*>(o + 8 * cb) = make_uint4(w[4], w[5], w[6], w[7]);
        }
      }
    } else {
      // ---- a block of keys or values --------------------------------------------------
      int pid = -1;
      if (page_pos < a.maxp) {
        pid = a.bt[static_cast<long long>(b) * a.maxp + page_pos];
        if (pid < 0 || pid >= a.num_pages) {
          if (lane == 0) atomicOr(a.err, kErrPage);
          pid = -1;
        }
      } else if (lane == 0) {
        atomicOr(a.err, kErrBlock);
      }
      if (pid >= 0) {                            // warp-uniform
        const long long blk = static_cast<long long>(pid) * a.H + h;
        uint8_t* codes = (kind == 0 ? a.kc : a.vc) + blk * (kPage * D);
        float* scale = (kind == 0 ? a.ks : a.vs) + blk;

        // largest value of the block's new tokens, and the largest bound on an error
        float amax = 0.0f, bmax = 0.0f;
        bool odd = false;                        // a value that is not finite
#pragma unroll 1
        for (int st = 0; st < steps; ++st) {
          const int t = st * kTok + sub;
          if (!there(t)) continue;
          pairs(t, [&](int, int, const Turned& r, float, float, float, float) {
            const float m1 = fabsf(r.r1), m2 = fabsf(r.r2);
            const bool f1 = finite32(m1), f2 = finite32(m2);
            odd |= !f1 || !f2;
            amax = fmaxf(amax, fmaxf(f1 ? m1 : 0.0f, f2 ? m2 : 0.0f));
            bmax = fmaxf(bmax, fmaxf(f1 ? r.b1 : 0.0f, f2 ? r.b2 : 0.0f));
          });
        }
        // non-negative floats order as their bits
        amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
        bmax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(bmax)));
        if (__any_sync(0xffffffffu, odd) && lane == 0) atomicOr(a.err, kErrNonFinite);
        int e = block_exp(amax);
        if (bmax > 0.0f && block_exp(fmaxf(amax - bmax, 0.0f)) != block_exp(fminf(amax + bmax, 3.4028234e38f))) {
          double m = 0.0;                        // next to a border: the maximum in fp64
#pragma unroll 1
          for (int st = 0; st < steps; ++st) {
            const int t = st * kTok + sub;
            if (!there(t)) continue;
            pairs(t, [&](int, int, const Turned& r, double x1, double x2, double c, double s) {
              if (finite32(r.r1)) m = fmax(m, fabs(x1 * c - x2 * s));
              if (finite32(r.r2)) m = fmax(m, fabs(x2 * c + x1 * s));
            });
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
          e = block_exp64(m);
        }
        if (slot0 > 0) {                         // earlier tokens keep at least the block's scale
          const uint32_t sb = __float_as_uint(*scale);
          int e_old = static_cast<int>(sb >> 23) - 127;
          if ((sb & 0x7FFFFFu) || e_old < kE8Min || e_old > kE8Max) {
            if (lane == 0) atomicOr(a.err, kErrScale);
            e_old = kE8Min;
          }
          if (e > e_old) {                       // their codes move down by an exact factor, rounded once more
            // below 2^-126 every code rounds to zero all the same
            const float f = pow2f(e_old - e < -126 ? -126 : e_old - e);
            for (int i = lane; i < slot0 * D / 4; i += 32) {
              const uint32_t w = reinterpret_cast<const uint32_t*>(codes)[i];
              float v0, v1, v2, v3;
              e4m3x2_to_float(w & 0xFFFFu, v0, v1);
              e4m3x2_to_float(w >> 16, v2, v3);
              reinterpret_cast<uint32_t*>(codes)[i] = cvt_e4m3x2(v1 * f, v0 * f) | (cvt_e4m3x2(v3 * f, v2 * f) << 16);
            }
          } else {
            e = e_old;
          }
          __syncwarp();                          // every lane has read the scale
        }
        if (lane == 0) *scale = pow2f(e);
        const float inv = pow2f(-e);
#pragma unroll 1
        for (int st = 0; st < steps; ++st) {
          const int t = st * kTok + sub;
          if (!there(t)) continue;
          uint32_t lo[8];                        // [pair]: code of the first channel | second << 8
          uint32_t open = 0u;
          if (kind == 0) {
            // codes of value +- bound agree: that is the code
            // (pairs at position 0 of their axis are exact, and one bf16 value in sixteen is half way between two codes:
            // taken again in fp64, they cost an image's tokens twice the call)
            pairs(t, [&](int i1, int, const Turned& r, float, float, float c, float s) {
              const bool exact = s == 0.0f && c == 1.0f;
              float r1 = r.r1, r2 = r.r2, b1 = exact ? 0.0f : r.b1, b2 = exact ? 0.0f : r.b2;
              tame(r1, b1);
              tame(r2, b2);
              const int j = INTER ? i1 / 2 : i1;
              lo[j] = cvt_e4m3x2((r2 - b2) * inv, (r1 - b1) * inv);
              // (a zero's two codes may differ too: exact values have no bound)
              if (lo[j] != cvt_e4m3x2((r2 + b2) * inv, (r1 + b1) * inv) && (b1 > 0.0f || b2 > 0.0f)) open |= 1u << j;
            });
            if (open) {
              pairs(t, [&](int i1, int, const Turned& r, double x1, double x2, double c, double s) {
                const int j = INTER ? i1 / 2 : i1;
                if ((open >> j) & 1u) {
                  // the nearest e4m3 of the fp64 value: rounded to fp32 towards odd, which keeps ties apart
                  auto code = [&](double y) {
                    float f = __double2float_rz(y * inv);
                    if (static_cast<double>(f) != y * inv) f = __uint_as_float(__float_as_uint(f) | 1u);
                    return cvt_e4m3x2(0.0f, f) & 0xFFu;
                  };
                  // an infinite half of the pair keeps its code
                  if (finite32(r.r1)) lo[j] = (lo[j] & 0xFF00u) | code(x1 * c - x2 * s);
                  if (finite32(r.r2)) lo[j] = (lo[j] & 0x00FFu) | (code(x2 * c + x1 * s) << 8);
                }
              });
            }
          } else {                               // values as they are
            pairs(t, [&](int i1, int, const Turned& r, float, float, float, float) {
              float r1 = r.r1, r2 = r.r2, b1 = 0.0f;
              tame(r1, b1);
              tame(r2, b1);
              lo[INTER ? i1 / 2 : i1] = cvt_e4m3x2(r2 * inv, r1 * inv);
            });
          }
          uint32_t w[4];                         // the sixteen codes in channel order
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (INTER) {
              w[i] = lo[2 * i] | (lo[2 * i + 1] << 16);
            } else {                             // bytes 0 of four pairs, then their bytes 1
              const int j = 4 * (i & 1);
              const uint32_t sel = i < 2 ? 0x0040u : 0x0051u;
              w[i] = __byte_perm(__byte_perm(lo[j], lo[j + 1], sel), __byte_perm(lo[j + 2], lo[j + 3], sel), 0x5410u);
            }
          }
          uint8_t* row = codes + (slot0 + t) * D;
          *reinterpret_cast<uint2*>(row + 8 * ca) = make_uint2(w[0], w[1]);
          *reinterpret_cast<uint2*>(row + 8 * cb) = make_uint2(w[2], w[3]);
        }
      }
    }
    if (S::N == 1 && task + kAWarps < task1) {
      __syncwarp();
      fetch(task + kAWarps, stages);
    }
    buf ^= S::N - 1;
  }
}

template <int D, bool F32, bool INTER>
cudaError_t launch_t(const Kv8Append& a, cudaStream_t s) {
  const int npg = (a.n_new + 2 * kPage - 2) / kPage;
  const long long pages = static_cast<long long>(a.batch) * npg;
  const int tasks = (a.k ? a.H : 0) + (a.v ? a.H : 0) + (a.q ? a.Hq : 0);
  // A block per warp up to three CTAs an SM, six where a warp has room for the next block's copy; more per warp beyond.
  // That is one wave (two) at d = 64 and 128; at d = 256 an SM holds two CTAs (fp32: one), and it is one and a half (three).
  // Inputs in L2: bf16, d = 128, 8 x 512 tokens of 32 + 8 + 8 heads: six CTAs an SM 21 us, three 25, twelve 25; fp32,
  // d = 128, 3 x 777 of 28 + 4 + 4, three axes: three 15.1, six 17.6.  d = 256, 32 + 8 + 8 heads: bf16, 4 x 256: three 15.0,
  // two 21.0, four 15.0; 16 x 64: three 21.1, two 21.1, four 15.3; fp32, 4 x 256: three 26, one 31, two 26; 3 x 777: three 60,
  // one 52, two 55.
  int groups = (tasks + kAWarps - 1) / kAWarps;
  int per = 1;
  using S = Stage<D, F32>;
  while (per < 8 && pages * ((groups + per - 1) / per) > (S::N == 2 ? 6LL : 3LL) * kv8_sm_count()) per *= 2;
  const int tpc = per * kAWarps;
  if (pages > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
  constexpr int kStages = kAWarps * S::N * S::BYTES;
  const size_t smem = kStages + sizeof(float) * kPage * static_cast<size_t>(a.rot);
  static std::atomic<unsigned long long> configured{0};
  const cudaError_t e = smem_attr_once(kv8_append_kernel<D, F32, INTER>, kStages + static_cast<int>(sizeof(float)) * kPage * D,
                                       configured);
  if (e != cudaSuccess) return e;
  return launch_pdl(kv8_append_kernel<D, F32, INTER>, dim3(static_cast<unsigned>(pages), (tasks + tpc - 1) / tpc),
                    dim3(32 * kAWarps), smem, s, a, tpc);
}

template <int D>
cudaError_t launch_d(const Kv8Append& a, bool f32, cudaStream_t s) {
  if (f32) return a.interleaved ? launch_t<D, true, true>(a, s) : launch_t<D, true, false>(a, s);
  return a.interleaved ? launch_t<D, false, true>(a, s) : launch_t<D, false, false>(a, s);
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8Append& a, int d, bool f32, cudaStream_t s) {
  switch (d) {
    case 64: return launch_d<64>(a, f32, s);
    case 128: return launch_d<128>(a, f32, s);
    case 256: return launch_d<256>(a, f32, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace tq
