// The launch of the tcgen05 form of attention over the 8-bit paged cache (tq_kv8_tc.cuh), and what the forms share on the
// host.

#include "tq_kv8_tc.cuh"

#include <cudaTypedefs.h>

namespace tq {
namespace {

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

cudaError_t launch_kv8_tc(const Kv8Attn& a, int d, cudaStream_t s) { return launch_tc(a, NoShare{}, d, s); }

}  // namespace tq
