// The launch of the mma.sync form of attention over the 8-bit paged cache (tq_kv8_rows.cuh).

#include "tq_kv8_rows.cuh"

namespace tq {

bool kv8_head_dim(int d) { return d == 64 || d == 128 || d == 256; }

size_t kv8_rows_workspace(int T, int G, int d) {
  const int R = rows_per_block(T, G, d);
  return static_cast<size_t>(ctas_per_sm(d, R)) * kv8_sm_count() * (sizeof(RSplit) + 2 * sizeof(float) * R * (d + 4));
}

cudaError_t launch_kv8_rows(const Kv8Attn& a, int d, bool f32, cudaStream_t s) { return launch_rows(a, NoShare{}, d, f32, s); }

}  // namespace tq
