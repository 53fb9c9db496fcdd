// The mma.sync form's passes of decode with shared prefixes (tq_kv8_rows.cuh, tq_kv8_shared.cu).

#include "tq_kv8_rows.cuh"

namespace tq {

cudaError_t launch_kv8_rows_shared(const Kv8Attn& a, const Kv8Share& share, int d, bool f32, cudaStream_t s) {
  return launch_rows(a, share, d, f32, s);
}
float kv8_rows_lift() { return kLift; }

}  // namespace tq
