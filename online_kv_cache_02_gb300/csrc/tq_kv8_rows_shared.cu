// The mma.sync form's passes of decode with shared prefixes (tq_kv8_rows.cuh, tq_kv8_shared.cu).

#include "tq_kv8_rows.cuh"

namespace tq {

cudaError_t launch_kv8_rows_shared(const Kv8Attn& a, const Kv8Share& share, int d, bool f32, cudaStream_t s) {
  return launch_rows(a, share, d, f32, s);
}
Kv8TcShape kv8_rows_shape(int T, int G, int d) {
  Kv8TcShape x;
  x.per = 1;
  x.rows = rows_per_block(T, G, d);
  x.dv = d;
  x.nqb = row_blocks(T, G, x.rows);
  x.ctas = ctas_per_sm(d, x.rows) * kv8_sm_count();
  x.records = x.ctas * sizeof(RSplit);
  x.lift = kLift;
  return x;
}

}  // namespace tq
