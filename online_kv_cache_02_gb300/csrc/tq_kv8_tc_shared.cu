// The tcgen05 form's prefix pass of decode with shared prefixes (tq_kv8_tc.cuh, tq_kv8_shared.cu).

#include "tq_kv8_tc.cuh"

namespace tq {

cudaError_t launch_kv8_tc_shared(const Kv8Attn& a, const Kv8Share& share, int d, cudaStream_t s) { return launch_tc(a, share, d, s); }
Kv8TcShape kv8_tc_shape(int B, int T, int G, int H, int max_seq_len, int d) {
  Kv8TcShape x;
  x.per = items_per_head(d);
  x.rows = rows_of(d);
  x.dv = d / x.per;
  x.nqb = query_blocks(T, G, d);
  x.ctas = ctas_for(B, H * x.per, x.nqb, max_seq_len);
  x.records = x.ctas * sizeof(TSplit);
  x.lift = kLift;
  return x;
}

}  // namespace tq
