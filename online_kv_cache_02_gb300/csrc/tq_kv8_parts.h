// What the join of shared prefixes reads of an item's record, apart from what touches the GPU (so that it also compiles for
// the host).
#ifndef TQ_KV8_PARTS_H_
#define TQ_KV8_PARTS_H_

#ifdef __CUDACC__
#define TQ_PARTS_FN __host__ __device__ __forceinline__
#else
#define TQ_PARTS_FN inline
#endif

namespace tq {

// A record holds the CTAs of its item's first and last part, or -1 for a whole item.  A pass that gave up a wait (and has flagged
// that) leaves records unwritten, and those may hold anything: what names no CTAs of the pass' `ctas` has no parts.
// The parts of an item that is not whole, whose first CTA is not negative.
TQ_PARTS_FN int kv8_item_parts(int first, int last, int ctas) { return first <= last && last < ctas ? last - first + 1 : 0; }

}  // namespace tq

#endif  // TQ_KV8_PARTS_H_
