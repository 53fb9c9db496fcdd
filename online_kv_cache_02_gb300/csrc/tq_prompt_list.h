// What attention over packed prompts counts before it lists its blocks of query rows, apart from what touches the GPU (so
// that it also compiles for the host).
#ifndef TQ_PROMPT_LIST_H_
#define TQ_PROMPT_LIST_H_

#ifdef __CUDACC__
#define TQ_LIST_FN __host__ __device__ __forceinline__
#else
#define TQ_LIST_FN inline
#endif

namespace tq {

constexpr int kPromptList = 2048;         // blocks and sequences that the list holds

// Whether a pair of offsets is a sequence of `total` rows, no more than `most` long.
TQ_LIST_FN bool prompt_pair(int x0, int x1, int total, int most) { return x0 >= 0 && x1 >= x0 && x1 <= total && x1 - x0 <= most; }
// Blocks of `rows` query rows that n queries of G rows make (n G is below 2^31).
TQ_LIST_FN int prompt_blocks(int n, int G, int rows) { return static_cast<int>((static_cast<long long>(n) * G + rows - 1) / rows); }
// Blocks that a call's sequences can have at most where the offsets ascend: a sequence's last block alone is not whole, and no
// row is in two sequences.
TQ_LIST_FN long long prompt_most_blocks(int S, int max_q, int total_q, int G, int rows) {
  const long long each = S * static_cast<long long>(prompt_blocks(max_q, G, rows)), whole = S + static_cast<long long>(total_q) * G / rows;
  return each < whole ? each : whole;
}
// Blocks that the list takes: its places, and no more than make 31 bits of units, a block taking `units` at most.
TQ_LIST_FN int prompt_list_room(long long units) {
  const long long n = 0x7FFFFFFFLL / units;
  return n < kPromptList ? static_cast<int>(n) : kPromptList;
}
// In offsets that fall the pairs around the falling one can be the same rows again, as often as there are pairs, and pass the
// bound above.  The list counts a sequence as one block too many where it has more than `most` (the list's room), so that no
// sum passes 31 bits, and takes the sequences from the first on for as long as they have `most` blocks together.  firsts:
// blocks before each of S sequences; total: of all of them.
TQ_LIST_FN int prompt_counted(int blocks, int most) { return blocks <= most ? blocks : most + 1; }
TQ_LIST_FN int prompt_taken(const int* firsts, int S, int total, int most) {
  if (total <= most) return S;
  int lo = 0, hi = S - 1;                 // the last sequence before which there are no more than `most`
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (firsts[mid] <= most) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

}  // namespace tq

#endif  // TQ_PROMPT_LIST_H_
