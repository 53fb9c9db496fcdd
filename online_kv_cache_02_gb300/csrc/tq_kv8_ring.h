// The bookkeeping of a warp's ring of pages in shared memory, apart from what touches the GPU (so that it also
// compiles for the host).
#ifndef TQ_KV8_RING_H_
#define TQ_KV8_RING_H_

#ifdef __CUDACC__
#define TQ_RING_FN __device__ __forceinline__
#else
#define TQ_RING_FN inline
#endif

namespace tq {

// A run of n pages passes through ST stages in order: the first ST are asked for at once, each is waited for (land),
// and once it has been read (pass) its stage takes the page ST further on.  A stage has one barrier, whose phase ends
// with each copy; the stages and phases go on over the runs.
//   send(ahead, stage)     asks for page k + ahead of the run
//   wait(stage, parity)    whether the stage's copy came, within a limit
// After a wait that gave up no copy is asked for any more: the stage's barrier still counts the one before.  Those
// under way are waited for once more, each in its own phase, so that none lands in memory that has another use by
// then; the run ends, and so does every later one.
template <int ST>
struct PageRing {
  int k = 0, n = 0;              // pages of the run that were taken, and all of them
  unsigned used = 0;             // stages taken, over all runs
  bool failed = false;

  template <class Send>
  TQ_RING_FN void start(int pages, Send&& send) {
    k = 0;
    n = failed ? 0 : pages;
    for (int i = 0; i < ST; ++i)
      if (i < n) send(i, (used + i) % ST);
  }
  template <class Wait>
  TQ_RING_FN bool land(Wait&& wait) {
    if (wait(used % ST, (used / ST) & 1)) return true;
    failed = true;
    for (int i = 0; i < ST && k + i < n; ++i) (void)wait((used + i) % ST, ((used + i) / ST) & 1);
    n = k;
    return false;
  }
  TQ_RING_FN unsigned stage() const { return used % ST; }
  template <class Send>
  TQ_RING_FN void pass(Send&& send) {
    if (k + ST < n) send(ST, used % ST);
    ++used;
    ++k;
  }
};

}  // namespace tq

#endif  // TQ_KV8_RING_H_
