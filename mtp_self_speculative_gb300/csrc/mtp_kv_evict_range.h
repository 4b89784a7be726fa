// How the thread blocks of a cluster share a request's slots when an eviction
// selects what stays; plain C++, so that it also runs on the host.
#pragma once

#ifdef __CUDACC__
#define MTP_RANGE_FN __host__ __device__ __forceinline__
#else
#define MTP_RANGE_FN inline
#endif

namespace mtp {

struct EvictRange {
  int s0, s1;   // this block's slots
  int c0, c1;   // its candidates: slots that are neither among the first `sink` nor the last `recent`
  int f0;       // where its loops over four slots at a time begin: c0 rounded down to four, not below s0; c1: no candidates
};

// Slots of a block at most: whole groups of 128.
MTP_RANGE_FN long long evict_share(long long L, int blocks) { return ((L + blocks - 1) / blocks + 127) & ~127ll; }

// Block c of `blocks`; a request of L slots, sink + recent <= L.  A block whose
// share begins at or behind the end has s0 = L, which need not be a multiple of
// four: rounded down it would lie in front of the block's keys.
MTP_RANGE_FN EvictRange evict_range(int L, int sink, int recent, int blocks, int c) {
  const int share = (int)evict_share(L, blocks), hi = L - recent;
  EvictRange r;
  r.s0 = (long long)c * share < L ? c * share : L;
  r.s1 = L - r.s0 < share ? L : r.s0 + share;
  r.c0 = sink > r.s0 ? sink : r.s0;
  r.c1 = hi < r.s1 ? hi : r.s1;
  r.f0 = r.c0 < r.c1 ? r.c0 & ~3 : r.c1;
  return r;
}

}  // namespace mtp
