// dl_seqs.cuh -- packed sequences: which token tile of which sequence a CTA
// (or thread) works on.  The host knows every length, so the table travels
// by value with the launch and a tile's sequence is found by bisection.
#pragma once

#include <stdint.h>

namespace dl {

// Sequence s holds tokens start[s] .. start[s+1]-1 and tiles tile0[s] ..
// tile0[s+1]-1 of the launch; every sequence has at least one tile (an empty
// one still passes its state on).
template <int N>
struct SeqTable {
  static constexpr int kMax = N;
  int n;
  int start[N + 1];
  int tile0[N + 1];

  __device__ __forceinline__ int index(int sl) const { return sl; }  // of a sequence in the call
  __device__ __forceinline__ int find(int tile) const {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tile0[mid] <= tile)
        lo = mid;
      else
        hi = mid - 1;
    }
    return lo;
  }
};

// Most batches fit the small table (a launch argument of about half a
// kilobyte); longer ones take the large table, at most kLargeSeqs a launch.
constexpr int kSmallSeqs = 64;
constexpr int kLargeSeqs = 1024;

// Fills the table from starts[s0 .. s0+n], tiles of `tile` tokens; returns
// the number of tiles.
template <int N>
inline long long fill_seqs(SeqTable<N>& t, const int32_t* starts, int s0, int n, int tile) {
  long long tiles = 0;
  t.n = n;
  for (int s = 0; s < n; ++s) {
    t.start[s] = starts[s0 + s];
    t.tile0[s] = int(tiles);
    const long long len = (long long)starts[s0 + s + 1] - starts[s0 + s];
    tiles += len > tile ? (len + tile - 1) / tile : 1;
  }
  t.start[n] = starts[s0 + n];
  t.tile0[n] = int(tiles);
  return tiles;
}

}  // namespace dl
