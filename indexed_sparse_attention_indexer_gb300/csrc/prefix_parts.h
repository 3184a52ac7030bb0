// Where the join of shared-prefix attention finds the parts of a query row.  Plain C++ (a host test
// drives it): the numbers of clusters come from the workspace, and after a wait that ran out they
// are whatever it held before, so they are held against the launch before anything is read by them.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define DSI_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define DSI_HOST_DEVICE inline
#endif

namespace dsi {

// Clusters that have a piece of a group: the first of them, and how many, one after another.  None
// unless from .. to are clusters of the launch.
struct Span {
  int first, pieces;
  DSI_HOST_DEVICE Span(int from, int to, int clusters) {
    const bool ok = from >= 0 && from <= to && to < clusters;
    first = ok ? from : 0;
    pieces = ok ? to - from + 1 : 0;
  }
};

// Part j of a query head (the prefix's, then its own rows'): a row of the pieces' slots, or -1 - p for
// the row p of whole groups' places.  prefix_row / own_row: its row of the groups; at / vectors: the
// query head and how many there are; own_slot0: the own pieces' first slot; m: rows of a slot.
DSI_HOST_DEVICE int64_t part_place(const Span& prefix, const Span& own, int j, int prefix_row, int own_row, int at,
                                   int vectors, int own_slot0, int m) {
  const bool second = j >= prefix.pieces;
  if (second) j -= prefix.pieces;
  if ((second ? own.pieces : prefix.pieces) == 1) return -1 - (second ? (int64_t)vectors + at : (int64_t)at);
  // (a cluster's first slot has the piece that goes on from the one before, its second the piece that starts)
  return (int64_t)((second ? own_slot0 + 2 * own.first : 2 * prefix.first) + 2 * j + (j == 0 ? 1 : 0)) * m +
         (second ? own_row : prefix_row);
}

}  // namespace dsi
