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

// Over the prefix (0) and over the sequence's own rows (1): the first cluster with a piece of the
// row's group, and pieces, one to a cluster from there on.
struct RowParts {
  int first[2], pieces[2];

  // first .. last as the clusters left them; none, and false, unless they are clusters of the launch.
  DSI_HOST_DEVICE bool set(int kind, int from, int to, int clusters) {
    const bool ok = from >= 0 && from <= to && to < clusters;
    first[kind] = ok ? from : 0;
    pieces[kind] = ok ? to - from + 1 : 0;
    return ok;
  }
  DSI_HOST_DEVICE int count() const { return pieces[0] + pieces[1]; }

  // Part j (the prefix's, then its own): a row of the pieces' slots, or -1 - p for the row p of
  // whole groups' places.  row: of its group, for both kinds; at / vectors: query head and how
  // many there are; own_slot0: the own pieces' first slot; m: rows of a slot.
  DSI_HOST_DEVICE int64_t place(int j, const int (&row)[2], int at, int vectors, int own_slot0, int m) const {
    const int kind = j >= pieces[0];
    if (kind) j -= pieces[0];
    if (pieces[kind] == 1) return -1 - (int64_t)at - (kind ? (int64_t)vectors : 0);
    // (a cluster's first slot has the piece that goes on from the one before, its second the piece that starts)
    return (int64_t)((kind ? own_slot0 : 0) + 2 * (first[kind] + j) + (j == 0)) * m + row[kind];
  }
};

}  // namespace dsi
