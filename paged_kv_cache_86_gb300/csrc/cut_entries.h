// cut_entries.h -- arithmetic of the cut line of decode_warp.cu that also compiles
// for the host, where it is tested.
#pragma once

#ifdef __CUDACC__
#define PKV_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define PKV_HOST_DEVICE inline
#endif

namespace pkv {

// Whether the merge follows its entry (sequence, first range, last range) number `at`:
// a sequence of the call that more than one range of the line works on. Where there is
// an entry for each sequence, entry `at` is sequence at's and no other one's. A walk
// that gave up a wait leaves the entries of its remaining sequences as the workspace had
// them, so anything may stand there; nothing that is refused here is followed, and
// what is not refused stays inside the records, the sequences and the work of one merge.
PKV_HOST_DEVICE bool merges_entry(int seq, int first, int last, int at, bool by_seq, int num_seqs, int ranges) {
  return seq >= 0 && seq < num_seqs && (!by_seq || seq == at) && first >= 0 && first < last && last < ranges;
}

// Tiles of a range: the line's `total`, below 2^31, over `ranges` of them rounded up, and at
// least `least`. (total + ranges - 1 may be past 2^31.)
PKV_HOST_DEVICE int range_length(int total, int ranges, int least) {
  const int n = total / ranges + (total % ranges > 0 ? 1 : 0);
  return n > least ? n : least;
}

}  // namespace pkv
