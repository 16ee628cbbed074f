// Index rules of the adapters' kernels that keep their accesses inside the caller's arrays, apart from the kernels so that
// a host program can check them over all sizes.
#pragma once

#ifdef __CUDACC__
#define NF4_INDEX __host__ __device__ __forceinline__
#else
#define NF4_INDEX inline
#endif

namespace nf4 {

// Four lanes share a row of B, lane t from value values * t on: whether the row has that value.  (At rank 8 lanes 2 and 3,
// at rank 24 lane 3, have none; behind the last row of the last adapter their place is past the end of B.)
NF4_INDEX bool lane_in_row(int values, int t, int rank) { return values * t < rank; }

// Columns of a projection, of which there are up to 2^31 - 1: a sum of two could pass that, their difference cannot.
// Whether so many blocks of 256 from column `first` on (below N) are whole; whether column from + more (from at most N + 255)
// is there.
NF4_INDEX bool whole_blocks(int first, int N, int blocks) { return N - first >= 256 * blocks; }
NF4_INDEX bool column_there(int from, int more, int N) { return more < N - from; }

// Whether a chunk of the plan (an adapter, its first place in the order, its tokens) is inside the lists, whatever its words say.
NF4_INDEX bool chunk_in_lists(int adapter, int first, int tokens, int most, long long adapters, int listed) {
    return adapter >= 0 && adapter < adapters && tokens > 0 && tokens <= most && first >= 0 && first <= listed - tokens;
}

}  // namespace nf4
