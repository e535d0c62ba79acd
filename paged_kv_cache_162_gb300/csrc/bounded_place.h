// Where the pieces of a unit lie in a split call of the bounded-cache
// attention.  Plain C++: the host tests it too.
#pragma once

#ifdef __CUDACC__
#define PKV_BOTH_SIDES __host__ __device__ __forceinline__
#else
#define PKV_BOTH_SIDES inline
#endif

namespace pkv {

// The pieces of a unit whose entry says that it begins in range `first` and ends
// in range `last` of a call's `ranges`: 0 where that cannot be so.  A wait that ran
// out leaves entries unwritten, and the workspace they are in has any contents:
// the pieces of such a unit are not looked for.
PKV_BOTH_SIDES int pieces_of(int first, int last, int ranges) {
    return first >= 0 && first <= last && last < ranges ? last - first + 1 : 0;
}

}  // namespace pkv
