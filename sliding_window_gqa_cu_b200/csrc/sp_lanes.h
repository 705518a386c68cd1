// How the units of a kernel of the shared-prefix attention are cut over its
// lanes.  Plain integer arithmetic, for the device and for the host's tests.
#pragma once

#ifdef __CUDACC__
#define SP_LANES_FN __host__ __device__ __forceinline__
#else
#define SP_LANES_FN inline
#endif

namespace thd {

// (32-bit division where it is enough: the 64-bit one takes some 100 instructions.)
// First unit of lane l when `units` are cut into `lanes` ranges (lanes <= units,
// so that none is empty).
SP_LANES_FN long long lane_begin(long long units, int lanes, int l) {
    const unsigned long long at = static_cast<unsigned long long>(units) * l;
    if (at >> 32 == 0) return static_cast<unsigned>(at) / static_cast<unsigned>(lanes);
    return static_cast<long long>(at / static_cast<unsigned>(lanes));
}

// The lane that holds unit x: the largest l with units * l / lanes < x + 1.  (The
// short division takes the number of units too, which may pass 2^32 while an early
// unit's dividend does not.)
SP_LANES_FN int lane_of(long long units, int lanes, long long x) {
    const unsigned long long at = static_cast<unsigned long long>(x + 1) * lanes - 1;
    if ((at | static_cast<unsigned long long>(units)) >> 32 == 0)
        return static_cast<int>(static_cast<unsigned>(at) / static_cast<unsigned>(units));
    return static_cast<int>(at / static_cast<unsigned long long>(units));
}

}  // namespace thd

#undef SP_LANES_FN
