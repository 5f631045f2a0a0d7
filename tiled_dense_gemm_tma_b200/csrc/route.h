// route.h -- how route.cu deals a row of experts out to a warp's lanes, and how
// close two keys may be before 64 bits decide.  Plain C++, also built by the host
// tests.
#pragma once

#if defined(__CUDACC__)
#define TG_HD_ROUTE __host__ __device__ __forceinline__
#else
#define TG_HD_ROUTE inline
#endif

namespace tg {

// Lanes that share a group (groups <= 32): 32 over the next power of two.
TG_HD_ROUTE int route_lanes(int groups) {
    int lanes = 32;
    for (int g = 1; g < groups; g <<= 1) lanes >>= 1;
    return lanes;
}

// Experts a lane takes: less than 64, as E is at most 1024 and the lanes of all groups more than 16.
TG_HD_ROUTE int route_values(int E, int groups) {
    return (E / groups + route_lanes(groups) - 1) / route_lanes(groups);
}

// What the difference of two keys of at most `size` may be off by, sums of a
// score (a sigmoid, or one of a softmax of at most `highest`) and a bias: the
// errors of both scores and of both sums (2^-24 each), twice over, and the bits that
// number a lane's `values` experts.
TG_HD_ROUTE float route_slack(int sigmoid, float highest, float size, int values) {
    return (sigmoid ? 0x1p-20f : highest * 0x1p-16f) + size * (0x1p-22f + 0x1p-23f * static_cast<float>(values));
}

}  // namespace tg
