// How many memory operations a wave of the large FP8 product may leave in flight at each of its waits (not
// installed).  No HIP in here: a host program can replay the order below and see that nothing is read too early.
//
// The stream is half tiles of k, tile after tile, through kRing slots of LDS: half g goes to slot g % kRing, 8 loads
// of a wave, and one more for the scales of a tile of k with each even half.  Halves 0 .. 3 are asked for at the start,
// and half 0 is waited for.  Then, for every half g in turn:
//   wait for half g + 1;  multiply half g, and meanwhile read half g + 1 from LDS, then ask for half g + kRing.
// Behind the half that is waited for, two have been asked for: 17 operations.  A tile's results are stored after its
// last half, with the next tile's first three halves on their way (the first of them has been read): the stores are
// behind those three, and the three waits for them may leave the stores in flight too.  The half of the fourth wait is
// asked for behind the stores, so that this wait, like all later ones, leaves the 17 only.
#pragma once

#if defined(__HIPCC__)
#define DOBB_STREAM_FN __host__ __device__ __forceinline__
#else
#define DOBB_STREAM_FN inline
#endif

namespace dobb {

constexpr int kRing = 4;                         // slots
constexpr int kHalfLoads = 8;                    // of a wave for a half's codes
constexpr int kScaleLoads = 1;                   // .. and for the scales, with an even half
constexpr int kMostLeft = 63;                    // the most that a wait can leave
constexpr int kStartLeft = (kRing - 1) * kHalfLoads + kScaleLoads;      // half 0 done, halves 1 .. 3 on their way
constexpr int kBehind = (kRing - 2) * kHalfLoads + kScaleLoads;         // two halves, one of them even
// a whole tile's stores of a wave, and what a wait for a half from before them may leave
constexpr int stream_stores(bool fp32) { return fp32 ? 64 : 32; }
constexpr int stream_left(bool fp32) { return kBehind + stream_stores(fp32) < kMostLeft ? kBehind + stream_stores(fp32) : kMostLeft; }

class StreamWaits {
    int before_ = 0;                             // halves from before the stores that have not been waited for
public:
    // a tile's results have left: `counted` if in stream_stores operations at least
    DOBB_STREAM_FN void stored(bool counted) { before_ = counted ? kRing - 1 : 0; }
    // whether the next wait may leave the stores in flight
    DOBB_STREAM_FN bool next() {
        const bool more = before_ > 0;
        before_ -= more;
        return more;
    }
};

}  // namespace dobb
