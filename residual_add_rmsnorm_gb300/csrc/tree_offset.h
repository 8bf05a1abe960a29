// tree_offset.h -- the offset of a row's running softmax in k_tree_tile: where
// it begins and how it moves.  Plain binary32 additions, the same on the host.
//
// A weight is 2^(score - off).  An offset, once chosen, moves up only where a
// weight passes 2^most; it then moves by a whole number, so that what the row
// has summed up is scaled by a power of two.  Offsets have binary32's steps:
// from |off| = 2^28 on, 32 and more, which a wanted move may be smaller than.
// So the offset moves at most kMoves times for the keys at hand, and what is
// over `most` after that counts as `most`: keys that tie for the largest score
// keep equal weights, and every key below them, at least a step of 32 away,
// has a weight of at most 2^-19 of theirs.
#pragma once

#include <math.h>
#include <stdint.h>
#include <string.h>

#ifdef __CUDACC__
#define RARN_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define RARN_HOST_DEVICE inline
#endif

namespace rarn {
namespace tree {

constexpr float kCentre = 4.f;    // log2 of a row's largest weight times value scale, to begin with
constexpr float kHighest = 15.f;  // and at most, so that binary16 holds it

// The next binary32 number above (up) or below a finite x that is not zero.
RARN_HOST_DEVICE float next_number(float x, bool up) {
    int32_t i;
    memcpy(&i, &x, 4);
    i += (x > 0.f) == up ? 1 : -1;
    memcpy(&x, &i, 4);
    return x;
}

// The offset of a row whose largest score is `top`: brings its weight to
// 2^centre, or to what the steps of binary32 allow, but not to less than 2^-8
// of that.
RARN_HOST_DEVICE float first_offset(float top, float centre) {
    const float off = top - centre;
    return top - off < centre - 8.f && off > -3e38f ? next_number(off, false) : off;
}

// Moves for one run of keys: one where scores differ by less than 2^23; each
// more leaves 2^-22 of the difference, of at most 2^128.
constexpr int kMoves = 8;

// Minus the offset (`sub`) after a move that brings a weight 2^high to
// 2^centre or up to a factor of two under it, or as near as binary32's steps
// allow from above; *down: by how much it moved, a whole number (0: not at all).
// From 2^23 on `high`, a rounded difference, does not say where the score is,
// and a move that went too far would lose the row's largest weight: it stops
// short of it by more than the rounding and any centre.
RARN_HOST_DEVICE float moved_offset(float sub, float high, float centre, float *down) {
    float s = sub - (high < 8388608.f ? ceilf(high - centre) : high * (1.f - 0x1p-22f) - 256.f);
    if (high - (sub - s) < centre - 9.f) s = next_number(s, true);
    *down = rintf(sub - s);
    return s;
}

}  // namespace tree
}  // namespace rarn
