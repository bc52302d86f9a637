// Sine and cosine of a rotary angle, shared by the rotation and the cache append.
#pragma once

#include "common.cuh"

namespace lsa {

// (cos, sin) of position * inv_freq, both times mscale.  rev_freq = inv_freq / (2 pi): the angle is
// formed in turns and in 64 bits, its whole turns dropped exactly, and what is left (at most half a turn)
// taken to 32 bits, an absolute error of 2^-25 of a half turn at any position.
__device__ __forceinline__ float2 rope_cs(int pos, double rev_freq, float mscale) {
    const double turns = (double)pos * rev_freq;
    float s, c;
    sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
    return make_float2(c * mscale, s * mscale);
}

// What the kernels take of an lsa_rope, by value.
struct RopeTable {
    int rot_dim, interleaved;
    float mscale;
    double rev_freq[LSA_ROPE_MAX_DIM / 2];       // inv_freq / (2 pi)
};

}  // namespace lsa
