// Rotary positions (rope.cu): a call's parameters, passed to the kernel by value.
#pragma once

#include <algorithm>

#include "internal.h"

namespace mita {

struct RopeArgs {
    int B, H, Hkv, T, d, rot;
    int back;   // the transposed map
    int heads;  // heads of a block
    float gain;
    const void* in[2];  // Q, K
    void* out[2];
    long long is[2][3], os[2][3];  // batch, head and row strides in elements
    bool same[2];                  // in place
    const int* pos;                // or null
    long long pos_stride;
    unsigned long long turns[MITA_ROPE_PAIRS];  // turns per position, as fractions of 2^64
};
cudaError_t launch_rope(RopeArgs& a, int dtype, bool interleaved, cudaStream_t st);

}  // namespace mita
