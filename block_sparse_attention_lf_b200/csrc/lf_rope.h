// lf_rope.h -- launch interface of the rotary-position kernel (lf_rope.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace lf {

constexpr int ROPE_MAX_IO = 3;
constexpr int ROPE_MAX_PAIRS = 128;  // head_dim <= 256

struct RopeIo {
    const void* x;
    void* out;
    long long xs[3], os[3];  // element strides of batch, head, token
    int heads, rotate;
};

struct RopeArgs {
    RopeIo io[ROPE_MAX_IO];
    int n_io, batch, tokens, head_dim, rot_dim, n_axes;
    int axis_end[2];       // pairs of axis 0, of axes 0 and 1
    float amplitude;
    int backward;
    const int* positions;  // [batch or 1][tokens][n_axes]
    long long pos_batch;   // 0: shared by the batch
    int heads_per_thread;
    double turns[ROPE_MAX_PAIRS];  // revolutions per position of each pair
};

// elems: elements of a load (1, 2, 4 or 8; at most 16 bytes), which every pointer, stride and span
// is a whole number of
cudaError_t launch_rope(const RopeArgs& a, int dtype, bool half_layout, int elems, cudaStream_t s);

}  // namespace lf
