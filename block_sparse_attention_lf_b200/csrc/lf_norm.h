// lf_norm.h -- launch interface of the gated residual norms (lf_norm.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace lf {

// Norm kinds of the C ABI (lf_norm_kind).
enum : int { NORM_NONE = 0, NORM_RMS = 1, NORM_LAYER = 2 };

constexpr int NORM_MAX_DIM = 16384;
constexpr int NORM_BWD_CTAS = 148;  // the gradient's CTAs, one an SM: bounds its workspace

struct NormVectors {  // fp32; gate, scale, shift [groups, dim], the rest [dim]; null where absent
    const float *gate, *scale, *shift, *pre_w, *pre_b, *post_w, *post_b;
};

struct NormArgs {
    const void *x, *y;
    void *r, *h;
    const void *dr, *dh;
    void *dx, *dy;
    NormVectors v;
    float *dgate, *dscale, *dshift, *dpre_w, *dpre_b, *dpost_w, *dpost_b;
    float* part;    // gradient: [slot][4][dim8] partial column sums; slot = CTA + group
    float* part_w;  // [CTA][4][dim8]: the same times 1 + scale or the gate, for the weights' gradients
    bool weights;   // any of those is wanted
    long long rows, per_group;
    int dim, pre, post;
    float eps, alpha;
    long long rows_per_cta;  // consecutive rows of a CTA
    int n_cta;
};

cudaError_t launch_norm_fwd(const NormArgs& a, int x_dtype, int y_dtype, cudaStream_t s);
cudaError_t launch_norm_bwd(const NormArgs& a, int x_dtype, int y_dtype, cudaStream_t s);

// Gradient kernel's CTAs for a call of `rows` rows.
inline int norm_bwd_ctas(long long rows) { return rows < NORM_BWD_CTAS ? static_cast<int>(rows) : NORM_BWD_CTAS; }

}  // namespace lf
