// lf_attn_bwd.h -- launch interface of the block-sparse attention's gradient (lf_attn_bwd.cu).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace lf {

struct AttnBwdArgs {
    const uint16_t* out;
    const uint16_t* out_lo;  // null: zeros
    const uint16_t* dout;
    const float* lse;
    const int* block_list;
    const int* block_count;
    float* delta;    // [BH, Lq]: <dout, out> of each row
    int* row_list;   // [BH, Nkv, Rq]: the query blocks that list each KV block, ascending
    int* row_count;  // [BH, Nkv]
    int* next_item;  // [2]: query and key items taken so far
    uint16_t* dq;
    uint16_t* dk;
    uint16_t* dv;
    int BH, list_cap, Rq, Nkv, bpf, F, rem, n_cur, NF, Lq;
    long long kv_stride;
    float scale, scale_log2;  // softmax scale, and it times log2(e)
    int* err;
};

struct AttnBwdMaps {
    CUtensorMap q, dout, k, v;  // 4-D views [head][frame][token][D], one 64 x 64 panel a box
};

cudaError_t launch_attn_bwd(const AttnBwdMaps& m, const AttnBwdArgs& a, int D, cudaStream_t s);

}  // namespace lf
