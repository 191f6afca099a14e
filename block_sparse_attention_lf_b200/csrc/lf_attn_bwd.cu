// lf_attn_bwd.cu -- gradient of the block-sparse attention in q, k and v on sm_100a tensor
// cores.
//
// With s the softmax scale, P = exp(s q k^T - lse) over a row's listed tokens and
// delta = <dout, out> per row:
//   dS = P * (dout v^T - delta),   dq = s dS k,   dk = s dS^T q,   dv = P^T dout.
// Where a row attends to few keys (or its softmax is sharp) dout v^T - delta cancels, and the
// roundings of out and of the forward's bf16 weights would put 2^-9 of |dout||v| into every dS
// of the row. So the forward also stores out_lo, and delta = <dout, out + out_lo> is the mean
// of dout v^T under weights that sum to one exactly: their roundings then weigh only the
// differences (dout v^T - delta), as dS's own rounding does.
//
// Two kernels of one shape, so that every sum has a fixed order and no value is added
// atomically: the query side (a CTA per query block, its KV block list streamed) forms dq,
// the key side (a CTA per KV block, the query blocks that list it streamed) forms dk and
// dv. Both form P and dS anew: 7 products instead of 5, for no fp32 dq in memory and the
// same bits on every run. The key side's lists are the transposed block lists, built by a
// small kernel before.
//
// One CTA holds the 64 rows of its own block (X0, Y0) in shared memory and streams tiles of
// two listed blocks (Xs, Ys, 128 rows):
//                 X0   Y0     Xs   Ys
//   query side    q    dout   k    v
//   key side      k    v      q    dout
//   S' = Xs X0^T and dP' = Ys Y0^T (M = 128 streamed rows, N = 64, K = head_dim) in TMEM;
//   a softmax thread owns one streamed row (TMEM lane) of the tile, forms P and dS in fp32
//   and writes them as bf16 rows of 64 to shared memory (128-byte swizzle);
//   acc0^T += Xs^T dS (dq^T or dk^T), and on the key side acc1^T += Ys^T P (dv^T):
//   M = head_dim (MN-major A: the streamed tile as it lies), N = 64 (MN-major B), K = 128.
// M is 128 in every product at head_dim 128 (M = 64 issues at half rate).
//
// Tensor maps run over [head][frame][token][D], so tokens past a frame's end and blocks that
// a list does not have read as zeros: every box has the same size and no row of a tile is
// ever stale. Rows that are not there get P = dS = 0.
//
// Warps: 0 loads, 1 issues MMAs, 2 owns TMEM, 4-11 are two softmax warpgroups that take the
// tiles in turn, so one tile's exponentials run under the other's products. Every wait is
// bounded, as in the forward kernel.
#include "lf_attn_bwd.h"
#include "lf_device.cuh"

#include <cuda_bf16.h>

#include <atomic>

namespace lf {
namespace {

constexpr int BWD_THREADS = 384;
constexpr int W_LOAD = 0, W_MMA = 1, W_TMEM = 2, W_SOFT0 = 4;
constexpr uint32_t TMEM_COLS = 512;  // S' of warpgroup g: 64 g; dP': 128 + 64 g; acc0^T: 256; acc1^T: 320
constexpr uint32_t TM_DP = 128, TM_ACC0 = 256, TM_ACC1 = 320;

template <int D, bool KV>
struct BwdLayout {
    static constexpr int NP = D / 64;                       // 64-element panels of a row
    static constexpr int NX = D == 64 ? 4 : (KV ? 2 : 3);   // tiles in the Xs and Ys rings: Ys is only read
    static constexpr int NY = D == 64 ? 4 : 2;              // by dP' on the query side and leaves early
    static constexpr uint32_t OWN_PANEL = 64u * 128u;
    static constexpr uint32_t OWN = NP * OWN_PANEL;
    static constexpr uint32_t PANEL = 128u * 128u;
    static constexpr uint32_t TILE = NP * PANEL;
    static constexpr uint32_t PBUF = 128u * 128u;           // 128 rows x 64 bf16
    static constexpr uint32_t OFF_X0 = 0;
    static constexpr uint32_t OFF_Y0 = OFF_X0 + OWN;
    static constexpr uint32_t OFF_X = OFF_Y0 + OWN;
    static constexpr uint32_t OFF_Y = OFF_X + NX * TILE;
    static constexpr uint32_t OFF_DS = OFF_Y + NY * TILE;
    static constexpr uint32_t OFF_P = OFF_DS + 2 * PBUF;    // key side only
    static constexpr uint32_t OFF_AUX = OFF_P + (KV ? 2 * PBUF : 0u);
};

struct BwdAux {
    uint64_t own_full;
    uint64_t x_full[4], x_empty[4], y_full[4], y_empty[4];
    uint64_t s_full[2], p_full[2], p_empty[2];
    uint64_t done;
    uint32_t tmem_base;
    int abort;
    alignas(16) float lse2[64];   // query side: log2(e) lse of the CTA's rows (+inf where P must be 0)
    alignas(16) float delta[64];
};

template <int D, bool KV>
constexpr uint32_t bwd_smem_bytes()
{
    return BwdLayout<D, KV>::OFF_AUX + static_cast<uint32_t>(sizeof(BwdAux)) + 1024u;
}

// A row's log-sum-exp in base 2; +inf (P = 0) for a row that attends to nothing.
__device__ __forceinline__ float lse_log2(float lse)
{
    return lse == -INFINITY ? INFINITY : lse * 1.4426950408889634f;
}

template <int D, bool KV>
__global__ void __launch_bounds__(BWD_THREADS, 1)
attn_bwd_kernel(const __grid_constant__ CUtensorMap tm_x0, const __grid_constant__ CUtensorMap tm_y0,
                const __grid_constant__ CUtensorMap tm_xs, const __grid_constant__ CUtensorMap tm_ys, const AttnBwdArgs a)
{
    using L = BwdLayout<D, KV>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    BwdAux& x = *reinterpret_cast<BwdAux*>(smem + L::OFF_AUX);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // This CTA's block: frame f0, block j0 of it; n0 valid rows starting at out_row of the output.
    const int per_head = KV ? a.Nkv : a.Rq;
    const int bh = blockIdx.x / per_head;
    const int own = blockIdx.x - bh * per_head;
    const int f0 = own / a.bpf, j0 = own - f0 * a.bpf;
    const int n0 = j0 == a.bpf - 1 ? a.rem : 64;
    const long long head_row = static_cast<long long>(bh) * (KV ? a.kv_stride : a.Lq);
    const long long out_row = head_row + static_cast<long long>(f0) * a.F + j0 * 64;
    const long long lrow = static_cast<long long>(bh) * per_head + own;
    const int* lst = KV ? a.row_list + lrow * a.Rq : a.block_list + lrow * a.list_cap;
    int cnt = KV ? a.row_count[lrow] : __ldg(a.block_count + lrow);
    if (!KV && (cnt < 0 || cnt > a.list_cap)) {
        if (tid == 0) record_error(a.err, DEVERR_LIST | 1);
        cnt = cnt < 0 ? 0 : a.list_cap;
    }
    const int n_it = (cnt + 1) >> 1;
    const int listed = KV ? a.Rq : a.Nkv;       // valid ids are [0, listed)
    const int frames = KV ? a.n_cur : a.NF;     // frames of the streamed side

    if (tid == 0) {
        mbar_init(&x.own_full, 1);
        for (int s = 0; s < 4; ++s) {
            mbar_init(&x.x_full[s], 1);
            mbar_init(&x.x_empty[s], 1);
            mbar_init(&x.y_full[s], 1);
            mbar_init(&x.y_empty[s], 1);
        }
        for (int g = 0; g < 2; ++g) {
            mbar_init(&x.s_full[g], 1);
            mbar_init(&x.p_full[g], 4);  // one arrival per warp of the warpgroup
            mbar_init(&x.p_empty[g], 1);
        }
        mbar_init(&x.done, 1);
        x.abort = 0;
        fence_mbar_init();
    }
    if (warp == W_TMEM) {
        tmem_alloc(&x.tmem_base, TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = x.tmem_base;
    volatile int* abort_flag = &x.abort;

    if (warp == W_LOAD) {
        if (n_it > 0) {
            mbar_arrive_expect_tx_elect(&x.own_full, 2 * L::OWN);
            for (int p = 0; p < L::NP; ++p) {
                tma_load_4d_elect(smem + L::OFF_X0 + p * L::OWN_PANEL, &tm_x0, p * 64, j0 * 64, f0, bh, &x.own_full);
                tma_load_4d_elect(smem + L::OFF_Y0 + p * L::OWN_PANEL, &tm_y0, p * 64, j0 * 64, f0, bh, &x.own_full);
            }
        }
        int armed = 0;
        for (int it = 0; it < n_it; ++it) {
            int tau[2], tok[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int e = 2 * it + h;
                const int id = e < cnt ? __ldg(lst + e) : -1;
                const bool good = id >= 0 && id < listed;
                if (e < cnt && !good && lane == 0) record_error(a.err, DEVERR_LIST | 2);
                tau[h] = good ? id / a.bpf : frames;  // past the last frame: the box reads zeros
                tok[h] = good ? (id - tau[h] * a.bpf) * 64 : 0;
            }
            const int xi = it % L::NX, yi = it % L::NY;
            if (!mbar_wait(&x.x_empty[xi], ((it / L::NX) & 1) ^ 1, abort_flag, a.err, 0x40)) break;
            mbar_arrive_expect_tx_elect(&x.x_full[xi], L::TILE);
            for (int h = 0; h < 2; ++h)
                for (int p = 0; p < L::NP; ++p)
                    tma_load_4d_elect(smem + L::OFF_X + xi * L::TILE + p * L::PANEL + h * 8192u, &tm_xs, p * 64,
                                          tok[h], tau[h], bh, &x.x_full[xi]);
            armed = 2 * it + 1;
            if (!mbar_wait(&x.y_empty[yi], ((it / L::NY) & 1) ^ 1, abort_flag, a.err, 0x41)) break;
            mbar_arrive_expect_tx_elect(&x.y_full[yi], L::TILE);
            for (int h = 0; h < 2; ++h)
                for (int p = 0; p < L::NP; ++p)
                    tma_load_4d_elect(smem + L::OFF_Y + yi * L::TILE + p * L::PANEL + h * 8192u, &tm_ys, p * 64,
                                          tok[h], tau[h], bh, &x.y_full[yi]);
            armed = 2 * it + 2;
        }
        if (*abort_flag && n_it > 0) {
            // let every copy already issued land before the CTA exits
            mbar_drain(&x.own_full, 0, 10000000ull);
            const int xs = (armed + 1) >> 1, ys = armed >> 1;
            for (int e = max(0, xs - L::NX); e < xs; ++e) mbar_drain(&x.x_full[e % L::NX], (e / L::NX) & 1, 10000000ull);
            for (int e = max(0, ys - L::NY); e < ys; ++e) mbar_drain(&x.y_full[e % L::NY], (e / L::NY) & 1, 10000000ull);
        }
    } else if (warp == W_MMA) {
        constexpr uint32_t IDESC_S = idesc_bf16_f32(128, 64, false, false);
        constexpr uint32_t IDESC_A = idesc_bf16_f32(D, 64, true, true);
        const uint64_t dX0 = sdesc_sw128(smem_u32(smem + L::OFF_X0), 16, 1024);
        const uint64_t dY0 = sdesc_sw128(smem_u32(smem + L::OFF_Y0), 16, 1024);
        const uint64_t dXk = sdesc_sw128(smem_u32(smem + L::OFF_X), 16, 1024);            // K-major: S'
        const uint64_t dYk = sdesc_sw128(smem_u32(smem + L::OFF_Y), 16, 1024);
        const uint64_t dXm = sdesc_sw128(smem_u32(smem + L::OFF_X), L::PANEL, 1024);      // MN-major: acc0
        const uint64_t dYm = sdesc_sw128(smem_u32(smem + L::OFF_Y), L::PANEL, 1024);
        const uint64_t dDS = sdesc_sw128(smem_u32(smem + L::OFF_DS), 1024, 1024);
        const uint64_t dP = sdesc_sw128(smem_u32(smem + L::OFF_P), 1024, 1024);
        bool ok = n_it > 0 && mbar_wait(&x.own_full, 0, abort_flag, a.err, 0x50);
        bool issued = false;
        // S' and dP' of tile it into warpgroup it & 1's buffers (its reads of tile it - 2 came
        // before p_full of that tile, which acc(it - 2) waited for)
        auto scores = [&](int it) -> bool {
            const int xi = it % L::NX, yi = it % L::NY;
            const uint32_t d = tmem + 64u * static_cast<uint32_t>(it & 1);
            if (!mbar_wait(&x.x_full[xi], (it / L::NX) & 1, abort_flag, a.err, 0x51)) return false;
            tc_fence_after();
            const uint64_t xb = dXk + ((xi * L::TILE) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                umma_bf16_elect(d, xb + (((kk >> 2) * L::PANEL + (kk & 3) * 32) >> 4),
                                dX0 + (((kk >> 2) * L::OWN_PANEL + (kk & 3) * 32) >> 4), IDESC_S, kk > 0 ? 1u : 0u);
            issued = true;
            if (!mbar_wait(&x.y_full[yi], (it / L::NY) & 1, abort_flag, a.err, 0x52)) return false;
            const uint64_t yb = dYk + ((yi * L::TILE) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                umma_bf16_elect(d + TM_DP, yb + (((kk >> 2) * L::PANEL + (kk & 3) * 32) >> 4),
                                dY0 + (((kk >> 2) * L::OWN_PANEL + (kk & 3) * 32) >> 4), IDESC_S, kk > 0 ? 1u : 0u);
            if (!KV) umma_commit_elect(&x.y_empty[yi]);
            umma_commit_elect(&x.s_full[it & 1]);
            return true;
        };
        auto accumulate = [&](int it) -> bool {
            const int g = it & 1, xi = it % L::NX, yi = it % L::NY;
            if (!mbar_wait(&x.p_full[g], (it >> 1) & 1, abort_flag, a.err, 0x53)) return false;
            tc_fence_after();
            const uint64_t xb = dXm + ((xi * L::TILE) >> 4), yb = dYm + ((yi * L::TILE) >> 4);
            const uint64_t sb = dDS + ((g * L::PBUF) >> 4), pb = dP + ((g * L::PBUF) >> 4);
            const int slices = 2 * it + 1 < cnt ? 8 : 4;  // 16 rows each; the second block may be missing
            for (int kk = 0; kk < slices; ++kk) {
                const uint32_t more = (it > 0 || kk > 0) ? 1u : 0u;
                umma_bf16_elect(tmem + TM_ACC0, xb + ((kk * 2048) >> 4), sb + ((kk * 2048) >> 4), IDESC_A, more);
                if (KV) umma_bf16_elect(tmem + TM_ACC1, yb + ((kk * 2048) >> 4), pb + ((kk * 2048) >> 4), IDESC_A, more);
            }
            umma_commit_elect(&x.x_empty[xi]);
            if (KV) umma_commit_elect(&x.y_empty[yi]);
            umma_commit_elect(&x.p_empty[g]);
            return true;
        };
        for (int it = 0; ok && it < n_it; ++it) {
            ok = scores(it);
            if (ok && it > 0) ok = accumulate(it - 1);
        }
        if (ok && n_it > 0) ok = accumulate(n_it - 1);
        if (ok || issued) umma_commit_elect(&x.done);
        if (*abort_flag && issued) mbar_drain(&x.done, 0, 10000000ull);
    } else if (warp >= W_SOFT0) {
        const int g = (warp - W_SOFT0) >> 2;       // this warpgroup takes the tiles it % 2 == g
        const int sp = warp & 3;                   // TMEM sub-partition
        const int rr = sp * 32 + lane;             // streamed row of the tile
        const int hb = rr >> 6, ri = rr & 63;      // its block in the tile and row of the block
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(sp * 32) << 16);
        const int st = tid - W_SOFT0 * 32;         // 0 .. 255

        if (!KV) {
            // delta of the CTA's 64 rows, eight rows a warp; the key side reads it from memory
            constexpr int EPL = D / 32;
            for (int i = 0; i < 8; ++i) {
                const int r = (warp - W_SOFT0) * 8 + i;
                float dot = 0.f;
                if (r < n0) {
                    const long long at = (out_row + r) * D + lane * EPL;
                    uint32_t o[EPL / 2], d[EPL / 2], lo[EPL / 2] = {};
                    if constexpr (EPL == 4) {
                        if (a.out_lo) {
                            const uint2 lu = __ldg(reinterpret_cast<const uint2*>(a.out_lo + at));
                            lo[0] = lu.x; lo[1] = lu.y;
                        }
                        const uint2 ou = __ldg(reinterpret_cast<const uint2*>(a.out + at));
                        const uint2 du = __ldg(reinterpret_cast<const uint2*>(a.dout + at));
                        o[0] = ou.x; o[1] = ou.y; d[0] = du.x; d[1] = du.y;
                    } else {
                        if (a.out_lo) lo[0] = __ldg(reinterpret_cast<const uint32_t*>(a.out_lo + at));
                        o[0] = __ldg(reinterpret_cast<const uint32_t*>(a.out + at));
                        d[0] = __ldg(reinterpret_cast<const uint32_t*>(a.dout + at));
                    }
#pragma unroll
                    for (int k = 0; k < EPL / 2; ++k) {
                        dot = fmaf(__uint_as_float(o[k] << 16) + __uint_as_float(lo[k] << 16), __uint_as_float(d[k] << 16), dot);
                        dot = fmaf(__uint_as_float(o[k] & 0xFFFF0000u) + __uint_as_float(lo[k] & 0xFFFF0000u),
                                   __uint_as_float(d[k] & 0xFFFF0000u), dot);
                    }
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
                if (lane == 0) {
                    x.delta[r] = dot;
                    x.lse2[r] = r < n0 ? lse_log2(__ldg(a.lse + out_row + r)) : INFINITY;
                    if (r < n0) a.delta[out_row + r] = dot;
                }
            }
            named_bar_sync(3, 256);
        }

        // The streamed row of tile `it`: is it there, and (key side) its lse and delta.
        float lse2 = INFINITY, delta = 0.f, lse2_next = INFINITY, delta_next = 0.f;
        bool valid = false, valid_next = false;
        auto fetch = [&](int it) {
            const int e = 2 * it + hb;
            valid_next = false;
            lse2_next = INFINITY;
            delta_next = 0.f;
            if (it < n_it && e < cnt) {
                const int id = __ldg(lst + e);
                if (id >= 0 && id < listed) {
                    const int f = id / a.bpf, j = id - f * a.bpf;
                    valid_next = ri < (j == a.bpf - 1 ? a.rem : 64);
                    if (KV && valid_next) {
                        const long long at = static_cast<long long>(bh) * a.Lq + f * a.F + j * 64 + ri;
                        lse2_next = lse_log2(__ldg(a.lse + at));
                        delta_next = a.delta[at];
                    }
                }
            }
        };
        fetch(g);
        int j = 0;
        for (int it = g; it < n_it; it += 2, ++j) {
            valid = valid_next;
            lse2 = lse2_next;
            delta = delta_next;
            fetch(it + 2);
            mbar_wait(&x.s_full[g], j & 1, abort_flag, a.err, 0x60);
            __syncwarp();
            tc_fence_after();
            if (j > 0) mbar_wait(&x.p_empty[g], (j - 1) & 1, abort_flag, a.err, 0x61);
            uint8_t* ds_row = smem + L::OFF_DS + g * L::PBUF + rr * 128;
            uint8_t* p_row = smem + L::OFF_P + g * L::PBUF + rr * 128;
            __syncwarp();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float sv[32], dp[32];
                tmem_ld32(lane_base + 64u * g + 32u * h, sv);
                tmem_ld32(lane_base + TM_DP + 64u * g + 32u * h, dp);
                tmem_ld_wait();
                uint32_t pk[16], dk[16];
#pragma unroll
                for (int c = 0; c < 32; c += 4) {
                    float4 l4, d4;
                    if (KV) {
                        l4 = make_float4(lse2, lse2, lse2, lse2);
                        d4 = make_float4(delta, delta, delta, delta);
                    } else {
                        l4 = *reinterpret_cast<const float4*>(&x.lse2[32 * h + c]);
                        d4 = *reinterpret_cast<const float4*>(&x.delta[32 * h + c]);
                    }
                    const float p0 = fast_exp2(fmaf(sv[c], a.scale_log2, -l4.x));
                    const float p1 = fast_exp2(fmaf(sv[c + 1], a.scale_log2, -l4.y));
                    const float p2 = fast_exp2(fmaf(sv[c + 2], a.scale_log2, -l4.z));
                    const float p3 = fast_exp2(fmaf(sv[c + 3], a.scale_log2, -l4.w));
                    if (KV) {
                        pk[c >> 1] = pack_bf16x2(p0, p1);
                        pk[(c >> 1) + 1] = pack_bf16x2(p2, p3);
                    }
                    dk[c >> 1] = pack_bf16x2(p0 * (dp[c] - d4.x), p1 * (dp[c + 1] - d4.y));
                    dk[(c >> 1) + 1] = pack_bf16x2(p2 * (dp[c + 2] - d4.z), p3 * (dp[c + 3] - d4.w));
                }
                // a streamed row that is not there contributes nothing, whatever its P came out as
                if (!valid) {
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        dk[c] = 0u;
                        if (KV) pk[c] = 0u;
                    }
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int chunk = (4 * h + c) ^ (rr & 7);
                    *reinterpret_cast<uint4*>(ds_row + chunk * 16) = make_uint4(dk[4 * c], dk[4 * c + 1], dk[4 * c + 2], dk[4 * c + 3]);
                    if (KV)
                        *reinterpret_cast<uint4*>(p_row + chunk * 16) = make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
                }
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&x.p_full[g]);
        }

        // Epilogue: acc^T [head_dim lanes][64 columns] -> bf16 rows through shared memory (the Xs
        // ring is idle once every MMA is done). Warpgroup g takes columns [32 g, 32 g + 32).
        constexpr int NOUT = KV ? 2 : 1;
        __nv_bfloat16* stage = reinterpret_cast<__nv_bfloat16*>(smem + L::OFF_X);
        if (n_it > 0) {
            mbar_wait(&x.done, 0, abort_flag, a.err, 0x62);
            __syncwarp();
            tc_fence_after();
            const int d = D == 128 ? rr : sp * 16 + (lane & 15);  // M = 64: 16 rows in each sub-partition's first lanes
            const bool has = D == 128 || lane < 16;
#pragma unroll
            for (int o = 0; o < NOUT; ++o) {
                float v[32];
                __syncwarp();
                tmem_ld32(lane_base + (o == 0 ? TM_ACC0 : TM_ACC1) + 32u * g, v);
                tmem_ld_wait();
                const float f = o == 0 ? a.scale : 1.f;
                if (has) {
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        stage[(o * 64 + 32 * g + c) * D + d] = __float2bfloat16_rn(v[c] * f);
                }
            }
            tc_fence_before();
            named_bar_sync(3, 256);
        }
        constexpr int CH = D / 8;  // 16-byte chunks of a row
        for (int i = st; i < NOUT * n0 * CH; i += 256) {
            const int o = i / (n0 * CH), q = i - o * (n0 * CH);
            const int row = q / CH, c8 = q - row * CH;
            uint16_t* dst = KV ? (o == 0 ? a.dk : a.dv) : a.dq;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (n_it > 0) v = *reinterpret_cast<const uint4*>(stage + (o * 64 + row) * D + c8 * 8);
            *reinterpret_cast<uint4*>(dst + (out_row + row) * D + c8 * 8) = v;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == W_TMEM) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

// Transposes the block lists of one head: for each KV block the query blocks that list it,
// ascending. A CTA owns 1024 KV blocks and walks the head's rows 32 at a time: each row's
// warp sets its bit for every block it lists, then each block's thread appends the bits it
// finds. (Bits are set atomically, but the set does not depend on the order.)
constexpr int TR_BLOCKS = 1024;

__global__ void __launch_bounds__(TR_BLOCKS) transpose_lists_kernel(const AttnBwdArgs a)
{
    __shared__ uint32_t bits[TR_BLOCKS];
    const int chunks = (a.Nkv + TR_BLOCKS - 1) / TR_BLOCKS;
    const int bh = blockIdx.x / chunks, g0 = (blockIdx.x - bh * chunks) * TR_BLOCKS, t = threadIdx.x;
    const int warp = t >> 5, lane = t & 31;
    int n = 0;
    int* mine = a.row_list + (static_cast<long long>(bh) * a.Nkv + g0 + t) * a.Rq;
    for (int w = 0; w * 32 < a.Rq; ++w) {
        bits[t] = 0u;
        __syncthreads();
        const int r = w * 32 + warp;
        if (r < a.Rq) {
            const long long lrow = static_cast<long long>(bh) * a.Rq + r;
            const int cnt = min(max(__ldg(a.block_count + lrow), 0), a.list_cap);
            const int* lst = a.block_list + lrow * a.list_cap;
            for (int e = lane; e < cnt; e += 32) {
                const int at = __ldg(lst + e) - g0;
                if (at >= 0 && at < TR_BLOCKS && at + g0 < a.Nkv) {
                    const uint32_t old = atomicOr(&bits[at], 1u << warp);
                    if (old >> warp & 1u) record_error(a.err, DEVERR_LIST | 3);  // a block named twice
                }
            }
        }
        __syncthreads();
        for (uint32_t m = bits[t]; m; m &= m - 1) mine[n++] = w * 32 + __ffs(m) - 1;
        __syncthreads();
    }
    if (g0 + t < a.Nkv) a.row_count[static_cast<long long>(bh) * a.Nkv + g0 + t] = n;
}

template <int D, bool KV>
cudaError_t launch_side(const AttnBwdMaps& m, const AttnBwdArgs& a, cudaStream_t s)
{
    constexpr uint32_t smem = bwd_smem_bytes<D, KV>();
    static_assert(smem <= 232448, "shared memory plan exceeds 227 KB");
    static std::atomic<bool> configured[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !configured[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(attn_bwd_kernel<D, KV>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev].store(true, std::memory_order_release);
    }
    const unsigned grid = static_cast<unsigned>(a.BH) * static_cast<unsigned>(KV ? a.Nkv : a.Rq);
    if (KV)
        attn_bwd_kernel<D, KV><<<grid, BWD_THREADS, smem, s>>>(m.k, m.v, m.q, m.dout, a);
    else
        attn_bwd_kernel<D, KV><<<grid, BWD_THREADS, smem, s>>>(m.q, m.dout, m.k, m.v, a);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const AttnBwdMaps& m, const AttnBwdArgs& a, cudaStream_t s)
{
    const unsigned chunks = static_cast<unsigned>((a.Nkv + TR_BLOCKS - 1) / TR_BLOCKS);
    transpose_lists_kernel<<<chunks * static_cast<unsigned>(a.BH), TR_BLOCKS, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if ((e = launch_side<D, false>(m, a, s)) != cudaSuccess) return e;
    return launch_side<D, true>(m, a, s);
}

}  // namespace

cudaError_t launch_attn_bwd(const AttnBwdMaps& m, const AttnBwdArgs& a, int D, cudaStream_t s)
{
    return D == 128 ? launch_d<128>(m, a, s) : launch_d<64>(m, a, s);
}

}  // namespace lf
