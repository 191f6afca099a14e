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
// Every sum has a fixed order and no value is added atomically. A query item (one query block,
// its KV block list streamed) forms dq, a key item (one KV block, the query blocks that list it
// streamed) forms dk and dv. Both form P and dS anew: 7 products instead of 5, for no fp32 dq in
// memory and the same bits on every run. The key items' lists are the transposed block lists,
// which a preparing kernel builds beside delta.
//
// An item keeps the 64 rows of its own block (X0, Y0) in shared memory and streams tiles of two
// listed blocks (Xs, Ys, 128 rows):
//                X0   Y0     Xs   Ys
//   query item   q    dout   k    v
//   key item     k    v      q    dout
//   S' = Xs X0^T and dP' = Ys Y0^T (M = 128 streamed rows, N = 64, K = head_dim) in TMEM;
//   a softmax thread owns one streamed row (TMEM lane) of the tile, forms P and dS in fp32
//   and writes them as bf16 rows of 64 to shared memory (128-byte swizzle; the one rounding
//   the tensor cores' operands need);
//   acc0^T += Xs^T dS (dq^T or dk^T), and for a key item acc1^T += Ys^T P (dv^T):
//   M = head_dim (MN-major A: the streamed tile as it lies), N = 64 (MN-major B), K = 128.
// M is 128 in every product at head_dim 128 (M = 64 issues at half rate).
//
// Tensor maps run over [head][frame][token][D], so tokens past a frame's end and blocks that
// a list does not have read as zeros: every box has the same size and no row of a tile is
// ever stale. Rows that are not there get P = dS = 0.
//
// One persistent CTA per SM takes query items, then key items, from two counters (which CTA
// takes an item changes no sum), so neither side has a last wave of its own. A key item is only
// some eight tiles long, so its boundaries must not drain the pipeline: roles run through the
// items independently, the loads of the next item start while the last one's sums are still
// formed, and accumulators are double-buffered in TMEM. Roles (16 warps):
//   0 Xs, X0, Y0 loads and the item counter; 1 Ys loads and row statistics (two issuing warps:
//   one alone reaches half the SM's ingest rate); 2 score products; 3 accumulating products;
//   4-11 two softmax warpgroups, half of every tile's columns each; 12-15 epilogue.
// Every wait is bounded, as in the forward kernel.
//
// Measured at layer480p (12 heads of 4680 queries, 21 frames of 1560 tokens, head_dim 128, 108 blocks a
// row; 1965 MHz): preparing kernel 20 us, this one 767 us, 884 TFLOP/s for its seven products; query
// items alone 308 us, key items alone 509. A key item's tile takes about 2950 cycles, boundaries among
// them, of which its MMAs are 1536 (M = 128, N = 64 products are bound by their operands' shared-memory
// bandwidth). A clock around every wait: the score warp stands 1084 cycles a key tile for Ys and 324 for
// Xs, the accumulating warp 1147 for P and dS, the softmax 828 for scores; a query tile of about 1840
// has 364 and 559 of the first and third. So two slots of a ring, which is what shared memory holds
// beside the own blocks, do not hide a key tile's chain load - scores - softmax - products (without the
// exponentials it still takes 495 us). Tried and left: S' and dP' on barriers of their own, a third Xs
// tile for key items in place of the second own block, dk before dv (each slower or within 20 us).
#include "lf_attn_bwd.h"
#include "lf_internal.h"
#include "lf_device.cuh"

#include <cuda_bf16.h>

#include <atomic>

namespace lf {
namespace {

constexpr int BWD_THREADS = 512;
constexpr int W_LOADX = 0, W_LOADY = 1, W_SCORE = 2, W_ACC = 3, W_SOFT0 = 4, W_EPI0 = 12;
constexpr int SCHED_READERS = 15;           // every warp but the one that publishes items
constexpr uint32_t TMEM_COLS = 512;         // S' of tile t: 64 (t % 2); dP': 128 more;
constexpr uint32_t TM_DP = 128;             // acc0^T of the n-th item with tiles: 256 + 128 (n % 2), acc1^T 64 more
constexpr uint32_t TM_ACC = 256;

template <int D, bool KV>
struct BwdLayout {
    static constexpr int NP = D / 64;                       // 64-element panels of a row
    // tiles in the Xs and Ys rings (a query item's Ys is only read by dP' and leaves early; it
    // needs no P buffers, so a third Xs tile fits)
    static constexpr int NX = D == 64 ? 4 : (KV ? 2 : 3);
    static constexpr int NY = D == 64 ? 4 : 2;
    // Key items are short, so the next item's X0 and Y0 load while the last one's tiles are still at
    // work (790 -> 767 us at layer480p); the room comes from second P and dS buffers, which two
    // tiles in flight hardly use.
    static constexpr int OWNS = KV ? 2 : 1;
    static constexpr int PBUFS = KV ? 1 : 2;
    static constexpr uint32_t OWN_PANEL = 64u * 128u;
    static constexpr uint32_t OWN = NP * OWN_PANEL;
    static constexpr uint32_t PANEL = 128u * 128u;
    static constexpr uint32_t TILE = NP * PANEL;
    static constexpr uint32_t PBUF = 128u * 128u;           // 128 rows x 64 bf16
    static constexpr uint32_t OFF_X0 = 0;                   // own buffers: X0, then Y0
    static constexpr uint32_t OFF_DS = OFF_X0 + OWNS * 2 * OWN;
    static constexpr uint32_t OFF_X = OFF_DS + PBUFS * PBUF;
    static constexpr uint32_t OFF_Y = OFF_X + NX * TILE;
    static constexpr uint32_t OFF_P = OFF_Y + NY * TILE;    // key items only
    static constexpr uint32_t END = OFF_P + (KV ? PBUFS * PBUF : 0u);
};

struct BwdBars {
    uint64_t own_full[2], own_empty[2];
    uint64_t x_full[4], x_empty[4], y_full[4], y_empty[4];
    uint64_t s_full[2], s_free[2], p_full[2], p_empty[2];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t info_full[2], info_empty[2];
    uint64_t sched_full[4], sched_empty[4];
    uint64_t drain_s, drain_a;
};

template <int D>
struct BwdAux {
    BwdBars bars[2];  // query items, key items: a barrier is initialised once
    uint32_t tmem_base;
    int abort;
    int sched_item[4], sched_cnt[4];  // item -1: no more
    int tile_rows[4][2];              // query side: valid rows of an Xs slot's two blocks
    // minus log2(e) lse (-inf: P = 0) and minus delta; query side: the item's 64 rows by item
    // parity; key side: an Ys slot's 128 rows
    alignas(16) float info[D == 64 ? 4 : 2][2][128];
};

template <int D>
constexpr uint32_t bwd_smem_bytes()
{
    constexpr uint32_t q = BwdLayout<D, false>::END, k = BwdLayout<D, true>::END;
    return (q > k ? q : k) + static_cast<uint32_t>(sizeof(BwdAux<D>));
}

// Minus a row's log-sum-exp in base 2; -inf (P = 0) for a row that attends to nothing.
__device__ __forceinline__ float neg_lse_log2(float lse)
{
    return lse == -INFINITY ? -INFINITY : lse * -1.4426950408889634f;
}

// A query item's count, clamped as the forward clamps it.
template <bool KV>
__device__ __forceinline__ int item_count(const AttnBwdArgs& a, int item)
{
    int cnt = KV ? a.row_count[item] : __ldg(a.block_count + item);
    if (!KV && (cnt < 0 || cnt > a.list_cap)) {
        record_error(a.err, DEVERR_LIST | 1);
        cnt = cnt < 0 ? 0 : a.list_cap;
    }
    return cnt;
}

struct Own {  // an item's own block
    int bh, f, j, n;       // head, frame, block of the frame, valid rows
    long long row;         // its first row in the output
    const int* list;
};

template <bool KV>
__device__ __forceinline__ Own own_of(const AttnBwdArgs& a, int item)
{
    const int per_head = KV ? a.Nkv : a.Rq;
    Own o;
    o.bh = item / per_head;
    const int g = item - o.bh * per_head;
    o.f = g / a.bpf;
    o.j = g - o.f * a.bpf;
    o.n = o.j == a.bpf - 1 ? a.rem : 64;
    o.row = static_cast<long long>(o.bh) * (KV ? a.kv_stride : a.Lq) + static_cast<long long>(o.f) * a.F + o.j * 64;
    o.list = KV ? a.row_list + static_cast<long long>(item) * a.Rq : a.block_list + static_cast<long long>(item) * a.list_cap;
    return o;
}

// One side's items, every role. Returns when the CTA has no more (or aborts).
template <int D, bool KV>
__device__ __forceinline__ void run_side(const CUtensorMap* tm_x0, const CUtensorMap* tm_y0, const CUtensorMap* tm_xs,
                                         const CUtensorMap* tm_ys, const AttnBwdArgs& a, uint8_t* smem, BwdAux<D>& x)
{
    using L = BwdLayout<D, KV>;
    BwdBars& m = x.bars[KV ? 1 : 0];
    // Values that steer a whole warp are taken through a shuffle: that tells the compiler that they
    // are uniform, so that the MMA and copy issue keeps its operands in uniform registers (without
    // it the key items took 650 us instead of 536 at layer480p).
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const uint32_t tmem = __shfl_sync(0xffffffffu, x.tmem_base, 0);
    volatile int* abort_flag = &x.abort;
    const int n_items = a.BH * (KV ? a.Nkv : a.Rq);
    const int listed = KV ? a.Rq : a.Nkv;      // valid ids are [0, listed)
    const int frames = KV ? a.n_cur : a.NF;    // frames of the streamed side
    const int list_len = KV ? a.Rq : a.list_cap;

    // The k-th published item; false: no more, or aborting.
    int k = 0, item = 0, cnt = 0;
    auto next_item = [&]() -> bool {
        const int s = k & 3;
        if (!mbar_wait(&m.sched_full[s], (k >> 2) & 1, abort_flag, a.err, 0x42)) return false;
        item = __shfl_sync(0xffffffffu, x.sched_item[s], 0);
        cnt = __shfl_sync(0xffffffffu, x.sched_cnt[s], 0);
        __syncwarp();
        if (lane == 0) mbar_arrive(&m.sched_empty[s]);
        ++k;
        return item >= 0;
    };

    if (warp == W_LOADX) {
        // Items are claimed one ahead, and their count and first ids loaded while the one before streams.
        auto claim = [&]() { return lane == 0 ? atomicAdd(a.next_item + (KV ? 1 : 0), 1) : 0; };
        int nitem = __shfl_sync(0xffffffffu, claim(), 0), ncnt = 0, nids = -1;
        auto look = [&]() {
            if (nitem < n_items) {
                ncnt = item_count<KV>(a, nitem);
                nids = lane < list_len ? __ldg(own_of<KV>(a, nitem).list + lane) : -1;
            }
        };
        look();
        int t = 0, ne = 0;  // tiles and items with tiles so far
        int armed_x = 0, armed_own = 0;
        bool ok = true;
        while (ok) {
            const bool more = nitem < n_items;
            item = nitem;
            cnt = ncnt;
            int ids = nids;
            const int s = k & 3;
            if (!mbar_wait(&m.sched_empty[s], ((k >> 2) & 1) ^ 1, abort_flag, a.err, 0x43)) break;
            if (lane == 0) {
                x.sched_item[s] = more ? item : -1;
                x.sched_cnt[s] = cnt;
            }
            __syncwarp();
            mbar_arrive_elect(&m.sched_full[s]);
            ++k;
            if (!more) break;
            const int claimed = claim();
            const Own o = own_of<KV>(a, item);
            const int n_it = (cnt + 1) >> 1;
            if (n_it > 0) {
                if (!KV) {
                    const int b = ne & 1;
                    if (!mbar_wait(&m.info_empty[b], ((ne >> 1) & 1) ^ 1, abort_flag, a.err, 0x44)) break;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int r = lane + 32 * i;
                        x.info[b][0][r] = r < o.n ? neg_lse_log2(__ldg(a.lse + o.row + r)) : -INFINITY;
                        x.info[b][1][r] = r < o.n ? -a.delta[o.row + r] : 0.f;
                    }
                    __syncwarp();
                    mbar_arrive_elect(&m.info_full[b]);
                }
                const int ob = ne % L::OWNS;
                if (!mbar_wait(&m.own_empty[ob], ((ne / L::OWNS) & 1) ^ 1, abort_flag, a.err, 0x45)) break;
                mbar_arrive_expect_tx_elect(&m.own_full[ob], 2 * L::OWN);
                uint8_t* own = smem + L::OFF_X0 + ob * 2 * L::OWN;
                for (int p = 0; p < L::NP; ++p) {
                    tma_load_4d_elect(own + p * L::OWN_PANEL, tm_x0, p * 64, o.j * 64, o.f, o.bh, &m.own_full[ob]);
                    tma_load_4d_elect(own + L::OWN + p * L::OWN_PANEL, tm_y0, p * 64, o.j * 64, o.f, o.bh, &m.own_full[ob]);
                }
                armed_own = ++ne;
            }
            for (int it = 0; it < n_it; ++it, ++t) {
                if (it > 0 && (it & 15) == 0) {
                    const int e = 2 * it + lane;
                    ids = e < cnt ? __ldg(o.list + e) : -1;
                }
                int tau[2], tok[2], rows[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int e = 2 * it + h;
                    const int id = __shfl_sync(0xffffffffu, ids, e & 31);
                    const bool good = e < cnt && id >= 0 && id < listed;
                    if (e < cnt && !good && lane == 0) record_error(a.err, DEVERR_LIST | 2);
                    tau[h] = good ? id / a.bpf : frames;  // past the last frame: the box reads zeros
                    const int j = good ? id - tau[h] * a.bpf : 0;
                    tok[h] = j * 64;
                    rows[h] = good ? (j == a.bpf - 1 ? a.rem : 64) : 0;
                }
                const int xi = t % L::NX;
                if (!(ok = mbar_wait(&m.x_empty[xi], ((t / L::NX) & 1) ^ 1, abort_flag, a.err, 0x46))) break;
                if (!KV && lane == 0) {
                    x.tile_rows[xi][0] = rows[0];
                    x.tile_rows[xi][1] = rows[1];
                }
                __syncwarp();
                mbar_arrive_expect_tx_elect(&m.x_full[xi], L::TILE);
                for (int h = 0; h < 2; ++h)
                    for (int p = 0; p < L::NP; ++p)
                        tma_load_4d_elect(smem + L::OFF_X + xi * L::TILE + p * L::PANEL + h * 8192u, tm_xs, p * 64, tok[h],
                                          tau[h], o.bh, &m.x_full[xi]);
                armed_x = t + 1;
                if (it == 0) {
                    nitem = __shfl_sync(0xffffffffu, claimed, 0);
                    look();
                }
            }
            if (n_it == 0) {
                nitem = __shfl_sync(0xffffffffu, claimed, 0);
                look();
            }
        }
        if (*abort_flag) {  // let every copy already issued land
            for (int n = max(0, armed_own - L::OWNS); n < armed_own; ++n)
                mbar_drain(&m.own_full[n % L::OWNS], (n / L::OWNS) & 1, 10000000ull);
            for (int e = max(0, armed_x - L::NX); e < armed_x; ++e)
                mbar_drain(&m.x_full[e % L::NX], (e / L::NX) & 1, 10000000ull);
        }
    } else if (warp == W_LOADY) {
        int t = 0;
        bool ok = true;
        while (ok && next_item()) {
            const Own o = own_of<KV>(a, item);
            const int n_it = (cnt + 1) >> 1;
            int ids = lane < cnt ? __ldg(o.list + lane) : -1;
            // key side: lse and delta of the lane's four rows of a tile, loaded a tile ahead
            float l4[4], d4[4];
            auto stats = [&](int it) {
                if (!KV || it >= n_it) return;
                const int e = 2 * it + (lane >> 4), r0 = (lane & 15) * 4;
                const int id = __shfl_sync(0xffffffffu, ids, e & 31);
                int rows = 0;
                long long at = 0;
                if (e < cnt && id >= 0 && id < listed) {
                    const int f = id / a.bpf, j = id - f * a.bpf;
                    rows = j == a.bpf - 1 ? a.rem : 64;
                    at = static_cast<long long>(o.bh) * a.Lq + f * a.F + j * 64 + r0;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool there = r0 + i < rows;
                    l4[i] = there ? __ldg(a.lse + at + i) : -INFINITY;
                    d4[i] = there ? a.delta[at + i] : 0.f;
                }
            };
            stats(0);
            for (int it = 0; it < n_it; ++it, ++t) {
                int tau[2], tok[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int e = 2 * it + h;
                    const int id = __shfl_sync(0xffffffffu, ids, e & 31);
                    const bool good = e < cnt && id >= 0 && id < listed;
                    tau[h] = good ? id / a.bpf : frames;
                    tok[h] = good ? (id - tau[h] * a.bpf) * 64 : 0;
                }
                const int yi = t % L::NY;
                if (!(ok = mbar_wait(&m.y_empty[yi], ((t / L::NY) & 1) ^ 1, abort_flag, a.err, 0x47))) break;
                if (KV) {
                    *reinterpret_cast<float4*>(&x.info[yi][0][lane * 4]) =
                        make_float4(neg_lse_log2(l4[0]), neg_lse_log2(l4[1]), neg_lse_log2(l4[2]), neg_lse_log2(l4[3]));
                    *reinterpret_cast<float4*>(&x.info[yi][1][lane * 4]) = make_float4(-d4[0], -d4[1], -d4[2], -d4[3]);
                }
                __syncwarp();
                mbar_arrive_expect_tx_elect(&m.y_full[yi], L::TILE);
                for (int h = 0; h < 2; ++h)
                    for (int p = 0; p < L::NP; ++p)
                        tma_load_4d_elect(smem + L::OFF_Y + yi * L::TILE + p * L::PANEL + h * 8192u, tm_ys, p * 64, tok[h],
                                          tau[h], o.bh, &m.y_full[yi]);
                if ((it & 15) == 15) {
                    const int e = 2 * (it + 1) + lane;
                    ids = e < cnt ? __ldg(o.list + e) : -1;
                }
                stats(it + 1);
            }
        }
        if (*abort_flag)
            for (int e = max(0, t - L::NY); e < t; ++e) mbar_drain(&m.y_full[e % L::NY], (e / L::NY) & 1, 10000000ull);
    } else if (warp == W_SCORE) {
        constexpr uint32_t IDESC = idesc_bf16_f32(128, 64, false, false);
        const uint64_t dOwn = sdesc_sw128(smem_u32(smem + L::OFF_X0), 16, 1024);
        const uint64_t dX = sdesc_sw128(smem_u32(smem + L::OFF_X), 16, 1024);
        const uint64_t dY = sdesc_sw128(smem_u32(smem + L::OFF_Y), 16, 1024);
        int t = 0, ne = 0;
        bool ok = true;
        while (ok && next_item()) {
            const int n_it = (cnt + 1) >> 1;
            if (n_it == 0) continue;
            const int ob = ne % L::OWNS;
            if (!mbar_wait(&m.own_full[ob], (ne / L::OWNS) & 1, abort_flag, a.err, 0x50)) break;
            const uint64_t dX0 = dOwn + ((ob * 2 * L::OWN) >> 4), dY0 = dX0 + (L::OWN >> 4);
            for (int it = 0; it < n_it; ++it, ++t) {
                const int xi = t % L::NX, yi = t % L::NY, b = t & 1, u = t >> 1;
                const uint32_t d = tmem + 64u * static_cast<uint32_t>(b);
                if (!(ok = mbar_wait(&m.s_free[b], (u & 1) ^ 1, abort_flag, a.err, 0x51))) break;
                // dP' first: Ys is released first, and so arrives first
                if (!(ok = mbar_wait(&m.y_full[yi], (t / L::NY) & 1, abort_flag, a.err, 0x52))) break;
                tc_fence_after();  // the softmax's TMEM reads of this buffer come first
                const uint64_t yb = dY + ((yi * L::TILE) >> 4);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    umma_bf16_elect(d + TM_DP, yb + (((kk >> 2) * L::PANEL + (kk & 3) * 32) >> 4),
                                    dY0 + (((kk >> 2) * L::OWN_PANEL + (kk & 3) * 32) >> 4), IDESC, kk > 0 ? 1u : 0u);
                if (!KV) umma_commit_elect(&m.y_empty[yi]);
                if (!(ok = mbar_wait(&m.x_full[xi], (t / L::NX) & 1, abort_flag, a.err, 0x53))) break;
                const uint64_t xb = dX + ((xi * L::TILE) >> 4);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    umma_bf16_elect(d, xb + (((kk >> 2) * L::PANEL + (kk & 3) * 32) >> 4),
                                    dX0 + (((kk >> 2) * L::OWN_PANEL + (kk & 3) * 32) >> 4), IDESC, kk > 0 ? 1u : 0u);
                umma_commit_elect(&m.s_full[b]);
            }
            if (ok) umma_commit_elect(&m.own_empty[ob]);
            ++ne;
        }
        if (*abort_flag) {
            umma_commit_elect(&m.drain_s);
            mbar_drain(&m.drain_s, 0, 10000000ull);
        }
    } else if (warp == W_ACC) {
        constexpr uint32_t IDESC = idesc_bf16_f32(D, 64, true, true);
        const uint64_t dX = sdesc_sw128(smem_u32(smem + L::OFF_X), L::PANEL, 1024);
        const uint64_t dY = sdesc_sw128(smem_u32(smem + L::OFF_Y), L::PANEL, 1024);
        const uint64_t dDS = sdesc_sw128(smem_u32(smem + L::OFF_DS), 1024, 1024);
        const uint64_t dP = sdesc_sw128(smem_u32(smem + L::OFF_P), 1024, 1024);
        int t = 0, ne = 0;
        bool ok = true;
        while (ok && next_item()) {
            const int n_it = (cnt + 1) >> 1;
            if (n_it == 0) continue;
            const int e = ne & 1;
            if (!mbar_wait(&m.acc_empty[e], ((ne >> 1) & 1) ^ 1, abort_flag, a.err, 0x54)) break;
            tc_fence_after();  // the epilogue's reads of these accumulators come first
            const uint32_t acc = tmem + TM_ACC + 128u * static_cast<uint32_t>(e);
            for (int it = 0; it < n_it; ++it, ++t) {
                const int xi = t % L::NX, yi = t % L::NY, b = t & 1;
                if (!(ok = mbar_wait(&m.x_full[xi], (t / L::NX) & 1, abort_flag, a.err, 0x55))) break;
                if (KV && !(ok = mbar_wait(&m.y_full[yi], (t / L::NY) & 1, abort_flag, a.err, 0x56))) break;
                if (!(ok = mbar_wait(&m.p_full[b], (t >> 1) & 1, abort_flag, a.err, 0x57))) break;
                tc_fence_after();
                const uint64_t xb = dX + ((xi * L::TILE) >> 4), yb = dY + ((yi * L::TILE) >> 4);
                const uint64_t sb = dDS + (((b % L::PBUFS) * L::PBUF) >> 4), pb = dP + (((b % L::PBUFS) * L::PBUF) >> 4);
                const uint32_t more = it > 0 ? 1u : 0u;
                const bool both = 2 * it + 1 < cnt;  // the tile's second block (the last four slices of 16 rows) may be missing
                if (KV) {  // dv first: Ys can be filled again while dk is summed
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_bf16_elect(acc + 64u, yb + ((kk * 2048) >> 4), pb + ((kk * 2048) >> 4), IDESC, kk > 0 ? 1u : more);
                    if (both)
#pragma unroll
                        for (int kk = 4; kk < 8; ++kk)
                            umma_bf16_elect(acc + 64u, yb + ((kk * 2048) >> 4), pb + ((kk * 2048) >> 4), IDESC, 1u);
                    umma_commit_elect(&m.y_empty[yi]);
                }
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    umma_bf16_elect(acc, xb + ((kk * 2048) >> 4), sb + ((kk * 2048) >> 4), IDESC, kk > 0 ? 1u : more);
                if (both)
#pragma unroll
                    for (int kk = 4; kk < 8; ++kk)
                        umma_bf16_elect(acc, xb + ((kk * 2048) >> 4), sb + ((kk * 2048) >> 4), IDESC, 1u);
                umma_commit_elect(&m.x_empty[xi]);
                umma_commit_elect(&m.p_empty[t % L::PBUFS]);
            }
            if (ok) umma_commit_elect(&m.acc_full[e]);
            ++ne;
        }
        if (*abort_flag) {
            umma_commit_elect(&m.drain_a);
            mbar_drain(&m.drain_a, 0, 10000000ull);
        }
    } else if (warp < W_EPI0) {
        // ---------------------------------------------------------------- softmax
        const int g = (warp - W_SOFT0) >> 2;       // this warpgroup takes columns [32 g, 32 g + 32) of every tile
        const int sp = warp & 3;                   // TMEM sub-partition
        const int rr = sp * 32 + lane;             // streamed row of the tile
        const uint32_t s_addr = tmem + (static_cast<uint32_t>(sp * 32) << 16) + 32u * g;
        uint8_t* ds_row = smem + L::OFF_DS + rr * 128;
        uint8_t* p_row = smem + L::OFF_P + rr * 128;
        int t = 0, ne = 0;
        bool ok = true;
        while (ok && next_item()) {
            const int n_it = (cnt + 1) >> 1;
            if (n_it == 0) continue;
            const int e = ne & 1;
            const int t_end = t + n_it;
            if (!KV && !(ok = mbar_wait(&m.info_full[e], (ne >> 1) & 1, abort_flag, a.err, 0x60))) break;
            for (; t < t_end; ++t) {
                const int xi = t % L::NX, yi = t % L::NY, b = t & 1, u = t >> 1;
                float nl = 0.f, nd = 0.f;
                bool valid = true;
                if (KV) {
                    if (!(ok = mbar_wait(&m.y_full[yi], (t / L::NY) & 1, abort_flag, a.err, 0x61))) break;
                    nl = x.info[yi][0][rr];
                    nd = x.info[yi][1][rr];
                } else {
                    if (!(ok = mbar_wait(&m.x_full[xi], (t / L::NX) & 1, abort_flag, a.err, 0x62))) break;
                    valid = (rr & 63) < x.tile_rows[xi][rr >> 6];
                }
                if (!(ok = mbar_wait(&m.s_full[b], u & 1, abort_flag, a.err, 0x63))) break;
                __syncwarp();
                tc_fence_after();
                float sv[32], dp[32];
                tmem_ld32(s_addr + 64u * b, sv);
                tmem_ld32(s_addr + TM_DP + 64u * b, dp);
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&m.s_free[b]);
                uint32_t pk[KV ? 16 : 1], dk[16];
#pragma unroll
                for (int c = 0; c < 32; c += 4) {
                    float4 l4, d4;
                    if (KV) {
                        l4 = make_float4(nl, nl, nl, nl);
                        d4 = make_float4(nd, nd, nd, nd);
                    } else {
                        l4 = *reinterpret_cast<const float4*>(&x.info[e][0][32 * g + c]);
                        d4 = *reinterpret_cast<const float4*>(&x.info[e][1][32 * g + c]);
                    }
                    const float2 sc = make_float2(a.scale_log2, a.scale_log2);
                    float2 e0 = __ffma2_rn(make_float2(sv[c], sv[c + 1]), sc, make_float2(l4.x, l4.y));
                    float2 e1 = __ffma2_rn(make_float2(sv[c + 2], sv[c + 3]), sc, make_float2(l4.z, l4.w));
                    e0 = make_float2(fast_exp2(e0.x), fast_exp2(e0.y));
                    e1 = make_float2(fast_exp2(e1.x), fast_exp2(e1.y));
                    if constexpr (KV) {
                        pk[c / 2] = pack_bf16x2(e0.x, e0.y);
                        pk[c / 2 + 1] = pack_bf16x2(e1.x, e1.y);
                    }
                    e0 = __fmul2_rn(e0, __fadd2_rn(make_float2(dp[c], dp[c + 1]), make_float2(d4.x, d4.y)));
                    e1 = __fmul2_rn(e1, __fadd2_rn(make_float2(dp[c + 2], dp[c + 3]), make_float2(d4.z, d4.w)));
                    // a streamed key that is not there contributes nothing, whatever its P came out as
                    // (a streamed query that is not there has P = 0)
                    dk[c / 2] = KV || valid ? pack_bf16x2(e0.x, e0.y) : 0u;
                    dk[c / 2 + 1] = KV || valid ? pack_bf16x2(e1.x, e1.y) : 0u;
                }
                if (!(ok = mbar_wait(&m.p_empty[t % L::PBUFS], ((t / L::PBUFS) & 1) ^ 1, abort_flag, a.err, 0x64))) break;
#pragma unroll
                for (int c8 = 0; c8 < 4; ++c8) {
                    const uint32_t at = (t % L::PBUFS) * L::PBUF + static_cast<uint32_t>(((4 * g + c8) ^ (rr & 7)) * 16);
                    *reinterpret_cast<uint4*>(ds_row + at) = make_uint4(dk[4 * c8], dk[4 * c8 + 1], dk[4 * c8 + 2], dk[4 * c8 + 3]);
                    if constexpr (KV)
                        *reinterpret_cast<uint4*>(p_row + at) = make_uint4(pk[4 * c8], pk[4 * c8 + 1], pk[4 * c8 + 2], pk[4 * c8 + 3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&m.p_full[b]);
            }
            t = t_end;
            if (!KV && ok) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&m.info_empty[e]);
            }
            ++ne;
        }
    } else {
        // ---------------------------------------------------------------- epilogue
        // acc^T [head_dim lanes][64 columns] -> bf16 rows. Neighbouring lanes (head_dim elements)
        // swap one of each two columns, so that a lane stores two elements of one row.
        const int sp = warp & 3;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(sp * 32) << 16);
        const int d = D == 128 ? sp * 32 + lane : sp * 16 + (lane & 15);  // M = 64: 16 rows in each sub-partition's first lanes
        const bool has = D == 128 || lane < 16;
        const bool odd = lane & 1;
        int ne = 0;
        while (next_item()) {
            const Own o = own_of<KV>(a, item);
            if (cnt == 0) {
                constexpr int CH = D / 8;
                for (int i = (warp - W_EPI0) * 32 + lane; i < o.n * CH; i += 128) {
                    const long long at = o.row * D + i * 8;
                    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
                    *reinterpret_cast<uint4*>((KV ? a.dk : a.dq) + at) = z;
                    if (KV) *reinterpret_cast<uint4*>(a.dv + at) = z;
                }
                continue;
            }
            const int e = ne & 1;
            if (!mbar_wait(&m.acc_full[e], (ne >> 1) & 1, abort_flag, a.err, 0x65)) break;
            ++ne;
            __syncwarp();
            tc_fence_after();
#pragma unroll
            for (int q = 0; q < (KV ? 4 : 2); ++q) {  // acc0 columns 0-31, 32-63, then acc1's
                float v[32];
                __syncwarp();
                tmem_ld32(lane_base + TM_ACC + 128u * e + 32u * q, v);
                tmem_ld_wait();
                if (q == (KV ? 3 : 1)) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&m.acc_empty[e]);
                }
                const float f = q < 2 ? a.scale : 1.f;
                uint16_t* dst = (KV ? (q < 2 ? a.dk : a.dv) : a.dq) + o.row * D + (d & ~1);
#pragma unroll
                for (int c = 0; c < 32; c += 2) {
                    const float keep = odd ? v[c + 1] : v[c], give = odd ? v[c] : v[c + 1];
                    const float got = __shfl_xor_sync(0xffffffffu, give, 1);
                    const int row = 32 * (q & 1) + c + (odd ? 1 : 0);
                    const uint32_t w = odd ? pack_bf16x2(got * f, keep * f) : pack_bf16x2(keep * f, got * f);
                    if (has && row < o.n) *reinterpret_cast<uint32_t*>(dst + static_cast<long long>(row) * D) = w;
                }
            }
        }
    }
}

template <int D>
__global__ void __launch_bounds__(BWD_THREADS, 1)
attn_bwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_dout,
                const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                const __grid_constant__ AttnBwdArgs a)
{
    extern __shared__ __align__(1024) uint8_t smem[];  // 128-byte swizzled tiles want 1024-byte boundaries
    constexpr uint32_t Q = BwdLayout<D, false>::END, K = BwdLayout<D, true>::END;
    BwdAux<D>& x = *reinterpret_cast<BwdAux<D>*>(smem + (Q > K ? Q : K));
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int side = 0; side < 2; ++side) {
            BwdBars& m = x.bars[side];
            for (int s = 0; s < 4; ++s) {
                mbar_init(&m.x_full[s], 1);
                mbar_init(&m.x_empty[s], 1);
                mbar_init(&m.y_full[s], 1);  // key side: the copies, and the rows' statistics
                mbar_init(&m.y_empty[s], 1);
                mbar_init(&m.sched_full[s], 1);
                mbar_init(&m.sched_empty[s], SCHED_READERS);
            }
            for (int b = 0; b < 2; ++b) {
                mbar_init(&m.own_full[b], 1);
                mbar_init(&m.own_empty[b], 1);
                mbar_init(&m.s_full[b], 1);
                mbar_init(&m.s_free[b], 8);      // the softmax warps
                mbar_init(&m.p_full[b], 8);
                mbar_init(&m.p_empty[b], 1);
                mbar_init(&m.acc_full[b], 1);
                mbar_init(&m.acc_empty[b], 4);   // the epilogue's warps
                mbar_init(&m.info_full[b], 1);
                mbar_init(&m.info_empty[b], 8);
            }
            mbar_init(&m.drain_s, 1);
            mbar_init(&m.drain_a, 1);
        }
        x.abort = (smem_u32(smem) & 1023u) != 0;
        if (x.abort) record_error(a.err, DEVERR_TIMEOUT | 0x7f);
        fence_mbar_init();
    }
    if (warp == W_SCORE) {
        tmem_alloc(&x.tmem_base, TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    asm volatile("griddepcontrol.wait;" ::: "memory");  // everything above overlaps the preparing kernel
    if (!x.abort) run_side<D, false>(&tm_q, &tm_dout, &tm_k, &tm_v, a, smem, x);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (!x.abort) run_side<D, true>(&tm_k, &tm_v, &tm_q, &tm_dout, a, smem, x);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == W_SCORE) {
        tc_fence_after();
        tmem_dealloc(x.tmem_base, TMEM_COLS);
    }
}

// The gradient's preparation, one launch: the first CTAs transpose the block lists, the others
// form delta.
//
// Transposition: for each KV block the query blocks that list it, ascending. A CTA owns 128 KV
// blocks of a head and walks the head's rows 256 at a time: each row's warp sets its bit for
// every block it lists, then each block's thread appends the bits it finds. (Bits are set
// atomically, but the set does not depend on the order.) 128 blocks a CTA spread the scattered
// stores of the lists over the machine; every CTA reads all lists of its head, from L2.
//
// Delta: <dout, out + out_lo> per row, a warp takes four rows at once.
constexpr int PREP_THREADS = 512;
constexpr int TR_BLOCKS = 128, TR_WORDS = 8;
constexpr int DELTA_ROWS = 4 * (PREP_THREADS / 32);

template <int D>
__global__ void __launch_bounds__(PREP_THREADS) attn_bwd_prep_kernel(const AttnBwdArgs a, int transposing)
{
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // only now: the gradient's CTAs take all of an SM's tensor memory, which the forward has left
    if (t == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (static_cast<int>(blockIdx.x) < transposing) {
        __shared__ uint32_t bits[TR_WORDS][TR_BLOCKS];
        if (blockIdx.x == 0 && t < 2) a.next_item[t] = 0;
        const int chunks = (a.Nkv + TR_BLOCKS - 1) / TR_BLOCKS;
        const int bh = blockIdx.x / chunks, g0 = (blockIdx.x - bh * chunks) * TR_BLOCKS;
        const int g1 = min(TR_BLOCKS, a.Nkv - g0);
        int n = 0;
        int* mine = a.row_list + (static_cast<long long>(bh) * a.Nkv + g0 + t) * a.Rq;
        for (int r0 = 0; r0 < a.Rq; r0 += 32 * TR_WORDS) {
            for (int i = t; i < TR_WORDS * TR_BLOCKS; i += PREP_THREADS) bits[i / TR_BLOCKS][i % TR_BLOCKS] = 0u;
            __syncthreads();
            for (int r = r0 + warp; r < min(a.Rq, r0 + 32 * TR_WORDS); r += PREP_THREADS / 32) {
                const long long lrow = static_cast<long long>(bh) * a.Rq + r;
                const int cnt = min(max(__ldg(a.block_count + lrow), 0), a.list_cap);
                const int* lst = a.block_list + lrow * a.list_cap;
                const uint32_t bit = 1u << (r & 31);
                uint32_t* word = bits[(r - r0) >> 5];
                for (int e = lane; e < cnt; e += 32) {
                    const int at = __ldg(lst + e) - g0;
                    if (at >= 0 && at < g1 && (atomicOr(word + at, bit) & bit))
                        record_error(a.err, DEVERR_LIST | 3);  // a block named twice
                }
            }
            __syncthreads();
            if (t < TR_BLOCKS)
                for (int w = 0; w < TR_WORDS; ++w)
                    for (uint32_t m = bits[w][t]; m; m &= m - 1) mine[n++] = r0 + 32 * w + __ffs(m) - 1;
            __syncthreads();
        }
        if (t < g1) a.row_count[static_cast<long long>(bh) * a.Nkv + g0 + t] = n;
        return;
    }
    constexpr int EPL = D / 32, W = EPL / 2;  // elements and words of a row a lane holds
    const long long rows = static_cast<long long>(a.BH) * a.Lq;
    const long long r0 = static_cast<long long>(blockIdx.x - transposing) * DELTA_ROWS + warp * 4;
    uint32_t o[4][W], d[4][W], lo[4][W];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const long long at = (r0 + i) * D + lane * EPL;
#pragma unroll
        for (int w = 0; w < W; ++w) o[i][w] = d[i][w] = lo[i][w] = 0u;
        if (r0 + i < rows) {
            if constexpr (W == 2) {
                *reinterpret_cast<uint2*>(o[i]) = __ldg(reinterpret_cast<const uint2*>(a.out + at));
                *reinterpret_cast<uint2*>(d[i]) = __ldg(reinterpret_cast<const uint2*>(a.dout + at));
                if (a.out_lo) *reinterpret_cast<uint2*>(lo[i]) = __ldg(reinterpret_cast<const uint2*>(a.out_lo + at));
            } else {
                o[i][0] = __ldg(reinterpret_cast<const uint32_t*>(a.out + at));
                d[i][0] = __ldg(reinterpret_cast<const uint32_t*>(a.dout + at));
                if (a.out_lo) lo[i][0] = __ldg(reinterpret_cast<const uint32_t*>(a.out_lo + at));
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float dot = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            dot = fmaf(__uint_as_float(o[i][w] << 16) + __uint_as_float(lo[i][w] << 16), __uint_as_float(d[i][w] << 16), dot);
            dot = fmaf(__uint_as_float(o[i][w] & 0xFFFF0000u) + __uint_as_float(lo[i][w] & 0xFFFF0000u),
                       __uint_as_float(d[i][w] & 0xFFFF0000u), dot);
        }
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, s);
        if (lane == 0 && r0 + i < rows) a.delta[r0 + i] = dot;
    }
}

template <int D>
cudaError_t launch_d(const AttnBwdMaps& m, const AttnBwdArgs& a, cudaStream_t s)
{
    constexpr uint32_t smem = bwd_smem_bytes<D>();
    static_assert(smem <= 232448, "shared memory plan exceeds 227 KB");
    static std::atomic<int> sms[64];  // SMs of a device once the kernel's shared memory is set there
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int sm = dev >= 0 && dev < 64 ? sms[dev].load(std::memory_order_acquire) : 0;
    if (sm == 0) {
        e = cudaFuncSetAttribute(attn_bwd_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
        if ((e = cudaDeviceGetAttribute(&sm, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) sms[dev].store(sm, std::memory_order_release);
    }
    const int transposing = (a.Nkv + TR_BLOCKS - 1) / TR_BLOCKS * a.BH;
    const long long rows = static_cast<long long>(a.BH) * a.Lq;
    const unsigned prep = static_cast<unsigned>(transposing + (rows + DELTA_ROWS - 1) / DELTA_ROWS);
    e = launch_dependent(attn_bwd_prep_kernel<D>, dim3(prep), PREP_THREADS, 0, s, a, transposing);
    if (e != cudaSuccess) return e;
    const long long items = static_cast<long long>(a.BH) * (a.Rq + a.Nkv);
    return launch_dependent(attn_bwd_kernel<D>, dim3(static_cast<unsigned>(items < sm ? items : sm)), BWD_THREADS, smem, s,
                            m.q, m.dout, m.k, m.v, a);
}

}  // namespace

cudaError_t launch_attn_bwd(const AttnBwdMaps& m, const AttnBwdArgs& a, int D, cudaStream_t s)
{
    return D == 128 ? launch_d<128>(m, a, s) : launch_d<64>(m, a, s);
}

}  // namespace lf
