// lf_norm.cu -- the step between two blocks of a transformer, fused: the norm after a
// block, its gate, the residual sum, the norm before the next block and its modulation,
//   u = post(y) w2 + b2          post, pre: none, RMS or layer norm over the row
//   r = alpha x + gate u         the residual stream
//   n = pre(r),  h = (n w1 + b1) (1 + scale) + shift
// with gate, scale and shift shared by groups of consecutive rows (a frame's tokens, a
// sample), and the gradients of all of it.
//
// Gradient (m = post(y), rs = 1 / deviation, mean over the row):
//   dn  = dh (1 + scale) w1
//   dr' = dr + rs1 (dn - [layer] mean(dn) - n mean(dn n))
//   dx  = alpha dr',   du = dr' gate,   dm = du w2
//   dy  = rs2 (dm - [layer] mean(dm) - m mean(dm m))
// and sums over the rows of a group: A1 = sum dh, A2 = sum dh n, A3 = sum dr', A4 = sum dr' m:
//   dshift = A1, dscale = w1 A2 + b1 A1, dgate = w2 A4 + b2 A3,
//   dw1 = sum_g (1 + scale_g) A2, db1 = sum_g (1 + scale_g) A1, dw2 = sum_g gate_g A4, db2 = sum_g gate_g A3.
// x and y are read again and r is formed anew in fp32, so that no gradient sees the
// rounding of a stored r; that costs the bytes a stored r would.
//
// Memory-bound. A team of threads holds a row in registers, NV groups of 8 elements a
// thread, so x, y (and dr, dh) are read once and the outputs written once; row sums go
// through warp shuffles and one shared-memory exchange. Deviations are taken about the
// mean, never as a difference of squares. Sums and statistics are fp32; the only
// roundings to fewer bits are the stores of r, h, dx and dy.
//
// CTAs are persistent and take consecutive rows, so the vectors of a group stay in
// registers or shared memory, folded to what a row needs (gate w2, gate b2, (1 + scale) w1,
// b1 (1 + scale) + shift), and rows are copied ahead into a ring in shared memory: a row has several
// dependent sums, and only loads that are rows ahead keep the memory busy meanwhile. Each thread
// copies what it will read itself, so the ring needs no barrier. Rows that do not start on 16-byte
// boundaries (dim not a multiple of 8), and rows too long for a ring, are loaded directly.
//
// The gradient kernel keeps its column sums in registers: a CTA writes one partial row per
// group it meets (slot = CTA + group, so no two coincide) and one of its weights' sums, and a
// second kernel adds them up in a fixed order -- no atomics, the same bits every time.
#include "lf_norm_rows.cuh"

namespace lf {
namespace {

// Two kernels, and rows too long for the first. The group kernel: one CTA of 512 threads an SM, the
// folded vectors of a group in shared memory for all its teams. A row's sums cost a warp the same
// whatever it holds of the row, so a thread holds up to 32 elements and a team is 64 threads at most.
// (fp32 rows of 2048, whose ring does not fit, are loaded directly: 113 us for 16384 rows; fewer teams
// with a ring 126.) At 32760 rows of 1536 bf16 it takes 80 us (402 MB, 5.0 TB/s); what is left is
// the row's dependent sums and the issue of its arithmetic by 16 warps, more than the memory.
// Vectors in registers took 94, read per row from L1 151-250; 768 threads of 80 registers 99 (they
// spill), every shared read before the sum that it follows 93 (likewise).
// The register kernel: every team goes its own way, the folded vectors in its registers, for groups
// too short to stop the CTA at (1024 elements a row, groups of 1 and 16 rows: 171 and 69 against 703
// and 94 us; 1536, groups of 64: 92 against 87, of 256: 87 against 77), and for few rows, where latency
// counts and more threads of one group of eight each share a row (one row of 1536: 4.2 us; with 24
// elements a thread 6.7).
// WIDE: a CTA of up to 512 threads for one row (4096: 105 us for 8192 rows, 2.6 TB/s; above 8192 its
// four groups a thread spill, 656 / 388 bytes and more: 118 us for 2048 rows of 16384).
constexpr int GRP_THREADS = 512, GRP_REGS = 128;
constexpr int FWD_THREADS = 128;
template <int NV, bool WIDE> constexpr int FWD_REGS = !WIDE && NV == 1 ? 80 : 128;
constexpr int FWD_CTAS[5] = {1, 6, 4, 1, 1};  // an SM's
constexpr long long FEW_ROWS = 592;           // four an SM
constexpr long long SHORT_GROUP = 64;

template <typename TX, typename TY, int NV, bool WIDE, bool FULL>
__global__ void __maxnreg__((FWD_REGS<NV, WIDE>)) norm_fwd_kernel(const NormArgs a, int team_threads, int stages)
{
    __shared__ __align__(16) float red[MAX_TEAMS][2][2][16];
    extern __shared__ __align__(16) uint8_t smem[];
    Team team = make_team(red, team_threads);
    const int teams = blockDim.x / team_threads;
    const int ti = threadIdx.x / team_threads, tt = threadIdx.x - ti * team_threads;
    const long long r0 = blockIdx.x * a.rows_per_cta, first = r0 + ti;
    const long long r1 = min(a.rows, r0 + a.rows_per_cta);
    const Place p{tt * 8, team_threads * 8, a.dim, team_threads, stages, static_cast<long long>(teams) * a.dim, a.dim % 8 == 0};
    __syncthreads();  // the sums' buffers are cleared
    if (first >= r1) return;
    const int rows = static_cast<int>((r1 - first + teams - 1) / teams);  // the team's
    Ring ring;
    ring.stage_bytes = 0;
    Source<TX, NV, FULL> x;
    Source<TY, NV, FULL> y;
    Sink<TX, NV, FULL> r;
    Sink<TY, NV, FULL> h;
    x.init(a.x, first, p, &ring.stage_bytes, tt);
    y.init(a.y, first, p, &ring.stage_bytes, tt);
    r.init(a.r, first, p);
    h.init(a.h, first, p);
    ring.stages = stages;
    ring.base = smem + static_cast<size_t>(ti) * stages * ring.stage_bytes;
    ring.start(rows, p, x, y);
    const float inv = 1.0f / static_cast<float>(a.dim);

    int same = 0;                         // rows left that share the vectors in registers
    Vec8 g2[NV], b2[NV], s1[NV], t1[NV];  // r = alpha x + m g2 + b2, h = n s1 + t1
    auto vectors = [&](int i) {
        const long long row = first + static_cast<long long>(i) * teams;
        const long long group = row / a.per_group, g = group * a.dim;
        same = static_cast<int>(min(((group + 1) * a.per_group - row + teams - 1) / teams, 1ll << 30));
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int col = p.col0 + k * p.stride;
            Vec8 v = load_param(a.v.gate ? a.v.gate + g : nullptr, col, a.dim, p.al, 1.f);
            g2[k] = mul(load_param(a.v.post_w, col, a.dim, p.al, 1.f), v);
            b2[k] = mul(load_param(a.v.post_b, col, a.dim, p.al, 0.f), v);
            v = add(load_param(a.v.scale ? a.v.scale + g : nullptr, col, a.dim, p.al, 0.f), 1.f);
            s1[k] = mul(load_param(a.v.pre_w, col, a.dim, p.al, 1.f), v);
            t1[k] = fma(load_param(a.v.pre_b, col, a.dim, p.al, 0.f), v,
                        load_param(a.v.shift ? a.v.shift + g : nullptr, col, a.dim, p.al, 0.f));
        }
    };
    vectors(0);  // while the first rows are on their way
    for (int i = 0; i < rows; ++i) {
        const uint8_t* st = ring.next(p, x, y);
        if (same == 0) vectors(i);
        --same;
        Vec8 t[NV];
        if (y.on) {
#pragma unroll
            for (int k = 0; k < NV; ++k) t[k] = y.get(st, k, p);
            if (a.post != NORM_NONE) normalise<NV, FULL>(team, t, a.post, inv, p, a.eps);
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const Vec8 v = x.get(st, k, p);
            t[k] = y.on ? fma(g2[k], t[k], fma(v, a.alpha, b2[k])) : mul(v, a.alpha);
            r.put(k, t[k], p);
        }
        x.done(p);
        y.done(p);
        r.done(p);
        ring.done();
        if (!h.on) continue;
        normalise<NV, FULL>(team, t, a.pre, inv, p, a.eps);
#pragma unroll
        for (int k = 0; k < NV; ++k) h.put(k, fma(t[k], s1[k], t1[k]), p);
        h.done(p);
    }
}

template <typename TX, typename TY, int NV, bool FULL>
__global__ void __maxnreg__(GRP_REGS) norm_fwd_group_kernel(const NormArgs a, int team_threads, int stages)
{
    __shared__ __align__(16) float red[MAX_TEAMS][2][2][16];
    extern __shared__ __align__(16) uint8_t smem[];  // the rings, then [4][dim8] vectors
    Team team = make_team(red, team_threads);
    const int teams = blockDim.x / team_threads;
    const int ti = threadIdx.x / team_threads, tt = threadIdx.x - ti * team_threads;
    const int dim = a.dim, dim8 = (dim + 7) & ~7;
    const long long r0 = blockIdx.x * a.rows_per_cta, first = r0 + ti;
    const long long r1 = min(a.rows, r0 + a.rows_per_cta);
    const Place p{tt * 8, team_threads * 8, dim, team_threads, stages, static_cast<long long>(teams) * dim, dim % 8 == 0};
    Ring ring;
    ring.stage_bytes = 0;
    Source<TX, NV, FULL> x;
    Source<TY, NV, FULL> y;
    Sink<TX, NV, FULL> r;
    Sink<TY, NV, FULL> h;
    x.init(a.x, first, p, &ring.stage_bytes, tt);
    y.init(a.y, first, p, &ring.stage_bytes, tt);
    r.init(a.r, first, p);
    h.init(a.h, first, p);
    ring.stages = stages;
    ring.base = smem + static_cast<size_t>(ti) * stages * ring.stage_bytes;
    ring.start(first < r1 ? static_cast<int>((r1 - first + teams - 1) / teams) : 0, p, x, y);
    float* vecs = reinterpret_cast<float*>(smem + static_cast<size_t>(teams) * stages * ring.stage_bytes);  // g2, b2, s1, t1
    const float inv = 1.0f / static_cast<float>(dim);
    auto vec = [&](int which, int k) {
        const int col = p.col0 + k * p.stride;
        return FULL || col < dim8 ? split_load(vecs + which * dim8, col, dim8) : fill8(0.f);
    };

    long long row = first;
    for (long long seg = r0; seg < r1;) {
        const long long gi = seg / a.per_group;
        const long long seg_end = min(r1, (gi + 1) * a.per_group);
        const long long g = gi * dim;
        __syncthreads();
        for (int col = threadIdx.x * 8; col < dim8; col += blockDim.x * 8) {
            Vec8 v = load_param(a.v.gate ? a.v.gate + g : nullptr, col, dim, p.al, 1.f);
            split_store(vecs, col, dim8, mul(load_param(a.v.post_w, col, dim, p.al, 1.f), v));
            split_store(vecs + dim8, col, dim8, mul(load_param(a.v.post_b, col, dim, p.al, 0.f), v));
            v = add(load_param(a.v.scale ? a.v.scale + g : nullptr, col, dim, p.al, 0.f), 1.f);
            split_store(vecs + 2 * dim8, col, dim8, mul(load_param(a.v.pre_w, col, dim, p.al, 1.f), v));
            split_store(vecs + 3 * dim8, col, dim8, fma(load_param(a.v.pre_b, col, dim, p.al, 0.f), v,
                                                        load_param(a.v.shift ? a.v.shift + g : nullptr, col, dim, p.al, 0.f)));
        }
        __syncthreads();
        for (; row < seg_end; row += teams) {
            const uint8_t* st = ring.next(p, x, y);
            Vec8 t[NV];
            if (y.on) {
#pragma unroll
                for (int k = 0; k < NV; ++k) t[k] = y.get(st, k, p);
                if (a.post != NORM_NONE) normalise<NV, FULL>(team, t, a.post, inv, p, a.eps);
            }
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const Vec8 v = x.get(st, k, p);
                t[k] = y.on ? fma(vec(0, k), t[k], fma(v, a.alpha, vec(1, k))) : mul(v, a.alpha);
                r.put(k, t[k], p);
            }
            x.done(p);
            y.done(p);
            r.done(p);
            ring.done();
            if (!h.on) continue;
            normalise<NV, FULL>(team, t, a.pre, inv, p, a.eps);
#pragma unroll
            for (int k = 0; k < NV; ++k) h.put(k, fma(t[k], vec(2, k), vec(3, k)), p);
            h.done(p);
        }
        seg = seg_end;
    }
}

template <typename TX, typename TY, int NV, bool FULL>
cudaError_t launch_group_full(NormArgs a, const NormPlan& p, cudaStream_t s)
{
    cudaError_t e = allow_smem<norm_fwd_group_kernel<TX, TY, NV, FULL>>(p.smem);
    if (e != cudaSuccess) return e;
    a.rows_per_cta = (a.rows + 147) / 148;
    const unsigned grid = static_cast<unsigned>((a.rows + a.rows_per_cta - 1) / a.rows_per_cta);
    norm_fwd_group_kernel<TX, TY, NV, FULL><<<grid, p.threads * p.teams, p.smem, s>>>(a, p.threads, p.stages);
    return cudaGetLastError();
}

template <typename TX, typename TY, int NV>
cudaError_t launch_group(const NormArgs& a, cudaStream_t s)
{
    const NormPlan p = plan_of(a.dim, NV, sizeof(TX) + (a.y ? sizeof(TY) : 0), GRP_THREADS, 1, 4, 0);
    return p.full ? launch_group_full<TX, TY, NV, true>(a, p, s) : launch_group_full<TX, TY, NV, false>(a, p, s);
}

template <typename TX, typename TY, int NV, bool WIDE, bool FULL>
cudaError_t launch_full(NormArgs a, const NormPlan& p, cudaStream_t s)
{
    cudaError_t e = allow_smem<norm_fwd_kernel<TX, TY, NV, WIDE, FULL>>(p.smem);
    if (e != cudaSuccess) return e;
    // all SMs' resident CTAs, the rows spread evenly over them
    const long long most = 148ll * (p.wide ? 1 : FWD_CTAS[NV]);
    const long long per = std::max<long long>(1, (a.rows + most - 1) / most);
    a.rows_per_cta = per < p.teams ? per : (per + p.teams - 1) / p.teams * p.teams;
    const unsigned grid = static_cast<unsigned>((a.rows + a.rows_per_cta - 1) / a.rows_per_cta);
    norm_fwd_kernel<TX, TY, NV, WIDE, FULL><<<grid, p.threads * p.teams, p.smem, s>>>(a, p.threads, p.stages);
    return cudaGetLastError();
}

template <typename TX, typename TY, int NV, bool WIDE>
cudaError_t launch_nv(const NormArgs& a, cudaStream_t s)
{
    const NormPlan p = plan_of(a.dim, NV, sizeof(TX) + (a.y ? sizeof(TY) : 0), FWD_THREADS, FWD_CTAS[NV], 0, 0);
    return p.full ? launch_full<TX, TY, NV, WIDE, true>(a, p, s) : launch_full<TX, TY, NV, WIDE, false>(a, p, s);
}

template <typename TX, typename TY>
cudaError_t launch_types(const NormArgs& a, cudaStream_t s)
{
    if (a.dim > 8192) return launch_nv<TX, TY, 4, true>(a, s);
    if (a.rows <= FEW_ROWS && a.dim <= 4096) return launch_nv<TX, TY, 1, false>(a, s);
    if (a.dim > 2048) return launch_nv<TX, TY, 2, true>(a, s);
    if (a.per_group < SHORT_GROUP) return a.dim <= 512 ? launch_nv<TX, TY, 1, false>(a, s) : launch_nv<TX, TY, 2, false>(a, s);
    if (a.dim <= 512) return launch_group<TX, TY, 1>(a, s);
    if (a.dim <= 1024) return launch_group<TX, TY, 2>(a, s);
    return a.dim <= 1536 ? launch_group<TX, TY, 3>(a, s) : launch_group<TX, TY, 4>(a, s);
}

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs& a, int x_dtype, int y_dtype, cudaStream_t s)
{
    return with_types(x_dtype, y_dtype, [&](auto x, auto y) { return launch_types<decltype(x), decltype(y)>(a, s); });
}

}  // namespace lf
