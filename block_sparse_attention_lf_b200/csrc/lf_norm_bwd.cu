// lf_norm_bwd.cu -- gradients of the gated residual norms (formulas and the rows' way through a
// team: lf_norm.cu).
#include "lf_norm_rows.cuh"
#include "lf_internal.h"

namespace lf {
namespace {

// One CTA an SM, so that few partial sums are written: 384 threads that hold two groups of eight
// (32760 rows of 1536 bf16, 604 MB: 202 us, 3.0 TB/s; one group in 192 threads 284, three in 64
// threads 266). What the row's first halves need is read before the sums that precede its use, as far
// as registers last (208 without; with every read so, 337: it spills). The bound is a row's chain of
// four dependent sums and the issue of its arithmetic by twelve warps; more warps would leave the column
// sums no registers. Rows that leave threads of a team idle spill where the post norm has a bias (460 /
// 792 bytes a thread stored and loaded; 768 wide: 298 us for 32760 rows).
// WIDE: longer rows take up to 512 threads, of two groups to 8192 and of four above. Their column sums,
// 64 and 128 registers of 128, spill (bf16: 424 / 636 to 3172 / 4064 bytes), and one row an SM is at
// work: 8192 rows of 4096 take 499 us, 2048 of 16384 564, where 16384 of 2048 take 145.
// Short groups are dear whatever the width: each stops its CTA and leaves four fp32 partial rows (32760
// rows of 1536 in groups of 16: 185 us and the finish 309; of one: 1227 and 4183).
template <bool WIDE> constexpr int BWD_REGS = WIDE ? 128 : 168;
constexpr int BWD_THREADS = 384;

__device__ __forceinline__ void vec_store(float* p, int col, const Vec8& x)
{
    float4* f = reinterpret_cast<float4*>(p + col);
    f[0] = make_float4(x.v[0].x, x.v[0].y, x.v[1].x, x.v[1].y);
    f[1] = make_float4(x.v[2].x, x.v[2].y, x.v[3].x, x.v[3].y);
}

__device__ __forceinline__ Vec8 vec_load(const float* p, int col)
{
    const float4* f = reinterpret_cast<const float4*>(p + col);
    const float4 a = f[0], b = f[1];
    Vec8 o;
    o.v[0] = make_float2(a.x, a.y);
    o.v[1] = make_float2(a.z, a.w);
    o.v[2] = make_float2(b.x, b.y);
    o.v[3] = make_float2(b.z, b.w);
    return o;
}

// BIAS: the post norm has a bias, or its gradient is wanted; without it b2 and A3 (sum dr') need
// no registers.
template <typename TX, typename TY, int NV, bool WIDE, bool FULL, bool BIAS>
__global__ void __maxnreg__(BWD_REGS<WIDE>) norm_bwd_kernel(const NormArgs a, int team_threads, int stages)
{
    __shared__ __align__(16) float red[MAX_TEAMS][2][2][16];
    extern __shared__ __align__(16) uint8_t smem[];  // the rings, then [3][dim8] vectors and [teams - 1][dim8] sums
    if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the finish, which waits
    Team team = make_team(red, team_threads);
    const int teams = blockDim.x / team_threads;
    const int ti = threadIdx.x / team_threads, tt = threadIdx.x - ti * team_threads;
    const int dim = a.dim, dim8 = (dim + 7) & ~7;
    const long long r0 = blockIdx.x * a.rows_per_cta, first = r0 + ti;
    const long long r1 = min(a.rows, r0 + a.rows_per_cta);
    const float inv = 1.0f / static_cast<float>(dim);
    const Place p{tt * 8, team_threads * 8, dim, team_threads, stages, static_cast<long long>(teams) * dim, dim % 8 == 0};
    Ring ring;
    ring.stage_bytes = 0;
    Source<TX, NV, FULL> x, dr;
    Source<TY, NV, FULL> y, dh;
    Sink<TX, NV, FULL> dx;
    Sink<TY, NV, FULL> dy;
    x.init(a.x, first, p, &ring.stage_bytes, tt);
    y.init(a.y, first, p, &ring.stage_bytes, tt);
    dr.init(a.dr, first, p, &ring.stage_bytes, tt);
    dh.init(a.dh, first, p, &ring.stage_bytes, tt);
    dx.init(a.dx, first, p);
    dy.init(a.dy, first, p);
    ring.stages = stages;
    ring.base = smem + static_cast<size_t>(ti) * stages * ring.stage_bytes;
    ring.start(first < r1 ? static_cast<int>((r1 - first + teams - 1) / teams) : 0, p, x, y, dr, dh);
    float* vecs = reinterpret_cast<float*>(smem + static_cast<size_t>(teams) * stages * ring.stage_bytes);  // g2, s1, b2
    float* fold = vecs + 3 * dim8;
    float* part_w = a.part_w + static_cast<long long>(blockIdx.x) * 4 * dim8;

    long long row = first;
    for (long long seg = r0; seg < r1;) {
        const long long gi = seg / a.per_group;
        const long long seg_end = min(r1, (gi + 1) * a.per_group);
        const long long g = gi * dim;
        // u gate = m g2 + b2; dn = dh s1: the same for every team, so in shared memory
        __syncthreads();
        for (int col = threadIdx.x * 8; col < dim8; col += blockDim.x * 8) {
            const Vec8 v = load_param(a.v.gate ? a.v.gate + g : nullptr, col, dim, p.al, 1.f);
            split_store(vecs, col, dim8, mul(load_param(a.v.post_w, col, dim, p.al, 1.f), v));
            split_store(vecs + dim8, col, dim8, mul(load_param(a.v.pre_w, col, dim, p.al, 1.f),
                                                    add(load_param(a.v.scale ? a.v.scale + g : nullptr, col, dim, p.al, 0.f), 1.f)));
            if (BIAS) split_store(vecs + 2 * dim8, col, dim8, mul(load_param(a.v.post_b, col, dim, p.al, 0.f), v));
        }
        __syncthreads();
        // a vector of the group at the thread's k-th eight columns
        auto vec = [&](int which, int k) {
            const int col = p.col0 + k * p.stride;
            return FULL || col < dim8 ? split_load(vecs + which * dim8, col, dim8) : fill8(0.f);
        };
        Vec8 A[4][NV];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < NV; ++k) A[j][k] = fill8(0.f);
        for (; row < seg_end; row += teams) {
            const uint8_t* st = ring.next(p, x, y, dr, dh);
            Vec8 m[NV], n[NV], d[NV];
            float rs1 = 1.f, rs2 = 1.f;
            // forward again: m = post(y), n = pre(r)
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                n[k] = x.get(st, k, p);
                n[k] = BIAS ? fma(n[k], a.alpha, vec(2, k)) : mul(n[k], a.alpha);
            }
            if (y.on) {
#pragma unroll
                for (int k = 0; k < NV; ++k) m[k] = y.get(st, k, p);
                if (a.post != NORM_NONE) rs2 = normalise<NV, FULL>(team, m, a.post, inv, p, a.eps);
            }
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                if (y.on) n[k] = fma(vec(0, k), m[k], n[k]);
            }
            float q1 = 0.f, q2 = 0.f;
            if (dh.on) {
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    d[k] = dh.get(st, k, p);
                    A[0][k] = add(A[0][k], d[k]);
                }
                rs1 = normalise<NV, FULL>(team, n, a.pre, inv, p, a.eps);
                float2 u = make_float2(0.f, 0.f), w = u;
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    A[1][k] = fma(d[k], n[k], A[1][k]);
                    d[k] = mul(d[k], vec(1, k));
                    acc(u, d[k]);
                    acc(w, d[k], n[k]);
                }
                q1 = u.x + u.y;
                q2 = w.x + w.y;
                team.sum(q1, q2);
                // minus rs1 times the means
                q1 = a.pre == NORM_LAYER ? q1 * inv * -rs1 : 0.f;
                q2 *= inv * -rs1;
            }
            // dr' in d
            float2 u = make_float2(0.f, 0.f), w = u;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const Vec8 v = dr.on ? dr.get(st, k, p) : fill8(0.f);
                d[k] = dh.on ? fma(n[k], q2, fma(d[k], rs1, add(v, q1))) : v;
                dx.put(k, mul(d[k], a.alpha), p);
                if (y.on) {
                    if (BIAS) A[2][k] = add(A[2][k], d[k]);
                    A[3][k] = fma(d[k], m[k], A[3][k]);
                    d[k] = mul(d[k], vec(0, k));  // dm (zero past dim, as g2 is)
                    acc(u, d[k]);
                    acc(w, d[k], m[k]);
                }
            }
            x.done(p);
            y.done(p);
            dr.done(p);
            dh.done(p);
            dx.done(p);
            ring.done();
            if (!dy.on) continue;
            if (a.post != NORM_NONE) {
                float p1 = u.x + u.y, p2 = w.x + w.y;
                team.sum(p1, p2);
                p1 = a.post == NORM_LAYER ? p1 * inv * -rs2 : 0.f;
                p2 *= inv * -rs2;
#pragma unroll
                for (int k = 0; k < NV; ++k) d[k] = fma(m[k], p2, fma(d[k], rs2, fill8(p1)));
            }
#pragma unroll
            for (int k = 0; k < NV; ++k) dy.put(k, d[k], p);
            dy.done(p);
        }
        // the CTA's sums for this group: teams added in order, one partial row each; and the
        // weights' sums so far
        float* slot = a.part + (blockIdx.x + gi) * 4 * dim8;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (teams > 1) {
                __syncthreads();
                if (ti > 0) {
#pragma unroll
                    for (int k = 0; k < NV; ++k)
                        if (p.col0 + k * p.stride < dim8) vec_store(fold + (ti - 1) * dim8, p.col0 + k * p.stride, A[j][k]);
                }
                __syncthreads();
            }
            if (ti == 0) {
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int col = p.col0 + k * p.stride;
                    if (col >= dim8) continue;
                    for (int o = 0; o < teams - 1; ++o) A[j][k] = add(A[j][k], vec_load(fold + o * dim8, col));
                    vec_store(slot + j * dim8, col, A[j][k]);
                    if (a.weights) {  // times 1 + scale, or the gate
                        const float* f = j < 2 ? a.v.scale : a.v.gate;
                        const Vec8 v = load_param(f ? f + g : nullptr, col, dim, p.al, j < 2 ? 0.f : 1.f);
                        const Vec8 before = seg > r0 ? vec_load(part_w + j * dim8, col) : fill8(0.f);
                        vec_store(part_w + j * dim8, col, fma(j < 2 ? add(v, 1.f) : v, A[j][k], before));
                    }
                }
            }
        }
        seg = seg_end;
    }
}

constexpr int FIN_COLS = 32, FIN_ROWS = 32, FIN_GROUPS = 4;

// Adds the partial rows up. A CTA takes 32 columns of four consecutive groups (dgate, dscale,
// dshift; 8 threads a column and group), or, blockIdx.y being the last, of the weights' gradients
// over all CTAs (32 threads a column).
__global__ void __launch_bounds__(FIN_COLS * FIN_ROWS) norm_bwd_finish_kernel(const NormArgs a, long long groups)
{
    __shared__ float red[4][FIN_ROWS][FIN_COLS];
    const int c = threadIdx.x % FIN_COLS, j = threadIdx.x / FIN_COLS;
    const int col = blockIdx.x * FIN_COLS + c;
    const int dim8 = (a.dim + 7) & ~7;
    const long long batches = (groups + FIN_GROUPS - 1) / FIN_GROUPS;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (long long batch = blockIdx.y; batch < batches + (a.weights ? 1 : 0); batch += gridDim.y) {
        const bool all = batch == batches;
        const int rows = all ? FIN_ROWS : FIN_ROWS / FIN_GROUPS, first = j % rows;
        const long long item = all ? 0 : batch * FIN_GROUPS + j / rows;
        // consecutive partial rows: a group's are those of the CTAs that met it
        int n = 0;
        const float* base = a.part_w + col;
        if (all) {
            n = a.n_cta;
        } else if (item < groups) {
            const long long row0 = item * a.per_group, row1 = min(a.rows, row0 + a.per_group);
            const long long c0 = row0 / a.rows_per_cta;
            n = static_cast<int>((row1 - 1) / a.rows_per_cta - c0) + 1;
            base = a.part + (c0 + item) * 4 * dim8 + col;
        }
        float A[4] = {0.f, 0.f, 0.f, 0.f};
        if (col < a.dim) {
#pragma unroll 4
            for (int s = first; s < n; s += rows) {
                const float* p = base + static_cast<long long>(s) * 4 * dim8;
                A[0] += p[0];
                A[1] += p[dim8];
                A[2] += p[2 * dim8];
                A[3] += p[3 * dim8];
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) red[i][j][c] = A[i];
        __syncthreads();
        if (first < 4) {  // a group's thread row i adds its sum i
            float s = 0.f;
            for (int o = 0; o < rows; ++o) s += red[first][j - first + o][c];
            __syncwarp();
            red[first][j - first][c] = s;
        }
        __syncthreads();
        if (first == 0 && col < a.dim && n > 0) {
            const float a1 = red[0][j][c], a2 = red[1][j][c], a3 = red[2][j][c], a4 = red[3][j][c];
            if (all) {
                if (a.dpre_w) a.dpre_w[col] = a2;
                if (a.dpre_b) a.dpre_b[col] = a1;
                if (a.dpost_w) a.dpost_w[col] = a4;
                if (a.dpost_b) a.dpost_b[col] = a3;
            } else {
                const long long at = item * a.dim + col;
                if (a.dshift) a.dshift[at] = a1;
                if (a.dscale) a.dscale[at] = fmaf(a.v.pre_w ? a.v.pre_w[col] : 1.f, a2, a.v.pre_b ? a.v.pre_b[col] * a1 : 0.f);
                if (a.dgate) a.dgate[at] = fmaf(a.v.post_w ? a.v.post_w[col] : 1.f, a4, a.v.post_b ? a.v.post_b[col] * a3 : 0.f);
            }
        }
    }
}

template <typename TX, typename TY, int NV, bool WIDE, bool FULL, bool BIAS>
cudaError_t launch_rows(const NormArgs& a, const NormPlan& p, cudaStream_t s)
{
    cudaError_t e = allow_smem<norm_bwd_kernel<TX, TY, NV, WIDE, FULL, BIAS>>(p.smem);
    if (e != cudaSuccess) return e;
    norm_bwd_kernel<TX, TY, NV, WIDE, FULL, BIAS><<<a.n_cta, p.threads * p.teams, p.smem, s>>>(a, p.threads, p.stages);
    return cudaGetLastError();
}

// BIAS: the post norm has a bias, or its gradient is wanted; without it b2 is not read and A3 (sum
// dr') needs no registers.
template <typename TX, typename TY, int NV, bool WIDE>
cudaError_t launch_nv(const NormArgs& a, cudaStream_t s)
{
    const size_t elem = sizeof(TX) * (a.dr ? 2 : 1) + sizeof(TY) * ((a.y ? 1 : 0) + (a.dh ? 1 : 0));
    const NormPlan p = plan_of(a.dim, NV, elem, WIDE ? 128 : BWD_THREADS, 1, 2, 1);  // 3 vectors, teams - 1 folded sums
    const bool bias = a.v.post_b || a.dpost_b;
    cudaError_t e;
    if (p.full)
        e = bias ? launch_rows<TX, TY, NV, WIDE, true, true>(a, p, s) : launch_rows<TX, TY, NV, WIDE, true, false>(a, p, s);
    else
        e = bias ? launch_rows<TX, TY, NV, WIDE, false, true>(a, p, s) : launch_rows<TX, TY, NV, WIDE, false, false>(a, p, s);
    if (e != cudaSuccess || (!a.dgate && !a.dscale && !a.dshift && !a.weights)) return e;
    const long long groups = (a.rows + a.per_group - 1) / a.per_group;
    const long long items = (groups + FIN_GROUPS - 1) / FIN_GROUPS + (a.weights ? 1 : 0);
    const dim3 grid((a.dim + FIN_COLS - 1) / FIN_COLS, static_cast<unsigned>(std::min<long long>(items, 65535)));
    return launch_dependent(norm_bwd_finish_kernel, grid, FIN_COLS * FIN_ROWS, 0, s, a, groups);
}

template <typename TX, typename TY>
cudaError_t launch_types(const NormArgs& a, cudaStream_t s)
{
    if (a.dim <= 2048) return launch_nv<TX, TY, 2, false>(a, s);
    return a.dim <= 8192 ? launch_nv<TX, TY, 2, true>(a, s) : launch_nv<TX, TY, 4, true>(a, s);
}

}  // namespace

cudaError_t launch_norm_bwd(const NormArgs& a, int x_dtype, int y_dtype, cudaStream_t s)
{
    return with_types(x_dtype, y_dtype, [&](auto x, auto y) { return launch_types<decltype(x), decltype(y)>(a, s); });
}

}  // namespace lf
