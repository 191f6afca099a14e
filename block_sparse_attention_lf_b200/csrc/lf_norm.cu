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
// The gradient kernel keeps its column sums in registers: a CTA takes consecutive rows,
// writes one partial row per group it meets (slot = CTA + group, so no two coincide), and
// a second kernel adds them up in a fixed order -- no atomics, the same bits every time.
#include "lf_norm.h"
#include "lf_device.cuh"
#include "lf_types.cuh"

namespace lf {
namespace {

// 8 consecutive elements of a row as loaded (16 or 32 bytes).
template <typename T> struct Raw8 { uint4 v[sizeof(T) / 2]; };

// Elements [col, col + 8) of a row; zeros past dim. `al`: rows start on 16-byte boundaries
// and dim is a multiple of 8, so the eight are all there and load as vectors.
template <typename T>
__device__ __forceinline__ Raw8<T> load_raw(const T* row, int col, int dim, bool al)
{
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) r.v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (al) {
        if (col < dim) {
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
                r.v[i] = *reinterpret_cast<const uint4*>(row + col + i * VEC_ELEMS<T>);
        }
    } else {
        T* e = reinterpret_cast<T*>(r.v);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col + i < dim) e[i] = row[col + i];
    }
    return r;
}

template <typename T>
__device__ __forceinline__ void unpack8(const Raw8<T>& r, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) {
        float t[VEC_ELEMS<T>];
        unpack<T>(r.v[i], t);
#pragma unroll
        for (int j = 0; j < VEC_ELEMS<T>; ++j) v[i * VEC_ELEMS<T> + j] = t[j];
    }
}

template <typename T>
__device__ __forceinline__ void store8(T* row, int col, int dim, bool al, const float (&v)[8])
{
    if (al) {
        if (col < dim) {
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) {
                float t[VEC_ELEMS<T>];
#pragma unroll
                for (int j = 0; j < VEC_ELEMS<T>; ++j) t[j] = v[i * VEC_ELEMS<T> + j];
                *reinterpret_cast<uint4*>(row + col + i * VEC_ELEMS<T>) = pack<T>(t);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col + i < dim) row[col + i] = from_f32<T>(v[i]);
    }
}

// A vector parameter's eight values (`other` where it is absent, zeros past dim).
__device__ __forceinline__ void load_param(const float* p, int col, int dim, bool al, float other, float (&v)[8])
{
    if (!p) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = other;
    } else {
        unpack8(load_raw(p, col, dim, al), v);
    }
}

// Row sums over a team of `threads` threads (whole warps): two values at once, in a fixed
// order. Consecutive calls alternate between two buffers, so one barrier a call is enough.
struct Team {
    float (*red)[2][32];  // [2 buffers][2 values][warps of the CTA]
    int warp0, warps, warp, lane, bar, threads, phase;

    __device__ __forceinline__ void sum(float& p, float& q)
    {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            p += __shfl_xor_sync(0xffffffffu, p, o);
            q += __shfl_xor_sync(0xffffffffu, q, o);
        }
        if (warps == 1) return;
        if (lane == 0) {
            red[phase][0][warp] = p;
            red[phase][1][warp] = q;
        }
        named_bar_sync(bar, threads);
        p = q = 0.f;
        for (int w = 0; w < warps; ++w) {
            p += red[phase][0][warp0 + w];
            q += red[phase][1][warp0 + w];
        }
        phase ^= 1;
    }
};

__device__ __forceinline__ Team make_team(float (*red)[2][32], int team_threads)
{
    Team t;
    const int team = threadIdx.x / team_threads;
    t.red = red;
    t.warps = team_threads >> 5;
    t.warp = threadIdx.x >> 5;
    t.warp0 = team * t.warps;
    t.lane = threadIdx.x & 31;
    t.bar = 1 + team;
    t.threads = team_threads;
    t.phase = 0;
    return t;
}

// Normalises the row in place (t -> (t - mean) / deviation) and returns 1 / deviation.
// Elements past dim are zero before and stay zero.
template <int NV>
__device__ __forceinline__ float normalise(Team& team, float (&t)[NV][8], int kind, int dim, int col0, int stride, float eps)
{
    const float inv = 1.0f / static_cast<float>(dim);
    float unused = 0.f;
    if (kind == NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) s += t[k][i];
        team.sum(s, unused);
        const float mean = s * inv;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) t[k][i] = col0 + k * stride + i < dim ? t[k][i] - mean : 0.f;
    }
    float q = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) q = fmaf(t[k][i], t[k][i], q);
    team.sum(q, unused);
    const float rs = 1.0f / sqrtf(q * inv + eps);
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) t[k][i] *= rs;
    return rs;
}

constexpr int NORM_THREADS = 512;

template <typename TX, typename TY, int NV>
__global__ void __launch_bounds__(NORM_THREADS) norm_fwd_kernel(const NormArgs a, int team_threads, bool al)
{
    __shared__ float red[2][2][32];
    Team team = make_team(red, team_threads);
    const int teams = blockDim.x / team_threads;
    const int ti = threadIdx.x / team_threads, tt = threadIdx.x - ti * team_threads;
    const long long row = static_cast<long long>(blockIdx.x) * teams + ti;
    if (row >= a.rows) return;  // whole teams leave
    const int col0 = tt * 8, stride = team_threads * 8;
    const long long at = row * a.dim;
    Raw8<TX> xr[NV];
    Raw8<TY> yr[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        xr[k] = load_raw(static_cast<const TX*>(a.x) + at, col0 + k * stride, a.dim, al);
        if (a.y) yr[k] = load_raw(static_cast<const TY*>(a.y) + at, col0 + k * stride, a.dim, al);
    }
    const long long g = (row / a.per_group) * a.dim;
    float t[NV][8];
    if (a.y) {
#pragma unroll
        for (int k = 0; k < NV; ++k) unpack8(yr[k], t[k]);
        if (a.post != NORM_NONE) normalise<NV>(team, t, a.post, a.dim, col0, stride, a.eps);
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int col = col0 + k * stride;
        float x[8], p[8];
        unpack8(xr[k], x);
        if (a.y) {
            if (a.v.post_w) {
                load_param(a.v.post_w, col, a.dim, al, 1.f, p);
#pragma unroll
                for (int i = 0; i < 8; ++i) t[k][i] *= p[i];
            }
            if (a.v.post_b) {
                load_param(a.v.post_b, col, a.dim, al, 0.f, p);
#pragma unroll
                for (int i = 0; i < 8; ++i) t[k][i] += p[i];
            }
            load_param(a.v.gate ? a.v.gate + g : nullptr, col, a.dim, al, 1.f, p);
#pragma unroll
            for (int i = 0; i < 8; ++i) t[k][i] = fmaf(p[i], t[k][i], a.alpha * x[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) t[k][i] = a.alpha * x[i];
        }
        if (a.r) store8(static_cast<TX*>(a.r) + at, col, a.dim, al, t[k]);
    }
    if (!a.h) return;
    normalise<NV>(team, t, a.pre, a.dim, col0, stride, a.eps);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int col = col0 + k * stride;
        float p[8], q[8];
        if (a.v.pre_w) {
            load_param(a.v.pre_w, col, a.dim, al, 1.f, p);
#pragma unroll
            for (int i = 0; i < 8; ++i) t[k][i] *= p[i];
        }
        if (a.v.pre_b) {
            load_param(a.v.pre_b, col, a.dim, al, 0.f, p);
#pragma unroll
            for (int i = 0; i < 8; ++i) t[k][i] += p[i];
        }
        load_param(a.v.scale ? a.v.scale + g : nullptr, col, a.dim, al, 0.f, p);
        load_param(a.v.shift ? a.v.shift + g : nullptr, col, a.dim, al, 0.f, q);
#pragma unroll
        for (int i = 0; i < 8; ++i) t[k][i] = fmaf(t[k][i], 1.f + p[i], q[i]);
        store8(static_cast<TY*>(a.h) + at, col, a.dim, al, t[k]);
    }
}

// Values past dim are kept at zero wherever they enter a sum.
template <typename TX, typename TY, int NV>
__global__ void __launch_bounds__(NORM_THREADS) norm_bwd_kernel(const NormArgs a, int team_threads, bool al)
{
    __shared__ float red[2][2][32];
    extern __shared__ float fold[];  // [teams - 1][dim8] while the teams' sums are added
    Team team = make_team(red, team_threads);
    const int teams = blockDim.x / team_threads;
    const int ti = threadIdx.x / team_threads, tt = threadIdx.x - ti * team_threads;
    const int col0 = tt * 8, stride = team_threads * 8, dim = a.dim;
    const int dim8 = (dim + 7) & ~7;
    const long long r0 = blockIdx.x * a.rows_per_cta;
    const long long r1 = min(a.rows, r0 + a.rows_per_cta);
    const float inv = 1.0f / static_cast<float>(dim);

    for (long long seg = r0; seg < r1;) {
        const long long gi = seg / a.per_group;
        const long long seg_end = min(r1, (gi + 1) * a.per_group);
        const long long g = gi * dim;
        float A[4][NV][8];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) A[j][k][i] = 0.f;
        for (long long row = seg + ti; row < seg_end; row += teams) {
            const long long at = row * dim;
            float m[NV][8], n[NV][8], d[NV][8], p[8];
            float rs1 = 1.f, rs2 = 1.f;
            // forward again: m = post(y), n = pre(r)
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                if (a.y) unpack8(load_raw(static_cast<const TY*>(a.y) + at, col0 + k * stride, dim, al), m[k]);
                unpack8(load_raw(static_cast<const TX*>(a.x) + at, col0 + k * stride, dim, al), n[k]);
            }
            if (a.y && a.post != NORM_NONE) rs2 = normalise<NV>(team, m, a.post, dim, col0, stride, a.eps);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = col0 + k * stride;
#pragma unroll
                for (int i = 0; i < 8; ++i) n[k][i] *= a.alpha;
                if (a.y) {
                    float u[8];
                    load_param(a.v.post_w, col, dim, al, 1.f, p);
#pragma unroll
                    for (int i = 0; i < 8; ++i) u[i] = m[k][i] * p[i];
                    load_param(a.v.post_b, col, dim, al, 0.f, p);
#pragma unroll
                    for (int i = 0; i < 8; ++i) u[i] += p[i];
                    load_param(a.v.gate ? a.v.gate + g : nullptr, col, dim, al, 1.f, p);
#pragma unroll
                    for (int i = 0; i < 8; ++i) n[k][i] = fmaf(p[i], u[i], n[k][i]);
                }
            }
            float s1 = 0.f, s2 = 0.f;
            if (a.dh) {
                rs1 = normalise<NV>(team, n, a.pre, dim, col0, stride, a.eps);
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int col = col0 + k * stride;
                    unpack8(load_raw(static_cast<const TY*>(a.dh) + at, col, dim, al), d[k]);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        A[0][k][i] += d[k][i];
                        A[1][k][i] = fmaf(d[k][i], n[k][i], A[1][k][i]);
                    }
                    load_param(a.v.scale ? a.v.scale + g : nullptr, col, dim, al, 0.f, p);
#pragma unroll
                    for (int i = 0; i < 8; ++i) d[k][i] *= 1.f + p[i];
                    load_param(a.v.pre_w, col, dim, al, 1.f, p);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        d[k][i] *= p[i];
                        s1 += d[k][i];
                        s2 = fmaf(d[k][i], n[k][i], s2);
                    }
                }
                team.sum(s1, s2);
                s1 = a.pre == NORM_LAYER ? s1 * inv : 0.f;
                s2 *= inv;
            }
            // dr' in d
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = col0 + k * stride;
                if (a.dr) unpack8(load_raw(static_cast<const TX*>(a.dr) + at, col, dim, al), p);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float dn = a.dh ? rs1 * (d[k][i] - s1 - n[k][i] * s2) : 0.f;
                    d[k][i] = (a.dr ? p[i] : 0.f) + dn;
                }
                if (a.dx) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) p[i] = a.alpha * d[k][i];
                    store8(static_cast<TX*>(a.dx) + at, col, dim, al, p);
                }
            }
            if (!a.y) continue;
            float t1 = 0.f, t2 = 0.f;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = col0 + k * stride;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    A[2][k][i] += d[k][i];
                    A[3][k][i] = fmaf(d[k][i], m[k][i], A[3][k][i]);
                }
                load_param(a.v.gate ? a.v.gate + g : nullptr, col, dim, al, 1.f, p);
#pragma unroll
                for (int i = 0; i < 8; ++i) d[k][i] *= p[i];
                load_param(a.v.post_w, col, dim, al, 1.f, p);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    d[k][i] = col + i < dim ? d[k][i] * p[i] : 0.f;
                    t1 += d[k][i];
                    t2 = fmaf(d[k][i], m[k][i], t2);
                }
            }
            if (!a.dy) continue;
            if (a.post != NORM_NONE) {
                team.sum(t1, t2);
                t1 = a.post == NORM_LAYER ? t1 * inv : 0.f;
                t2 *= inv;
#pragma unroll
                for (int k = 0; k < NV; ++k)
#pragma unroll
                    for (int i = 0; i < 8; ++i) d[k][i] = rs2 * (d[k][i] - t1 - m[k][i] * t2);
            }
#pragma unroll
            for (int k = 0; k < NV; ++k) store8(static_cast<TY*>(a.dy) + at, col0 + k * stride, dim, al, d[k]);
        }
        // the CTA's sums for this group: teams added in order, one partial row each
        float* slot = a.part + (blockIdx.x + gi) * 4 * dim8;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (teams > 1) {
                __syncthreads();
                if (ti > 0) {
#pragma unroll
                    for (int k = 0; k < NV; ++k) {
                        const int col = col0 + k * stride;
                        if (col < dim8) {
                            float* f = fold + (ti - 1) * dim8 + col;
#pragma unroll
                            for (int i = 0; i < 8; ++i) f[i] = A[j][k][i];
                        }
                    }
                }
                __syncthreads();
            }
            if (ti == 0) {
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int col = col0 + k * stride;
                    if (col < dim8) {
                        for (int o = 0; o < teams - 1; ++o)
#pragma unroll
                            for (int i = 0; i < 8; ++i) A[j][k][i] += fold[o * dim8 + col + i];
                        *reinterpret_cast<float4*>(slot + j * dim8 + col) = make_float4(A[j][k][0], A[j][k][1], A[j][k][2], A[j][k][3]);
                        *reinterpret_cast<float4*>(slot + j * dim8 + col + 4) = make_float4(A[j][k][4], A[j][k][5], A[j][k][6], A[j][k][7]);
                    }
                }
            }
        }
        seg = seg_end;
    }
}

constexpr int FIN_COLS = 32, FIN_ROWS = 16;

// Adds the partial rows up: blockIdx.y < groups is a group's dgate, dscale and dshift, the
// last one the weights' gradients over all groups. A CTA takes 32 columns, 16 threads each.
__global__ void __launch_bounds__(FIN_COLS * FIN_ROWS) norm_bwd_finish_kernel(const NormArgs a, long long groups)
{
    __shared__ float red[FIN_ROWS][4][FIN_COLS];
    const int c = threadIdx.x % FIN_COLS, j = threadIdx.x / FIN_COLS;
    const int col = blockIdx.x * FIN_COLS + c;
    const int dim8 = (a.dim + 7) & ~7;
    const bool weights = a.dpre_w || a.dpre_b || a.dpost_w || a.dpost_b;
    for (long long item = blockIdx.y; item < groups + (weights ? 1 : 0); item += gridDim.y) {
        const bool all = item == groups;
        const long long row0 = all ? 0 : item * a.per_group;
        const long long row1 = all ? a.rows : min(a.rows, row0 + a.per_group);
        float A[4] = {0.f, 0.f, 0.f, 0.f};
        if (col < a.dim && row1 > row0) {
            const long long c0 = row0 / a.rows_per_cta, c1 = (row1 - 1) / a.rows_per_cta;
            for (long long cta = c0 + j; cta <= c1; cta += FIN_ROWS) {
                // the groups this CTA met, of those wanted
                const long long first = cta * a.rows_per_cta, last = min(a.rows, first + a.rows_per_cta) - 1;
                const long long g0 = all ? first / a.per_group : item, g1 = all ? last / a.per_group : item;
                for (long long g = g0; g <= g1; ++g) {
                    const float* p = a.part + (cta + g) * 4 * dim8 + col;
                    float w1 = 1.f, w2 = 1.f;
                    if (all) {
                        w1 = a.v.scale ? 1.f + a.v.scale[g * a.dim + col] : 1.f;
                        w2 = a.v.gate ? a.v.gate[g * a.dim + col] : 1.f;
                    }
                    A[0] = fmaf(w1, p[0], A[0]);
                    A[1] = fmaf(w1, p[dim8], A[1]);
                    A[2] = fmaf(w2, p[2 * dim8], A[2]);
                    A[3] = fmaf(w2, p[3 * dim8], A[3]);
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) red[j][i][c] = A[i];
        __syncthreads();
        if (j < 4 && col < a.dim) {  // thread row i adds sum i
            float s = 0.f;
            for (int o = 0; o < FIN_ROWS; ++o) s += red[o][j][c];
            red[0][j][c] = s;
        }
        __syncthreads();
        if (j == 0 && col < a.dim) {
            const float a1 = red[0][0][c], a2 = red[0][1][c], a3 = red[0][2][c], a4 = red[0][3][c];
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

// Threads of a team and groups of 8 a thread: as few elements a thread as 256 threads
// allow, then two groups, then four (dim <= 16384 = 512 * 4 * 8).
int team_of(int dim, int* nv)
{
    const int vecs = (dim + 7) / 8;
    *nv = vecs <= 256 ? 1 : (vecs <= 1024 ? 2 : 4);
    const int t = (vecs + *nv - 1) / *nv;
    return (t + 31) / 32 * 32;
}

bool aligned_rows(const NormArgs& a) { return a.dim % 8 == 0; }  // pointers are 16-byte aligned

template <typename TX, typename TY>
cudaError_t launch_fwd(const NormArgs& a, cudaStream_t s)
{
    int nv;
    const int t = team_of(a.dim, &nv);
    const int teams = t >= 256 ? 1 : 256 / t;
    const unsigned grid = static_cast<unsigned>((a.rows + teams - 1) / teams);
    const bool al = aligned_rows(a);
    if (nv == 1)
        norm_fwd_kernel<TX, TY, 1><<<grid, t * teams, 0, s>>>(a, t, al);
    else if (nv == 2)
        norm_fwd_kernel<TX, TY, 2><<<grid, t * teams, 0, s>>>(a, t, al);
    else
        norm_fwd_kernel<TX, TY, 4><<<grid, t * teams, 0, s>>>(a, t, al);
    return cudaGetLastError();
}

template <typename TX, typename TY>
cudaError_t launch_bwd(const NormArgs& a, cudaStream_t s)
{
    int nv;
    const int t = team_of(a.dim, &nv);
    const int teams = t >= 256 ? 1 : 256 / t;
    const bool al = aligned_rows(a);
    const size_t fold = static_cast<size_t>(teams - 1) * ((a.dim + 7) / 8 * 8) * sizeof(float);
    if (nv == 1)
        norm_bwd_kernel<TX, TY, 1><<<a.n_cta, t * teams, fold, s>>>(a, t, al);
    else if (nv == 2)
        norm_bwd_kernel<TX, TY, 2><<<a.n_cta, t * teams, fold, s>>>(a, t, al);
    else
        norm_bwd_kernel<TX, TY, 4><<<a.n_cta, t * teams, fold, s>>>(a, t, al);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (!a.dgate && !a.dscale && !a.dshift && !a.dpre_w && !a.dpre_b && !a.dpost_w && !a.dpost_b) return cudaSuccess;
    const long long groups = (a.rows + a.per_group - 1) / a.per_group;
    const long long items = groups + 1;
    norm_bwd_finish_kernel<<<dim3((a.dim + FIN_COLS - 1) / FIN_COLS, static_cast<unsigned>(items < 65535 ? items : 65535)),
                             FIN_COLS * FIN_ROWS, 0, s>>>(a, groups);
    return cudaGetLastError();
}

template <bool BWD, typename TX, typename TY>
cudaError_t launch_one(const NormArgs& a, cudaStream_t s)
{
    if constexpr (BWD) return launch_bwd<TX, TY>(a, s);
    else return launch_fwd<TX, TY>(a, s);
}

template <bool BWD>
cudaError_t launch_any(const NormArgs& a, int xd, int yd, cudaStream_t s)
{
    if (xd == DT_BF16) return launch_one<BWD, __nv_bfloat16, __nv_bfloat16>(a, s);
    if (xd == DT_F16) return launch_one<BWD, __half, __half>(a, s);
    if (yd == DT_BF16) return launch_one<BWD, float, __nv_bfloat16>(a, s);
    if (yd == DT_F16) return launch_one<BWD, float, __half>(a, s);
    return launch_one<BWD, float, float>(a, s);
}

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs& a, int x_dtype, int y_dtype, cudaStream_t s)
{
    return launch_any<false>(a, x_dtype, y_dtype, s);
}

cudaError_t launch_norm_bwd(const NormArgs& a, int x_dtype, int y_dtype, cudaStream_t s)
{
    return launch_any<true>(a, x_dtype, y_dtype, s);
}

}  // namespace lf
