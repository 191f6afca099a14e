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
// registers, folded to what a row needs (gate w2, gate b2, (1 + scale) w1, b1 (1 + scale) +
// shift), and rows arrive ahead through a ring of bulk copies: a row has several dependent
// sums, and only loads that are many rows ahead keep the memory busy meanwhile. Rows that do
// not start on 16-byte boundaries (dim not a multiple of 8), and rows too long for a ring,
// are loaded directly.
//
// The gradient kernel keeps its column sums in registers: a CTA writes one partial row per
// group it meets (slot = CTA + group, so no two coincide) and one of its weights' sums, and a
// second kernel adds them up in a fixed order -- no atomics, the same bits every time.
#include "lf_norm.h"
#include "lf_device.cuh"
#include "lf_types.cuh"

#include <algorithm>
#include <atomic>

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

// Eight values of a vector (`other` where it is absent, zeros past dim).
__device__ __forceinline__ void load_param(const float* p, int col, int dim, bool al, float other, float (&v)[8])
{
    if (!p) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = col + i < dim ? other : 0.f;
    } else {
        unpack8(load_raw(p, col, dim, al), v);
    }
}

constexpr int MAX_TEAMS = 8, MAX_STAGES = 4;

// (d0, d1) = (a0, a1) * (b0, b1) + (c0, c1), packed
__device__ __forceinline__ void ffma2(float& d0, float& d1, float a0, float a1, float b0, float b1, float c0, float c1)
{
    asm("{\n\t.reg .b64 ra, rb, rc;\n\t"
        "mov.b64 ra, {%2, %3};\n\t"
        "mov.b64 rb, {%4, %5};\n\t"
        "mov.b64 rc, {%6, %7};\n\t"
        "fma.rn.f32x2 rc, ra, rb, rc;\n\t"
        "mov.b64 {%0, %1}, rc;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}

// Row sums over a team of whole warps, in a fixed order. Consecutive calls alternate between two
// buffers, so one barrier a call is enough; unused places of a buffer stay zero.
struct Team {
    float (*red)[2][16];  // this team's [2 buffers][2 values][warps]
    int warps, warp, lane, bar, threads, phase;

    __device__ __forceinline__ void sync()
    {
        if (warps == 1) __syncwarp();
        else named_bar_sync(bar, threads);
    }

    __device__ __forceinline__ float gather(int which)
    {
        const float4* f = reinterpret_cast<const float4*>(red[phase][which]);
        const float4 u = f[0], v = f[1];
        float s = ((u.x + u.y) + (u.z + u.w)) + ((v.x + v.y) + (v.z + v.w));
        if (warps > 8) {
            const float4 w = f[2], x = f[3];
            s += ((w.x + w.y) + (w.z + w.w)) + ((x.x + x.y) + (x.z + x.w));
        }
        return s;
    }

    __device__ __forceinline__ void sum(float& p, float& q)
    {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float a = __shfl_xor_sync(0xffffffffu, p, o), b = __shfl_xor_sync(0xffffffffu, q, o);
            fadd2_acc(p, q, a, b);
        }
        if (warps == 1) return;
        if (lane == 0) {
            red[phase][0][warp] = p;
            red[phase][1][warp] = q;
        }
        named_bar_sync(bar, threads);
        p = gather(0);
        q = gather(1);
        phase ^= 1;
    }

    __device__ __forceinline__ void sum(float& p)
    {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) p += __shfl_xor_sync(0xffffffffu, p, o);
        if (warps == 1) return;
        if (lane == 0) red[phase][0][warp] = p;
        named_bar_sync(bar, threads);
        p = gather(0);
        phase ^= 1;
    }
};

__device__ __forceinline__ Team make_team(float (*red)[2][2][16], int team_threads)
{
    Team t;
    const int team = threadIdx.x / team_threads, in = threadIdx.x - team * team_threads;
    t.red = red[team];
    t.warps = team_threads >> 5;
    t.warp = in >> 5;
    t.lane = threadIdx.x & 31;
    t.bar = 1 + team;
    t.threads = team_threads;
    t.phase = 0;
    for (int i = in; i < 2 * 2 * 16; i += team_threads) (&t.red[0][0][0])[i] = 0.f;
    return t;
}

// Normalises the row in place (t -> (t - mean) / deviation) and returns 1 / deviation.
// Elements past dim are zero before and stay zero; `mine[k]` of a group's eight are within dim.
template <int NV>
__device__ __forceinline__ float normalise(Team& team, float (&t)[NV][8], int kind, float inv, const int (&mine)[NV], float eps)
{
    float a = 0.f, b = 0.f;
    if (kind == NORM_LAYER) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < 8; i += 2) fadd2_acc(a, b, t[k][i], t[k][i + 1]);
        float s = a + b;
        team.sum(s);
        const float mean = -s * inv;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) fadd2_acc(t[k][i], t[k][i + 1], mean, mean);
            if (mine[k] < 8) {
#pragma unroll
                for (int i = 0; i < 8; ++i) t[k][i] = i < mine[k] ? t[k][i] : 0.f;
            }
        }
        a = b = 0.f;
    }
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 8; i += 2) ffma2(a, b, t[k][i], t[k][i + 1], t[k][i], t[k][i + 1], a, b);
    float q = a + b;
    team.sum(q);
    const float rs = rsqrtf(fmaf(q, inv, eps));
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 8; i += 2) fmul2(t[k][i], t[k][i + 1], rs, rs);
    return rs;
}

// One untiled bulk copy, issued by one thread.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// A team's rows, arriving through a ring of `stages` rows of N streams in shared memory (or
// loaded directly when stages == 0). Stream n of a row has esize[n] bytes an element; a null
// stream is skipped. Rows are first, first + step, ... below end.
template <int N>
struct Rows {
    const uint8_t* src[N];
    uint32_t bytes[N], at[N];  // bytes of a row, offset in a stage
    uint32_t stage_bytes;
    uint8_t* ring;
    uint64_t* full;
    int stages, slot, parity;  // the next row's stage and its phase
    long long step, end;
    bool leader;

    __device__ __forceinline__ void issue(long long row, int s)
    {
        uint32_t sum = 0;
#pragma unroll
        for (int n = 0; n < N; ++n) sum += src[n] ? bytes[n] : 0u;
        mbar_arrive_expect_tx(&full[s], sum);
#pragma unroll
        for (int n = 0; n < N; ++n)
            if (src[n]) bulk_load(ring + s * stage_bytes + at[n], src[n] + row * bytes[n], bytes[n], &full[s]);
    }

    __device__ __forceinline__ void start(long long first)
    {
        slot = parity = 0;
        if (leader)
            for (int s = 0; s < stages; ++s)
                if (first + s * step < end) issue(first + s * step, s);
    }

    // Waits for the next row; its stage's address.
    __device__ __forceinline__ const uint8_t* wait(volatile int* abort_flag, int* err, bool* ok)
    {
        *ok = mbar_wait(&full[slot], parity, abort_flag, err, 0x70);
        return ring + slot * stage_bytes;
    }

    // The whole team has read `row`'s stage: its next use is filled.
    __device__ __forceinline__ void release(long long row)
    {
        if (leader && row + stages * step < end) issue(row + stages * step, slot);
        if (++slot == stages) {
            slot = 0;
            parity ^= 1;
        }
    }

    // After an expired wait: every copy issued lands before the CTA leaves.
    __device__ __forceinline__ void drain()
    {
        if (leader)
            for (int s = 0; s < stages; ++s)
                for (int p = 0; p < 2; ++p) mbar_drain(&full[s], p, 10000000ull);
    }
};

template <int N>
__device__ __forceinline__ Rows<N> make_rows(const void* const (&src)[N], const int (&esize)[N], int dim, uint8_t* smem,
                                             uint64_t* full, int stages, int team, int team_thread, int teams, long long end)
{
    Rows<N> r;
    uint32_t at = 0;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        r.src[n] = static_cast<const uint8_t*>(src[n]);
        r.bytes[n] = static_cast<uint32_t>(dim) * esize[n];
        r.at[n] = at;
        at += src[n] ? r.bytes[n] : 0u;
    }
    r.stage_bytes = at;
    r.ring = smem + static_cast<size_t>(team) * stages * at;
    r.full = full + team * MAX_STAGES;
    r.stages = stages;
    r.step = teams;
    r.end = end;
    r.leader = team_thread == 0;
    return r;
}

template <typename T>
__device__ __forceinline__ Raw8<T> stage_raw(const uint8_t* stage, uint32_t at, int col, int dim)
{
    return load_raw(reinterpret_cast<const T*>(stage + at), col, dim, true);
}

// A CTA has up to 256 threads where a thread holds one group of eight, 512 where it holds more.
// Registers a thread: what lets NORM_FWD_CTAS_PER_SM and NORM_BWD_CTAS_PER_SM CTAs of 192 threads
// (1536 columns) share an SM; all there are where one CTA has the SM to itself.
template <int NV> constexpr int FWD_REGS = NV == 1 ? 80 : 128;
template <int NV> constexpr int BWD_REGS = NV == 1 ? 96 : 128;

template <typename TX, typename TY, int NV>
__global__ void __maxnreg__(FWD_REGS<NV>) norm_fwd_kernel(const NormArgs a, int team_threads, int stages, bool al)
{
    __shared__ __align__(16) float red[MAX_TEAMS][2][2][16];
    __shared__ uint64_t full[MAX_TEAMS * MAX_STAGES];
    __shared__ int abort_word;
    extern __shared__ __align__(16) uint8_t smem[];
    Team team = make_team(red, team_threads);
    const int teams = blockDim.x / team_threads;
    const int ti = threadIdx.x / team_threads, tt = threadIdx.x - ti * team_threads;
    const int col0 = tt * 8, stride = team_threads * 8, dim = a.dim;
    const long long r0 = blockIdx.x * a.rows_per_cta;
    const long long r1 = min(a.rows, r0 + a.rows_per_cta);
    if (threadIdx.x == 0) {
        for (int i = 0; i < teams * MAX_STAGES; ++i) mbar_init(&full[i], 1);
        abort_word = 0;
        fence_mbar_init();
    }
    __syncthreads();
    volatile int* abort_flag = &abort_word;
    const void* src[2] = {a.x, a.y};
    const int esize[2] = {sizeof(TX), sizeof(TY)};
    Rows<2> in = make_rows<2>(src, esize, dim, smem, full, stages, ti, tt, teams, r1);
    in.start(r0 + ti);

    const float inv = 1.0f / static_cast<float>(dim);
    int mine[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) mine[k] = min(max(dim - (col0 + k * stride), 0), 8);
    long long group_end = 0;  // rows below it share the vectors in registers
    float g2[NV][8], b2[NV][8], s1[NV][8], t1[NV][8];  // r = alpha x + m g2 + b2, h = n s1 + t1
    for (long long row = r0 + ti; row < r1; row += teams) {
        Raw8<TX> xr[NV];
        Raw8<TY> yr[NV];
        if (stages) {
            bool ok;
            const uint8_t* st = in.wait(abort_flag, a.err, &ok);
            if (!ok) {
                in.drain();
                return;  // the whole team: it waits on one barrier
            }
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                xr[k] = stage_raw<TX>(st, in.at[0], col0 + k * stride, dim);
                if (a.y) yr[k] = stage_raw<TY>(st, in.at[1], col0 + k * stride, dim);
            }
            team.sync();
            in.release(row);
        } else {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                xr[k] = load_raw(static_cast<const TX*>(a.x) + row * dim, col0 + k * stride, dim, al);
                if (a.y) yr[k] = load_raw(static_cast<const TY*>(a.y) + row * dim, col0 + k * stride, dim, al);
            }
        }
        if (row >= group_end) {
            const long long group = row / a.per_group, g = group * dim;
            group_end = (group + 1) * a.per_group;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = col0 + k * stride;
                float p[8];
                load_param(a.v.gate ? a.v.gate + g : nullptr, col, dim, al, 1.f, p);
                load_param(a.v.post_w, col, dim, al, 1.f, g2[k]);
                load_param(a.v.post_b, col, dim, al, 0.f, b2[k]);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    g2[k][i] *= p[i];
                    b2[k][i] *= p[i];
                }
                load_param(a.v.scale ? a.v.scale + g : nullptr, col, dim, al, 0.f, p);
                load_param(a.v.pre_w, col, dim, al, 1.f, s1[k]);
                load_param(a.v.pre_b, col, dim, al, 0.f, t1[k]);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    s1[k][i] *= 1.f + p[i];
                    t1[k][i] *= 1.f + p[i];
                }
                load_param(a.v.shift ? a.v.shift + g : nullptr, col, dim, al, 0.f, p);
#pragma unroll
                for (int i = 0; i < 8; ++i) t1[k][i] += p[i];
            }
        }
        float t[NV][8];
        if (a.y) {
#pragma unroll
            for (int k = 0; k < NV; ++k) unpack8(yr[k], t[k]);
            if (a.post != NORM_NONE) normalise<NV>(team, t, a.post, inv, mine, a.eps);
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float x[8];
            unpack8(xr[k], x);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                if (a.y) {
                    ffma2(x[i], x[i + 1], x[i], x[i + 1], a.alpha, a.alpha, b2[k][i], b2[k][i + 1]);
                    ffma2(t[k][i], t[k][i + 1], g2[k][i], g2[k][i + 1], t[k][i], t[k][i + 1], x[i], x[i + 1]);
                } else {
                    t[k][i] = a.alpha * x[i];
                    t[k][i + 1] = a.alpha * x[i + 1];
                }
            }
            if (a.r) store8(static_cast<TX*>(a.r) + row * dim, col0 + k * stride, dim, al, t[k]);
        }
        if (!a.h) continue;
        normalise<NV>(team, t, a.pre, inv, mine, a.eps);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
#pragma unroll
            for (int i = 0; i < 8; i += 2)
                ffma2(t[k][i], t[k][i + 1], t[k][i], t[k][i + 1], s1[k][i], s1[k][i + 1], t1[k][i], t1[k][i + 1]);
            store8(static_cast<TY*>(a.h) + row * dim, col0 + k * stride, dim, al, t[k]);
        }
    }
}

// BIAS: the post norm has a bias, or its gradient is wanted; without it b2 and A3 (sum dr') need
// no registers.
template <typename TX, typename TY, int NV, bool BIAS>
__global__ void __maxnreg__(BWD_REGS<NV>) norm_bwd_kernel(const NormArgs a, int team_threads, int stages, bool al)
{
    __shared__ __align__(16) float red[MAX_TEAMS][2][2][16];
    __shared__ uint64_t full[MAX_TEAMS * MAX_STAGES];
    __shared__ int abort_word;
    extern __shared__ __align__(16) uint8_t smem[];  // the rings, then [teams - 1][dim8] floats
    Team team = make_team(red, team_threads);
    const int teams = blockDim.x / team_threads;
    const int ti = threadIdx.x / team_threads, tt = threadIdx.x - ti * team_threads;
    const int col0 = tt * 8, stride = team_threads * 8, dim = a.dim;
    const int dim8 = (dim + 7) & ~7;
    const long long r0 = blockIdx.x * a.rows_per_cta;
    const long long r1 = min(a.rows, r0 + a.rows_per_cta);
    const float inv = 1.0f / static_cast<float>(dim);
    if (threadIdx.x == 0) {
        for (int i = 0; i < teams * MAX_STAGES; ++i) mbar_init(&full[i], 1);
        abort_word = 0;
        fence_mbar_init();
    }
    __syncthreads();
    volatile int* abort_flag = &abort_word;
    const void* src[4] = {a.x, a.y, a.dr, a.dh};
    const int esize[4] = {sizeof(TX), sizeof(TY), sizeof(TX), sizeof(TY)};
    Rows<4> in = make_rows<4>(src, esize, dim, smem, full, stages, ti, tt, teams, r1);
    in.start(r0 + ti);
    float* fold = reinterpret_cast<float*>(smem + static_cast<size_t>(teams) * stages * in.stage_bytes);
    float* part_w = a.part_w + static_cast<long long>(blockIdx.x) * 4 * dim8;

    int mine[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) mine[k] = min(max(dim - (col0 + k * stride), 0), 8);
    long long row = r0 + ti;
    bool broken = false;
    for (long long seg = r0; seg < r1;) {
        const long long gi = seg / a.per_group;
        const long long seg_end = min(r1, (gi + 1) * a.per_group);
        const long long g = gi * dim;
        float g2[NV][8], b2[BIAS ? NV : 1][8], s1[NV][8];  // u gate = m g2 + b2; dn = dh s1
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int col = col0 + k * stride;
            float p[8];
            load_param(a.v.gate ? a.v.gate + g : nullptr, col, dim, al, 1.f, p);
            load_param(a.v.post_w, col, dim, al, 1.f, g2[k]);
#pragma unroll
            for (int i = 0; i < 8; ++i) g2[k][i] *= p[i];
            if constexpr (BIAS) {
                load_param(a.v.post_b, col, dim, al, 0.f, b2[k]);
#pragma unroll
                for (int i = 0; i < 8; ++i) b2[k][i] *= p[i];
            }
            load_param(a.v.scale ? a.v.scale + g : nullptr, col, dim, al, 0.f, p);
            load_param(a.v.pre_w, col, dim, al, 1.f, s1[k]);
#pragma unroll
            for (int i = 0; i < 8; ++i) s1[k][i] *= 1.f + p[i];
        }
        float A[4][NV][8];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) A[j][k][i] = 0.f;
        for (; row < seg_end && !broken; row += teams) {
            const long long at = row * dim;
            const TX *x_row = static_cast<const TX*>(a.x) + at, *dr_row = static_cast<const TX*>(a.dr) + at;
            const TY *y_row = static_cast<const TY*>(a.y) + at, *dh_row = static_cast<const TY*>(a.dh) + at;
            if (stages) {
                bool ok;
                const uint8_t* st = in.wait(abort_flag, a.err, &ok);
                if (!ok) {
                    in.drain();
                    broken = true;
                    break;
                }
                x_row = reinterpret_cast<const TX*>(st + in.at[0]);
                y_row = reinterpret_cast<const TY*>(st + in.at[1]);
                dr_row = reinterpret_cast<const TX*>(st + in.at[2]);
                dh_row = reinterpret_cast<const TY*>(st + in.at[3]);
            }
            float m[NV][8], n[NV][8], d[NV][8];
            float rs1 = 1.f, rs2 = 1.f;
            // forward again: m = post(y), n = pre(r)
            if (a.y) {
#pragma unroll
                for (int k = 0; k < NV; ++k) unpack8(load_raw(y_row, col0 + k * stride, dim, al), m[k]);
                if (a.post != NORM_NONE) rs2 = normalise<NV>(team, m, a.post, inv, mine, a.eps);
            }
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                unpack8(load_raw(x_row, col0 + k * stride, dim, al), n[k]);
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    if constexpr (BIAS)
                        ffma2(n[k][i], n[k][i + 1], n[k][i], n[k][i + 1], a.alpha, a.alpha, b2[k][i], b2[k][i + 1]);
                    else
                        fmul2(n[k][i], n[k][i + 1], a.alpha, a.alpha);
                    if (a.y)
                        ffma2(n[k][i], n[k][i + 1], g2[k][i], g2[k][i + 1], m[k][i], m[k][i + 1], n[k][i], n[k][i + 1]);
                }
            }
            float q1 = 0.f, q2 = 0.f;
            if (a.dh) {
                rs1 = normalise<NV>(team, n, a.pre, inv, mine, a.eps);
                float q3 = 0.f, q4 = 0.f;
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    unpack8(load_raw(dh_row, col0 + k * stride, dim, al), d[k]);
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        fadd2_acc(A[0][k][i], A[0][k][i + 1], d[k][i], d[k][i + 1]);
                        ffma2(A[1][k][i], A[1][k][i + 1], d[k][i], d[k][i + 1], n[k][i], n[k][i + 1], A[1][k][i], A[1][k][i + 1]);
                        fmul2(d[k][i], d[k][i + 1], s1[k][i], s1[k][i + 1]);
                        fadd2_acc(q1, q3, d[k][i], d[k][i + 1]);
                        ffma2(q2, q4, d[k][i], d[k][i + 1], n[k][i], n[k][i + 1], q2, q4);
                    }
                }
                q1 += q3;
                q2 += q4;
                team.sum(q1, q2);
                // minus rs1 times the means
                q1 = a.pre == NORM_LAYER ? q1 * inv * -rs1 : 0.f;
                q2 *= inv * -rs1;
            }
            // dr' in d
            float p1 = 0.f, p2 = 0.f, p3 = 0.f, p4 = 0.f;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = col0 + k * stride;
                float p[8] = {};
                if (a.dr) unpack8(load_raw(dr_row, col, dim, al), p);
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    if (a.dh) {
                        fadd2_acc(p[i], p[i + 1], q1, q1);
                        ffma2(p[i], p[i + 1], d[k][i], d[k][i + 1], rs1, rs1, p[i], p[i + 1]);
                        ffma2(d[k][i], d[k][i + 1], n[k][i], n[k][i + 1], q2, q2, p[i], p[i + 1]);
                    } else {
                        d[k][i] = p[i];
                        d[k][i + 1] = p[i + 1];
                    }
                }
                if (a.dx) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) p[i] = a.alpha * d[k][i];
                    store8(static_cast<TX*>(a.dx) + at, col, dim, al, p);
                }
                if (a.y) {
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        if constexpr (BIAS) fadd2_acc(A[2][k][i], A[2][k][i + 1], d[k][i], d[k][i + 1]);
                        ffma2(A[3][k][i], A[3][k][i + 1], d[k][i], d[k][i + 1], m[k][i], m[k][i + 1], A[3][k][i], A[3][k][i + 1]);
                        fmul2(d[k][i], d[k][i + 1], g2[k][i], g2[k][i + 1]);  // dm (zero past dim, as g2 is)
                        fadd2_acc(p1, p3, d[k][i], d[k][i + 1]);
                        ffma2(p2, p4, d[k][i], d[k][i + 1], m[k][i], m[k][i + 1], p2, p4);
                    }
                }
            }
            if (stages) {
                team.sync();
                in.release(row);
            }
            if (!a.dy) continue;
            if (a.post != NORM_NONE) {
                p1 += p3;
                p2 += p4;
                team.sum(p1, p2);
                p1 = a.post == NORM_LAYER ? p1 * inv * -rs2 : 0.f;
                p2 *= inv * -rs2;
#pragma unroll
                for (int k = 0; k < NV; ++k)
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        ffma2(d[k][i], d[k][i + 1], d[k][i], d[k][i + 1], rs2, rs2, p1, p1);
                        ffma2(d[k][i], d[k][i + 1], m[k][i], m[k][i + 1], p2, p2, d[k][i], d[k][i + 1]);
                    }
            }
#pragma unroll
            for (int k = 0; k < NV; ++k) store8(static_cast<TY*>(a.dy) + at, col0 + k * stride, dim, al, d[k]);
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
                    for (int k = 0; k < NV; ++k) {
                        const int col = col0 + k * stride;
                        if (col < dim8) {
                            float4* f = reinterpret_cast<float4*>(fold + (ti - 1) * dim8 + col);
                            f[0] = make_float4(A[j][k][0], A[j][k][1], A[j][k][2], A[j][k][3]);
                            f[1] = make_float4(A[j][k][4], A[j][k][5], A[j][k][6], A[j][k][7]);
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
                        float4* to = reinterpret_cast<float4*>(slot + j * dim8 + col);
                        to[0] = make_float4(A[j][k][0], A[j][k][1], A[j][k][2], A[j][k][3]);
                        to[1] = make_float4(A[j][k][4], A[j][k][5], A[j][k][6], A[j][k][7]);
                        if (a.weights) {  // times 1 + scale, or the gate
                            const float* f = j < 2 ? a.v.scale : a.v.gate;
                            float p[8];
                            load_param(f ? f + g : nullptr, col, dim, al, j < 2 ? 0.f : 1.f, p);
                            float4* w = reinterpret_cast<float4*>(part_w + j * dim8 + col);
                            float o[8] = {};
                            if (seg > r0) {
                                const float4 lo = w[0], hi = w[1];
                                o[0] = lo.x; o[1] = lo.y; o[2] = lo.z; o[3] = lo.w;
                                o[4] = hi.x; o[5] = hi.y; o[6] = hi.z; o[7] = hi.w;
                            }
#pragma unroll
                            for (int i = 0; i < 8; ++i) o[i] = fmaf(j < 2 ? 1.f + p[i] : p[i], A[j][k][i], o[i]);
                            w[0] = make_float4(o[0], o[1], o[2], o[3]);
                            w[1] = make_float4(o[4], o[5], o[6], o[7]);
                        }
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

// How a call's rows are taken: threads of a team and groups of 8 a thread (as few as 256
// threads allow, then two, then four: dim <= 16384 = 512 * 4 * 8), teams of a CTA, stages of
// the ring (as many as leave `ctas` CTAs an SM; fewer than two are not worth a ring).
struct NormPlan {
    int nv, threads, teams, stages;
    size_t smem;
};

NormPlan plan_of(const NormArgs& a, size_t row_bytes, int ctas, bool fold)
{
    NormPlan p;
    const int vecs = (a.dim + 7) / 8;
    p.nv = vecs <= 256 ? 1 : (vecs <= 1024 ? 2 : 4);
    p.threads = ((vecs + p.nv - 1) / p.nv + 31) / 32 * 32;
    p.teams = p.nv > 1 ? 1 : std::min(MAX_TEAMS, 256 / p.threads);
    const size_t extra = fold ? static_cast<size_t>(p.teams - 1) * vecs * 8 * sizeof(float) : 0;
    const size_t room = (220u * 1024u) / ctas - 2048 - extra;
    const int fit = static_cast<int>(std::min<size_t>(room / (row_bytes * p.teams), MAX_STAGES));
    p.stages = a.dim % 8 == 0 && fit >= 2 ? fit : 0;
    p.smem = p.stages * row_bytes * p.teams + extra;
    return p;
}

// Dynamic shared memory past the default limit (48 KB with the kernel's static part), asked for
// once a device: the most that a plan uses.
template <auto KERNEL>
cudaError_t allow_smem(size_t bytes)
{
    if (bytes <= 40 * 1024) return cudaSuccess;
    static std::atomic<bool> set[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64 && set[dev].load(std::memory_order_acquire)) return cudaSuccess;
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024);
    if (e == cudaSuccess && dev >= 0 && dev < 64) set[dev].store(true, std::memory_order_release);
    return e;
}

template <typename TX, typename TY, int NV>
cudaError_t launch_fwd(NormArgs a, const NormPlan& p, cudaStream_t s)
{
    cudaError_t e = allow_smem<norm_fwd_kernel<TX, TY, NV>>(p.smem);
    if (e != cudaSuccess) return e;
    // CTAs for all SMs' worth of resident ones; rows are spread evenly over them
    const long long most = 148ll * (NV == 1 ? NORM_FWD_CTAS_PER_SM : 1);
    const long long per = std::max<long long>(p.teams, (a.rows + most - 1) / most);
    a.rows_per_cta = (per + p.teams - 1) / p.teams * p.teams;
    const unsigned grid = static_cast<unsigned>((a.rows + a.rows_per_cta - 1) / a.rows_per_cta);
    norm_fwd_kernel<TX, TY, NV><<<grid, p.threads * p.teams, p.smem, s>>>(a, p.threads, p.stages, a.dim % 8 == 0);
    return cudaGetLastError();
}

template <typename TX, typename TY, int NV>
cudaError_t launch_bwd(const NormArgs& a, const NormPlan& p, cudaStream_t s)
{
    const bool bias = a.v.post_b || a.dpost_b;
    cudaError_t e = bias ? allow_smem<norm_bwd_kernel<TX, TY, NV, true>>(p.smem) : allow_smem<norm_bwd_kernel<TX, TY, NV, false>>(p.smem);
    if (e != cudaSuccess) return e;
    if (bias)
        norm_bwd_kernel<TX, TY, NV, true><<<a.n_cta, p.threads * p.teams, p.smem, s>>>(a, p.threads, p.stages, a.dim % 8 == 0);
    else
        norm_bwd_kernel<TX, TY, NV, false><<<a.n_cta, p.threads * p.teams, p.smem, s>>>(a, p.threads, p.stages, a.dim % 8 == 0);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (!a.dgate && !a.dscale && !a.dshift && !a.weights) return cudaSuccess;
    const long long groups = (a.rows + a.per_group - 1) / a.per_group;
    const long long items = (groups + FIN_GROUPS - 1) / FIN_GROUPS + (a.weights ? 1 : 0);
    norm_bwd_finish_kernel<<<dim3((a.dim + FIN_COLS - 1) / FIN_COLS, static_cast<unsigned>(std::min<long long>(items, 65535))),
                             FIN_COLS * FIN_ROWS, 0, s>>>(a, groups);
    return cudaGetLastError();
}

template <bool BWD, typename TX, typename TY>
cudaError_t launch_one(const NormArgs& a, cudaStream_t s)
{
    const size_t x = static_cast<size_t>(a.dim) * sizeof(TX), y = static_cast<size_t>(a.dim) * sizeof(TY);
    const size_t row = BWD ? x + (a.y ? y : 0) + (a.dr ? x : 0) + (a.dh ? y : 0) : x + (a.y ? y : 0);
    const bool small = a.dim <= 2048;
    const NormPlan p = plan_of(a, row, small ? (BWD ? NORM_BWD_CTAS_PER_SM : NORM_FWD_CTAS_PER_SM) : 1, BWD);
    if constexpr (BWD) {
        if (p.nv == 1) return launch_bwd<TX, TY, 1>(a, p, s);
        return p.nv == 2 ? launch_bwd<TX, TY, 2>(a, p, s) : launch_bwd<TX, TY, 4>(a, p, s);
    } else {
        if (p.nv == 1) return launch_fwd<TX, TY, 1>(a, p, s);
        return p.nv == 2 ? launch_fwd<TX, TY, 2>(a, p, s) : launch_fwd<TX, TY, 4>(a, p, s);
    }
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
