// lf_norm_rows.cuh -- what the forward and gradient kernels of the gated residual norms share:
// rows of 8-element groups in registers, team sums, the ring of rows copied ahead, launch plans.
#pragma once

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

// A group of eight as four packed pairs: their products and sums are one instruction a pair.
struct Vec8 {
    float2 v[4];
};

template <typename T>
__device__ __forceinline__ Vec8 unpack8(const Raw8<T>& r)
{
    Vec8 o;
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) {
        float t[VEC_ELEMS<T>];
        unpack<T>(r.v[i], t);
#pragma unroll
        for (int j = 0; j < VEC_ELEMS<T>; j += 2) o.v[(i * VEC_ELEMS<T> + j) / 2] = make_float2(t[j], t[j + 1]);
    }
    return o;
}

template <typename T>
__device__ __forceinline__ void store8(T* row, int col, int dim, bool al, const Vec8& x)
{
    if (al) {
        if (col < dim) {
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) {
                float t[VEC_ELEMS<T>];
#pragma unroll
                for (int j = 0; j < VEC_ELEMS<T>; j += 2) {
                    t[j] = x.v[(i * VEC_ELEMS<T> + j) / 2].x;
                    t[j + 1] = x.v[(i * VEC_ELEMS<T> + j) / 2].y;
                }
                *reinterpret_cast<uint4*>(row + col + i * VEC_ELEMS<T>) = pack<T>(t);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (col + 2 * i < dim) row[col + 2 * i] = from_f32<T>(x.v[i].x);
            if (col + 2 * i + 1 < dim) row[col + 2 * i + 1] = from_f32<T>(x.v[i].y);
        }
    }
}

__device__ __forceinline__ Vec8 mul(const Vec8& a, const Vec8& b)
{
    Vec8 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.v[i] = __fmul2_rn(a.v[i], b.v[i]);
    return o;
}
__device__ __forceinline__ Vec8 mul(const Vec8& a, float b)
{
    Vec8 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.v[i] = __fmul2_rn(a.v[i], make_float2(b, b));
    return o;
}
__device__ __forceinline__ Vec8 add(const Vec8& a, const Vec8& b)
{
    Vec8 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.v[i] = __fadd2_rn(a.v[i], b.v[i]);
    return o;
}
__device__ __forceinline__ Vec8 add(const Vec8& a, float b)
{
    Vec8 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.v[i] = __fadd2_rn(a.v[i], make_float2(b, b));
    return o;
}
// a b + c
__device__ __forceinline__ Vec8 fma(const Vec8& a, const Vec8& b, const Vec8& c)
{
    Vec8 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.v[i] = __ffma2_rn(a.v[i], b.v[i], c.v[i]);
    return o;
}
__device__ __forceinline__ Vec8 fma(const Vec8& a, float b, const Vec8& c)
{
    Vec8 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.v[i] = __ffma2_rn(a.v[i], make_float2(b, b), c.v[i]);
    return o;
}
// s += the eight elements of a, of a b
__device__ __forceinline__ void acc(float2& s, const Vec8& a)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) s = __fadd2_rn(s, a.v[i]);
}
__device__ __forceinline__ void acc(float2& s, const Vec8& a, const Vec8& b)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) s = __ffma2_rn(a.v[i], b.v[i], s);
}
__device__ __forceinline__ Vec8 fill8(float x)
{
    Vec8 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.v[i] = make_float2(x, x);
    return o;
}
// The first n of the eight, zeros behind them.
__device__ __forceinline__ Vec8 head8(const Vec8& a, int n)
{
    Vec8 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.v[i] = make_float2(2 * i < n ? a.v[i].x : 0.f, 2 * i + 1 < n ? a.v[i].y : 0.f);
    return o;
}

// Eight values of a vector (`other` where it is absent, zeros past dim).
__device__ __forceinline__ Vec8 load_param(const float* p, int col, int dim, bool al, float other)
{
    return p ? unpack8(load_raw(p, col, dim, al)) : head8(fill8(other), dim - col);
}

// A vector of the CTA's in shared memory: the first fours of all eights, then the second fours, so
// that neighbouring threads meet different banks.
__device__ __forceinline__ void split_store(float* p, int col, int dim8, const Vec8& x)
{
    *reinterpret_cast<float4*>(p + col / 2) = make_float4(x.v[0].x, x.v[0].y, x.v[1].x, x.v[1].y);
    *reinterpret_cast<float4*>(p + dim8 / 2 + col / 2) = make_float4(x.v[2].x, x.v[2].y, x.v[3].x, x.v[3].y);
}

__device__ __forceinline__ Vec8 split_load(const float* p, int col, int dim8)
{
    const float4 a = *reinterpret_cast<const float4*>(p + col / 2), b = *reinterpret_cast<const float4*>(p + dim8 / 2 + col / 2);
    Vec8 o;
    o.v[0] = make_float2(a.x, a.y);
    o.v[1] = make_float2(a.z, a.w);
    o.v[2] = make_float2(b.x, b.y);
    o.v[3] = make_float2(b.z, b.w);
    return o;
}

constexpr int MAX_TEAMS = 12, MAX_STAGES = 4;

// Row sums over a team of whole warps, in a fixed order. Consecutive calls alternate between two
// buffers, so one barrier a call is enough; unused places of a buffer stay zero.
struct Team {
    float (*red)[2][16];  // this team's [2 buffers][2 values][warps]
    int warps, warp, lane, bar, threads, phase;

    __device__ __forceinline__ float gather(int which)
    {
        const float4* f = reinterpret_cast<const float4*>(red[phase][which]);
        const float4 u = f[0];
        float s = (u.x + u.y) + (u.z + u.w);
        if (warps <= 4) return s;
        const float4 v = f[1];
        s += (v.x + v.y) + (v.z + v.w);
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

__device__ __forceinline__ void copy16_async(void* dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// How a thread meets its team's rows: `col0` its first column, `stride` columns from one of its
// groups of eight to the next, `step` elements from one of the team's rows to the next.
// Where every thread's every group lies within dim (FULL, chosen at the launch) no column is tested.
struct Place {
    int col0, stride, dim, threads, stages;
    long long step;
    bool al;
};

// One tensor's rows, read. A thread copies exactly what it will read ahead into a ring of stages in
// shared memory, so no barrier and no other thread is involved; where stages is 0 rows are loaded
// when asked for.
template <typename T, int NV, bool FULL>
struct Source {
    const T* ahead;  // the thread's column of the next row to copy (or to load)
    uint32_t at;     // offset in a stage, the thread's 16 bytes included
    bool on;

    __device__ __forceinline__ void init(const void* base, long long row, const Place& p, uint32_t* stage_bytes, int team_thread)
    {
        on = base != nullptr;
        ahead = static_cast<const T*>(base) + row * p.dim + p.col0;
        at = *stage_bytes + team_thread * 16;
        if (on) *stage_bytes += p.threads * NV * 8 * static_cast<uint32_t>(sizeof(T));
    }

    __device__ __forceinline__ void copy(uint8_t* stage, const Place& p)
    {
        if (!on) return;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (!FULL && p.col0 + k * p.stride >= p.dim) continue;
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
                copy16_async(stage + at + (k * static_cast<int>(sizeof(T) / 2) + i) * p.threads * 16,
                             ahead + k * p.stride + i * VEC_ELEMS<T>);
        }
        ahead += p.step;
    }

    __device__ __forceinline__ Vec8 get(const uint8_t* stage, int k, const Place& p) const
    {
        if (!FULL && p.stages == 0) return unpack8(load_raw(ahead - p.col0, p.col0 + k * p.stride, p.dim, p.al));
        Raw8<T> r;
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
            r.v[i] = FULL || p.col0 + k * p.stride < p.dim
                         ? *reinterpret_cast<const uint4*>(stage + at + (k * static_cast<int>(sizeof(T) / 2) + i) * p.threads * 16)
                         : make_uint4(0u, 0u, 0u, 0u);
        return unpack8(r);
    }

    __device__ __forceinline__ void done(const Place& p)
    {
        if (!FULL && p.stages == 0) ahead += p.step;
    }
};

// One tensor's rows, written.
template <typename T, int NV, bool FULL>
struct Sink {
    T* to;
    bool on;

    __device__ __forceinline__ void init(void* base, long long row, const Place& p)
    {
        on = base != nullptr;
        to = static_cast<T*>(base) + row * p.dim + p.col0;
    }
    __device__ __forceinline__ void put(int k, const Vec8& x, const Place& p)
    {
        if (!on) return;
        if (FULL) store8(to, k * p.stride, 1 << 30, true, x);
        else store8(to - p.col0, p.col0 + k * p.stride, p.dim, p.al, x);
    }
    __device__ __forceinline__ void done(const Place& p) { to += p.step; }
};

// The ring's turn: `rows` of the team's rows are still to be copied.
struct Ring {
    uint8_t* base;
    uint32_t stage_bytes, slot;
    int rows, stages;

    template <typename... S>
    __device__ __forceinline__ void ask(uint32_t to, const Place& p, S&... s)
    {
        if (rows > 0) {
            --rows;
            (s.copy(base + to, p), ...);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");  // one a row, so that the count of groups tells the row
    }
    template <typename... S>
    __device__ __forceinline__ void start(int team_rows, const Place& p, S&... s)
    {
        rows = team_rows;
        slot = 0;
        for (int i = 0; i < stages - 1; ++i) ask(i * stage_bytes, p, s...);
    }
    // The thread's part of the next row is there; the row stages - 1 further on is asked for.
    template <typename... S>
    __device__ __forceinline__ const uint8_t* next(const Place& p, S&... s)
    {
        if (stages == 0) return nullptr;
        ask(slot == 0 ? (stages - 1) * stage_bytes : slot - stage_bytes, p, s...);
        if (stages == 4) asm volatile("cp.async.wait_group 3;" ::: "memory");
        else if (stages == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
        else asm volatile("cp.async.wait_group 1;" ::: "memory");
        return base + slot;
    }
    __device__ __forceinline__ void done()
    {
        slot += stage_bytes;
        if (slot == stages * stage_bytes) slot = 0;
    }
};

// Normalises the row in place (t -> (t - mean) / deviation) and returns 1 / deviation.
// Elements past dim are zero before and stay zero.
template <int NV, bool FULL>
__device__ __forceinline__ float normalise(Team& team, Vec8 (&t)[NV], int kind, float inv, const Place& p, float eps)
{
    if (kind == NORM_LAYER) {
        float2 a = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < NV; ++k) acc(a, t[k]);
        float s = a.x + a.y;
        team.sum(s);
        const float mean = -s * inv;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            t[k] = add(t[k], mean);
            if (!FULL && p.col0 + k * p.stride + 8 > p.dim) t[k] = head8(t[k], p.dim - p.col0 - k * p.stride);
        }
    }
    float2 b = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < NV; ++k) acc(b, t[k], t[k]);
    float q = b.x + b.y;
    team.sum(q);
    const float rs = rsqrtf(fmaf(q, inv, eps));
#pragma unroll
    for (int k = 0; k < NV; ++k) t[k] = mul(t[k], rs);
    return rs;
}

// How a call's rows are taken: threads of a team, teams of a CTA, stages of the ring (as many as leave `ctas` CTAs an SM; fewer than two are not worth a ring).
struct NormPlan {
    int threads, teams, stages;
    bool wide, full;
    size_t smem;
};

// nv groups of a thread; elem_bytes: of the streams read, together; vectors of a row's length that the
// CTA, and each of its teams, keeps in shared memory beside the rings.
NormPlan plan_of(int dim, int nv, size_t elem_bytes, int cta_threads, int ctas, int vectors, int team_vectors)
{
    NormPlan p;
    const int vecs = (dim + 7) / 8;
    p.threads = ((vecs + nv - 1) / nv + 31) / 32 * 32;
    p.wide = p.threads > cta_threads;
    p.teams = p.wide ? 1 : std::min(MAX_TEAMS, cta_threads / p.threads);
    const size_t extra = static_cast<size_t>(vectors + team_vectors * p.teams) * vecs * 8 * sizeof(float);
    const size_t room = (220u * 1024u) / (p.wide ? 1 : ctas) - 4096 - extra;
    const size_t stage = elem_bytes * p.threads * nv * 8;  // a team's row
    const int fit = static_cast<int>(std::min<size_t>(room / (stage * p.teams), MAX_STAGES));
    p.stages = dim % 8 == 0 && fit >= 2 ? fit : 0;
    p.full = p.stages > 0 && dim == p.threads * nv * 8;
    p.smem = p.stages * stage * p.teams + extra;
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

// Calls f with the element types of x and y as two values.
template <typename F>
cudaError_t with_types(int xd, int yd, F f)
{
    if (xd == DT_BF16) return f(__nv_bfloat16(), __nv_bfloat16());
    if (xd == DT_F16) return f(__half(), __half());
    if (yd == DT_BF16) return f(float(), __nv_bfloat16());
    if (yd == DT_F16) return f(float(), __half());
    return f(float(), float());
}

}  // namespace
}  // namespace lf
