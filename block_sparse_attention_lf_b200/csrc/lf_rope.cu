// lf_rope.cu -- rotary positions of up to three tensors in one launch, with the change of
// layout between a projection's token-major output and the head-major tensors of an HSA
// call, and the gradient.
//
// A pair (a, b) of a head's rotated elements -- (2i, 2i+1) in the interleaved layout,
// (i, i + rot/2) in the half layout -- turns by theta = position * frequency:
//   a' = m (a cos - b sin),  b' = m (a sin + b cos),
// and its gradient is the same with -theta. Elements past rot_dim, and tensors with
// rotate = 0 (a value projection that only moves), are copied.
//
// The angle. Frequencies arrive as revolutions per position in fp64, so the whole turns
// of a far position are dropped exactly (t - rint(t)) before anything is rounded to fp32;
// the remaining half turn goes to sincospif. A thread computes the angles of one token's
// unit (a 16-byte vector, or two half a head apart) once and uses them for every head
// it takes, so the fp64 work is spread over heads * tensors vectors.
//
// Memory-bound: each element is read and written once. A unit is one 16-byte vector
// wherever pointers, strides and spans allow it; otherwise one pair at a time.
#include "lf_rope.h"
#include "lf_types.cuh"

namespace lf {
namespace {

constexpr int ROPE_THREADS = 256;

__device__ __forceinline__ void turn_of(double turns, int pos, float& c, float& s)
{
    double t = static_cast<double>(pos) * turns;
    t -= rint(t);
    sincospif(2.0f * static_cast<float>(t), &s, &c);
}

// Elements of a unit and how many units a head has: rotated ones first, then copied ones.
// VEC: a unit is a 16-byte vector (interleaved, copied) or two of them half a head's rotated
// part apart (half). Otherwise a pair, or one copied element.
template <typename T, bool HALF, bool VEC>
struct RopeUnits {
    static constexpr int E = VEC ? VEC_ELEMS<T> : 1;              // elements of a load
    static constexpr int PAIRS = HALF ? E : (VEC ? E / 2 : 1);    // pairs of a rotated unit
    static constexpr int SPAN = HALF ? E : (VEC ? E : 2);         // elements between rotated units' starts
    __host__ __device__ static int rotated(int rot) { return (HALF ? rot / 2 : rot) / SPAN; }
    __host__ __device__ static int all(int D, int rot) { return rotated(rot) + (D - rot) / E; }
};

template <typename T, int E>
__device__ __forceinline__ void load_elems(float (&v)[E], const T* p)
{
    if constexpr (E == 1)
        v[0] = to_f32(*p);
    else
        unpack<T>(*reinterpret_cast<const uint4*>(p), v);
}

template <typename T, int E>
__device__ __forceinline__ void store_elems(T* p, const float (&v)[E])
{
    if constexpr (E == 1)
        *p = from_f32<T>(v[0]);
    else
        *reinterpret_cast<uint4*>(p) = pack<T>(v);
}

// The two operands of a rotated unit: in the half layout two loads, interleaved one load
// whose even and odd elements are the pair's members.
template <typename T, bool HALF, bool VEC>
__global__ void __launch_bounds__(ROPE_THREADS) rope_kernel(const __grid_constant__ RopeArgs a)
{
    using U = RopeUnits<T, HALF, VEC>;
    constexpr int E = U::E, NP = U::PAIRS;
    constexpr int UNROLL = 4;  // heads loaded before any is stored
    const int rot_units = U::rotated(a.rot_dim), units = U::all(a.head_dim, a.rot_dim);
    const unsigned item = blockIdx.x * ROPE_THREADS + threadIdx.x;
    const unsigned bt = item / units;
    if (bt >= static_cast<unsigned>(a.batch) * a.tokens) return;
    const int u = item - bt * units;
    const int b = bt / a.tokens, t = bt - b * a.tokens;
    const bool turned = u < rot_units;
    const int e0 = turned ? u * U::SPAN : a.rot_dim + (u - rot_units) * E;  // first element
    const int half = a.rot_dim >> 1;

    float c[NP], s[NP];
    if (turned) {
        const int* pos = a.positions + b * a.pos_batch + static_cast<long long>(t) * a.n_axes;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int p = u * NP + i;
            const int ax = (p >= a.axis_end[0]) + (p >= a.axis_end[1]);
            turn_of(a.turns[p], __ldg(pos + ax), c[i], s[i]);
            c[i] *= a.amplitude;
            s[i] *= a.backward ? -a.amplitude : a.amplitude;
        }
    }
    int h0 = blockIdx.y * a.heads_per_thread;
    int left = a.heads_per_thread;
    for (int k = 0; k < a.n_io && left > 0; ++k) {
        const RopeIo& io = a.io[k];
        if (h0 >= io.heads) {
            h0 -= io.heads;
            continue;
        }
        const int n = min(left, io.heads - h0);
        const T* x = static_cast<const T*>(io.x) + b * io.xs[0] + h0 * io.xs[1] + t * io.xs[2] + e0;
        T* o = static_cast<T*>(io.out) + b * io.os[0] + h0 * io.os[1] + t * io.os[2] + e0;
        const bool rotate = turned && io.rotate;
        for (int h = 0; h < n; h += UNROLL) {
            float va[UNROLL][E], vb[UNROLL][E];  // vb: the second operand (half layout, or the scalar pair's)
#pragma unroll
            for (int i = 0; i < UNROLL; ++i)
                if (h + i < n) {
                    const T* p = x + (h + i) * io.xs[1];
                    load_elems<T, E>(va[i], p);
                    if constexpr (HALF) {
                        if (turned) load_elems<T, E>(vb[i], p + half);
                    } else if constexpr (!VEC) {
                        if (turned) load_elems<T, E>(vb[i], p + 1);
                    }
                }
#pragma unroll
            for (int i = 0; i < UNROLL; ++i)
                if (h + i < n) {
                    T* p = o + (h + i) * io.os[1];
                    if (rotate) {
                        if constexpr (HALF || !VEC) {
#pragma unroll
                            for (int j = 0; j < E; ++j) {
                                const float xa = va[i][j], xb = vb[i][j];
                                va[i][j] = xa * c[j] - xb * s[j];
                                vb[i][j] = xa * s[j] + xb * c[j];
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < NP; ++j) {
                                const float xa = va[i][2 * j], xb = va[i][2 * j + 1];
                                va[i][2 * j] = xa * c[j] - xb * s[j];
                                va[i][2 * j + 1] = xa * s[j] + xb * c[j];
                            }
                        }
                    }
                    store_elems<T, E>(p, va[i]);
                    if constexpr (HALF) {
                        if (turned) store_elems<T, E>(p + half, vb[i]);
                    } else if constexpr (!VEC) {
                        if (turned) store_elems<T, E>(p + 1, vb[i]);
                    }
                }
        }
        left -= n;
        h0 = 0;
    }
}

template <typename T, bool HALF, bool VEC>
cudaError_t launch_t(RopeArgs& a, cudaStream_t s)
{
    const long long items = static_cast<long long>(a.batch) * a.tokens * RopeUnits<T, HALF, VEC>::all(a.head_dim, a.rot_dim);
    int heads = 0;
    for (int k = 0; k < a.n_io; ++k) heads += a.io[k].heads;
    // Heads are spread over threads until the machine is full: 148 SMs * 1024 threads.
    const long long want = (148ll * 1024 + items - 1) / items;
    const int groups = static_cast<int>(want < 1 ? 1 : (want > heads ? heads : want));
    a.heads_per_thread = (heads + groups - 1) / groups;
    const dim3 grid(static_cast<unsigned>((items + ROPE_THREADS - 1) / ROPE_THREADS),
                    static_cast<unsigned>((heads + a.heads_per_thread - 1) / a.heads_per_thread));
    rope_kernel<T, HALF, VEC><<<grid, ROPE_THREADS, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_l(RopeArgs& a, bool half_layout, bool vec, cudaStream_t s)
{
    if (half_layout) return vec ? launch_t<T, true, true>(a, s) : launch_t<T, true, false>(a, s);
    return vec ? launch_t<T, false, true>(a, s) : launch_t<T, false, false>(a, s);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a0, int dtype, bool half_layout, bool vec, cudaStream_t s)
{
    RopeArgs a = a0;
    if (dtype == DT_F32) return launch_l<float>(a, half_layout, vec, s);
    if (dtype == DT_BF16) return launch_l<__nv_bfloat16>(a, half_layout, vec, s);
    return launch_l<__half>(a, half_layout, vec, s);
}

}  // namespace lf
