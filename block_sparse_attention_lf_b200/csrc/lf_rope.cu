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
// Memory-bound: each element is read and written once (32760 tokens of 12 x 128 bf16, 201 MB:
// 34.5 us, 5.8 TB/s). A unit is the widest vector (16, 8, 4 or
// 2 bytes) that pointers, strides and spans allow; a thread asks for several heads' units before
// it forms the angles, which take longer than a head's arithmetic, and for the next heads' before
// it stores these. Frequencies are staged in shared memory: lanes need different ones, which the
// constant bank would serve one by one.
#include "lf_rope.h"
#include "lf_types.cuh"

namespace lf {
namespace {

constexpr int ROPE_THREADS = 256;

__device__ __forceinline__ void turn_of(double turns, double pos, float& c, float& s)
{
    // t - rint(t) by adding and taking off 1.5 * 2^52 (|t| < 2^31)
    const double t = pos * turns;
    const double whole = __dadd_rn(__dadd_rn(t, 6755399441055744.0), -6755399441055744.0);
    sincospif(2.0f * static_cast<float>(t - whole), &s, &c);
}

template <int BYTES> struct RopeWord;
template <> struct RopeWord<16> { using type = uint4; };
template <> struct RopeWord<8> { using type = uint2; };
template <> struct RopeWord<4> { using type = uint32_t; };
template <> struct RopeWord<2> { using type = uint16_t; };

// E elements of T as loaded.
template <typename T, int E>
struct Chunk {
    typename RopeWord<E * static_cast<int>(sizeof(T))>::type w;
    __device__ __forceinline__ void load(const T* p) { w = *reinterpret_cast<const decltype(w)*>(p); }
    __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<decltype(w)*>(p) = w; }
    __device__ __forceinline__ float get(int i) const { return to_f32(reinterpret_cast<const T*>(&w)[i]); }
    __device__ __forceinline__ void set(int i, float x) { reinterpret_cast<T*>(&w)[i] = from_f32<T>(x); }
};

// A unit of E elements and, where its pairs' second members lie apart (half layout, or single
// elements), the E elements that hold them.
template <typename T, bool HALF, int E>
struct RopeUnits {
    static constexpr bool TWO = HALF || E == 1;
    static constexpr int PAIRS = TWO ? E : E / 2;               // pairs of a rotated unit
    static constexpr int SPAN = !HALF && E == 1 ? 2 : E;        // elements between rotated units' starts
    __host__ __device__ static int rotated(int rot) { return (HALF ? rot / 2 : rot) / SPAN; }
    __host__ __device__ static int all(int D, int rot) { return rotated(rot) + (D - rot) / E; }
};

template <typename T, bool HALF, int E>
__global__ void __launch_bounds__(ROPE_THREADS) rope_kernel(const __grid_constant__ RopeArgs a)
{
    using U = RopeUnits<T, HALF, E>;
    constexpr int NP = U::PAIRS;
    constexpr int AHEAD = 3;  // heads asked for at once (1, 2, 3, 4: 39.9, 35.0, 34.5, 35.3 us for 32760 tokens of 12 x 128 bf16)
    __shared__ double turns[ROPE_MAX_PAIRS];
    for (int i = threadIdx.x; i < a.rot_dim / 2; i += ROPE_THREADS) turns[i] = a.turns[i];
    __syncthreads();
    const int rot_units = U::rotated(a.rot_dim), units = U::all(a.head_dim, a.rot_dim);
    const unsigned item = blockIdx.x * ROPE_THREADS + threadIdx.x;
    const unsigned bt = item / units;
    if (bt >= static_cast<unsigned>(a.batch) * a.tokens) return;
    const int u = item - bt * units;
    const int b = bt / a.tokens, t = bt - b * a.tokens;
    const bool turned = u < rot_units;
    const int e0 = turned ? u * U::SPAN : a.rot_dim + (u - rot_units) * E;  // first element
    const int apart = HALF ? a.rot_dim >> 1 : 1;
    const bool two = U::TWO && turned;

    // This thread's heads: `left` of them from head h0 of tensor k on.
    int h0 = blockIdx.y * a.heads_per_thread, left = a.heads_per_thread, k = 0;
    while (h0 >= a.io[k].heads) h0 -= a.io[k++].heads;
    Chunk<T, E> va[AHEAD], vb[AHEAD];
    auto ask = [&](const RopeIo& io, int h, int n) {  // heads [h, h + n) of a tensor, n <= AHEAD
        const T* x = static_cast<const T*>(io.x) + b * io.xs[0] + h * io.xs[1] + t * io.xs[2] + e0;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (i < n) {
                va[i].load(x + i * io.xs[1]);
                if (U::TWO && two) vb[i].load(x + i * io.xs[1] + apart);
            }
    };
    int n = min(min(left, a.io[k].heads - h0), AHEAD);
    ask(a.io[k], h0, n);

    float c[NP], s[NP];
    if (turned) {
        const int* pos = a.positions + b * a.pos_batch + static_cast<long long>(t) * a.n_axes;
        const double p0 = __ldg(pos);
        const double p1 = a.n_axes > 1 ? __ldg(pos + 1) : 0, p2 = a.n_axes > 2 ? __ldg(pos + 2) : 0;
        const float sa = a.backward ? -a.amplitude : a.amplitude;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int p = u * NP + i;
            turn_of(turns[p], p < a.axis_end[0] ? p0 : (p < a.axis_end[1] ? p1 : p2), c[i], s[i]);
            c[i] *= a.amplitude;
            s[i] *= sa;
        }
    }
    while (n > 0) {
        const RopeIo& io = a.io[k];
        T* o = static_cast<T*>(io.out) + b * io.os[0] + h0 * io.os[1] + t * io.os[2] + e0;
        Chunk<T, E> ra[AHEAD], rb[AHEAD];
        const bool rotate = turned && io.rotate;
        const long long step = io.os[1];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            ra[i] = va[i];
            rb[i] = vb[i];
        }
        const int done = n;
        // the next heads, before these are stored
        left -= n;
        h0 += n;
        if (h0 == io.heads) {
            h0 = 0;
            ++k;
        }
        n = left > 0 && k < a.n_io ? min(min(left, a.io[k].heads - h0), AHEAD) : 0;
        if (n > 0) ask(a.io[k], h0, n);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (i < done) {
                if (rotate) {
#pragma unroll
                    for (int j = 0; j < NP; ++j) {
                        const float xa = U::TWO ? ra[i].get(j) : ra[i].get(2 * j);
                        const float xb = U::TWO ? rb[i].get(j) : ra[i].get(2 * j + 1);
                        const float ya = xa * c[j] - xb * s[j], yb = xa * s[j] + xb * c[j];
                        if (U::TWO) {
                            ra[i].set(j, ya);
                            rb[i].set(j, yb);
                        } else {
                            ra[i].set(2 * j, ya);
                            ra[i].set(2 * j + 1, yb);
                        }
                    }
                }
                ra[i].store(o + i * step);
                if (U::TWO && two) rb[i].store(o + i * step + apart);
            }
    }
}

template <typename T, bool HALF, int E>
cudaError_t launch_t(RopeArgs& a, cudaStream_t s)
{
    const long long items = static_cast<long long>(a.batch) * a.tokens * RopeUnits<T, HALF, E>::all(a.head_dim, a.rot_dim);
    int heads = 0;
    for (int k = 0; k < a.n_io; ++k) heads += a.io[k].heads;
    // Heads are spread over threads until the machine is full: 148 SMs * 1024 threads.
    const long long want = (148ll * 1024 + items - 1) / items;
    const int groups = static_cast<int>(want < 1 ? 1 : (want > heads ? heads : want));
    a.heads_per_thread = (heads + groups - 1) / groups;
    const dim3 grid(static_cast<unsigned>((items + ROPE_THREADS - 1) / ROPE_THREADS),
                    static_cast<unsigned>((heads + a.heads_per_thread - 1) / a.heads_per_thread));
    rope_kernel<T, HALF, E><<<grid, ROPE_THREADS, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T, bool HALF>
cudaError_t launch_e(RopeArgs& a, int elems, cudaStream_t s)
{
    if constexpr (sizeof(T) == 2) {
        if (elems == 8) return launch_t<T, HALF, 8>(a, s);
    }
    if (elems == 4) return launch_t<T, HALF, 4>(a, s);
    return elems == 2 ? launch_t<T, HALF, 2>(a, s) : launch_t<T, HALF, 1>(a, s);
}

template <typename T>
cudaError_t launch_l(RopeArgs& a, bool half_layout, int elems, cudaStream_t s)
{
    return half_layout ? launch_e<T, true>(a, elems, s) : launch_e<T, false>(a, elems, s);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a0, int dtype, bool half_layout, int elems, cudaStream_t s)
{
    RopeArgs a = a0;
    if (dtype == DT_F32) return launch_l<float>(a, half_layout, elems, s);
    if (dtype == DT_BF16) return launch_l<__nv_bfloat16>(a, half_layout, elems, s);
    return launch_l<__half>(a, half_layout, elems, s);
}

}  // namespace lf
