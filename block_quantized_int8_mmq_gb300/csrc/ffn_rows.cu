// The rows of a feed-forward call as operands of its product: k_ffn_rows (x as it is) and k_ffn_gradients
// (dz = dy act'(z); for the gated block dg = dh u act'(g) and du = dh act(g), side by side).
//
// A row is scaled by a power of two that brings its largest magnitude into [2^13, 2^14), so that f16 holds all
// but what lies 2^-38 below it, and written as f16 (bf16 rows exactly, f16 rows as they are but for the
// scaling; f32 rows in two terms) in the order in which the tensor cores read them: per 64 values and 8 rows 1024
// bytes, eight core matrices of 8 rows x 16 bytes.  `up` takes the scaling back, and the 2^8 of the weights.
// HBM-bound; a CTA per row, the row read twice (the second time from L1 or L2) where it does not fit in registers.
#include "ffn.cuh"
#include "kv.cuh"
#include "umma.cuh"

namespace mmq {
namespace {

using namespace ffn;

struct Scale {
    float down, up;
};
__device__ __forceinline__ Scale row_scale(float amax) {
    // biased exponent; NaN and infinity count as the largest
    const int e = max(22, min(254, (int)((__float_as_uint(amax) >> 23) & 255)));
    return {__uint_as_float((uint32_t)(267 - e) << 23), __uint_as_float((uint32_t)(e - 21) << 23)};
}

template <int THREADS>
__device__ __forceinline__ float max_cta(float v, float* scratch) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    v = scratch[0];
#pragma unroll
    for (int i = 1; i < THREADS / 32; ++i) v = fmaxf(v, scratch[i]);
    return v;
}

// Eight values of a row to their place(s).
__device__ __forceinline__ void put(const Rows& r, int m, int step, int chunk, const float (&v)[8], float down) {
    uint8_t* p = r.tiles + ((long long)step * r.groups + (m >> 3)) * 1024 + chunk * 128 + (m & 7) * 16;
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = v[2 * i] * down, b = v[2 * i + 1] * down;
        const __half2 h = __floats2half2_rn(a, b);
        const float2 back = __half22float2(h);
        hi[i] = umma::h2_bits(h);
        lo[i] = umma::h2_bits(__floats2half2_rn(a - back.x, b - back.y));
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    if (r.dtype == MMQ_F32) *reinterpret_cast<uint4*>(p + r.term) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
}

__device__ __forceinline__ void clear_counters(const Rows& r) {
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < r.n_counters; i += blockDim.x) r.counters[i] = 0u;
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
    if (sizeof(T) == 2) {
        kv::load_run<T, 8>(p, v);
    } else {
        const float4 a = kv::Elem<T>::load4(p), b = kv::Elem<T>::load4(p + 4);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
}

constexpr int HELD = 4;  // runs of 8 values a thread keeps

template <typename T, int THREADS>
__global__ void __launch_bounds__(THREADS) k_ffn_rows(const Rows r) {
    __shared__ float s_max[THREADS / 32];
    ptx::grid_dep_wait();
    ptx::grid_dep_launch_dependents();
    clear_counters(r);
    const int m = blockIdx.x, runs = r.width / 8, places = (r.width + 63) / 64 * 8;  // K is a multiple of 32
    const T* x = static_cast<const T*>(r.x) + m * r.stride;
    float held[HELD][8], amax = 0.f;
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
        const int c = threadIdx.x + i * THREADS;
        if (c < runs) load8(x + 8ll * c, held[i]);
    }
#pragma unroll
    for (int i = 0; i < HELD; ++i)
        if (threadIdx.x + i * THREADS < runs)
#pragma unroll
            for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(held[i][k]));
    for (int c = threadIdx.x + HELD * THREADS; c < runs; c += THREADS) {
        float v[8];
        load8(x + 8ll * c, v);
#pragma unroll
        for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(v[k]));
    }
    const Scale s = row_scale(max_cta<THREADS>(amax, s_max));
    if (threadIdx.x == 0) r.up[m] = s.up;
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
        const int c = threadIdx.x + i * THREADS;
        if (c < runs) put(r, m, c >> 3, c & 7, held[i], s.down);
    }
    for (int c = threadIdx.x + HELD * THREADS; c < places; c += THREADS) {
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (c < runs) load8(x + 8ll * c, v);
        put(r, m, c >> 3, c & 7, v, s.down);
    }
    // the last step's places past K, where all runs are held
    const float none[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int c = runs + threadIdx.x; c < min(places, HELD * THREADS); c += THREADS) put(r, m, c >> 3, c & 7, none, s.down);
}

// Eight values from an address that is aligned to its elements, as one load where it is aligned to 16 bytes.
template <typename T>
__device__ __forceinline__ void get8(const T* p, int left, bool vector, float (&v)[8]) {
    if (vector && left >= 8) {
        load8(p, v);
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = k < left ? get_one(p + k) : 0.f;
}
template <typename T>
__device__ __forceinline__ void put8(T* p, int left, bool vector, const float (&v)[8]) {
    if (vector && left >= 8) {
        if (sizeof(T) == 2) {
            kv::store_run<T, 8>(p, v);
        } else {
            kv::Elem<T>::store4(p, make_float4(v[0], v[1], v[2], v[3]));
            kv::Elem<T>::store4(p + 4, make_float4(v[4], v[5], v[6], v[7]));
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k < left) put_one(p + k, v[k]);
}

template <typename T, int THREADS>
__global__ void __launch_bounds__(THREADS) k_ffn_gradients(const Rows r) {
    __shared__ float s_max[THREADS / 32];
    ptx::grid_dep_wait();
    ptx::grid_dep_launch_dependents();
    clear_counters(r);
    const int m = blockIdx.x, N = r.width, steps = (N + 63) / 64;
    const long long at = (long long)m * N;
    const T* x = static_cast<const T*>(r.x) + m * r.stride;
    const T* pre[2] = {static_cast<const T*>(r.pre[0]) + at, static_cast<const T*>(r.pre[1]) + at};
    T* dz[2] = {static_cast<T*>(r.dz[0]) + at, static_cast<T*>(r.dz[1]) + at};
    auto aligned = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
    const bool vx = aligned(x), v0 = aligned(pre[0]), v1 = aligned(pre[1]), w0 = aligned(dz[0]), w1 = aligned(dz[1]);
    // the gradients of values n .. n + 7, 0 past the row
    auto form = [&](int n, float (&g)[8], float (&u)[8]) {
        const int left = N - n;
        get8(x + n, left, vx, g);
        if (!r.pre[0]) return;
        float z[8], y[8];
        get8(pre[0] + n, left, v0, z);
        if (r.mats == 2) get8(pre[1] + n, left, v1, y);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float a, d;
            activate(r.act, z[k], a, d);
            u[k] = g[k] * a;
            g[k] *= d;
            if (r.mats == 2) g[k] *= y[k];
        }
    };
    float amax = 0.f, g[8], u[8];
#pragma unroll 2
    for (int c = threadIdx.x; c < (N + 7) / 8; c += THREADS) {
        form(8 * c, g, u);
#pragma unroll
        for (int k = 0; k < 8; ++k) amax = fmaxf(amax, r.mats == 2 ? fmaxf(fabsf(g[k]), fabsf(u[k])) : fabsf(g[k]));
    }
    const Scale s = row_scale(max_cta<THREADS>(amax, s_max));
    if (threadIdx.x == 0) r.up[m] = s.up;
#pragma unroll 2
    for (int c = threadIdx.x; c < steps * 8; c += THREADS) {
        form(8 * c, g, u);
        put(r, m, c >> 3, c & 7, g, s.down);
        if (r.mats == 2) put(r, m, steps + (c >> 3), c & 7, u, s.down);
        if (r.dz[0]) put8(dz[0] + 8 * c, N - 8 * c, w0, g);
        if (r.dz[1]) put8(dz[1] + 8 * c, N - 8 * c, w1, u);
    }
}

template <typename T>
int launch(const Rows& r, bool back, const char* fn, cudaStream_t s) {
    ProfScope ps(back ? "k_ffn_gradients" : "k_ffn_rows", s);
    constexpr int T0 = 256;
    const dim3 grid((unsigned)r.rows);
    return pdl_status(back ? launch_pdl(&k_ffn_gradients<T, T0>, grid, dim3(T0), 0, s, r)
                           : launch_pdl(&k_ffn_rows<T, T0>, grid, dim3(T0), 0, s, r),
                      fn);
}

}  // namespace

int ffn_rows_launch(const Rows& r, bool back, const char* fn, cudaStream_t s) {
    if (r.dtype == MMQ_F32) return launch<float>(r, back, fn, s);
    if (r.dtype == MMQ_BF16) return launch<__nv_bfloat16>(r, back, fn, s);
    return launch<__half>(r, back, fn, s);
}

}  // namespace mmq
