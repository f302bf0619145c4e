// The rows of a feed-forward call as operands of its product: k_ffn_rows (x as it is) and k_ffn_gradients
// (dz = dy act'(z); for the gated block dg = dh u act'(g) and du = dh act(g), side by side).
//
// Bound: HBM.  k_ffn_rows 2048 bf16 rows of 18944 values, 155 MB, 28 us (5.5 TB/s); k_ffn_gradients below.
//
// A row is scaled by a power of two that brings its largest magnitude into [2^13, 2^14), so that f16 holds all
// but what lies 2^-38 below it, and written as f16 (bf16 rows exactly, f16 rows as they are but for the
// scaling; f32 rows in two terms) in the order in which the tensor cores read them: per 64 values and 8 rows 1024
// bytes, a row 128 of them, its 16-byte pieces exchanged by the row's number (piece c at c ^ row: 128-byte swizzle).  `up` takes
// the scaling back, and the 2^8 of the weights.  f16 rows are operands as they are: no scaling, so they are cut at will; but
// where blocks' sums are wanted too they are scaled as the others, since the two f16 terms of a sum hold 2^-19 of it only
// where x is of the size of one (unscaled rows of 1e-4: 4.6e-3 of the outputs' norm).
#include "ffn_rows.cuh"

namespace mmq {
namespace {

using namespace ffn;

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

__device__ __forceinline__ void clear_counters(const Rows& r) {
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int i = threadIdx.x; i < r.n_counters; i += blockDim.x) r.counters[i] = 0u;
}

// A CTA per row (rows that are not scaled: several), a thread per run of eight values; eight neighbouring threads write a line.
constexpr int GRADIENT_THREADS = 256;
constexpr int HELD = 5;  // runs a thread keeps between looking for the largest value and writing

template <typename T, int THREADS, bool SCALED>
__global__ void __launch_bounds__(THREADS) k_ffn_rows(const Rows r) {
    __shared__ float s_max[THREADS / 32];
    ptx::grid_dep_wait();
    ptx::grid_dep_launch_dependents();
    clear_counters(r);
    const int m = blockIdx.x, first = threadIdx.x + blockIdx.y * THREADS, step = THREADS * gridDim.y;
    const int runs = r.width / 8, places = (r.width + 63) / 64 * 8;  // K is a multiple of 32; whole steps: zeros past K
    const T* x = static_cast<const T*>(r.x) + m * r.stride;
    float held[HELD][8], down = 1.f;
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
        const int c = first + i * step;
#pragma unroll
        for (int k = 0; k < 8; ++k) held[i][k] = 0.f;
        if (c < runs) load8(x + 8ll * c, held[i]);
    }
    if (SCALED) {
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < HELD; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(held[i][k]));
#pragma unroll 4
        for (int c = first + HELD * step; c < runs; c += step) {
            float v[8];
            load8(x + 8ll * c, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(v[k]));
        }
        const Scale s = row_scale(max_cta<THREADS>(amax, s_max));
        if (threadIdx.x == 0) r.up[m] = s.up;
        down = s.down;
    } else if (blockIdx.y == 0 && threadIdx.x == 0) {
        r.up[m] = 1.f / 256.f;  // the weights' 2^8
    }
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
        const int c = first + i * step;
        if (c < places) {
            put(r, m, c >> 3, c & 7, held[i], down);
            if (r.sums) put_sum(r.sums, r.groups, m, c, held[i], down);  // (whole warps: K is a multiple of 256 then)
        }
    }
#pragma unroll 4
    for (int c = first + HELD * step; c < places; c += step) {
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (c < runs) load8(x + 8ll * c, v);
        put(r, m, c >> 3, c & 7, v, down);
        if (r.sums) put_sum(r.sums, r.groups, m, c, v, down);
    }
}

// Eight values as they lie, from an address that is aligned to its elements, as one load where it is aligned to 16 bytes.
template <typename T>
struct Run {
    alignas(16) T v[8];
};
template <typename T>
__device__ __forceinline__ void get8(const T* p, int left, bool vector, Run<T>& r) {
    if (vector && left >= 8) {
        const uint4* q = reinterpret_cast<const uint4*>(p);
        uint4* to = reinterpret_cast<uint4*>(r.v);
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) to[i] = q[i];
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) r.v[k] = k < left ? p[k] : T(0.f);
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

// The largest of a cluster of CTAS, which every one of them reads where its own stands: no peer's memory is touched once
// the second barrier is behind, so that a CTA may end.
template <int CTAS>
__device__ __forceinline__ float max_cluster(float v, float* s_all) {
    if (CTAS == 1) return v;
    const uint32_t here = ptx::smem_u32(s_all + blockIdx.x % CTAS);
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");  // every peer has begun
    if (threadIdx.x < CTAS) {
        uint32_t there;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(here), "r"(threadIdx.x));
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(there), "f"(v) : "memory");
    }
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
#pragma unroll
    for (int i = 0; i < CTAS; ++i) v = fmaxf(v, s_all[i]);
    return v;
}

// CTAS CTAs per row, a cluster, each its share of whole steps.  KEEP: the gradients stay in shared memory between looking for
// the largest and writing (f32, 8 bytes a value of the gated block); rows that are too wide for that are formed twice.
// Four CTAs on an SM, so that one's loads go on while another waits for its row's largest.  Measured on 2048 bf16 rows of
// 18944, gated, 543 MB: formed twice 198 us, kept by one CTA a row 152, by a cluster of four 151, with the next run's loads
// under way while one is formed 123 (4.4 TB/s; its bound is what is in flight: at five CTAs of 48 registers it spills, 265).
template <typename T, bool KEEP, int CTAS>
__global__ void __launch_bounds__(GRADIENT_THREADS) k_ffn_gradients(const Rows r) {
    constexpr int THREADS = GRADIENT_THREADS;
    extern __shared__ __align__(16) float s_keep[];
    __shared__ float s_max[THREADS / 32], s_all[CTAS];
    if (CTAS > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
    ptx::grid_dep_wait();
    ptx::grid_dep_launch_dependents();
    clear_counters(r);
    const int m = blockIdx.x / CTAS, N = r.width, steps = (N + 63) / 64, share = (steps + CTAS - 1) / CTAS;
    const int first = blockIdx.x % CTAS * share, last = min(steps, first + share);
    const long long at = (long long)m * N;
    const T* x = static_cast<const T*>(r.x) + m * r.stride;
    const T* pre[2] = {nullptr, nullptr};
    T* dz[2] = {nullptr, nullptr};
    for (int g = 0; g < 2; ++g) {
        if (r.pre[g]) pre[g] = static_cast<const T*>(r.pre[g]) + at;
        if (r.dz[g]) dz[g] = static_cast<T*>(r.dz[g]) + at;
    }
    auto aligned = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
    const bool vx = aligned(x), v0 = aligned(pre[0]), v1 = aligned(pre[1]), w0 = aligned(dz[0]), w1 = aligned(dz[1]);
    with_act(r.pre[0] ? r.act : MMQ_ACT_NONE, [&](auto A) {
        struct Values {
            Run<T> x, pre, up;
        };
        auto load = [&](int n, Values& in) {
            get8(x + n, N - n, vx, in.x);
            if (r.pre[0]) get8(pre[0] + n, N - n, v0, in.pre);
            if (r.mats == 2) get8(pre[1] + n, N - n, v1, in.up);
        };
        // the gradients of a run, 0 past the row
        auto form = [&](const Values& in, auto fast, float (&g)[8], float (&u)[8]) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                g[k] = (float)in.x.v[k];
                if (!r.pre[0]) continue;
                float a, d;
                activate<decltype(A)::value, decltype(fast)::value>((float)in.pre.v[k], a, d);
                u[k] = g[k] * a;
                g[k] *= d;
                if (r.mats == 2) g[k] *= (float)in.up.v[k];
            }
        };
        float amax = 0.f, g[8], u[8];
        float* keep_u = s_keep + share * STEP;
        Values in, next;  // the next run's loads are under way while one is formed
        if (first * 8 + (int)threadIdx.x < last * 8) load(8 * (first * 8 + threadIdx.x), in);
#pragma unroll 1
        for (int c = first * 8 + threadIdx.x; c < last * 8; c += THREADS) {
            const int kept = 8 * (c - first * 8);
            if (c + THREADS < last * 8) load(8 * (c + THREADS), next);
            // (where the row is formed again the largest value's exponent is all that is wanted)
            form(in, std::integral_constant<bool, !KEEP || sizeof(T) == 2>{}, g, u);
            in = next;
#pragma unroll
            for (int k = 0; k < 8; ++k) amax = fmaxf(amax, r.mats == 2 ? fmaxf(fabsf(g[k]), fabsf(u[k])) : fabsf(g[k]));
            if (KEEP) {
                put8(s_keep + kept, 8, true, g);
                if (r.mats == 2) put8(keep_u + kept, 8, true, u);
            }
        }
        const Scale s = row_scale(max_cluster<CTAS>(max_cta<THREADS>(amax, s_max), s_all));
        if (first == 0 && threadIdx.x == 0) r.up[m] = s.up;
#pragma unroll 1
        for (int c = first * 8 + threadIdx.x; c < last * 8; c += THREADS) {
            const int kept = 8 * (c - first * 8);
            if (KEEP) {
                load8(s_keep + kept, g);
                if (r.mats == 2) load8(keep_u + kept, u);
            } else {
                load(8 * c, in);
                form(in, std::integral_constant<bool, sizeof(T) == 2>{}, g, u);
            }
            put(r, m, c >> 3, c & 7, g, s.down);
            if (r.mats == 2) put(r, m, steps + (c >> 3), c & 7, u, s.down);
            if (r.dz[0]) put8(dz[0] + 8 * c, N - 8 * c, w0, g);
            if (r.dz[1]) put8(dz[1] + 8 * c, N - 8 * c, w1, u);
        }
    });
}

constexpr int KEEP_MOST = 50 * 1024;  // of a CTA, so that four share an SM

template <typename T, bool KEEP, int CTAS>
int gradients(const Rows& r, int smem, bool go, const char* fn, cudaStream_t s) {
    static SmemAttr attr;
    auto k = &k_ffn_gradients<T, KEEP, CTAS>;
    if (smem > 48 * 1024)
        if (const int st = ensure_smem(reinterpret_cast<const void*>(k), KEEP_MOST, attr)) {
            report(fn, st, "the gradients' shared memory was refused");
            return st;
        }
    if (!go) return MMQ_OK;
    ProfScope ps("k_ffn_gradients", s);
    return pdl_status(ffn_cluster_launch(k, r.rows * CTAS, GRADIENT_THREADS, CTAS, smem, s, r), fn);
}

template <typename T, int THREADS, bool SCALED>
int rows(const Rows& r, const char* fn, cudaStream_t s) {
    // not scaled: CTAs enough for every SM's threads, as long as each has what its threads hold
    const int each = THREADS * HELD, runs = r.width / 8, want = 4 * device_shape().sms / r.rows + 1;
    const int most = (runs + each - 1) / each, cuts = SCALED ? 1 : want < most ? want : most;
    ProfScope ps("k_ffn_rows", s);
    return pdl_status(launch_pdl(&k_ffn_rows<T, THREADS, SCALED>, dim3((unsigned)r.rows, (unsigned)cuts), dim3(THREADS), 0, s, r), fn);
}

template <typename T>
int launch(const Rows& r, bool back, bool go, const char* fn, cudaStream_t s) {
    if (back) {
        constexpr int CTAS = 4;
        const int steps = (r.width + STEP - 1) / STEP, keep = STEP * 4 * r.mats;
        if (r.width <= 4096) return gradients<T, true, 1>(r, steps * keep, go, fn, s);
        const int each = (steps + CTAS - 1) / CTAS * keep;
        return each <= KEEP_MOST ? gradients<T, true, CTAS>(r, each, go, fn, s) : gradients<T, false, CTAS>(r, 0, go, fn, s);
    }
    if (!go) return MMQ_OK;
    constexpr bool SCALED = !std::is_same<T, __half>::value;
    if (!SCALED && r.sums) return rows<T, 512, true>(r, fn, s);
    // a narrow row in small CTAs where there are many; one row's latency in a large one
    return r.rows >= 2 * device_shape().sms && r.width <= 8 * 128 * HELD ? rows<T, 128, SCALED>(r, fn, s) : rows<T, 512, SCALED>(r, fn, s);
}

}  // namespace

int ffn_rows_launch(const Rows& r, bool back, bool go, const char* fn, cudaStream_t s) {
    if (r.dtype == MMQ_F32) return launch<float>(r, back, go, fn, s);
    if (r.dtype == MMQ_BF16) return launch<__nv_bfloat16>(r, back, go, fn, s);
    return launch<__half>(r, back, go, fn, s);
}

}  // namespace mmq
