// Attention over the 8-bit key/value cache, plain form: one warp per (row, query head), one
// block of 32 tokens at a time, a lane per token for the scores and D / 32 values per lane for
// the output, with the running maximum and sum of the softmax in f32.
#include <math.h>

#include "kv_attend.cuh"

namespace mmq {

int kv_stream_rows(int dim);
int kv_stream_launch(const kv::Attend& a, int rows, cudaStream_t s);
unsigned kv_stream_take_error();

namespace {

using namespace kv;

constexpr int WARPS = 4;

__device__ unsigned g_kv_attend_error;

template <typename T, int D>
__global__ void __launch_bounds__(WARPS * 32)
k_kv_attend(Cache c, Batch bt, Rows qr, int q_heads, float scale, int window, T* __restrict__ out,
            float* __restrict__ lse) {
    __shared__ float qs[WARPS][D];
    ptx::grid_dep_wait();
    ptx::grid_dep_launch_dependents();
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const long long unit = (long long)blockIdx.x * WARPS + wid;
    if (unit >= (long long)bt.tokens * q_heads) return;
    const int row = (int)(unit / q_heads), h = (int)(unit % q_heads), hk = h / (q_heads / c.heads);
    int b = -1;
    for (int i0 = 0; i0 < bt.seqs; i0 += 32) {
        const int i = i0 + lane;
        b += __popc(__ballot_sync(0xffffffffu, i < bt.seqs && bt.starts[min(i, bt.seqs - 1)] <= row));
    }
    int start = 0, n = 0, len = 0;
    if (b < 0 || !seq_range(c, bt, b, start, n, len, &g_kv_attend_error) || row >= start + n) return;
    const int pos = len - n + row - start;
    const T* q = static_cast<const T*>(qr.data) + (long long)row * qr.token_stride + (long long)h * qr.head_stride;
    for (int d = 4 * lane; d < D; d += 128) {
        const float4 v = Elem<T>::load4(q + d);
        *reinterpret_cast<float4*>(&qs[wid][d]) = v;
    }
    __syncwarp();
    float m = -INFINITY, l = 0.f, acc[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[i] = 0.f;
    const int lo = window > 0 ? max(0, pos - window + 1) : 0;
    for (int blk = lo / BT; blk * BT <= pos; ++blk) {
        const uint8_t* rec = record(c, bt, b, blk, hk, &g_kv_attend_error);
        if (!rec) break;
        const float2 d = *reinterpret_cast<const float2*>(rec + 2 * BT * D);
        float s = 0.f;
        const uint32_t* kc = reinterpret_cast<const uint32_t*>(rec + lane * D);
        for (int e = 0; e < D / 4; ++e) {
            const uint32_t w = kc[e];
            const float4 v = *reinterpret_cast<const float4*>(&qs[wid][4 * e]);
            s += v.x * (float)(int8_t)w + v.y * (float)(int8_t)(w >> 8) + v.z * (float)(int8_t)(w >> 16) +
                 v.w * (float)(int8_t)(w >> 24);
        }
        const int j = blk * BT + lane;
        s = j >= lo && j <= pos ? s * d.x * scale : -INFINITY;
        float mx = s;
#pragma unroll
        for (int off = 16; off; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float mn = fmaxf(m, mx), f = expf(m - mn);
        const float p = expf(s - mn);
        m = mn;
        l = l * f + p;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) acc[i] *= f;
        for (int t = 0; t < BT; ++t) {
            const float pt = __shfl_sync(0xffffffffu, p, t) * d.y;
            if (blk * BT + t > pos) break;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) acc[i] += pt * (float)(int8_t)rec[BT * D + t * D + lane + 32 * i];
        }
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
    T* o = out + unit * D;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[lane + 32 * i] = (T)(l > 0.f ? acc[i] / l : 0.f);
    if (lse && lane == 0) lse[unit] = l > 0.f ? m + logf(l) : -INFINITY;
}

template <typename T>
int attend_t(const Cache& c, const Batch& b, const Rows& q, int q_heads, float scale, int window, void* out, float* lse,
             cudaStream_t s) {
    const long long units = (long long)b.tokens * q_heads;
    const dim3 grid((unsigned)((units + WARPS - 1) / WARPS));
    ProfScope ps("k_kv_attend", s);
    auto go = [&](auto kernel) {
        return pdl_status(launch_pdl(kernel, grid, dim3(WARPS * 32), 0, s, c, b, q, q_heads, scale, window,
                                     static_cast<T*>(out), lse),
                          "mmq_kv_attend");
    };
    return c.dim == 64 ? go(k_kv_attend<T, 64>) : c.dim == 128 ? go(k_kv_attend<T, 128>) : go(k_kv_attend<T, 256>);
}

}  // namespace

int kv_attend_launch(const Cache& c, const Batch& b, int dtype, const Rows& q, int q_heads, float scale, int window,
                     void* out, float* lse, void* ws, cudaStream_t s) {
    const int group = q_heads / c.heads;
    const Attend a{c, b, q, q_heads, group, dtype, window, scale * 1.44269504088896341f, out, lse,
                   static_cast<uint8_t*>(ws)};
    if ((long long)b.max_new * group <= kv_stream_rows(c.dim)) return kv_stream_launch(a, b.max_new * group, s);
    return dtype == MMQ_F32    ? attend_t<float>(c, b, q, q_heads, scale, window, out, lse, s)
           : dtype == MMQ_BF16 ? attend_t<__nv_bfloat16>(c, b, q, q_heads, scale, window, out, lse, s)
                               : attend_t<__half>(c, b, q, q_heads, scale, window, out, lse, s);
}

// two partial results of up to 256 rows for every SM, behind the counters
size_t kv_attend_workspace(int dim) { return 4096 + (size_t)device_shape().sms * 2 * 256 * (dim + 2) * 4; }

unsigned kv_attend_take_error() {
    unsigned v = 0;
    if (cudaMemcpyFromSymbol(&v, g_kv_attend_error, sizeof(v)) != cudaSuccess) return 0;
    if (v) {
        const unsigned zero = 0;
        cudaMemcpyToSymbol(g_kv_attend_error, &zero, sizeof(zero));
    }
    return v | kv_stream_take_error();
}

}  // namespace mmq
