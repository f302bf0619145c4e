// What the two attention kernels over the 8-bit cache share: the arguments, the sharing-out of
// the work and the joining of partial results.
//
// The work is the list of all (sequence, [row tile,] head) units, each a run of key/value
// tiles, laid end to end: T tiles in all.  Worker w of W takes tiles floor(T w / W) ..
// floor(T (w + 1) / W) - 1, whatever the lengths are, so every SM streams the same number of
// tiles and no length has to be known on the host.  A unit that lies in one CTA's range is
// finished there; one that spans CTAs leaves, per CTA, a partial result (O, m, l) in the
// workspace (a CTA can have one unit that came in, slot 0, and one that goes out, slot 1), and
// the last CTA to arrive adds the parts in CTA order: the order of summation depends on the
// lengths alone.  The stream's parts, a few rows each, are added in one go; the tiles', up to 64 KB a
// row tile, eight at a time: the last arriver of eight neighbours puts their sum in the first
// one's place and arrives for them one level up.  An arrival counter belongs to the CTA, and to
// the slot, where the parts that it counts begin, and the last arriver sets it back to zero.
//
// The softmax, in base 2, with the value scale folded into the exponent: for a block with
// scales dk, dv and a query scaled by a = scale * log2(e) * dk,
//   t_j = a (q . kc_j) + log2 dv,  P_j = 2^(t_j - m),  O = sum P_j vc_j,  l = sum P_j / dv,
// out = O / l.  The value codes enter the second product as they are, and 1 / dv is applied
// once per block and row, not once per weight.  m only has to keep 2^(t - m) inside f16: it is
// set SHIFT below the running maximum and moved when a t passes m + LIMIT, so the accumulators
// are rescaled a few times per row, not once per tile; weights below 2^-(25 + SHIFT) of the
// largest vanish in f16.  A block whose values are all zero (dv = 0) stands in with 2^-60.
#pragma once

#include <math.h>

#include "kv.cuh"

namespace mmq {
namespace kv {

constexpr float SHIFT = 7.f, LIMIT = 15.f;  // weights up to 2^15 < 65504
constexpr float M_NONE = -1e30f;            // m of a row that has seen nothing
constexpr int WS_COUNTERS = 16384;          // bytes of arrival counters before the partial results
constexpr int WS_ROWS = 256;                // rows a partial result holds at most,
constexpr int WS_ROW_STATS = 6;             // values beside O: m and l, for each level of joining

struct Attend {
    Cache c;
    Batch bt;
    Rows q;
    int q_heads, group, dtype, window;
    float scale2;  // scale * log2(e)
    void* out;
    float* lse;
    uint8_t* ws;
};

__device__ __forceinline__ int work_start(long long total, int w, int workers) { return (int)(total * w / workers); }
// the worker whose range holds tile x
__device__ __forceinline__ int work_owner(int total, int x, int workers) {
    return (int)((((long long)x + 1) * workers - 1) / total);
}

__device__ __forceinline__ float* part_slot(const Attend& a, int cta, int slot) {
    return reinterpret_cast<float*>(a.ws + WS_COUNTERS) + ((long long)cta * 2 + slot) * WS_ROWS * (a.c.dim + WS_ROW_STATS);
}

// first key that row 0 of a sequence (at position first) sees
__device__ __forceinline__ int first_key(const Attend& a, int first) { return a.window > 0 ? max(0, first - a.window + 1) : 0; }

__device__ __forceinline__ void store_out4(const Attend& a, long long row, int h, int d, float4 v) {
    const long long at = (row * a.q_heads + h) * a.c.dim + d;
    if (a.dtype == MMQ_F32)
        Elem<float>::store4(static_cast<float*>(a.out) + at, v);
    else if (a.dtype == MMQ_BF16)
        Elem<__nv_bfloat16>::store4(static_cast<__nv_bfloat16*>(a.out) + at, v);
    else
        Elem<__half>::store4(static_cast<__half*>(a.out) + at, v);
}
__device__ __forceinline__ void store_out8(const Attend& a, long long row, int h, int d, float4 u, float4 v) {
    const long long at = (row * a.q_heads + h) * a.c.dim + d;
    if (a.dtype == MMQ_F32) {
        Elem<float>::store4(static_cast<float*>(a.out) + at, u);
        Elem<float>::store4(static_cast<float*>(a.out) + at + 4, v);
    } else if (a.dtype == MMQ_BF16) {
        using E = Elem<__nv_bfloat16>;
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at) =
            make_uint4(E::pack2(u.x, u.y), E::pack2(u.z, u.w), E::pack2(v.x, v.y), E::pack2(v.z, v.w));
    } else {
        using E = Elem<__half>;
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at) =
            make_uint4(E::pack2(u.x, u.y), E::pack2(u.z, u.w), E::pack2(v.x, v.y), E::pack2(v.z, v.w));
    }
}
__device__ __forceinline__ void store_lse(const Attend& a, long long row, int h, float m, float l) {
    if (a.lse) a.lse[row * a.q_heads + h] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// log2 of a block's value scale and its reciprocal, as the exponent and the sum take them
__device__ __forceinline__ void value_scale(float dv, float& lv, float& rv) {
    const float d = dv >= MIN_SCALE ? dv : 0x1p-60f;
    lv = __log2f(d);
    rv = __fdividef(1.f, d);
}

// Powers of two: `down` brings a row's largest magnitude into [2^8, 2^9) (exactly; f16 then keeps
// what lies down to 2^-33 below it), `up` takes it back.
__device__ __forceinline__ void row_scale(float amax, float& down, float& up) {
    const int e = max(9, min(253, (int)((__float_as_uint(amax) >> 23) & 255)));  // biased
    down = __uint_as_float((uint32_t)(262 - e) << 23);
    up = __uint_as_float((uint32_t)(e - 8) << 23);
}

// Parts of one row's result as they are added up.
struct Joined {
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float m = M_NONE, l = 0.f;
    __device__ __forceinline__ void add(float4 x, float mx, float lx) {
        const float mn = fmaxf(m, mx), f = exp2_approx(m - mn), g = exp2_approx(mx - mn);
        o = make_float4(o.x * f + x.x * g, o.y * f + x.y * g, o.z * f + x.z * g, o.w * f + x.w * g);
        l = l * f + lx * g;
        m = mn;
    }
    __device__ __forceinline__ float4 out() const {
        const float inv = l > 0.f ? __frcp_rn(l) : 0.f;
        return make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    }
};

__device__ __forceinline__ uint32_t pack_h2(float a, float b) { return Elem<__half>::pack2(a, b); }
__device__ __forceinline__ float2 unpack_h2(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }
// the two f16 terms of a pair
__device__ __forceinline__ void split_h2(float a, float b, uint32_t& hi, uint32_t& lo) {
    hi = pack_h2(a, b);
    const float2 f = unpack_h2(hi);
    lo = pack_h2(a - f.x, b - f.y);
}

// Exclusive scan over the CTA; total: the sum.
template <int WARPS>
__device__ __forceinline__ int scan_cta(int v, int& total, int* scratch) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) scratch[wid] = x;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
        if (i < wid) before += scratch[i];
        total += scratch[i];
    }
    __syncthreads();
    return before + x - v;
}

}  // namespace kv
// The two kernels: up to kv_stream_rows(dim, dtype) query rows per sequence and head (kv_stream.cu), any
// number (kv_tile.cu).
int kv_stream_rows(int dim, int dtype);
int kv_stream_launch(const kv::Attend& a, int rows, cudaStream_t s);
int kv_tile_launch(const kv::Attend& a, cudaStream_t s);

}  // namespace mmq
