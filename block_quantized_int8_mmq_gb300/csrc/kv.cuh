// Shared pieces of the 8-bit key/value cache kernels: the views the launchers pass, the
// checks of what a kernel reads from device memory (never followed when out of range), and
// the element conversions of the row arrays.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "kv_ptx.cuh"

namespace mmq {

constexpr unsigned ERR_RANGE = 2u;  // error bit beside ERR_TIMEOUT: a value in device memory outside its range

namespace kv {

constexpr int BT = 32;                 // tokens per block (one scale per head)
constexpr int REC_TAIL = 16;           // dk, dv and 8 reserved bytes after the codes
constexpr float MIN_SCALE = 0x1p-100f;  // scales below it count as 0
__host__ __device__ constexpr int rec_bytes(int dim) { return 2 * BT * dim + REC_TAIL; }

struct Cache {
    uint8_t* data;
    long long pages;
    int page, heads, dim, blocks;  // blocks: records per page and head
};
struct Batch {
    const int32_t* starts;
    const int32_t* lens;
    const int32_t* table;
    long long table_stride;
    int seqs, tokens, max_new, table_pages;
};
struct Rows {
    const void* data;
    long long token_stride, head_stride;
};
struct Rope {
    const float *cos, *sin;
    long long rows;
    int rotary, interleaved;  // rotary 0: no rotation
};

// Sequence b: first row, new tokens and length, or false (all 0, the error word set) where
// they are out of range.
__device__ __forceinline__ bool seq_range(const Cache& c, const Batch& bt, int b, int& start, int& n, int& len,
                                          unsigned* err) {
    const int s0 = bt.starts[b], s1 = bt.starts[b + 1], l = bt.lens[b];
    if (s0 < 0 || s1 < s0 || s1 > bt.tokens || s1 - s0 > bt.max_new || l < 0 ||
        l > (long long)bt.table_pages * c.page) {
        atomicOr(err, ERR_RANGE);
        start = n = len = 0;
        return false;
    }
    start = s0;
    n = s1 - s0;
    len = l;
    return true;
}

// Record of block blk of sequence b and head h, or nullptr (the error word set) where the
// table names no page.
__device__ __forceinline__ uint8_t* record(const Cache& c, const Batch& bt, int b, int blk, int h, unsigned* err) {
    const int pg = blk / c.blocks, in = blk - pg * c.blocks;
    const int id = bt.table[(long long)b * bt.table_stride + pg];
    if (id < 0 || id >= c.pages) {
        atomicOr(err, ERR_RANGE);
        return nullptr;
    }
    return c.data + (((long long)id * c.heads + h) * c.blocks + in) * rec_bytes(c.dim);
}

// Four and eight consecutive elements of a row as f32 and back (one rounding).
template <typename T>
struct Elem;
template <>
struct Elem<float> {
    static __device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
    static __device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
    static __device__ __forceinline__ float4 widen(uint2) { return make_float4(0.f, 0.f, 0.f, 0.f); }  // 16-bit types only
    static __device__ __forceinline__ uint32_t pack2(float, float) { return 0u; }
};
template <>
struct Elem<__nv_bfloat16> {
    static __device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
        return widen(*reinterpret_cast<const uint2*>(p));
    }
    static __device__ __forceinline__ float4 widen(uint2 u) {
        return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                           __uint_as_float(u.y & 0xffff0000u));
    }
    static __device__ __forceinline__ uint32_t pack2(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static __device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack2(v.x, v.y), pack2(v.z, v.w));
    }
};
template <>
struct Elem<__half> {
    static __device__ __forceinline__ float4 load4(const __half* p) { return widen(*reinterpret_cast<const uint2*>(p)); }
    static __device__ __forceinline__ float4 widen(uint2 u) {
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
        return make_float4(a.x, a.y, b.x, b.y);
    }
    static __device__ __forceinline__ uint32_t pack2(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static __device__ __forceinline__ void store4(__half* p, float4 v) {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack2(v.x, v.y), pack2(v.z, v.w));
    }
};

// V consecutive elements of a row (V = 4, or 8 of a 16-bit type: one 16-byte load) as f32.
template <typename T, int V>
__device__ __forceinline__ void load_run(const T* p, float (&x)[V]) {
    if (V == 8) {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        const float4 a = Elem<T>::widen(make_uint2(u.x, u.y)), b = Elem<T>::widen(make_uint2(u.z, u.w));
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
        x[V - 4] = b.x, x[V - 3] = b.y, x[V - 2] = b.z, x[V - 1] = b.w;
    } else {
        const float4 a = Elem<T>::load4(p);
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    }
}
template <typename T, int V>
__device__ __forceinline__ void store_run(T* p, const float (&x)[V]) {
    if (V == 8)
        *reinterpret_cast<uint4*>(p) = make_uint4(Elem<T>::pack2(x[0], x[1]), Elem<T>::pack2(x[2], x[3]),
                                                  Elem<T>::pack2(x[V - 4], x[V - 3]), Elem<T>::pack2(x[V - 2], x[V - 1]));
    else
        Elem<T>::store4(p, make_float4(x[0], x[1], x[2], x[3]));
}

}  // namespace kv

int kv_append_launch(const kv::Cache& c, const kv::Batch& b, int dtype, const kv::Rows& k, const kv::Rows& v,
                     const kv::Rows& q, int q_heads, const kv::Rope& rope, void* q_out, cudaStream_t s);
int kv_read_launch(const kv::Cache& c, const kv::Batch& b, int dtype, void* k_out, void* v_out, cudaStream_t s);
unsigned kv_cache_take_error();

}  // namespace mmq
