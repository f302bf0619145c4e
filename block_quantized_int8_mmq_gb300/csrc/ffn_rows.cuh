// Rows of x as f16 operands: their scaling and their places in a tile, for the row kernels (ffn_rows.cu) and for the
// stream of weights, which lays few rows out by itself.
#pragma once

#include "ffn.cuh"
#include "kv.cuh"
#include "umma.cuh"

namespace mmq {
// A launch as launch_pdl's, its CTAs in clusters (1: none), of which `ctas` is a multiple.
template <class Args>
cudaError_t ffn_cluster_launch(void (*kernel)(Args), int ctas, int threads, int cluster, int smem, cudaStream_t s,
                               const std::remove_const_t<Args>& args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args);
}

namespace ffn {

struct Scale {
    float down, up;
};
__device__ __forceinline__ Scale row_scale(float amax) {
    // biased exponent; NaN and infinity count as the largest
    const int e = max(22, min(254, (int)((__float_as_uint(amax) >> 23) & 255)));
    return {__uint_as_float((uint32_t)(267 - e) << 23), __uint_as_float((uint32_t)(e - 21) << 23)};
}

// Eight values of a row to their place, and what f16 leaves of them `term` bytes on.
__device__ __forceinline__ void put_at(uint8_t* p, long long term, bool two, const float (&v)[8], float down) {
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
    if (two) *reinterpret_cast<uint4*>(p + term) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
}
__device__ __forceinline__ void put(const Rows& r, int m, int step, int chunk, const float (&v)[8], float down) {
    put_at(r.tiles + ((long long)step * r.groups + (m >> 3)) * 1024 + (m & 7) * 128 + ((chunk ^ (m & 7)) << 4), r.term,
           r.dtype == MMQ_F32, v, down);
}

// The sum of a block of 32 values, held by four neighbouring threads, in two f16 terms, times 2^-6 so that they fit (rows are
// scaled to [2^13, 2^14) here, so what the terms leave, 2^-19, is 2^-32 of the row's largest value): in the order in which
// k_ffn_stream's product takes them, per 256 values and eight rows 256 bytes.
__device__ __forceinline__ void put_sum(uint8_t* sums, int groups, int m, int run, const float (&v)[8], float down) {
    float s = ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    if (run & 3) return;
    s *= down * 0x1p-6f;
    const int block = run >> 2, j = block & 7;
    uint8_t* p = sums + (((long long)(block >> 3) * groups + (m >> 3)) * 32 + (m & 7) * 4 + (j >> 1)) * 8 + (j & 1) * 2;
    const __half hi = __float2half_rn(s);
    *reinterpret_cast<__half*>(p) = hi;
    *reinterpret_cast<__half*>(p + 4) = __float2half_rn(s - __half2float(hi));
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

}  // namespace ffn
}  // namespace mmq
