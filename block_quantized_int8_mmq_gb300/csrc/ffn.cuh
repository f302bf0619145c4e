// Shared pieces of the feed-forward operators over block-quantized weights: the arguments that
// the C entry points hand to the launchers, and the activations with their derivatives.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace mmq {
namespace ffn {

// One call.  Forward: rows x [M][K], `mats` weights [N][K] (one, or gate and up), out [M][N].
// Backward: rows dz [M][N] of each weight (formed from dy and pre), out = dx [M][K].
struct Call {
    const char* fn;
    int fmt, dtype, act, mats;
    bool backward;
    long long M, N, K;
    const void* w[2];
    const void* x;  // forward: the rows; backward: dy
    long long x_stride;
    const float* bias[2];
    const void* residual;
    long long residual_stride;
    void* pre[2];  // forward: where z (or g, u) go, or nullptr; backward: read, nullptr where act is none
    void* dz[2];   // backward: where dz (or dg, du) go, or nullptr
    void* out;
};

__device__ __forceinline__ float load(const void* p, int dtype, long long i) {
    if (dtype == MMQ_F32) return static_cast<const float*>(p)[i];
    if (dtype == MMQ_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    return __half2float(static_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ void store(void* p, int dtype, long long i, float v) {
    if (dtype == MMQ_F32)
        static_cast<float*>(p)[i] = v;
    else if (dtype == MMQ_BF16)
        static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else
        static_cast<__half*>(p)[i] = __float2half_rn(v);
}

// act(z) and act'(z).  A NaN stays one.
__device__ __forceinline__ void activate(int act, float z, float& a, float& d) {
    if (act == MMQ_ACT_NONE) {
        a = z;
        d = 1.f;
    } else if (act == MMQ_ACT_RELU) {
        a = z < 0.f ? 0.f : z;
        d = z > 0.f ? 1.f : 0.f;
    } else if (act == MMQ_ACT_SILU) {
        const float s = 1.f / (1.f + expf(-z));
        a = z * s;
        d = s * (1.f + z * (1.f - s));
    } else if (act == MMQ_ACT_GELU) {
        const float s = 0.5f * erfcf(-0.70710678118654752f * z);
        a = z * s;
        d = s + z * 0.39894228040143268f * expf(-0.5f * z * z);
    } else {  // gelu, by tanh: (1 + tanh(t)) / 2 = 1 / (1 + exp(-2 t))
        const float z2 = z * z, s = 1.f / (1.f + expf(-1.5957691216057308f * z * (1.f + 0.044715f * z2)));
        a = z * s;
        d = s + z * s * (1.f - s) * 1.5957691216057308f * (1.f + 0.134145f * z2);
    }
}

}  // namespace ffn

int ffn_launch(const ffn::Call& c, cudaStream_t s);
unsigned ffn_take_error();

}  // namespace mmq
