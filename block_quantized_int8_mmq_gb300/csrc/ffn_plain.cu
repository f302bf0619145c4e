// The feed-forward operators in their simplest form: a thread per output value, f32 sums, every
// weight decoded where it is used.
#include "ffn.cuh"

namespace mmq {
namespace {

using namespace ffn;

// Value k of the weight row at `row`.
__device__ float weight(int fmt, const uint8_t* row, int k) {
    if (fmt == FMT_Q8_0) {
        const uint8_t* b = row + (long long)(k / QK) * Q8_0_BYTES;
        return f16_bits_to_f32(b[0] | b[1] << 8) * (float)(int8_t)b[2 + k % QK];
    }
    const uint8_t* b = row + (long long)(k / QK_K) * kq_bytes(fmt);
    const int v = k % QK_K;
    if (fmt == FMT_Q6_K) {
        const int h = v / 128, t = v % 128 / 32, l = v % 32;
        const int q = ((b[64 * h + 32 * (t % 2) + l] >> (4 * (t / 2))) & 15) | ((b[128 + 32 * h + l] >> (2 * t)) & 3) << 4;
        return f16_bits_to_f32(b[208] | b[209] << 8) * (float)((int8_t)b[192 + v / 16] * (q - 32));
    }
    const int c = v / 64, h = v % 64 / 32, i = v % 32;
    int q = (b[kq_qs_off(fmt) + 32 * c + i] >> (4 * h)) & 15, sc, mn;
    if (fmt == FMT_Q5_K) q |= ((b[16 + i] >> (2 * c + h)) & 1) << 4;
    uint32_t s[3];
    for (int j = 0; j < 3; ++j) s[j] = b[4 + 4 * j] | b[5 + 4 * j] << 8 | b[6 + 4 * j] << 16 | (uint32_t)b[7 + 4 * j] << 24;
    q4_k_scale_min(s[0], s[1], s[2], v / 32, sc, mn);
    return f16_bits_to_f32(b[0] | b[1] << 8) * (float)(sc * q) - f16_bits_to_f32(b[2] | b[3] << 8) * (float)mn;
}

__device__ __forceinline__ long long row_bytes(const Call& c) {
    return c.fmt == FMT_Q8_0 ? c.K / QK * Q8_0_BYTES : c.K / QK_K * kq_bytes(c.fmt);
}

__global__ void __launch_bounds__(256) k_ffn_forward(const Call c) {
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < c.M * c.N; i += gridDim.x * 256ll) {
        const long long m = i / c.N, n = i - m * c.N;
        float z[2] = {0.f, 0.f};
        for (int g = 0; g < c.mats; ++g) {
            const uint8_t* row = static_cast<const uint8_t*>(c.w[g]) + n * row_bytes(c);
            float sum = 0.f;
            for (int k0 = 0; k0 < c.K; k0 += QK) {
                float part = 0.f;
                for (int k = k0; k < k0 + QK; ++k) part += load(c.x, c.dtype, m * c.x_stride + k) * weight(c.fmt, row, k);
                sum += part;
            }
            z[g] = sum + (c.bias[g] ? c.bias[g][n] : 0.f);
            if (c.pre[g]) store(c.pre[g], c.dtype, i, z[g]);
        }
        float a, d;
        activate(c.act, z[0], a, d);
        if (c.mats == 2) a *= z[1];
        if (c.residual) a += load(c.residual, c.dtype, m * c.residual_stride + n);
        store(c.out, c.dtype, i, a);
    }
}

__device__ __forceinline__ void gradient(const Call& c, long long m, long long n, float (&dz)[2]) {
    const float dy = load(c.x, c.dtype, m * c.x_stride + n);
    dz[0] = dy;
    dz[1] = 0.f;
    if (!c.pre[0]) return;
    float a, d;
    activate(c.act, load(c.pre[0], c.dtype, m * c.N + n), a, d);
    dz[0] = dy * d;
    if (c.mats == 2) {
        dz[0] *= load(c.pre[1], c.dtype, m * c.N + n);
        dz[1] = dy * a;
    }
}

__global__ void __launch_bounds__(256) k_ffn_backward(const Call c) {
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < c.M * c.K; i += gridDim.x * 256ll) {
        const long long m = i / c.K, k = i - m * c.K;
        float sum = 0.f, part = 0.f;
        for (long long n = 0; n < c.N; ++n) {
            float dz[2];
            gradient(c, m, n, dz);
            for (int g = 0; g < c.mats; ++g)
                part += dz[g] * weight(c.fmt, static_cast<const uint8_t*>(c.w[g]) + n * row_bytes(c), (int)k);
            if (n % QK == QK - 1) {
                sum += part;
                part = 0.f;
            }
        }
        store(c.out, c.dtype, i, sum + part);
    }
}

__global__ void __launch_bounds__(256) k_ffn_gradient(const Call c) {
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < c.M * c.N; i += gridDim.x * 256ll) {
        float dz[2];
        gradient(c, i / c.N, i % c.N, dz);
        for (int g = 0; g < c.mats; ++g)
            if (c.dz[g]) store(c.dz[g], c.dtype, i, dz[g]);
    }
}

unsigned grid(long long values) {
    const long long g = (values + 255) / 256, most = device_shape().sms * 64ll;
    return (unsigned)(g < most ? g : most);
}

}  // namespace

int ffn_launch(const Call& c, cudaStream_t s) {
    if (!c.backward) {
        ProfScope ps("k_ffn_forward", s);
        k_ffn_forward<<<grid(c.M * c.N), 256, 0, s>>>(c);
        return launch_status(c.fn);
    }
    if (c.dz[0] || c.dz[1]) {
        ProfScope ps("k_ffn_gradient", s);
        k_ffn_gradient<<<grid(c.M * c.N), 256, 0, s>>>(c);
        if (const int st = launch_status(c.fn)) return st;
    }
    ProfScope ps("k_ffn_backward", s);
    k_ffn_backward<<<grid(c.M * c.K), 256, 0, s>>>(c);
    return launch_status(c.fn);
}

}  // namespace mmq
