// Shared pieces of the feed-forward operators over block-quantized weights: the arguments that
// the C entry points hand to the launchers, and the activations with their derivatives.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

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

// What the row kernels write: f16 tiles, per step of 64 values and group of 8 rows 1024 bytes.
struct Rows {
    const void* x;
    long long stride;
    int dtype, act, mats, rows, width, groups;
    const void* pre[2];
    void* dz[2];
    uint8_t* tiles;
    long long term;  // bytes from the first terms to the second
    uint8_t* sums;   // where the sums of 32-value blocks go (k_ffn_stream), or nullptr
    float* up;
    unsigned* counters;
    int n_counters;
};

struct Tile {
    CUtensorMap map[2];            // of the weight matrices, where rows begin on 16 bytes
    const uint8_t* w[2];
    long long row_bytes;           // of a weight row
    const uint8_t* x;              // the rows' tiles
    long long x_term;
    const float* up;
    float* parts;
    unsigned* counters;
    int mats, M, N, K, width;    // width: of the output
    int sub;                     // 64-value pieces of the reduction in a step
    int groups, mtiles, nt;      // groups of 8 rows, row tiles, rows in a tile (a multiple of 16)
    int units, steps, chunks;    // steps (64 or 128 values of the reduction) and chunks of a unit
    int rounds, rest;            // rounds of whole units, then `rest` units cut into equal runs of chunks
    int aligned, slot, rs, xs;   // weight rows begin on 16 bytes; bytes of a chunk's place; ring lengths
    int dtype, act;
    const float* bias[2];
    const void* residual;
    long long residual_stride;
    void* pre[2];
    void* out;
};

// The products of few rows (k_ffn_stream).
struct Stream {
    CUtensorMap map[2];            // of the weight matrices, where rows begin on 16 bytes
    const uint8_t* w[2];
    long long row_bytes;           // of a weight row
    const void* rows;              // x where it is held in shared memory, else
    long long rows_stride;
    const uint8_t* x;              // its tiles
    long long x_term;
    const uint8_t* sums;           // Q4_K, Q5_K: the blocks' sums
    const float* up;
    int mats, M, N, K, chunks, xgroups;  // xgroups: of 8 rows
    int groups, splits;            // of a CTA: runs of 16 weight rows, shares of the reduction
    int cluster;                   // CTAs that share the same runs' reduction
    int aligned, slot, rs, held;   // bytes of a chunk's row in shared memory, places of a warp's ring, whether x is held there too
    int dtype, act;
    const float* bias[2];
    const void* residual;
    long long residual_stride;
    void* pre[2];
    void* out;
};
constexpr int STREAM_ROWS = 16, STREAM_WARPS = 16, STREAM_SLAB = 16;  // rows of x at most, warps, weight rows of a warp

constexpr int W_WARPS = 16, C_WARPS = 1, I_WARPS = 2, THREADS = (W_WARPS + C_WARPS + 1 + I_WARPS) * 32;
constexpr int STEP = 64;     // values of the reduction that are multiplied together
constexpr int CHUNK = 256;   // values of a weight row that are copied together
constexpr int RING = 8, R_MOST = 8;  // barriers of steps; longest ring of weight chunks
// SUB: 64-value pieces of the reduction in a step.  Two where TMEM has the room (16-bit rows, forward, up to 128 rows
// a tile): a step costs its warps some 600 cycles of waits and loops, which few rows' products do not cover.
template <bool SPLIT, bool BACK, int SUB = 1>
struct Shape {
    static constexpr int TERMS = SPLIT ? 2 : 1;
    static constexpr int NT = SPLIT ? 64 : SUB == 2 ? 128 : 192;  // rows of x in a tile, at most
    static constexpr int DB = SPLIT ? 2 : 1;          // accumulator buffers
    static constexpr int D_COLS = 2 * NT;             // of a buffer: two weight tiles
    static constexpr int COL_A = DB * D_COLS;         // forward: weights, two stages
    static constexpr int A_COLS = 64 * TERMS * SUB;   // of a stage: two tiles, 32 columns a term and piece
    static constexpr int A_BYTES = STEP * CHUNK * 2;  // backward: a stage's term in shared memory
    static_assert(COL_A + (BACK ? 0 : 2 * A_COLS) <= 512, "TMEM columns");
};
// Rings of weight chunks, 32 rows each: forward, one for each 32 of the 256 weight rows, which two warps share;
// backward, one for each half of a step's 64 rows and each of the two sets of warps.
__host__ __device__ constexpr int rings(bool back) { return back ? 4 : 8; }
constexpr int SMEM_MOST = 232448 - 2048;  // less what is static

__device__ __forceinline__ float get_one(const float* p) { return *p; }
__device__ __forceinline__ float get_one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float get_one(const __half* p) { return __half2float(*p); }
__device__ __forceinline__ void put_one(float* p, float v) { *p = v; }
__device__ __forceinline__ void put_one(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put_one(__half* p, float v) { *p = __float2half_rn(v); }

// e^x.  FAST: 2^(x log2 e) with the argument rounded to f32: 2^-23 of it off, which is nothing beside a 16-bit value.
template <bool FAST>
__device__ __forceinline__ float exponential(float x) {
    return FAST ? __expf(x) : expf(x);
}

// act(z) and act'(z).  A NaN stays one.  The quotients are 1 / (1 + e) with two ulp, and 0 where e is above 2^126.
template <int ACT, bool FAST>
__device__ __forceinline__ void activate(float z, float& a, float& d) {
    if (ACT == MMQ_ACT_NONE) {
        a = z;
        d = 1.f;
    } else if (ACT == MMQ_ACT_RELU) {
        a = z < 0.f ? 0.f : z;
        d = z > 0.f ? 1.f : 0.f;
    } else if (ACT == MMQ_ACT_SILU) {
        const float s = __fdividef(1.f, 1.f + exponential<FAST>(-z));
        a = z * s;
        d = s * (1.f + z * (1.f - s));
    } else if (ACT == MMQ_ACT_GELU) {
        const float s = 0.5f * erfcf(-0.70710678118654752f * z);
        a = z * s;
        d = s + z * 0.39894228040143268f * exponential<FAST>(-0.5f * z * z);
    } else {  // gelu, by tanh: (1 + tanh(t)) / 2 = 1 / (1 + exp(-2 t))
        const float z2 = fminf(z * z, 1e30f);  // (infinite, it would make NaN of the derivative's s (1 - s), which is 0 there)
        const float s = __fdividef(1.f, 1.f + exponential<FAST>(-1.5957691216057308f * z * (1.f + 0.044715f * z2)));
        a = z * s;
        d = s + z * s * (1.f - s) * 1.5957691216057308f * (1.f + 0.134145f * z2);
    }
}
// f(integral_constant of the activation): one branch for a loop of them
template <class F>
__device__ __forceinline__ void with_act(int act, F&& f) {
    if (act == MMQ_ACT_SILU)
        f(std::integral_constant<int, MMQ_ACT_SILU>{});
    else if (act == MMQ_ACT_GELU)
        f(std::integral_constant<int, MMQ_ACT_GELU>{});
    else if (act == MMQ_ACT_GELU_TANH)
        f(std::integral_constant<int, MMQ_ACT_GELU_TANH>{});
    else if (act == MMQ_ACT_RELU)
        f(std::integral_constant<int, MMQ_ACT_RELU>{});
    else
        f(std::integral_constant<int, MMQ_ACT_NONE>{});
}

}  // namespace ffn

int ffn_launch(const ffn::Call& c, cudaStream_t s);
// go: false asks for the shared memory that the kernel needs and launches nothing, so that a refusal comes before any launch
int ffn_rows_launch(const ffn::Rows& r, bool back, bool go, const char* fn, cudaStream_t s);
int ffn_forward_launch(int fmt, const ffn::Tile& a, int smem, int ctas, bool go, const char* fn, cudaStream_t s);
int ffn_backward_launch(int fmt, const ffn::Tile& a, int smem, int ctas, bool go, const char* fn, cudaStream_t s);
int ffn_stream_launch(int fmt, const ffn::Stream& a, int smem, int ctas, bool go, const char* fn, cudaStream_t s);

}  // namespace mmq
