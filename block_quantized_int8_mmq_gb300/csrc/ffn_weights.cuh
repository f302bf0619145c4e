// 64 consecutive values of a weight row, from the bytes of its 256-value chunk in shared memory to
// f16 operands: exact integer codes (their bits under 1024's exponent, 1024 and the format's own centre
// taken off again), times the block's scale, less its minimum.
//
// Weights enter the product times 2^8: f16 is then normal from 2^-22 up, and whatever a weight is formed
// from, |scale| times the largest code and the minimum, has to stay below 255 (`bad` otherwise).
// For 16-bit rows the scale and the minimum are rounded to f16 first and the weight once more, 2^-11 each: no more
// than the rows' own type loses, and four instructions for two weights.  For f32 rows the weight is formed in
// f32 and split in two f16 terms (2^-22).
#pragma once

#include "ffn.cuh"
#include "umma.cuh"

namespace mmq {
namespace ffn {

__host__ __device__ constexpr int chunk_bytes(int fmt) { return fmt == FMT_Q8_0 ? 8 * Q8_0_BYTES : kq_bytes(fmt); }
// Bytes from row to row of a chunk in shared memory: an odd number of 16-byte units, so that eight lanes' 16-byte
// reads at one place of their rows touch all banks.  Rows that do not begin on 16 bytes are copied from the
// boundary before to the one behind (Q6_K always, Q8_0 where K % 256 != 0).
__host__ __device__ constexpr int slot_bytes(int fmt, bool aligned) {
    return fmt == FMT_Q8_0 ? (aligned ? 272 : 304) : fmt == FMT_Q6_K ? 240 : kq_bytes(fmt);
}
constexpr float W_UP = 256.f, W_MOST = 65504.f;

// A linear map of codes, s q + m.
struct Lin {
    __half2 s2, m2;
    float s, m;
    __device__ __forceinline__ Lin(float s_, float m_, float most, bool valid, bool& bad) {
        s = valid ? s_ : 0.f;  // rows that are not there: whatever is in their place counts for nothing
        m = valid ? m_ : 0.f;
        bad |= !(fabsf(s) * most + fabsf(m) <= W_MOST);
        s2 = __float2half2_rn(s);
        m2 = __float2half2_rn(m);
    }
};

__device__ __forceinline__ uint32_t h2(__half2 h) { return umma::h2_bits(h); }

// Four codes (one per byte) to two pairs of f16: hi, and for SPLIT what hi leaves in lo.
template <bool SPLIT, bool MIN>
__device__ __forceinline__ void four(uint32_t codes, uint32_t bias, const Lin& l, uint32_t* hi, uint32_t* lo) {
    const __half2 b = umma::bits_h2(bias);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const __half2 q = __hsub2(umma::bits_h2(__byte_perm(codes, 0x64646464u, i ? 0x4342 : 0x4140)), b);
        if (!SPLIT) {
            hi[i] = h2(MIN ? __hfma2(q, l.s2, l.m2) : __hmul2(q, l.s2));
        } else {
            const float2 f = __half22float2(q);
            const float a = MIN ? fmaf(f.x, l.s, l.m) : f.x * l.s, c = MIN ? fmaf(f.y, l.s, l.m) : f.y * l.s;
            const __half2 h = __floats2half2_rn(a, c);
            const float2 back = __half22float2(h);
            hi[i] = h2(h);
            lo[i] = h2(__floats2half2_rn(a - back.x, c - back.y));
        }
    }
}

// W words at an even byte offset, from 8-byte reads: two lanes of sixteen share a bank then.
template <int W>
__device__ __forceinline__ void read_run(const uint8_t* p, int off, uint32_t (&out)[W]) {
    constexpr int N = (4 * W + 13) / 8;
    const uint2* src = reinterpret_cast<const uint2*>(p + (off & ~7));
    uint32_t w[2 * N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint2 v = src[i];
        w[2 * i] = v.x;
        w[2 * i + 1] = v.y;
    }
    const bool odd = off & 4;
    const int sh = (off & 2) * 8;
#pragma unroll
    for (int i = 0; i <= W; ++i) w[i] = odd ? w[i + 1 < 2 * N ? i + 1 : i] : w[i];
#pragma unroll
    for (int i = 0; i < W; ++i) out[i] = __funnelshift_r(w[i], w[i + 1], sh);
}

// Values 64 J .. 64 J + 63 of the chunk at `slot` (mis: bytes before its first, 0 .. 14).  emit(half, hi, lo)
// takes 32 values at a time as 16 pairs.  blocks: Q8_0's 32-value blocks that exist here (0 .. 2), the others are zero.
template <int FMT, bool SPLIT, int J, class Emit>
__device__ __forceinline__ void quarter(const uint8_t* slot, int mis, bool aligned, int blocks, bool valid, bool& bad,
                                        Emit&& emit) {
    uint32_t hi[16], lo[16];
    if (FMT == FMT_Q8_0) {
        uint32_t w[17];
        if (aligned) {
            uint32_t r[20];
#pragma unroll
            for (int i = 0; i < 5; ++i) {
                const uint4 v = *reinterpret_cast<const uint4*>(slot + 64 * J + 16 * i);
                r[4 * i] = v.x, r[4 * i + 1] = v.y, r[4 * i + 2] = v.z, r[4 * i + 3] = v.w;
            }
#pragma unroll
            for (int i = 0; i < 17; ++i) w[i] = r[J + i];
        } else {
            read_run<17>(slot, 68 * J + mis, w);
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const Lin l(f16_bits_to_f32(b ? w[8] >> 16 : w[0]) * W_UP, 0.f, 128.f, valid && b < blocks, bad);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t c = b ? w[9 + i] : __funnelshift_r(w[i], w[i + 1], 16);
                four<SPLIT, false>(c ^ 0x80808080u, 0x64806480u, l, hi + 2 * i, lo + 2 * i);
            }
            emit(b, hi, lo);
        }
    } else if (FMT == FMT_Q6_K) {
        constexpr int H = J >> 1, T = 2 * (J & 1);
        uint32_t ql[16], qh[8], sc[1];
        read_run<16>(slot, 64 * H + mis, ql);
        read_run<8>(slot, 128 + 32 * H + mis, qh);
        read_run<1>(slot, 192 + 4 * J + mis, sc);
        const float d = f16_bits_to_f32(*reinterpret_cast<const uint16_t*>(slot + 208 + mis)) * W_UP;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const Lin l(d * (float)(int8_t)(sc[0] >> (16 * b + 8 * g)), 0.f, 32.f, valid, bad);
#pragma unroll
                for (int i = 4 * g; i < 4 * g + 4; ++i) {
                    const uint32_t low = (ql[8 * b + i] >> (2 * T)) & 0x0f0f0f0fu;
                    const uint32_t top = T + b >= 2 ? qh[i] >> (2 * (T + b) - 4) : qh[i] << (4 - 2 * (T + b));
                    four<SPLIT, false>(low | (top & 0x30303030u), 0x64206420u, l, hi + 2 * i, lo + 2 * i);
                }
            }
            emit(b, hi, lo);
        }
    } else {
        const uint4 head = *reinterpret_cast<const uint4*>(slot);
        uint32_t q[8], qh[8];
        const uint4* src = reinterpret_cast<const uint4*>(slot + kq_qs_off(FMT) + 32 * J);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 v = src[i];
            q[4 * i] = v.x, q[4 * i + 1] = v.y, q[4 * i + 2] = v.z, q[4 * i + 3] = v.w;
        }
        if (FMT == FMT_Q5_K) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint4 v = *reinterpret_cast<const uint4*>(slot + 16 + 16 * i);
                qh[4 * i] = v.x, qh[4 * i + 1] = v.y, qh[4 * i + 2] = v.z, qh[4 * i + 3] = v.w;
            }
        }
        const float d = f16_bits_to_f32(head.x) * W_UP, dmin = f16_bits_to_f32(head.x >> 16) * -W_UP;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            int sc, mn;
            q4_k_scale_min(head.y, head.z, head.w, 2 * J + b, sc, mn);
            const Lin l(d * (float)sc, dmin * (float)mn, FMT == FMT_Q5_K ? 31.f : 15.f, valid, bad);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t c = (b ? q[i] >> 4 : q[i]) & 0x0f0f0f0fu;
                if (FMT == FMT_Q5_K) {
                    constexpr int S = 2 * J;
                    c |= (S + b >= 4 ? qh[i] >> (S + b - 4) : qh[i] << (4 - S - b)) & 0x10101010u;
                }
                four<SPLIT, true>(c, 0x64006400u, l, hi + 2 * i, lo + 2 * i);
            }
            emit(b, hi, lo);
        }
    }
}

}  // namespace ffn
}  // namespace mmq
