// 64 consecutive values of a weight row, from the bytes of its 256-value chunk in shared memory to
// f16 operands: exact integer codes (their bits under 1024's exponent, 1024 and the format's own centre
// taken off again), times the block's scale, less its minimum.
//
// Weights enter the product times 2^8: f16 is then normal from 2^-22 up, and whatever a weight is formed
// from, |scale| times the largest code and the minimum, has to stay below 255 (Check).
// For bf16 rows a block's scale is rounded to f16 first and the weight once more, 2^-11 each: little beside what the rows' own
// type loses (2^-8), and four instructions for two weights.  For f16 rows only the weight is (Fine).  Minimums: Centred.
// For f32 rows the weight is formed in f32 and split in two f16 terms (2^-22).
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
// 16 bytes to shared memory, the first `bytes` of them from src, the others zero; an arrival at a barrier once this
// thread's copies so far have landed.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

constexpr float W_UP = 256.f, W_MOST = 65504.f;

__device__ __forceinline__ uint32_t h2(__half2 h) { return umma::h2_bits(h); }
__device__ __forceinline__ __half2 low2(__half2 h) { return __lows2half2(h, h); }
__device__ __forceinline__ __half2 high2(__half2 h) { return __highs2half2(h, h); }

// What became of the range: NaN or an infinity once a scale was too large.
struct Check {
    float f = 0.f;
    __half2 h = __half2{__half_raw{0}, __half_raw{0}};
    __device__ __forceinline__ void add(__half2 s, __half2 m, float most) {
        const __half2 t = __hfma2(__habs2(s), __float2half2_rn(most), __habs2(m));
        h = __hfma2(t, __float2half2_rn(0.f), h);  // an infinity times 0 stays in the sum
    }
    __device__ __forceinline__ void add(float s, float m, float most) {
        if (!(fabsf(s) * most + fabsf(m) <= W_MOST)) f = 1.f;
    }
    __device__ __forceinline__ bool bad() const { return f != 0.f || !__hbeq2(h, __float2half2_rn(0.f)); }
};

// Q4_K, Q5_K, 16-bit rows: s q - m as s (q - c) + r, c a whole number near m / s that the codes' placing takes off with their
// 1024 and r = c s - m, at most some 0.6 s.  s q and m are each many times what they leave; a rounding of either alone is
// the same for 32 weights, and rows of one sign add it up (bf16 rows, |normal|: 3.4e-3 of the outputs' norm with s and m rounded
// by themselves).  Of two blocks, side by side: s = s1 + s2 and m = m1 + m2 exactly (products of 11 and 6 bits, multiples of
// 2^-16), r from all four.  (m / s beyond 1000: r is most of the weight.)
struct Centred {
    __half2 s1, s2, r, bias;
    __device__ __forceinline__ Centred(uint32_t sc, uint32_t mn, uint32_t dd, float most, Check& check) {
        const __half2 up2 = __float2half2_rn(W_UP), b = umma::bits_h2(0x64006400u), d2 = umma::bits_h2(dd);
        const __half2 sq = __hmul2(__hsub2(umma::bits_h2(__byte_perm(sc, 0x64646464u, 0x4140)), b), up2);
        const __half2 mq = __hmul2(__hsub2(umma::bits_h2(__byte_perm(mn, 0x64646464u, 0x4140)), b), up2);
        s1 = __hmul2(sq, low2(d2));
        s2 = __hfma2(sq, low2(d2), __hneg2(s1));
        const __half2 m1 = __hmul2(mq, high2(d2)), m2 = __hfma2(mq, high2(d2), __hneg2(m1));
        check.add(s1, m1, most);
        // (the quotient of what is not rounded yet: c from s1 would follow its rounding, whose product with q - c then has one sign
        // where m / s lies between two numbers: 1e-5 of the weights' size on the average, 1.2e-3 of a sum of 18944 |normal|)
        const float2 d = __half22float2(d2), s = __half22float2(sq), m = __half22float2(mq);
        const float by = __fdividef(d.y, d.x);
        const __half2 t = __floats2half2_rn(by * __fdividef(m.x, s.x), by * __fdividef(m.y, s.y));
        const __half2 c = h2rint(__hmax2(__hmin2(t, __float2half2_rn(1000.f)), __float2half2_rn(-1000.f)));  // (0 / 0: any will do)
        r = __hadd2(__hfma2(c, s1, __hneg2(m1)), __hfma2(c, s2, __hneg2(m2)));
        bias = __hadd2(__float2half2_rn(1024.f), c);
    }
};

// f16 rows: no rounding but the weight's own (2^-11, 2.1e-4 of the weights' norm; with the scale in one term 2.5e-4), the
// scale in two terms: s1 (q - c) + (s2 (q - c) + r).
struct Fine {
    __half2 s1, s2, r;
    uint32_t bias;
    __device__ __forceinline__ Fine(const Centred& w, int b)
        : s1(b ? high2(w.s1) : low2(w.s1)), s2(b ? high2(w.s2) : low2(w.s2)), r(b ? high2(w.r) : low2(w.r)),
          bias(h2(b ? high2(w.bias) : low2(w.bias))) {}
    __device__ __forceinline__ explicit Fine(float s) : r(__float2half2_rn(0.f)), bias(0x64206420u) {  // Q6_K: no minimum, codes centred on 32
        s1 = __float2half2_rn(s);
        s2 = __float2half2_rn(s - __low2float(s1));
    }
};
__device__ __forceinline__ void four(uint32_t codes, const Fine& l, uint32_t* hi) {
    const __half2 b = umma::bits_h2(l.bias);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const __half2 q = __hsub2(umma::bits_h2(__byte_perm(codes, 0x64646464u, i ? 0x4342 : 0x4140)), b);
        hi[i] = h2(__hfma2(q, l.s1, __hfma2(q, l.s2, l.r)));
    }
}

// Four codes (one per byte) to two pairs of f16, s (q - bias) + m: bf16 rows.
template <bool MIN>
__device__ __forceinline__ void four(uint32_t codes, uint32_t bias, __half2 s, __half2 m, uint32_t* hi) {
    const __half2 b = umma::bits_h2(bias);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const __half2 q = __hsub2(umma::bits_h2(__byte_perm(codes, 0x64646464u, i ? 0x4342 : 0x4140)), b);
        hi[i] = h2(MIN ? __hfma2(q, s, m) : __hmul2(q, s));
    }
}
// The same for f32 rows: hi, and what it leaves in lo.  With a minimum in f32; without one in f16 alone: s = s1 + s2
// (f16 each), hi = q s1 rounded, what that leaves is a product's remainder and an f16 value itself, and q s2 joins it.
struct Scale2 {
    float s, m;
    __half2 s1, s2;
    __device__ __forceinline__ Scale2(float s_, float m_, bool min) : s(s_), m(m_) {
        if (min) return;
        s1 = __float2half2_rn(s_);
        s2 = __float2half2_rn(s_ - __low2float(s1));
    }
};
template <bool MIN>
__device__ __forceinline__ void four(uint32_t codes, uint32_t bias, const Scale2& l, uint32_t* hi, uint32_t* lo) {
    const __half2 b = umma::bits_h2(bias);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const __half2 q = __hsub2(umma::bits_h2(__byte_perm(codes, 0x64646464u, i ? 0x4342 : 0x4140)), b);
        if (!MIN) {
            const __half2 h = __hmul2(q, l.s1);
            hi[i] = h2(h);
            lo[i] = h2(__hfma2(q, l.s2, __hfma2(q, l.s1, __hneg2(h))));
            continue;
        }
        const float2 f = __half22float2(q);
        const unsigned long long w = ptx::fma_f32x2(ptx::f2_bits(f.x, f.y), ptx::f2_bits(l.s, l.s), ptx::f2_bits(l.m, l.m));
        const __half2 h = __floats2half2_rn(__uint_as_float((uint32_t)w), __uint_as_float((uint32_t)(w >> 32)));
        const float2 back = __half22float2(h);
        const unsigned long long r = ptx::add_f32x2(w, ptx::f2_bits(-back.x, -back.y));
        hi[i] = h2(h);
        lo[i] = h2(__floats2half2_rn(__uint_as_float((uint32_t)r), __uint_as_float((uint32_t)(r >> 32))));
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

// Half of a Q6_K chunk, 128 values, as it is read: two quarters share its bytes.
struct Q6Half {
    uint32_t ql[16], qh[8], sc[2], d;
    __device__ __forceinline__ void load(const uint8_t* slot, int H, int mis, bool valid) {
        read_run<16>(slot, 64 * H + mis, ql);
        read_run<8>(slot, 128 + 32 * H + mis, qh);
        read_run<2>(slot, 192 + 8 * H + mis, sc);
        d = valid ? *reinterpret_cast<const uint16_t*>(slot + 208 + mis) * 0x10001u : 0u;
    }
};
// Its first (P = 0) or second quarter: emit(half, hi, lo) as below.
template <bool SPLIT, bool FINE, class Emit>
__device__ __forceinline__ void quarter_q6(const Q6Half& w, int P, Check& check, Emit&& emit) {
    uint32_t hi[16], lo[16];
    const uint32_t sc = P ? w.sc[1] : w.sc[0];
    const float d = f16_bits_to_f32(w.d) * W_UP;
    __half2 sp[2];
    if (!SPLIT && !FINE) {
        const __half2 d2 = umma::bits_h2(w.d), up2 = __float2half2_rn(W_UP), bias = umma::bits_h2(0x64806480u);
        const uint32_t u = sc ^ 0x80808080u;
        // (the sub-scale times 2^8 first, which f16 holds exactly whatever d is)
        sp[0] = __hmul2(__hmul2(__hsub2(umma::bits_h2(__byte_perm(u, 0x64646464u, 0x4140)), bias), up2), d2);
        sp[1] = __hmul2(__hmul2(__hsub2(umma::bits_h2(__byte_perm(u, 0x64646464u, 0x4342)), bias), up2), d2);
        check.add(sp[0], __float2half2_rn(0.f), 32.f);
        check.add(sp[1], __float2half2_rn(0.f), 32.f);
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const int turn = 4 - 2 * (2 * P + b);  // the two high bits of each byte to bits 4 and 5
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const float s = d * (float)(int8_t)(sc >> (16 * b + 8 * g));
            const __half2 s2 = g ? high2(sp[b]) : low2(sp[b]);
            if (SPLIT || FINE) check.add(s, 0.f, 32.f);
            const Scale2 w2(s, 0.f, false);
            const Fine fine(s);
#pragma unroll
            for (int i = 4 * g; i < 4 * g + 4; ++i) {
                const uint32_t c = ((w.ql[8 * b + i] >> (4 * P)) & 0x0f0f0f0fu) |
                                   (__funnelshift_l(w.qh[i], w.qh[i], turn) & 0x30303030u);
                if (SPLIT)
                    four<false>(c, 0x64206420u, w2, hi + 2 * i, lo + 2 * i);
                else if (FINE)
                    four(c, fine, hi + 2 * i);
                else
                    four<false>(c, 0x64206420u, s2, s2, hi + 2 * i);
            }
        }
        emit(b, hi, lo);
    }
}

// Values 64 J .. 64 J + 63 of the chunk at `slot` (mis: bytes before its first, 0 .. 14).  emit(half, hi, lo)
// takes 32 values at a time as 16 pairs.  blocks: Q8_0's 32-value blocks that exist here (0 .. 2), the others are
// zero.  valid: whether there is such a row; where not, zeros come out of whatever is in its place.  J is a constant
// for Q8_0 (its blocks of 34 bytes lie at another word offset in each quarter).
template <int FMT, bool SPLIT, bool FINE, class Emit>
__device__ __forceinline__ void quarter(const uint8_t* slot, int J, int mis, bool aligned, int blocks, bool valid,
                                        Check& check, Emit&& emit) {
    uint32_t hi[16], lo[16];
    const __half2 up2 = __float2half2_rn(W_UP);
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
        uint32_t dd = __byte_perm(w[0], w[8], 0x7610);  // the two blocks' scales
        dd &= (valid && blocks > 0 ? 0xffffu : 0u) | (valid && blocks > 1 ? 0xffff0000u : 0u);
        const __half2 d2 = __hmul2(umma::bits_h2(dd), up2);
        if (!SPLIT) check.add(d2, d2, 127.f);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const float s = f16_bits_to_f32(b ? dd >> 16 : dd) * W_UP;
            if (SPLIT) check.add(s, 0.f, 128.f);
            const Scale2 w2(s, 0.f, false);
            const __half2 s2 = b ? high2(d2) : low2(d2);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t c = (b ? w[9 + i] : __funnelshift_r(w[i], w[i + 1], 16)) ^ 0x80808080u;
                if (SPLIT)
                    four<false>(c, 0x64806480u, w2, hi + 2 * i, lo + 2 * i);
                else
                    four<false>(c, 0x64806480u, s2, s2, hi + 2 * i);
            }
            emit(b, hi, lo);
        }
    } else if (FMT == FMT_Q6_K) {
        Q6Half w;
        w.load(slot, J >> 1, mis, valid);
        quarter_q6<SPLIT, FINE>(w, J & 1, check, emit);
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
        // sub-scales and minimums 2J, 2J + 1 (q4_k_scale_min for two at a time), in the low two bytes
        uint32_t sc, mn;
        if (J < 2) {
            sc = head.y & 0x3f3f3f3fu;
            mn = head.z & 0x3f3f3f3fu;
        } else {
            sc = (head.w & 0x0f0f0f0fu) | ((head.y >> 2) & 0x30303030u);
            mn = ((head.w >> 4) & 0x0f0f0f0fu) | ((head.z >> 2) & 0x30303030u);
        }
        sc >>= 16 * (J & 1);
        mn >>= 16 * (J & 1);
        constexpr float MOST = FMT == FMT_Q5_K ? 31.f : 15.f;
        const uint32_t dd = valid ? head.x : 0u;
        Check none;
        const Centred two(sc, mn, dd, MOST, SPLIT ? none : check);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const float s = f16_bits_to_f32(dd) * W_UP * (float)((sc >> (8 * b)) & 63);
            const float m = f16_bits_to_f32(dd >> 16) * -W_UP * (float)((mn >> (8 * b)) & 63);
            if (SPLIT) check.add(s, m, MOST);
            const Scale2 w2(s, m, true);
            const Fine fine(two, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t c = (b ? q[i] >> 4 : q[i]) & 0x0f0f0f0fu;
                if (FMT == FMT_Q5_K) c |= __funnelshift_l(qh[i], qh[i], 4 - 2 * J - b) & 0x10101010u;
                if (SPLIT)
                    four<true>(c, 0x64006400u, w2, hi + 2 * i, lo + 2 * i);
                else if (FINE)
                    four(c, fine, hi + 2 * i);
                else
                    four<true>(c, fine.bias, fine.s1, fine.r, hi + 2 * i);
            }
            emit(b, hi, lo);
        }
    }
}

}  // namespace ffn
}  // namespace mmq
