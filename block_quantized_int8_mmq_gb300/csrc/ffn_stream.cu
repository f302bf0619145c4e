// The forward products of a few rows (up to 16): k_ffn_stream.
//
// Bound: HBM, the weights once.  A warp takes 16 weight rows and a run of 256-value chunks, which it streams
// through a ring of its own (TMA boxes of 16 rows; rows that do not begin on 16 bytes by asynchronous copies) and
// multiplies with m16n8k16 products: weights on the M side, rows of x, as k_ffn_rows has laid them out, on the N
// side.  The codes enter as they are, exact in f16 (Q4_K and Q5_K of 16-bit rows as subnormals, code x 2^-24, with no instruction
// beyond the bytes' placing; Q6_K and Q8_0 less their centre), and every block's sum is scaled in f32, so f32 rows take two
// terms of x but one of the weights.  The order of the values within a block is free as long as both sides
// share it: a thread's share of a block's codes are the bytes it reads at once.  Q4_K's and Q5_K's minimums multiply
// the blocks' sums of x (16 values of the reduction: eight sums in two terms): one product a chunk.
// The products leave the tensor core every 32 values (16 for Q6_K).
// Measured, weights not in L2: gated 1 x 18944 x 3584 of Q4_K 22.5 us (3.4 TB/s), 1 x 3584 x 18944 of Q8_0 18.8 (3.8 TB/s), what
// starts and ends included; 1 x 512 x 3584 4.8.
//
// A CTA is `groups` runs of 16 weight rows (gate and up of the same columns are two) times `splits` shares of the
// reduction, added up in shared memory in their order.  Few columns and a long reduction: a cluster of CTAs shares it, and
// each adds up its part of the outputs from all of them (9 x 3584 x 18944 of Q6_K 34.7 -> 28.4 us in pairs, on 150 SMs
// instead of 112; 3 x 333 x 13824 of Q4_K 16 -> 9.8 in fours).
#include "ffn_rows.cuh"
#include "ffn_weights.cuh"

namespace mmq {
namespace {

using namespace ffn;

__device__ unsigned g_ffn_stream_error;

constexpr int WARPS = STREAM_WARPS, SLAB = STREAM_SLAB;

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_fresh(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// What stands in the shared memory of the cluster's CTA `rank` where p does in this one's.
__device__ __forceinline__ float peer_value(const float* p, int rank) {
    uint32_t at;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(ptx::smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}

// A word at an even byte offset.
__device__ __forceinline__ uint32_t word_at(const uint8_t* p, int off) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(p + (off & ~3));
    return off & 2 ? __funnelshift_r(w[0], w[1], 16) : w[0];
}

// Two codes of a word as f16: bytes 0, 1 (i = 0) or 2, 3; as subnormals, or less a centre.
__device__ __forceinline__ uint32_t small(uint32_t codes, int i) { return __byte_perm(codes, 0u, i ? 0x4342 : 0x4140); }
__device__ __forceinline__ uint32_t centred(uint32_t codes, int i, uint32_t bias) {
    return h2(__hsub2(umma::bits_h2(__byte_perm(codes, 0x64646464u, i ? 0x4342 : 0x4140)), umma::bits_h2(bias)));
}

template <int FMT, int NT, int TERMS, bool HELD>
__global__ void __launch_bounds__(32 * WARPS, 1) k_ffn_stream(const __grid_constant__ Stream a) {
    constexpr int CB = chunk_bytes(FMT);
    constexpr bool MINS = is_kquant(FMT), ROWS = !MINS;  // ROWS: rows may be off 16 bytes
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ __align__(8) uint64_t s_bar[WARPS * R_MOST];
    __shared__ int s_abort;
    __shared__ unsigned s_top[STREAM_ROWS];  // HELD: bits of the rows' largest magnitudes
    const int tid = threadIdx.x, lane = tid & 31, wid = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int g = lane >> 2, t = lane & 3;
    const int group = wid / a.splits, split = wid - group * a.splits;
    const bool works = group < a.groups;
    const uint32_t bars = ptx::smem_u32(s_bar) + 8 * wid * R_MOST;
    if (lane < a.rs) ptx::mbar_init(bars + 8 * lane, a.aligned ? 1 : 32);
    if (tid == 0) s_abort = 0;
    if (tid < STREAM_ROWS) s_top[tid] = 0u;
    ptx::fence_barrier_init();
    __syncthreads();
    volatile int* abort = &s_abort;
    unsigned* err = &g_ffn_stream_error;

    // this warp's rows and chunks
    const int per = a.mats == 2 ? a.groups / 2 : a.groups;       // column runs of a CTA
    const int mat = a.mats == 2 && group >= per ? 1 : 0;
    const int rank = blockIdx.x % a.cluster, run0 = blockIdx.x / a.cluster * per, shares = a.cluster * a.splits;
    const int n0 = (run0 + group - mat * per) * SLAB, share = rank * a.splits + split;
    const int c0 = works && n0 < a.N ? (int)((long long)a.chunks * share / shares) : 0;
    const int c1 = works && n0 < a.N ? (int)((long long)a.chunks * (share + 1) / shares) : 0;
    const int stage = SLAB * a.slot;
    uint8_t* ring = smem + wid * a.rs * stage;
    int asked = c0, f_slot = 0;
    auto fetch = [&]() {
        if (asked >= c1) return;
        const uint32_t bar = bars + 8 * f_slot, dst = ptx::smem_u32(ring) + f_slot * stage;
        if (!ROWS || a.aligned) {
            if (ptx::elect_one()) {
                ptx::mbar_arrive_expect_tx(bar, SLAB * CB);
                ptx::tma_load_2d(dst, &a.map[mat], bar, asked * (CB / 2), n0);
            }
            __syncwarp();
        } else {
            const int sub = 16 * (lane & 7), r0 = lane >> 3, in_row = asked * CB, len = min(CB, (int)a.row_bytes - in_row);
            const uint8_t* p = a.w[mat] + (n0 + r0) * a.row_bytes + in_row;
            // the matrix's last bytes do not fill 16: a copy there takes what there is
            const bool tail = in_row + len == (int)a.row_bytes;
#pragma unroll
            for (int r = 0; r < SLAB; r += 4, p += 4 * a.row_bytes) {
                const int mis = (int)(reinterpret_cast<uintptr_t>(p) & 15), need = n0 + r0 + r < a.N ? mis + len - sub : 0;
                const uint8_t* src = p - mis + sub;
#pragma unroll
                for (int k = 0; k < slot_bytes(FMT, false); k += 128)
                    if (k < need) cp_async16(dst + (r0 + r) * a.slot + sub + k, src + k, tail ? min(16, need - k) : 16);
            }
            cp_async_arrive(bar);
        }
        ++asked;
        if (++f_slot == a.rs) f_slot = 0;
    };
    for (int i = 0; i < a.rs; ++i) fetch();

    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
    ptx::grid_dep_wait();  // the rows are there
    // (not before: the next call asks for its weights before it waits, and must find those that any kernel but this one wrote)
    ptx::grid_dep_launch_dependents();
    // HELD: all of x in shared memory, after the rings, laid out here while the first weights are on their way; so there
    // is no other kernel and no memory beside
    const int x_steps = (a.K + STEP - 1) / STEP;
    uint8_t* x_held = smem + WARPS * a.rs * stage;
    const int x_step = HELD ? a.M * 128 : NT * 1024;  // bytes of a step's rows (held: only those that there are)
    const long long x_term = HELD ? (long long)x_steps * x_step : a.x_term;
    uint8_t* held_sums = x_held + x_term * TERMS;
    if (HELD) {
        // a cluster's CTA: its chunks' share of the rows, whose largest is of the whole
        const int runs = a.K / 8, places = x_steps * 8;
        const int from = (int)((long long)a.chunks * rank / a.cluster) * 32, to = min(places, (int)((long long)a.chunks * (rank + 1) / a.cluster) * 32);
        auto lay_out = [&](auto type) {
            using T = decltype(type);
            constexpr bool SCALED = !std::is_same<T, __half>::value || MINS;
            const T* x = static_cast<const T*>(a.rows);
            if (SCALED) {
                for (int m = 0; m < a.M; ++m) {
                    float top = 0.f;
#pragma unroll 4
                    for (int c = tid; c < runs; c += 32 * WARPS) {
                        float v[8];
                        load8(x + m * a.rows_stride + 8ll * c, v);
#pragma unroll
                        for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(v[k]));
                    }
                    const unsigned bits = __reduce_max_sync(0xffffffffu, __float_as_uint(top));  // (magnitudes order as their bits)
                    if (lane == 0 && bits) atomicMax(&s_top[m], bits);
                }
                __syncthreads();
            }
            for (int m = 0; m < a.M; ++m) {
                const float down = SCALED ? row_scale(__uint_as_float(s_top[m])).down : 1.f;
                for (int c = from + tid; c < to; c += 32 * WARPS) {
                    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                    if (c < runs) load8(x + m * a.rows_stride + 8ll * c, v);
                    put_at(x_held + (c >> 3) * x_step + m * 128 + (((c ^ m) & 7) << 4), x_term, TERMS == 2, v, down);
                    if (MINS) put_sum(held_sums, NT, m, c, v, down);  // (whole warps: K is a multiple of 256 then)
                }
            }
            __syncthreads();
        };
        if (TERMS == 2)
            lay_out(float{});
        else if (a.dtype == MMQ_BF16)
            lay_out(__nv_bfloat16{});
        else
            lay_out(__half{});
    }
    const uint8_t* x_sums = HELD ? held_sums : a.sums;
    // x for this lane, AHEAD blocks of 32 values at a time and as many ahead of their use: 16 bytes a block and term (Q6_K:
    // two of 8, of its two halves).  Measured one block ahead, from L2: most of a decode's cycles waited for it.
    constexpr int AHEAD = HELD ? 1 : 4 / (NT * TERMS);
    const int x_lane = FMT == FMT_Q6_K ? g * 128 + (((t >> 1) ^ g) << 4) + (t & 1) * 8 : g * 128 + ((t ^ g) << 4);
    const uint8_t* xt = HELD ? x_held : a.x;
    const int b_end = min(8 * c1, a.K / QK);
    const int lane_rows = g < a.M ? g + 8 < a.M ? 2 : 1 : 0;  // rows of x that this lane reads: g, g + 8
    uint4 xv[2][AHEAD][NT][TERMS];
#pragma unroll
    for (int i = 0; i < 2 * AHEAD * NT * TERMS; ++i) (&xv[0][0][0][0])[i] = make_uint4(0u, 0u, 0u, 0u);
    auto load_x = [&](int block, uint4 (&v)[AHEAD][NT][TERMS]) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (block + i >= b_end || lane_rows == 0) break;
            const int at = x_lane ^ ((block + i) & 1) * 64;  // (pieces 4 .. 7 of a step)
            const uint8_t* p = xt + (long long)((block + i) >> 1) * x_step;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (n >= lane_rows) break;
#pragma unroll
                for (int e = 0; e < TERMS; ++e) {
                    const uint8_t* q = p + n * 1024 + e * x_term;
                    if (FMT == FMT_Q6_K) {
                        const uint2 *w0 = reinterpret_cast<const uint2*>(q + at), *w1 = reinterpret_cast<const uint2*>(q + (at ^ 32));
                        const uint2 lo = HELD ? *w0 : __ldg(w0), hi = HELD ? *w1 : __ldg(w1);
                        v[i][n][e] = make_uint4(lo.x, lo.y, hi.x, hi.y);
                    } else {
                        const uint4* w = reinterpret_cast<const uint4*>(q + at);
                        v[i][n][e] = HELD ? *w : __ldg(w);
                    }
                }
            }
        }
    };
    // before block `block` (0 .. 7) of chunk c: the next batch is asked for where one begins
    auto next_x = [&](int c, int block) {
        if (block % AHEAD == 0) load_x(8 * c + block + AHEAD, xv[(block / AHEAD + 1) & 1]);
    };
    // D of a block from its two products (Q6_K: of one 16-value half)
    auto block_sum = [&](const uint32_t (&a0)[4], const uint32_t (&a1)[4], const uint4 (&v)[TERMS], float (&d)[4]) {
#pragma unroll
        for (int e = TERMS - 1; e >= 0; --e) {  // the small terms first
            e == TERMS - 1 ? mma_fresh(d, a0, v[e].x, v[e].y) : mma(d, a0, v[e].x, v[e].y);
            mma(d, a1, v[e].z, v[e].w);
        }
    };

    // Q4_K's and Q5_K's codes: f32 rows take them as normal f16 (the tensor core cuts what lies 2^-24 below a product's exponent as
    // its operands' fields give it, and a subnormal's is up to 2^10 too large: 2e-6 of the outputs' norm, against 2e-7)
    constexpr float CODE_UP = TERMS == 2 ? 1.f : 0x1p24f;
    auto code = [&](uint32_t codes, int i) { return TERMS == 2 ? centred(codes, i, 0x64006400u) : small(codes, i); };

    int st = 0;
    uint32_t par = 0;
    bool ok = true;
    load_x(8 * c0, xv[0]);
#pragma unroll 1
    for (int c = c0; c < c1 && ok; ++c) {
        if (!umma::warp_wait(bars + 8 * st, par, abort, err)) {
            ok = false;
            break;
        }
        const uint8_t* rows[2] = {ring + st * stage + g * a.slot, ring + st * stage + (g + 8) * a.slot};
        int mis[2] = {0, 0};
        if (ROWS && !a.aligned)
#pragma unroll
            for (int r = 0; r < 2; ++r) mis[r] = (int)(((uint32_t)(n0 + g + 8 * r) * (uint32_t)a.row_bytes + (uint32_t)c * CB) & 15u);
        const int last = min(8 * c + 8, b_end);  // Q8_0: the last chunk may be short
        if (MINS) {
            uint2 xs[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n)
                xs[n] = *reinterpret_cast<const uint2*>(x_sums + (((long long)c * NT + n) * 32 + lane) * 8);
            uint4 head[2];
            uint32_t sc[2][2], mn[2][2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                head[r] = *reinterpret_cast<const uint4*>(rows[r]);
                sc[r][0] = head[r].y & 0x3f3f3f3fu;
                mn[r][0] = head[r].z & 0x3f3f3f3fu;
                sc[r][1] = (head[r].w & 0x0f0f0f0fu) | ((head[r].y >> 2) & 0x30303030u);
                mn[r][1] = ((head[r].w >> 4) & 0x0f0f0f0fu) | ((head[r].z >> 2) & 0x30303030u);
            }
            float part[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) part[n][i] = 0.f;
            uint2 qh[2];
            if (FMT == FMT_Q5_K)
#pragma unroll
                for (int r = 0; r < 2; ++r) qh[r] = *reinterpret_cast<const uint2*>(rows[r] + 16 + 8 * t);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint2 q[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) q[r] = *reinterpret_cast<const uint2*>(rows[r] + kq_qs_off(FMT) + 32 * j + 8 * t);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const int block = 2 * j + b;
                    next_x(c, block);
                    uint32_t a0[4], a1[4];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        uint32_t lo = (b ? q[r].x >> 4 : q[r].x) & 0x0f0f0f0fu, hi = (b ? q[r].y >> 4 : q[r].y) & 0x0f0f0f0fu;
                        if (FMT == FMT_Q5_K) {
                            lo |= (block >= 4 ? qh[r].x >> (block - 4) : qh[r].x << (4 - block)) & 0x10101010u;
                            hi |= (block >= 4 ? qh[r].y >> (block - 4) : qh[r].y << (4 - block)) & 0x10101010u;
                        }
                        a0[r] = code(lo, 0), a0[2 + r] = code(lo, 1);
                        a1[r] = code(hi, 0), a1[2 + r] = code(hi, 1);
                    }
                    const float s0 = (float)((sc[0][block >> 2] >> (8 * (block & 3))) & 63u);
                    const float s1 = (float)((sc[1][block >> 2] >> (8 * (block & 3))) & 63u);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float d[4];
                        block_sum(a0, a1, xv[(block / AHEAD) & 1][block % AHEAD][n], d);
                        part[n][0] = fmaf(s0, d[0], part[n][0]);
                        part[n][1] = fmaf(s0, d[1], part[n][1]);
                        part[n][2] = fmaf(s1, d[2], part[n][2]);
                        part[n][3] = fmaf(s1, d[3], part[n][3]);
                    }
                }
            }
            // minimums times the blocks' sums of x (which are stored times 2^-6)
            uint32_t m[4];
#pragma unroll
            for (int r = 0; r < 2; ++r) m[r] = m[2 + r] = code(mn[r][t >> 1], t & 1);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float d[4];
                mma_fresh(d, m, xs[n].x, xs[n].y);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t dd = head[i >> 1].x;
                    acc[n][i] = fmaf(f16_bits_to_f32(dd) * CODE_UP, part[n][i],
                                     fmaf(f16_bits_to_f32(dd >> 16) * (-64.f * CODE_UP), d[i], acc[n][i]));
                }
            }
        } else if (FMT == FMT_Q8_0) {
#pragma unroll
            for (int block = 0; block < 8; ++block) {
                if (8 * c + block >= last) break;
                next_x(c, block);
                uint32_t a0[4], a1[4];
                float s[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int at = 34 * block + mis[r];
                    const uint32_t* w = reinterpret_cast<const uint32_t*>(rows[r] + ((at + 2 + 8 * t) & ~3));
                    const int sh = (at + 2) & 2 ? 16 : 0;
                    const uint32_t w0 = w[0], w1 = w[1], w2 = sh ? w[2] : 0u;
                    const uint32_t lo = __funnelshift_r(w0, w1, sh) ^ 0x80808080u, hi = __funnelshift_r(w1, w2, sh) ^ 0x80808080u;
                    a0[r] = centred(lo, 0, 0x64806480u), a0[2 + r] = centred(lo, 1, 0x64806480u);
                    a1[r] = centred(hi, 0, 0x64806480u), a1[2 + r] = centred(hi, 1, 0x64806480u);
                    s[r] = f16_bits_to_f32(*reinterpret_cast<const uint16_t*>(rows[r] + at));
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float d[4];
                    block_sum(a0, a1, xv[(block / AHEAD) & 1][block % AHEAD][n], d);
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[n][i] = fmaf(s[i >> 1], d[i], acc[n][i]);
                }
            }
        } else {
            float part[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) part[n][i] = 0.f;
            float d[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) d[r] = f16_bits_to_f32(*reinterpret_cast<const uint16_t*>(rows[r] + 208 + mis[r]));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t ql[2][4], qh[2][2], sc[2][2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) ql[r][i] = word_at(rows[r], 64 * h + 16 * i + 4 * t + mis[r]);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        qh[r][i] = word_at(rows[r], 128 + 32 * h + 16 * i + 4 * t + mis[r]);
                        sc[r][i] = word_at(rows[r], 192 + 8 * h + 4 * i + mis[r]);
                    }
                }
#pragma unroll
                for (int T = 0; T < 4; ++T) {
                    const int block = 4 * h + T;
                    next_x(c, block);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {  // a 16-value half of the block
                        uint32_t w[4];
                        float s[2];
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const uint32_t low = (ql[r][2 * (T & 1) + i] >> (4 * (T >> 1))) & 0x0f0f0f0fu;
                            const uint32_t top = (T >= 2 ? qh[r][i] >> (2 * T - 4) : qh[r][i] << (4 - 2 * T)) & 0x30303030u;
                            w[r] = centred(low | top, 0, 0x64206420u), w[2 + r] = centred(low | top, 1, 0x64206420u);
                            s[r] = (float)(int8_t)(sc[r][T >> 1] >> (16 * (T & 1) + 8 * i));
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            float e4[4];
#pragma unroll
                            for (int e = TERMS - 1; e >= 0; --e) {
                                const uint4 v = xv[(block / AHEAD) & 1][block % AHEAD][n][e];
                                const uint32_t b0 = i ? v.z : v.x, b1 = i ? v.w : v.y;
                                e == TERMS - 1 ? mma_fresh(e4, w, b0, b1) : mma(e4, w, b0, b1);
                            }
#pragma unroll
                            for (int k = 0; k < 4; ++k) part[n][k] = fmaf(s[k >> 1], e4[k], part[n][k]);
                        }
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[n][i] = fmaf(d[i >> 1], part[n][i], acc[n][i]);
        }
        __syncwarp();  // the chunk has been read
        fetch();
        if (++st == a.rs) {
            st = 0;
            par ^= 1;
        }
    }
    if (ROWS) cp_async_wait_all();
    if (!ok && (!ROWS || a.aligned))  // let the boxes in flight land before the shared memory goes
        for (int i = 0; i < a.rs; ++i) {
            const int n = asked - c0;
            if (n > i) umma::drain_bar(bars + 8 * i, ((n - i + a.rs - 1) / a.rs - 1) & 1, err);
        }
    // ---- the shares of the reduction in their order, then the outputs: 16 columns side by side
    __syncthreads();
    float* sums = reinterpret_cast<float*>(smem);  // [warp][8 NT rows of x][16 columns]
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) sums[(wid * 8 * NT + 8 * n + 2 * t + (i & 1)) * SLAB + g + 8 * (i >> 1)] = acc[n][i];
    __syncthreads();
    if (a.cluster > 1) cluster_sync();  // (a CTA that gave up comes here too)
    // the sum of a run's shares at row m and column k
    auto total = [&](int group, int m, int k) {
        float z = 0.f;
        for (int c = 0; c < a.cluster; ++c) {
            const float* p = sums + (group * a.splits * 8 * NT + m) * SLAB + k;
            for (int s = 0; s < a.splits; ++s, p += 8 * NT * SLAB) z += a.cluster > 1 ? peer_value(p, c) : *p;
        }
        return z;
    };
    auto output = [&](auto type) {
        using T = decltype(type);
        for (int i = rank * 32 * WARPS + tid; i < per * a.M * SLAB; i += a.cluster * 32 * WARPS) {
            const int k = i % SLAB, m = i / SLAB % a.M, run = i / SLAB / a.M;
            const int n = (run0 + run) * SLAB + k;
            if (n >= a.N) continue;
            const long long at = (long long)m * a.N + n;
            // (the weights' 2^8, which `up` takes back, these weights have not)
            const float up = (!HELD ? __ldg(a.up + m) : !MINS && std::is_same<T, __half>::value ? 1.f / 256.f : row_scale(__uint_as_float(s_top[m])).up) * 256.f;
            float z[2] = {0.f, 0.f};
            for (int w = 0; w < a.mats; ++w) {
                z[w] = fmaf(total(w * per + run, m, k), up, a.bias[w] ? __ldg(a.bias[w] + n) : 0.f);
                if (a.pre[w]) put_one(static_cast<T*>(a.pre[w]) + at, z[w]);
            }
            float y = 0.f;
            with_act(a.act, [&](auto A) {
                float d;
                activate<decltype(A)::value, sizeof(T) == 2>(z[0], y, d);
            });
            if (a.mats == 2) y *= z[1];
            if (a.residual) y += get_one(static_cast<const T*>(a.residual) + m * a.residual_stride + n);
            put_one(static_cast<T*>(a.out) + at, y);
        }
    };
    if (*abort == 0) {
        if (TERMS == 2)
            output(float{});
        else if (a.dtype == MMQ_BF16)
            output(__nv_bfloat16{});
        else
            output(__half{});
    }
    if (a.cluster > 1) cluster_sync();  // its sums have been read
}

template <int FMT, int NT, int TERMS, bool HELD>
int launch(const Stream& a, int smem, int ctas, bool go, const char* fn, cudaStream_t s) {
    static SmemAttr attr;
    auto k = &k_ffn_stream<FMT, NT, TERMS, HELD>;
    const int st = ensure_smem(reinterpret_cast<const void*>(k), SMEM_MOST, attr);
    if (st != MMQ_OK) {
        report(fn, st, "the stream's shared memory was refused");
        return st;
    }
    if (!go) return MMQ_OK;
    ProfScope ps("k_ffn_stream", s);
    return pdl_status(ffn_cluster_launch(k, ctas, 32 * WARPS, a.cluster, smem, s, a), fn);
}

template <int FMT, int NT, int TERMS>
int launch(const Stream& a, int smem, int ctas, bool go, const char* fn, cudaStream_t s) {
    return a.held ? launch<FMT, NT, TERMS, true>(a, smem, ctas, go, fn, s) : launch<FMT, NT, TERMS, false>(a, smem, ctas, go, fn, s);
}

template <int FMT>
int launch(const Stream& a, int smem, int ctas, bool go, const char* fn, cudaStream_t s) {
    if (a.dtype == MMQ_F32) return a.xgroups == 1 ? launch<FMT, 1, 2>(a, smem, ctas, go, fn, s) : launch<FMT, 2, 2>(a, smem, ctas, go, fn, s);
    return a.xgroups == 1 ? launch<FMT, 1, 1>(a, smem, ctas, go, fn, s) : launch<FMT, 2, 1>(a, smem, ctas, go, fn, s);
}

}  // namespace

int ffn_stream_launch(int fmt, const Stream& a, int smem, int ctas, bool go, const char* fn, cudaStream_t s) {
    if (fmt == FMT_Q8_0) return launch<FMT_Q8_0>(a, smem, ctas, go, fn, s);
    if (fmt == FMT_Q4_K) return launch<FMT_Q4_K>(a, smem, ctas, go, fn, s);
    if (fmt == FMT_Q5_K) return launch<FMT_Q5_K>(a, smem, ctas, go, fn, s);
    return launch<FMT_Q6_K>(a, smem, ctas, go, fn, s);
}

unsigned ffn_stream_take_error() {
    unsigned v = 0;
    if (cudaMemcpyFromSymbol(&v, g_ffn_stream_error, sizeof(v)) != cudaSuccess) return 0;
    if (v) {
        const unsigned zero = 0;
        cudaMemcpyToSymbol(g_ffn_stream_error, &zero, sizeof(zero));
    }
    return v;
}

}  // namespace mmq
