// The products of the feed-forward operators: k_ffn_tile.
//
// A unit is 256 weight rows (forward: 128 of gate and the same 128 of up, or 256 in a row; backward: 256
// columns) by up to NT_MOST rows of x, summed over the whole reduction.  Weights are the M side of the tensor
// cores' products (two tiles of 128), rows of x the N side, so one row costs what sixteen do, an output's
// epilogue finds gate and up in one TMEM lane, and a warp stores 32 neighbouring columns at a time.  Roles of a CTA:
//   a copy warp       chunks of 256 values of the weight rows into rings, as TMA boxes of 32 rows; where rows do not
//                     begin on 16 bytes the weight warps copy them themselves;
//   weight warps (16) turn them into f16 (ffn_weights.cuh): forward, a thread per weight row, straight
//                     into TMEM as the A operand; backward, where the reduction runs over weight rows, into shared
//                     memory as an MN-major A operand (8 x 16-byte core matrices, no transpose).  Then the
//                     epilogue, a thread per lane;
//   a loader warp     the rows' tiles, which k_ffn_rows has laid out, one bulk copy a step and term;
//   issuer warps (2)  the products of a weight tile each, 64 values of the reduction a step.
// f32 rows (SPLIT): rows and weights in two f16 terms each, three products, and the accumulators move to registers
// every 128 values of the reduction: the tensor core's additions round towards zero, and over a long sum that
// would be more than f32 allows.
//
// Bound: the tensor cores at 192 rows (a 64-value step 0.50 us of 0.59; gated 2048 x 18944 x 3584 of Q4_K, bf16, 371 us in a graph
// and 400 called back to back, under the power cap: 1.50 and 1.39 PFLOP/s), the weights' way to f16 at few rows (0.55 us a step, f32
// rows 1.1; Q6_K 0.9: 9.4 instructions a weight, the ALU pipe 0.66 busy) and for Q5_K and Q6_K at all; backward 0.65 us a step,
// both operands read from shared memory (2048 rows 390 to 400 us, 1.4 PFLOP/s).
//
// The work is dealt unit by unit in rounds; where the last round would leave too many SMs idle it and the one before
// are laid end to end instead and cut into equal runs.  A unit that is cut leaves its parts in scratch memory, and the
// last CTA to arrive adds them in their order: the order of summation depends on the sizes alone.
#pragma once

#include "ffn_weights.cuh"
#include "kv.cuh"

namespace mmq {
namespace ffn {

static __device__ unsigned g_ffn_tile_error;  // of each translation unit its own
// the bound of the weight warps' wait for a unit's sums, in ns (mmq_debug_set_wait_limit)
static __device__ unsigned long long g_ffn_tile_wait_limit = umma::WAIT_LIMIT_NS;

// SPLIT: steps between two moves of the accumulators.  Measured two against four: 8.4e-7 -> 3.8e-7 of a projection's norm,
// 66 -> 69 us (517 x 3584 x 3584 of Q5_K; 70 by now).
constexpr int PERIOD = 2;

// The pieces of work of a CTA: (unit, first chunk, end).
struct Pieces {
    int r = 0;
    long long x, x1;
    __device__ __forceinline__ explicit Pieces(const Tile& a) {
        const long long all = (long long)a.rest * a.chunks;
        x = all * blockIdx.x / gridDim.x;
        x1 = all * (blockIdx.x + 1) / gridDim.x;
    }
    __device__ __forceinline__ bool next(const Tile& a, int& unit, int& c0, int& c1) {
        if (r < a.rounds) {
            unit = r++ * (int)gridDim.x + (int)blockIdx.x;
            c0 = 0;
            c1 = a.chunks;
            if (unit < a.units - a.rest) return true;
        }
        if (x >= x1) return false;
        const int u = (int)(x / a.chunks);
        unit = a.units - a.rest + u;
        c0 = (int)(x - (long long)u * a.chunks);
        c1 = (int)min((long long)a.chunks, c0 + (x1 - x));
        x += c1 - c0;
        return true;
    }
};
// the CTA whose run holds chunk x of the units that are cut
__device__ __forceinline__ int run_owner(const Tile& a, long long x) {
    return (int)(((x + 1) * gridDim.x - 1) / ((long long)a.rest * a.chunks));
}

// A barrier of the weight warps: whether all of them came with ok.  One whose wait gave up comes too, wherever another
// may be waiting for it.
__device__ __forceinline__ bool sync_weight_warps(bool ok) {
    uint32_t all;
    __syncwarp();
    asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.and.pred q, 1, 512, p;\n selp.u32 %0, 1, 0, q;\n}"
                 : "=r"(all)
                 : "r"((uint32_t)ok)
                 : "memory");
    return all != 0u;
}
// A barrier of all warps, each at the end of its role: no wait is left that could give up.
__device__ __forceinline__ void sync_roles() {
    __syncwarp();
    asm volatile("bar.sync 2, %0;" ::"n"(THREADS) : "memory");
}

template <bool FAST>
__device__ __forceinline__ void activate8(int act, float (&v)[8]) {
    if (act == MMQ_ACT_NONE) return;
    with_act(act, [&](auto A) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float a, d;
            activate<decltype(A)::value, FAST>(v[i], a, d);
            v[i] = a;
        }
    });
}

// Eight rows of x (m .. m + count - 1) of an output column: stored with `stride` elements between them.
template <typename T>
__device__ __forceinline__ void store8(void* p, long long at, long long stride, int count, const float (&v)[8]) {
    T* q = static_cast<T*>(p) + at;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (i < count) put_one(q, v[i]);
        q += stride;
    }
}

// What an output column needs beside its sums, asked for before they are there.
struct Beside {
    float up[8], r[2][8];
};
template <typename T, bool BACK>
__device__ __forceinline__ void beside8(const Tile& a, int pair, int lane_row, int m, int count, Beside& w) {
    if (count == 8) {
        const float4 u = __ldg(reinterpret_cast<const float4*>(a.up + m)), v = __ldg(reinterpret_cast<const float4*>(a.up + m + 4));
        w.up[0] = u.x, w.up[1] = u.y, w.up[2] = u.z, w.up[3] = u.w, w.up[4] = v.x, w.up[5] = v.y, w.up[6] = v.z, w.up[7] = v.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) w.up[i] = i < count ? __ldg(a.up + m + i) : 0.f;
    }
    if (BACK || !a.residual) return;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        const int n = pair * 256 + g * 128 + lane_row;
        const T* q = static_cast<const T*>(a.residual) + m * a.residual_stride + n;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w.r[g][i] = i < count && n < a.width ? get_one(q) : 0.f;
            q += a.residual_stride;
        }
    }
}

// The outputs of a lane's columns: z0, z1 are the sums of its two tiles.
template <typename T, bool BACK>
__device__ __forceinline__ void finish8(const Tile& a, int pair, int lane_row, int m, int count, const Beside& w,
                                        float (&z0)[8], float (&z1)[8]) {
    if (!BACK && a.mats == 2) {
        const int n = pair * 128 + lane_row;
        if (n >= a.width) return;
        const long long at = (long long)m * a.width + n;
        const float b0 = a.bias[0] ? __ldg(a.bias[0] + n) : 0.f, b1 = a.bias[1] ? __ldg(a.bias[1] + n) : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            z0[i] = fmaf(z0[i], w.up[i], b0);
            z1[i] = fmaf(z1[i], w.up[i], b1);
        }
        if (a.pre[0]) store8<T>(a.pre[0], at, a.width, count, z0);
        if (a.pre[1]) store8<T>(a.pre[1], at, a.width, count, z1);
        activate8<sizeof(T) == 2>(a.act, z0);
#pragma unroll
        for (int i = 0; i < 8; ++i) z0[i] *= z1[i];
        store8<T>(a.out, at, a.width, count, z0);
        return;
    }
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        float(&z)[8] = g ? z1 : z0;
        const int n = pair * 256 + g * 128 + lane_row;
        if (n >= a.width) continue;
        const long long at = (long long)m * a.width + n;
        const float b = !BACK && a.bias[0] ? __ldg(a.bias[0] + n) : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = fmaf(z[i], w.up[i], b);
        if (!BACK) {
            if (a.pre[0]) store8<T>(a.pre[0], at, a.width, count, z);
            activate8<sizeof(T) == 2>(a.act, z);
            if (a.residual)
#pragma unroll
                for (int i = 0; i < 8; ++i) z[i] += w.r[g][i];
        }
        store8<T>(a.out, at, a.width, count, z);
    }
}

// Forward, one piece a step: the steps of a chunk take its quarters in the order 0, 2, 1, 3, so that a set's two are
// side by side (Q6_K's share their bytes); Q8_0, whose last chunk may be short, as they come.
__host__ __device__ constexpr int step_of(int fmt, int q) { return fmt == FMT_Q8_0 || q == 0 || q == 3 ? q : 3 - q; }

template <int FMT, bool SPLIT, bool BACK, int SUB, bool FINE>
__global__ void __launch_bounds__(THREADS, 1) k_ffn_tile(const __grid_constant__ Tile a) {
    using S = Shape<SPLIT, BACK, SUB>;
    constexpr int PER = CHUNK / STEP / SUB;  // forward: steps of a chunk
    constexpr int TERMS = S::TERMS;
    constexpr int NG = rings(BACK), GW = W_WARPS / NG;  // rings, weight warps that share one
    constexpr int CB = chunk_bytes(FMT);
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ __align__(8) uint64_t s_bar[2 * RING + 4 + 2 * NG * R_MOST + 2];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_last;
    const int tid = threadIdx.x, lane = tid & 31, wid = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const uint32_t bars = ptx::smem_u32(s_bar);
    // Steps are counted through all pieces: full (the rows' tile and the set's weights are there) and empty (its products
    // are done) of step n at n % RING.
    const uint32_t full = bars, empty = full + 8 * RING, d_full = empty + 8 * RING, d_empty = d_full + 16;
    const uint32_t raw_full = d_empty + 16, raw_empty = raw_full + 8 * NG * R_MOST, done = raw_empty + 8 * NG * R_MOST;
    const int xb = a.nt * 128 * TERMS * SUB;  // bytes of a step's rows
    const uint32_t xs_addr = ptx::smem_u32(smem), as_addr = xs_addr + a.xs * xb;
    const uint32_t raw_addr = as_addr + (BACK ? 2 * TERMS * S::A_BYTES : 0);
    uint8_t* a_smem = smem + a.xs * xb;
    uint8_t* raw = a_smem + (BACK ? 2 * TERMS * S::A_BYTES : 0);
    if (tid < RING) {
        ptx::mbar_init(full + 8 * tid, W_WARPS / 2 + 1);
        ptx::mbar_init(empty + 8 * tid, I_WARPS);
    } else if (tid < RING + 2) {
        const int i = tid - RING;
        ptx::mbar_init(d_full + 8 * i, I_WARPS);
        ptx::mbar_init(d_empty + 8 * i, W_WARPS);
        ptx::mbar_init(done + 8 * i, 1);
        if (a.aligned && i < a.mats) ptx::tma_prefetch_desc(&a.map[i]);
        if (i == 0) s_abort = 0;
    } else if (tid >= 32 && tid < 32 + NG * R_MOST) {
        const int i = tid - 32;
        ptx::mbar_init(raw_full + 8 * i, a.aligned ? 1 : 32 * GW);
        ptx::mbar_init(raw_empty + 8 * i, GW);
    }
    ptx::fence_barrier_init();
    if (wid == W_WARPS + C_WARPS + 1) {
        ptx::tmem_alloc(ptx::smem_u32(&s_tmem), 512);
        ptx::tmem_relinquish();
    }
    __syncthreads();
    ptx::tc_fence_after();
    ptx::grid_dep_launch_dependents();
    const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
    volatile int* abort = &s_abort;
    unsigned* err = &g_ffn_tile_error;
    auto step_range = [&](int c0, int c1, int& s0, int& s1) {
        s0 = BACK ? c0 : c0 * PER;
        s1 = BACK ? c1 : min(a.steps, c1 * PER);
    };

    if (wid < W_WARPS) {
        // ------------------------------------------------ weights, then the epilogue
        // Two sets of eight warps take the steps by turns, each with a stage of its own.
        const int e = wid >> 3;                                   // set and stage
        const int g = (wid >> 2) & 1, lane_row = 32 * (wid & 3) + lane;  // forward: weight tile and row of it
        const int grp = BACK ? 2 * e + (wid & 1) : wid & 7;       // ring; backward: of 32 of a step's 64 weight rows
        const int q = (wid & 7) >> 1;                             // backward: the quarter of the 256 columns
        uint8_t* ring = raw + grp * a.rs * 32 * a.slot + lane * a.slot;
        const int nsteps = (a.N + STEP - 1) / STEP;  // backward: steps of a matrix
        // byte offset of this lane's row at a chunk, or -1
        auto row_at = [&](int pair, int c, int& mat) -> long long {
            if (BACK) {
                mat = c >= nsteps;
                const int n = (c - mat * nsteps) * STEP + 32 * (wid & 1) + lane;
                return n < a.N ? n * a.row_bytes + (long long)pair * CB : -1;
            }
            mat = a.mats == 2 ? g : 0;
            const int n = (a.mats == 2 ? pair * 128 : pair * 256 + g * 128) + lane_row;
            return n < a.N ? n * a.row_bytes + (long long)c * CB : -1;
        };
        // the chunks of a piece that are this ring's: all; backward, those of its set
        auto first_of = [&](int c) { return BACK ? c + ((c ^ e) & 1) : c; };
        constexpr int NEXT = BACK ? 2 : 1;
        // ---- rows that do not begin on 16 bytes: each warp of a ring copies its share of them, eight lanes a row, whole
        // 16-byte units (bulk copies of single rows take 24 to 46 cycles each, whatever is in flight)
        constexpr bool ROWS = FMT == FMT_Q8_0 || FMT == FMT_Q6_K;
        Pieces pf(a);
        int f_unit = 0, f_c = 0, f_c1 = 0, f_slot = 0;
        const int f_row = (BACK ? 8 * q : 16 * e) + (lane >> 3);
        auto fetch = [&]() {
            while (f_c >= f_c1) {
                if (!pf.next(a, f_unit, f_c, f_c1)) return;
                f_c = first_of(f_c);
            }
            const int pair = f_unit / a.mtiles, mat = BACK ? f_c >= nsteps : a.mats == 2 ? g : 0;
            const int n0 = f_row + (BACK ? (f_c - mat * nsteps) * STEP + 32 * (wid & 1)
                                         : (a.mats == 2 ? pair * 128 : pair * 256 + g * 128) + 32 * (wid & 3));
            const int in_row = (BACK ? pair : f_c) * CB, len = min(CB, (int)a.row_bytes - in_row), sub = 16 * (lane & 7);
            const uint32_t dst = raw_addr + ((grp * a.rs + f_slot) * 32 + f_row) * a.slot + sub;
            const uint8_t* p = a.w[mat] + n0 * a.row_bytes + in_row;
            // the matrix's last bytes do not fill 16: a copy there takes what there is
            const bool tail = in_row + len == (int)a.row_bytes;
#pragma unroll
            for (int t = 0; t < (BACK ? 2 : 4); ++t, p += 4 * a.row_bytes) {
                const int mis = (int)(reinterpret_cast<uintptr_t>(p) & 15), need = n0 + 4 * t < a.N ? mis + len - sub : 0;
                const uint8_t* src = p - mis + sub;
#pragma unroll
                for (int k = 0; k < slot_bytes(FMT, false); k += 128)
                    if (k < need) cp_async16(dst + 4 * t * a.slot + k, src + k, tail ? min(16, need - k) : 16);
            }
            cp_async_arrive(raw_full + 8 * (grp * R_MOST + f_slot));
            f_c += NEXT;
            if (++f_slot == a.rs) f_slot = 0;
        };
        if (ROWS && !a.aligned)
            for (int i = 0; i < a.rs; ++i) fetch();
        bool ok = true, waited = false, bad = false;
        int taken = 0;                     // chunks read
        Check check;
        int slot = 0;                      // the ring's place
        uint32_t par = 0;                  // its parity
        uint32_t n_d = 0;                  // accumulator periods so far
        int base = 0, before = -1;         // steps of the pieces before, this set's last step
        constexpr int RUN = SPLIT ? S::NT / 2 : 1;
        float run[RUN];                    // SPLIT: sums of this thread's lane of tile g, half of its columns
        auto wait_sums = [&](uint32_t bar, uint32_t parity) {
            return __all_sync(0xffffffffu, umma::wait_bar_bounded(bar, parity, abort, err, g_ffn_tile_wait_limit)) != 0;
        };
        auto drain = [&](uint32_t period, bool last) {
            const uint32_t b = S::DB == 2 ? period & 1 : 0;
            const uint32_t parity = (S::DB == 2 ? period >> 1 : period) & 1;
            if (!(last ? wait_sums(d_full + 8 * b, parity) : umma::warp_wait(d_full + 8 * b, parity, abort, err))) return false;
            ptx::tc_fence_after();
#pragma unroll
            for (int c = 0; c < RUN / 16; ++c) {
                if (e * RUN + 16 * c >= a.nt) break;
                uint32_t v[16];
                ptx::tmem_ld16(tmem + ((uint32_t)(32 * (wid & 3)) << 16) + b * S::D_COLS + g * S::NT + e * RUN + 16 * c, v);
                ptx::tmem_ld_wait(v);
#pragma unroll
                for (int k = 0; k < 16; ++k) run[SPLIT ? 16 * c + k : 0] += __uint_as_float(v[k]);
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (!last && lane == 0) ptx::mbar_arrive(d_empty + 8 * b);
            return true;
        };
        Pieces pc(a);
        int unit, c0, c1;
        // A warp whose wait gave up skips the work that is left, but not the barriers: it leaves with the others at the first
        // one, or at the end.
        while (pc.next(a, unit, c0, c1)) {
            const int pair = unit / a.mtiles, mt = unit - pair * a.mtiles;
            int s0, s1;
            step_range(c0, c1, s0, s1);
            if (SPLIT)
#pragma unroll
                for (int k = 0; k < RUN; ++k) run[k] = 0.f;
            int drained = 0, mine = 0;  // SPLIT: periods moved to registers; steps that this set has taken
#pragma unroll 1
            for (int c = first_of(c0); c < c1 && ok; c += NEXT) {
                int mat;
                const long long at = row_at(pair, c, mat);
                const bool valid = at >= 0;
                const int mis = valid ? (int)(at & 15) : 0;
                if (ROWS && !a.aligned && taken > 0) {
                    // the place before this one is filled again as soon as the ring's other warps have left it too
                    const int prev = taken - 1;
                    ok = umma::warp_wait(raw_empty + 8 * (grp * R_MOST + prev % a.rs), (prev / a.rs) & 1, abort, err);
                    if (!ok) break;
                    fetch();
                }
                if (!umma::warp_wait(raw_full + 8 * (grp * R_MOST + slot), par, abort, err)) {
                    ok = false;
                    break;
                }
                const uint8_t* src = ring + slot * 32 * a.slot;
                // the quarter j: piece `sub` of this set's step
                Q6Half q6;
                if (FMT == FMT_Q6_K && !BACK) q6.load(src, e, mis, true);
                auto one = [&](int j, int sub) {
                    const int k0 = (BACK ? pair : c) * CHUNK + j * STEP;
                    const int blocks = min(2, max(0, (a.K - k0) / QK));
                    auto put = [&](int half, const uint32_t (&hi)[16], const uint32_t (&lo)[16]) {
                        if (half == 0 && sub == 0 && ok && before >= 0)
                            ok = umma::warp_wait(empty + 8 * (before % RING), (before / RING) & 1, abort, err);
                        if (!BACK) {
                            if (half == 0) ptx::tc_fence_after();
                            const uint32_t t = tmem + ((uint32_t)(32 * (wid & 3)) << 16) + S::COL_A + e * S::A_COLS +
                                               (g * SUB + sub) * 32 * TERMS + 16 * half;
                            ptx::tmem_st16(t, hi);
                            if (SPLIT) ptx::tmem_st16(t + 32, lo);
                        } else {
                            const int n = 32 * (wid & 1) + lane;
                            uint8_t* p = a_smem + e * TERMS * S::A_BYTES + (n >> 3) * 4096 + (8 * j + 4 * half) * 128 + (n & 7) * 16;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                *reinterpret_cast<uint4*>(p + 128 * i) = make_uint4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
                                if (SPLIT)
                                    *reinterpret_cast<uint4*>(p + S::A_BYTES + 128 * i) =
                                        make_uint4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
                            }
                        }
                    };
                    if (FMT == FMT_Q6_K && !BACK)
                        quarter_q6<SPLIT, FINE>(q6, j & 1, check, put);
                    else
                        quarter<FMT, SPLIT, FINE>(src, j, mis, a.aligned, blocks, !BACK || valid, check, put);
                    if (sub + 1 < SUB) return;
                    if (!BACK) {
                        ptx::tmem_st_wait();
                        ptx::tc_fence_before();
                    } else {
                        ptx::fence_proxy_async_smem();
                    }
                    __syncwarp();
                    before = base + (BACK ? c - c0 : PER * (c - c0) + (SUB == 2 ? e : step_of(FMT, j)));
                    if (lane == 0) ptx::mbar_arrive(full + 8 * (before % RING));
                    ++mine;
                    // SPLIT: a period (a step of each set) behind, whose sums the other buffer holds
                    if (SPLIT && mine >= PERIOD / 2 * (drained + S::DB)) {
                        ok = ok && drain(n_d++, false);
                        ++drained;
                    }
                };
                if (BACK) {
                    if (FMT == FMT_Q8_0) {
                        if (q == 0) one(0, 0);
                        if (q == 1) one(1, 0);
                        if (q == 2) one(2, 0);
                        if (q == 3) one(3, 0);
                    } else {
                        one(q, 0);
                    }
                } else if (FMT == FMT_Q8_0) {
                    // the set's quarters: e and e + 2, or 2 e and 2 e + 1
                    if (e == 0) {
                        one(0, 0);
                        if (SUB == 2)
                            one(1, 1);
                        else if (ok && 4 * c + 2 < a.steps)
                            one(2, 0);
                    } else if (SUB == 2) {
                        if (2 * c + 1 < a.steps) {
                            one(2, 0);
                            one(3, 1);
                        }
                    } else {
                        if (4 * c + 1 < a.steps) one(1, 0);
                        if (ok && 4 * c + 3 < a.steps) one(3, 0);
                    }
                } else {
#pragma unroll 1
                    for (int i = 0; i < 2 && ok; ++i) one(2 * e + i, SUB == 2 ? i : 0);
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(raw_empty + 8 * (grp * R_MOST + slot));  // the chunk has been read
                ++taken;
                if (++slot == a.rs) {
                    slot = 0;
                    par ^= 1;
                }
            }
            base += s1 - s0;
            int any;
            bad |= check.bad() && (BACK || row_at(pair, 0, any) >= 0);  // (lanes past the last row hold anything)
            check = Check();
            if (!waited) ptx::grid_dep_wait();  // what follows reads and writes the call's rows
            waited = true;
            const bool whole = c0 == 0 && c1 == a.chunks;
            uint32_t buf = 0;
            if (SPLIT) {
                // the periods that are left: the last stays in its buffer's hands
                for (; ok && drained + 1 < (s1 - s0 + PERIOD - 1) / PERIOD; ++drained) ok = drain(n_d++, false);
                buf = S::DB == 2 ? n_d & 1 : 0;
                ok = ok && drain(n_d++, true);
                if (ok) {
#pragma unroll
                    for (int c = 0; c < RUN / 16; ++c) {
                        if (e * RUN + 16 * c >= a.nt) break;
                        uint32_t v[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(run[SPLIT ? 16 * c + k : 0]);
                        ptx::tmem_st16(tmem + ((uint32_t)(32 * (wid & 3)) << 16) + buf * S::D_COLS + g * S::NT + e * RUN + 16 * c, v);
                    }
                    ptx::tmem_st_wait();
                    ptx::tc_fence_before();
                }
                ok = sync_weight_warps(ok);
                if (!ok) break;
                ptx::tc_fence_after();
            } else {
                ok = ok && wait_sums(d_full, n_d & 1);
                ++n_d;
                if (!ok && whole) continue;
                ptx::tc_fence_after();
            }
            // ---- the output, or this CTA's part of it: the lane's row, half of the tile's columns
            const int m0 = mt * a.nt, m1 = min(a.M, m0 + a.nt);
            const uint32_t src = tmem + ((uint32_t)(32 * (wid & 3)) << 16) + buf * S::D_COLS;
            auto part = [&](int cta, int which, int tile) {
                return a.parts + ((((long long)cta * 2 + which) * 2 + tile) * a.nt) * 128 + lane_row;
            };
            const int b0 = 8 * (wid >> 2);  // the four warps of a lane take columns by turns
            auto output = [&](auto type) {
                using T = decltype(type);
#pragma unroll 1
                for (int b = b0; m0 + b < m1; b += 32) {
                    const int count = min(8, m1 - m0 - b);
                    Beside w;
                    beside8<T, BACK>(a, pair, lane_row, m0 + b, count, w);
                    uint32_t v0[8], v1[8];
                    ptx::tmem_ld8(src + b, v0);
                    ptx::tmem_ld8(src + S::NT + b, v1);
                    ptx::tmem_ld_wait(v0);
                    ptx::tmem_ld_wait(v1);
                    float z0[8], z1[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        z0[i] = __uint_as_float(v0[i]);
                        z1[i] = __uint_as_float(v1[i]);
                    }
                    finish8<T, BACK>(a, pair, lane_row, m0 + b, count, w, z0, z1);
                    __syncwarp();
                }
            };
            if (whole) {
                if (SPLIT)
                    output(float{});
                else if (a.dtype == MMQ_BF16)
                    output(__nv_bfloat16{});
                else
                    output(__half{});
            } else if (ok) {
#pragma unroll 1
                for (int b = b0; m0 + b < m1; b += 32) {
                    uint32_t v0[8], v1[8];
                    ptx::tmem_ld8(src + b, v0);
                    ptx::tmem_ld8(src + S::NT + b, v1);
                    ptx::tmem_ld_wait(v0);
                    ptx::tmem_ld_wait(v1);
                    float* p0 = part(blockIdx.x, c0 == 0, 0) + b * 128;
                    float* p1 = part(blockIdx.x, c0 == 0, 1) + b * 128;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        p0[i * 128] = __uint_as_float(v0[i]);
                        p1[i * 128] = __uint_as_float(v1[i]);
                    }
                }
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (ok && lane == 0) ptx::mbar_arrive(d_empty + 8 * buf);
            if (!whole) {
                ok = sync_weight_warps(ok);  // every warp's part is written; the counter releases and acquires them
                if (!ok) break;
                const int u = unit - (a.units - a.rest);
                const int first = run_owner(a, (long long)u * a.chunks), last = run_owner(a, (long long)(u + 1) * a.chunks - 1);
                if (tid == 0) s_last = ptx::atom_inc_acq_rel(a.counters + u) == (unsigned)(last - first);
                sync_weight_warps(true);
                auto join = [&](auto type) {
                    using T = decltype(type);
#pragma unroll 1
                    for (int b = b0; m0 + b < m1; b += 32) {
                        const int count = min(8, m1 - m0 - b);
                        Beside w;
                        beside8<T, BACK>(a, pair, lane_row, m0 + b, count, w);
                        float z0[8], z1[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) z0[i] = z1[i] = 0.f;
#pragma unroll 2
                        for (int cta = first; cta <= last; ++cta) {
                            // a run that begins inside the unit is its CTA's first piece, one that begins with it the last
                            const int which = cta == first;
                            const float* p0 = part(cta, which, 0) + b * 128;
                            const float* p1 = part(cta, which, 1) + b * 128;
                            float x0[8], x1[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                x0[i] = __ldcg(p0 + i * 128);
                                x1[i] = __ldcg(p1 + i * 128);
                            }
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                z0[i] += x0[i];
                                z1[i] += x1[i];
                            }
                        }
                        finish8<T, BACK>(a, pair, lane_row, m0 + b, count, w, z0, z1);
                        __syncwarp();
                    }
                };
                if (s_last) {
                    if (SPLIT)
                        join(float{});
                    else if (a.dtype == MMQ_BF16)
                        join(__nv_bfloat16{});
                    else
                        join(__half{});
                }
            }
        }
        if (bad) atomicOr(err, ERR_RANGE);
        if (ROWS) cp_async_wait_all();
        sync_roles();
    } else if (wid < W_WARPS + C_WARPS) {
        // ------------------------------------------------ weight chunks as boxes of 32 rows
        Pieces pc(a);
        int unit, c0, c1, slot[BACK ? 2 : 1] = {};  // the ring's place (of each set)
        uint32_t par[BACK ? 2 : 1];
        par[0] = par[BACK ? 1 : 0] = 1;
        bool ok = a.aligned;
        int asked[NG] = {};  // boxes of each ring
        const int nsteps = (a.N + STEP - 1) / STEP;
        while (ok && pc.next(a, unit, c0, c1)) {
            const int pair = unit / a.mtiles;
#pragma unroll 1
            for (int c = c0; c < c1 && ok; ++c) {
                const int e = BACK ? c & 1 : 0, k = BACK ? e : 0;
                const int mat0 = BACK ? c >= nsteps : 0, x = (BACK ? pair : c) * (CB / 2);
                const int n0 = BACK ? (c - mat0 * nsteps) * STEP : a.mats == 2 ? pair * 128 : pair * 256;
#pragma unroll 1
                for (int i = 0; i < (BACK ? 2 : NG); ++i) {
                    const int r = BACK ? 2 * e + i : i, place = (BACK && k ? slot[BACK ? 1 : 0] : slot[0]);
                    ok = umma::warp_wait(raw_empty + 8 * (r * R_MOST + place), BACK && k ? par[BACK ? 1 : 0] : par[0], abort, err);
                    if (!ok) break;
                    const bool up = BACK ? mat0 : a.mats == 2 && i >= 4;
                    if (ptx::elect_one()) {
                        const uint32_t bar = raw_full + 8 * (r * R_MOST + place);
                        ptx::mbar_arrive_expect_tx(bar, 32 * CB);
                        ptx::tma_load_2d(raw_addr + (r * a.rs + place) * 32 * CB, &a.map[up], bar, x,
                                         n0 + 32 * (BACK || a.mats == 1 ? i : i & 3));
                    }
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < NG; ++j) asked[j] += j == r;
                }
                int& s = BACK && k ? slot[BACK ? 1 : 0] : slot[0];
                if (++s == a.rs) {
                    s = 0;
                    (BACK && k ? par[BACK ? 1 : 0] : par[0]) ^= 1;
                }
            }
        }
        sync_roles();
        if (*abort && a.aligned)  // let the boxes in flight land before the shared memory goes
            for (int r = 0; r < NG; ++r)
                for (int i = 0; i < a.rs; ++i)
                    if (const int n = (asked[r] - i + a.rs - 1) / a.rs; asked[r] > i)
                        umma::drain_bar(raw_full + 8 * (r * R_MOST + i), (n - 1) & 1, err);
    } else if (wid == W_WARPS + C_WARPS) {
        // ------------------------------------------------ the rows' tiles
        ptx::grid_dep_wait();
        Pieces pc(a);
        int unit, c0, c1, st = 0, n = 0;
        bool ok = true;
        while (ok && pc.next(a, unit, c0, c1)) {
            const int mt = unit % a.mtiles, g0 = mt * (a.nt / 8);
            const uint32_t bytes = min(a.nt / 8, a.groups - g0) * 1024;
            int s0, s1;
            step_range(c0, c1, s0, s1);
#pragma unroll 1
            for (int s = s0; s < s1; ++s, ++n) {
                const int piece = !BACK && SUB == 1 ? (s & ~3) + step_of(FMT, s & 3) : s * SUB;
                const uint8_t* src = a.x + ((long long)piece * a.groups + g0) * 1024;
                const int free = n - a.xs;  // the step whose products have read this place
                if (free >= 0 && !umma::warp_wait(empty + 8 * (free % RING), (free / RING) & 1, abort, err)) {
                    ok = false;
                    break;
                }
                if (ptx::elect_one()) {
                    const uint32_t bar = full + 8 * (n % RING);
                    ptx::mbar_arrive_expect_tx(bar, bytes * TERMS * SUB);
                    ptx::bulk_load(xs_addr + st * xb, src, bytes, bar);
                    if (SUB == 2) ptx::bulk_load(xs_addr + st * xb + a.nt * 128, src + (long long)a.groups * 1024, bytes, bar);
                    if (SPLIT) ptx::bulk_load(xs_addr + st * xb + a.nt * 128, src + a.x_term, bytes, bar);
                }
                __syncwarp();
                if (++st == a.xs) st = 0;
            }
        }
        sync_roles();
        if (*abort) {
            // let the copies in flight land before the shared memory goes (a step's barrier counts the weights too, which may
            // never come: the copies are given the time of a wait)
            const uint64_t t0 = ptx::globaltimer_ns();
            while (ptx::globaltimer_ns() - t0 < 1000000ull) {
            }
        }
    } else {
        // ------------------------------------------------ the products, a warp for each weight tile
        // The tensor core's queue is short, so what a warp does between two steps counts (measured with one warp for both
        // tiles and barriers of their own for rows and weights: 450 cycles of waits and loops beside 750 of products at
        // nt = 192, with weights and rows never late).  Products issue from uniform registers in an elected lane.
        const int g = wid - (W_WARPS + C_WARPS + 1);
        Pieces pc(a);
        int unit, c0, c1, xst = 0;
        uint32_t n = 0, n_d = 0;
        bool ok = true;
        const uint32_t idesc = umma::make_idesc(128, a.nt) | (BACK ? 1u << 15 : 0u);
        const uint32_t term_x = a.nt * 128 >> 4;
        // 8-column groups 128 B apart (stride offset), 8-row groups 4096 B (leading offset)
        const uint64_t a_desc = (uint64_t)(((as_addr + g * 2048) & 0x3FFFFu) >> 4) | ((uint64_t)(4096 >> 4) << 16) |
                                ((uint64_t)(128 >> 4) << 32) | (1ull << 46);
        while (ok && pc.next(a, unit, c0, c1)) {
            int s0, s1;
            step_range(c0, c1, s0, s1);
#pragma unroll 1
            for (int s = s0; s < s1; ++s, ++n) {
                const int i = s - s0;
                const bool fresh = SPLIT ? i % PERIOD == 0 : i == 0, last = s + 1 == s1 || (SPLIT && i % PERIOD == PERIOD - 1);
                const uint32_t buf = S::DB == 2 ? n_d & 1 : 0;
                const uint32_t st = s & 1;  // (a chunk of two or four steps begins on an even one)
                if (fresh) ok = umma::warp_wait(d_empty + 8 * buf, ((S::DB == 2 ? n_d >> 1 : n_d) & 1) ^ 1, abort, err);
                ok = ok && umma::warp_wait(full + 8 * (n % RING), (n / RING) & 1, abort, err);
                if (!ok) break;
                ptx::tc_fence_after();
                const uint32_t x_at = __shfl_sync(0xffffffffu, xs_addr + xst * xb, 0);
                if (ptx::elect_one()) {
                    const uint64_t xd = umma::sdesc(x_at, 1024) | (2ull << 61);  // 128-byte swizzle
                    const uint32_t d = tmem + buf * S::D_COLS + g * S::NT;
                    uint32_t acc = fresh ? 0u : 1u;
                    // the products of small terms first
#pragma unroll
                    for (int e = SPLIT ? 2 : 0; e >= 0; --e) {
                        const int ea = e == 2, ex = e == 1;
#pragma unroll
                        for (int kk = 0; kk < SUB * STEP / 16; ++kk) {
                            if (!BACK)
                                ptx::umma_f16_ts(d, tmem + S::COL_A + st * S::A_COLS + (g * SUB * TERMS + ea) * 32 + 8 * kk,
                                                 xd + (ex + kk / 4) * term_x + 2 * (kk % 4), idesc, acc);
                            else
                                ptx::umma_f16(d, a_desc + (uint32_t)((st * TERMS + ea) * (S::A_BYTES >> 4) + kk * 512),
                                              xd + ex * term_x + 2 * kk, idesc, acc);
                            acc = 1u;
                        }
                    }
                    ptx::umma_commit(empty + 8 * (n % RING));
                    if (last) ptx::umma_commit(d_full + 8 * buf);
                }
                __syncwarp();
                if (last) ++n_d;
                if (++xst == a.xs) xst = 0;
            }
        }
        sync_roles();
        if (*abort) {  // let the products in flight end: those whose sums nobody waited for
            if (ptx::elect_one()) ptx::umma_commit(done + 8 * g);
            __syncwarp();
            umma::drain_bar(done + 8 * g, 0, err);
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (wid == W_WARPS + C_WARPS + 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------------------------------ host
template <int FMT, bool SPLIT, bool BACK, int SUB, bool FINE>
int launch_tile(const Tile& a, int smem, int ctas, bool go, const char* fn, cudaStream_t s) {
    static SmemAttr attr;
    auto k = &k_ffn_tile<FMT, SPLIT, BACK, SUB, FINE>;
    const int st = ensure_smem(reinterpret_cast<const void*>(k), SMEM_MOST, attr);
    if (st != MMQ_OK) {
        report(fn, st, "the tiles' shared memory was refused");
        return st;
    }
    if (!go) return MMQ_OK;
    ProfScope ps(BACK ? "k_ffn_tile_back" : "k_ffn_tile", s);
    return pdl_status(launch_pdl(k, dim3((unsigned)ctas), dim3(THREADS), smem, s, a), fn);
}

static int set_tile_wait_limit(unsigned long long ns) {
    return cudaMemcpyToSymbol(g_ffn_tile_wait_limit, &ns, sizeof(ns)) == cudaSuccess ? MMQ_OK : MMQ_ERR_CUDA;
}
static unsigned take_tile_error() {
    unsigned v = 0;
    if (cudaMemcpyFromSymbol(&v, g_ffn_tile_error, sizeof(v)) != cudaSuccess) return 0;
    if (v) {
        const unsigned zero = 0;
        cudaMemcpyToSymbol(g_ffn_tile_error, &zero, sizeof(zero));
    }
    return v;
}

}  // namespace ffn
}  // namespace mmq
