// Attention of a few query rows per sequence and key/value head (single tokens, drafted tokens)
// over the 8-bit cache: k_kv_attend_stream.
//
// Bound: HBM.  Every record in reach is read once (64 D + 16 bytes per 32 tokens and head) and
// used for 8 NT of the head's query rows; more rows are units of their own, next to each other in the
// list of work, so that they read the records from the L2.  A warp is a worker (kv_attend.cuh)
// with a ring of its own: one bulk copy per record, S records in flight, no barrier but its own;
// the ring runs on over the ends of heads and sequences, so short sequences stream like long
// ones.  Codes go from shared memory to f16 MMA operands exactly (|c| <= 127), tokens on the
// M side of both products:
//   S^T [32 tokens x 8 queries] = K [tokens x d] Q^T,   O^T [d x 8 queries] += V^T [d x tokens] P^T
// (m16n8k16).  k is permuted alike in both operands of a product, so every lane reads 16
// consecutive bytes of a record's row; V^T's token pairs are put side by side by byte permutes
// and P^T comes from S^T's accumulators by 8x8 transposes within the warp.  The queries stay in
// registers, scaled per row by a power of two into f16's range: one f16 term for bf16 and f16
// rows (exact but for bits 2^-25 below the row's largest), two for f32 rows (SPLIT), whose
// weights are split into two f16 terms as well.
//
// The tensor core's accumulation rounds towards zero: a sum falls short by about 2^-22.7 of itself for every
// record added to it.  For f32 rows the products of 16 tokens therefore start at zero and are added in f32, to
// nearest: 65500 tokens of one sign, 400 to 2000 records a warp, come within 7e-7 to 3e-6 of 64 bits, where one long
// chain was 9e-5 to 4e-4 off (64 sequences of 1000 to 8191 tokens, 4 rows a head of 64 / 128 / 256: 69 / 104 / 227 ->
// 72 / 107 / 245 us).  For 16-bit rows the chain stays: 400 records are 6e-5 off, a quarter of f16's own rounding
// (2^-12), and the additions cost 1 to 8 % (62.9 -> 63.5 us, 24 rows of 128 on long runs 1365 -> 1480).
//
// Measured (GB300): 64 sequences of 1000 to 8191 tokens, 4 rows a head, 614 MB of records: 108 us,
// 5.7 TB/s, 0.84 of the copy rate, with an issue slot used in 0.45 of the cycles and the tensor pipe in
// 0.14.  One sequence of 131069 tokens, 135 MB: 36 us; of 777 tokens, f32: 12.8 us, which are a CTA's prologue
// (lengths, first table entries, first records: three dependent trips to memory), a record's chain, its parts'
// join and the CTAs'.  The two large calls are 16 to 17 us above their bytes; how much of that is the same
// prologue and joins was not taken apart.  Past 8 rows the warps' instructions bound it: a record
// takes a warp 2.6 us at 24 rows of 128 where eight share an SM.
// Registers: all but 24 rows of 128 (16-bit), 8 and 16 of 128 and 8 of 256 (f32) fit without a spill; those
// keep 12 to 108 bytes a thread on the stack.
#include "kv_attend.cuh"
#include "umma.cuh"

namespace mmq {
namespace {

using namespace kv;

__device__ unsigned g_kv_stream_error;

template <int D, int NT>
struct Stream {
    // as many warps as shared memory holds rings of two records for (dim 64: four), and registers
    // for two tiles of rows: a block is a chain of dependent steps, and only other warps fill its gaps
    static constexpr int WARPS = D == 256 ? 6 : NT > 1 ? 8 : 12, THREADS = WARPS * 32;
    static constexpr int STAGES = D == 64 ? 4 : D == 128 && NT > 1 ? 3 : 2;
    static constexpr int ROWS = 8 * NT, REC = rec_bytes(D);
    static constexpr int RING = WARPS * STAGES * REC, SMEM = RING + WARPS * STAGES * 8;
    // a kept result: rows of O, then m and l.  16-byte piece i of the values that lane group g holds of a row
    // is at 8 i + g, and two rows are 8 floats past a multiple of 32 apart: stores and loads without conflicts
    static constexpr int KD = D + 4, KEPT = ROWS * (KD + 2);
    static constexpr int RUN = D < 128 ? D / 8 : 16;  // consecutive values of O that a lane group holds
    static __device__ __forceinline__ int column(int piece) { return 128 * (piece / 32) + RUN * (piece % 8) + piece % 32 / 8 * 4; }
    static_assert(KEPT * 4 <= STAGES * REC && ROWS * D + WARPS * KEPT <= WS_ROWS * D, "room for a warp's partial results");
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// as mma16816, from zero
__device__ __forceinline__ void mma16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t o;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(o) : "r"(v));
    return o;
}
// Where a warp keeps an incomplete unit's result: at the beginning of its
// ring, or (ring: nullptr) in a place of its own in the CTA's first slot of the workspace, behind the
// rows that the CTA's own partial result takes there.
template <class C, int D>
__device__ __forceinline__ float* kept_at(uint8_t* ring, const Attend& a, int warp) {
    return ring ? reinterpret_cast<float*>(ring) : part_slot(a, blockIdx.x, 0) + C::ROWS * D + warp * C::KEPT;
}

// Adds parts c .. c + B - 1, c1 at most, of the unit whose first part is CTA c0's, all of them in flight.
template <int B, int D>
__device__ __forceinline__ void add_parts(const Attend& a, Joined& j, int r, int piece, int c, int c0, int c1) {
    float4 x[B];
    float m[B], l[B];
#pragma unroll
    for (int k = 0; k < B; ++k) {
        const float* ps = part_slot(a, min(c + k, c1), min(c + k, c1) == c0);
        x[k] = __ldcg(reinterpret_cast<const float4*>(ps + r * D + 4 * piece));
        m[k] = __ldcg(ps + WS_ROWS * D + r);
        l[k] = __ldcg(ps + WS_ROWS * (D + 1) + r);
    }
#pragma unroll
    for (int k = 0; k < B; ++k)
        if (c + k <= c1) j.add(x[k], m[k], l[k]);
}

// A sequence as the units see it: heads * groups units, unit h of head h / groups and rows
// (h % groups) * ROWS ..
struct Seq {
    int start, n, len, lo_blk, groups, tiles;  // tiles: records in reach, or 1 for a sequence of padding rows; 0: none
};
template <int ROWS>
__device__ __forceinline__ Seq load_seq(const Attend& a, int b) {
    Seq s;
    seq_range(a.c, a.bt, b, s.start, s.n, s.len, &g_kv_stream_error);
    s.lo_blk = s.len > 0 ? first_key(a, s.len - s.n) / BT : 0;
    s.tiles = s.n == 0 ? 0 : max(1, (s.len + BT - 1) / BT - s.lo_blk);
    s.groups = a.bt.max_new * a.group <= ROWS ? 1 : max(1, (s.n * a.group + ROWS - 1) / ROWS);
    return s;
}
// the unit after (b, h): the sequence's next, or the first of the next sequence that has rows
template <int ROWS>
__device__ __forceinline__ void next_unit(const Attend& a, int& b, int& h, Seq& s) {
    if (++h < a.c.heads * s.groups) return;
    h = 0;
    do ++b;
    while (b < a.bt.seqs && (s = load_seq<ROWS>(a, b)).tiles == 0);
}

template <int D, int NT, bool SPLIT>
__global__ void __launch_bounds__(Stream<D, NT>::THREADS, 1)
k_kv_attend_stream(const Attend a) {
    using C = Stream<D, NT>;
    constexpr int KS = D / 16;  // k steps of the first product, row tiles of the second
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_scan[C::WARPS], s_b[C::WARPS], s_off[C::WARPS], s_x[C::WARPS + 1], s_abort;
    __shared__ int s_out[2], s_first[2], s_final[2];  // the unit that came in, the one that goes out: slot, its CTAs
    // the incomplete units of the CTA in work order, two slots per warp (the second: its range's end)
    __shared__ int s_unit[2 * C::WARPS], s_end[2 * C::WARPS], s_head[2 * C::WARPS], s_row[2 * C::WARPS];
    __shared__ Seq s_sq[2 * C::WARPS];
    // its parts in work order, and where in them and in the slots each unit begins
    __shared__ const float* s_part[2 * C::WARPS];
    __shared__ int s_runs, s_run[2 * C::WARPS + 1], s_slot[2 * C::WARPS];
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, g = lane >> 2, tq = lane & 3;
    uint8_t* ring = smem + wid * C::STAGES * C::REC;
    const uint32_t bars = ptx::smem_u32(smem + C::RING) + wid * C::STAGES * 8;
    if (lane < C::STAGES) ptx::mbar_init(bars + 8 * lane, 1);
    ptx::fence_barrier_init();
    if (tid == 0) s_abort = 0;
    if (lane < 2) s_unit[2 * wid + lane] = -1;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch_dependents();

    // ---- this warp's range of the work
    const int seqs = a.bt.seqs;
    auto places = [&](int i) {
        const Seq s = load_seq<C::ROWS>(a, i);
        return s.tiles * s.groups * a.c.heads;
    };
    const int v0 = tid < seqs ? places(tid) : 0;
    int total;
    const int e0 = scan_cta<C::WARPS>(v0, total, s_scan);
    const int total0 = total;
    int T = total;
    for (int base = C::THREADS; base < seqs; base += C::THREADS) {
        const int i = base + tid;
        scan_cta<C::WARPS>(i < seqs ? places(i) : 0, total, s_scan);
        T += total;
    }
    const int W = min((int)gridDim.x * C::WARPS, T), w0 = blockIdx.x * C::WARPS;
    if (w0 >= W) return;
    if (tid <= C::WARPS) s_x[tid] = work_start(T, min(w0 + tid, W), W);  // the warps' ranges
    __syncthreads();
    for (int base = 0, carry = 0; base < seqs; base += C::THREADS) {
        const int i = base + tid;
        int v = v0, e = e0;
        total = total0;
        if (base > 0) {
            v = i < seqs ? places(i) : 0;
            e = carry + scan_cta<C::WARPS>(v, total, s_scan);
        }
        carry += total;
        for (int k = 0; k < C::WARPS && w0 + k < W; ++k) {
            const int x = s_x[k];
            if (x >= e && x < e + v) {
                s_b[k] = i;
                s_off[k] = x - e;
            }
        }
    }
    __syncthreads();

    if (w0 + wid < W) {
        const int x0 = s_x[wid], x1 = s_x[wid + 1];
        int b = s_b[wid];
        Seq sq = load_seq<C::ROWS>(a, b);
        int h = s_off[wid] / sq.tiles, o = s_off[wid] - h * sq.tiles;
        // the fetching side runs STAGES records ahead; within a page it only steps to the next record
        int fb = b, fh = h, fo = o, fx = x0, left = 0, pg = 0, tab0 = 0, tabn = 0, tab = -1;
        Seq fs = sq;
        const uint8_t* src = nullptr;   // the next record (nullptr: on no page)
        uint32_t live = 0, phase = 0;   // stages that a copy was started into, parities
        auto fetch = [&](int st) {      // the next record of the range into stage st
            if (fs.len > 0) {
                if (left == 0) {  // a new unit or page
                    const int blk = fs.lo_blk + fo;
                    pg = blk / a.c.blocks;
                    const int in = blk - pg * a.c.blocks;
                    left = a.c.blocks - in;
                    if (pg < tab0 || pg >= tab0 + tabn) {  // 32 page numbers at a time, one per lane
                        tab0 = pg;
                        tabn = min(32, (fs.len + a.c.page - 1) / a.c.page - pg);
                        tab = lane < tabn ? a.bt.table[(long long)fb * a.bt.table_stride + pg + lane] : -1;
                    }
                    const int id = __shfl_sync(0xffffffffu, tab, pg - tab0);
                    src = nullptr;
                    if (id >= 0 && id < a.c.pages)
                        src = a.c.data + (((long long)id * a.c.heads + fh / fs.groups) * a.c.blocks + in) * C::REC;
                    else if (lane == 0)
                        atomicOr(&g_kv_stream_error, ERR_RANGE);
                }
                if (src) {
                    if (lane == 0) {
                        ptx::mbar_arrive_expect_tx(bars + 8 * st, C::REC);
                        ptx::bulk_load(ptx::smem_u32(ring + st * C::REC), src, C::REC, bars + 8 * st);
                    }
                    live |= 1u << st;
                    src += C::REC;
                }
                --left;
            }
            ++fx;
            if (++fo == fs.tiles) {
                const int was = fb;
                next_unit<C::ROWS>(a, fb, fh, fs);
                fo = left = 0;
                if (fb != was) tabn = 0;
            }
        };
        uint32_t qf[SPLIT ? 2 : 1][NT][KS][2];
        float acc[KS][NT][4], m[NT][2], l[NT][2], fq[NT][2];
        int hi[NT][2], lo[NT][2], hi_min = 0, lo_max = 0, o_from = 0;
        int head = 0, row0 = 0;  // of the unit
        bool fresh = true, ok = true;
        int st = 0;
#pragma unroll 1
        for (int x = x0; x < x1; ++x) {
            if (fresh) {  // a new unit: its queries as B operands, its rows' limits
                fresh = false;
                o_from = o;
                head = h / sq.groups;
                row0 = (h - head * sq.groups) * C::ROWS;
                const int rows = sq.n * a.group, first = sq.len - sq.n;
                hi_min = 0x7fffffff;
                lo_max = 0;
                // 16 consecutive values of each 64 per lane: one run of loads, whatever the type; the first
                // unit's go out before the first records, or they would queue behind them
                uint4 raw[NT][D / 64][SPLIT ? 4 : 2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int r = row0 + 8 * nt + g, t = r / a.group;
                    const uint8_t* src = static_cast<const uint8_t*>(a.q.data) +
                                         ((sq.start + t) * a.q.token_stride + (head * a.group + r - t * a.group) * a.q.head_stride +
                                          16 * tq) * (SPLIT ? 4 : 2);
#pragma unroll
                    for (int sg = 0; sg < D / 64; ++sg)
#pragma unroll
                        for (int e = 0; e < (SPLIT ? 4 : 2); ++e)
                            raw[nt][sg][e] = r < rows ? *reinterpret_cast<const uint4*>(src + sg * (SPLIT ? 256 : 128) + 16 * e)
                                                      : make_uint4(0u, 0u, 0u, 0u);
                }
                if (x == x0) {
#pragma unroll 1
                    for (int i = 0; i < C::STAGES && fx < x1; ++i) fetch(i);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float4 v[KS];
                    float am = 0.f;
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        const uint4 p = raw[nt][ks >> 2][SPLIT ? ks & 3 : (ks & 3) >> 1];
                        const uint2 w = ks & 1 ? make_uint2(p.z, p.w) : make_uint2(p.x, p.y);
                        v[ks] = SPLIT ? make_float4(__uint_as_float(p.x), __uint_as_float(p.y), __uint_as_float(p.z),
                                                    __uint_as_float(p.w))
                                : a.dtype == MMQ_BF16 ? Elem<__nv_bfloat16>::widen(w)
                                                      : Elem<__half>::widen(w);
                        am = fmaxf(am, fmaxf(fmaxf(fabsf(v[ks].x), fabsf(v[ks].y)), fmaxf(fabsf(v[ks].z), fabsf(v[ks].w))));
                    }
                    am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
                    am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
                    float down, up;
                    row_scale(am, down, up);
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        if (SPLIT) {
                            split_h2(v[ks].x * down, v[ks].y * down, qf[0][nt][ks][0], qf[SPLIT ? 1 : 0][nt][ks][0]);
                            split_h2(v[ks].z * down, v[ks].w * down, qf[0][nt][ks][1], qf[SPLIT ? 1 : 0][nt][ks][1]);
                        } else {
                            qf[0][nt][ks][0] = pack_h2(v[ks].x * down, v[ks].y * down);
                            qf[0][nt][ks][1] = pack_h2(v[ks].z * down, v[ks].w * down);
                        }
                    }
#pragma unroll
                    for (int c = 0; c < 2; ++c) {  // this lane's columns of S^T and O^T: rows 2 tq, 2 tq + 1
                        fq[nt][c] = __shfl_sync(0xffffffffu, up, 4 * (2 * tq + c)) * a.scale2;
                        const int rc = row0 + 8 * nt + 2 * tq + c, pos = first + rc / a.group;
                        hi[nt][c] = rc < rows ? pos + 1 : 0x7fffffff;
                        lo[nt][c] = rc < rows && a.window > 0 ? max(0, pos - a.window + 1) : 0;
                        hi_min = min(hi_min, hi[nt][c]);
                        lo_max = max(lo_max, lo[nt][c]);
                        m[nt][c] = M_NONE;
                        l[nt][c] = 0.f;
                    }
#pragma unroll
                    for (int j = 0; j < KS; ++j)
#pragma unroll
                        for (int c = 0; c < 4; ++c) acc[j][nt][c] = 0.f;
                }
#pragma unroll
                for (int off = 1; off <= 2; off <<= 1) {
                    hi_min = min(hi_min, __shfl_xor_sync(0xffffffffu, hi_min, off));
                    lo_max = max(lo_max, __shfl_xor_sync(0xffffffffu, lo_max, off));
                }
            }

            if (live >> st & 1) {
                if (!umma::warp_wait(bars + 8 * st, phase >> st & 1, &s_abort, &g_kv_stream_error)) {
                    ok = false;
                    break;
                }
                phase ^= 1u << st;
                live &= ~(1u << st);
                const uint8_t* rec = ring + st * C::REC;
                // S^T: token slots g and g + 8 of two 16-token tiles, query columns 2 tq and 2 tq + 1
                float s[2][NT][4];
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 4; ++c) s[mt][nt][c] = 0.f;
#pragma unroll
                for (int sg = 0; sg < D / 64; ++sg) {
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
                        const uint8_t* p = rec + (16 * mt + g) * D + 64 * sg + 16 * tq;
                        const uint4 ra = *reinterpret_cast<const uint4*>(p);
                        const uint4 rb = *reinterpret_cast<const uint4*>(p + 8 * D);
                        const uint32_t wa[4] = {ra.x, ra.y, ra.z, ra.w}, wb[4] = {rb.x, rb.y, rb.z, rb.w};
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const uint2 ca = umma::i8x4_to_f16x4(wa[u]), cb = umma::i8x4_to_f16x4(wb[u]);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < (SPLIT ? 2 : 1); ++e)
                                    mma16816(s[mt][nt], ca.x, cb.x, ca.y, cb.y, qf[e][nt][4 * sg + u][0],
                                             qf[e][nt][4 * sg + u][1]);
                        }
                    }
                }
                const float2 d = *reinterpret_cast<const float2*>(rec + 2 * BT * D);
                float lv, rv;
                value_scale(d.y, lv, rv);
                const int j0 = (sq.lo_blk + o) * BT;
                const bool edge = j0 + BT > hi_min || j0 < lo_max;
                bool over = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float a0 = fq[nt][0] * d.x, a1 = fq[nt][1] * d.x;
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            float t = fmaf(s[mt][nt][c], c & 1 ? a1 : a0, lv);
                            if (edge) {
                                const int j = j0 + 16 * mt + g + 8 * (c >> 1);
                                if (j >= hi[nt][c & 1] || j < lo[nt][c & 1]) t = -INFINITY;
                            }
                            s[mt][nt][c] = t;
                            over |= t > m[nt][c & 1] + LIMIT;
                        }
                }
                if (__any_sync(0xffffffffu, over)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float mx = fmaxf(fmaxf(s[0][nt][c], s[0][nt][c + 2]), fmaxf(s[1][nt][c], s[1][nt][c + 2]));
#pragma unroll
                            for (int off = 4; off <= 16; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                            const float mn = fmaxf(m[nt][c], mx - SHIFT), f = exp2_approx(m[nt][c] - mn);
                            m[nt][c] = mn;
                            l[nt][c] *= f;
#pragma unroll
                            for (int j = 0; j < KS; ++j) {
                                acc[j][nt][c] *= f;
                                acc[j][nt][c + 2] *= f;
                            }
                        }
                }
                uint32_t pf[SPLIT ? 2 : 1][2][NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float p0 = exp2_approx(s[mt][nt][2 * r] - m[nt][0]);
                            const float p1 = exp2_approx(s[mt][nt][2 * r + 1] - m[nt][1]);
                            sum0 += p0;
                            sum1 += p1;
                            if (SPLIT) {
                                uint32_t ph, pl;
                                split_h2(p0, p1, ph, pl);
                                pf[0][mt][nt][r] = transpose8x8(ph);
                                pf[SPLIT ? 1 : 0][mt][nt][r] = transpose8x8(pl);
                            } else {
                                pf[0][mt][nt][r] = transpose8x8(pack_h2(p0, p1));
                            }
                        }
                    l[nt][0] = fmaf(sum0, rv, l[nt][0]);
                    l[nt][1] = fmaf(sum1, rv, l[nt][1]);
                }
                // O^T: lane (g, tq) takes the value columns 16 g .. 16 g + 15 of each 128 (8 g .. of
                // 64), of tokens 2 tq, 2 tq + 1, 2 tq + 8, 2 tq + 9 of each 16-token tile; row tile j
                // holds columns 2j (rows 0..7) and 2j + 1 (rows 8..15) of every lane's run
                constexpr int RUN = D < 128 ? D / 8 : 16, RUNS = D / (8 * RUN), WORDS = RUN / 4;
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int hh = 0; hh < RUNS; ++hh) {
                        const uint8_t* p = rec + BT * D + (16 * mt + 2 * tq) * D + 128 * hh + RUN * g;
                        uint32_t wv[4][WORDS];
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const uint8_t* pu = p + ((u & 1) + 8 * (u >> 1)) * D;
                            if (WORDS == 4) {
                                const uint4 t4 = *reinterpret_cast<const uint4*>(pu);
                                wv[u][0] = t4.x;
                                wv[u][1] = t4.y;
                                wv[u][WORDS == 4 ? 2 : 0] = t4.z;
                                wv[u][WORDS == 4 ? 3 : 0] = t4.w;
                            } else {
                                const uint2 t2 = *reinterpret_cast<const uint2*>(pu);
                                wv[u][0] = t2.x;
                                wv[u][1] = t2.y;
                            }
                        }
#pragma unroll
                        for (int j = 0; j < RUN / 2; ++j) {
                            const uint32_t sel = j & 1 ? 0x7362 : 0x5140;
                            const uint2 c0 = umma::i8x4_to_f16x4(__byte_perm(wv[0][j >> 1], wv[1][j >> 1], sel));
                            const uint2 c1 = umma::i8x4_to_f16x4(__byte_perm(wv[2][j >> 1], wv[3][j >> 1], sel));
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                float (&to)[4] = acc[hh * (RUN / 2) + j][nt];
                                if (SPLIT) {  // the small terms first
                                    float part[4];
                                    mma16816_first(part, c0.x, c0.y, c1.x, c1.y, pf[SPLIT ? 1 : 0][mt][nt][0],
                                                   pf[SPLIT ? 1 : 0][mt][nt][1]);
                                    mma16816(part, c0.x, c0.y, c1.x, c1.y, pf[0][mt][nt][0], pf[0][mt][nt][1]);
#pragma unroll
                                    for (int c = 0; c < 4; ++c) to[c] += part[c];
                                } else {
                                    mma16816(to, c0.x, c0.y, c1.x, c1.y, pf[0][mt][nt][0], pf[0][mt][nt][1]);
                                }
                            }
                        }
                    }
                __syncwarp();  // the stage is read
            }
            if (fx < x1) fetch(st);
            if (++st == C::STAGES) st = 0;

            if (++o == sq.tiles || x + 1 == x1) {  // the unit ends, or the range does
                const int ustart = x + 1 - o, uend = ustart + sq.tiles, rows = sq.n * a.group;
                const bool whole = o_from == 0 && o == sq.tiles;
                // incomplete: kept in the ring if the range ends (nothing is in flight any more), else, a
                // unit that came in and ends here, in the warp's rows of the workspace
                float* kept = kept_at<C, D>(x + 1 == x1 ? ring : nullptr, a, wid);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float sum = l[nt][c];
#pragma unroll
                        for (int off = 4; off <= 16; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                        const int r = 8 * nt + 2 * tq + c, rs = row0 + r;  // in the unit, in the sequence
                        constexpr int RUN = C::RUN, RUNS = D / (8 * RUN);
                        const float inv = whole ? (sum > 0.f ? __frcp_rn(sum) : 0.f) : 1.f;
                        const int t = rs / a.group, hq = head * a.group + rs - t * a.group;
                        if (rs >= rows) continue;
#pragma unroll
                        for (int hh = 0; hh < RUNS; ++hh)
#pragma unroll
                            for (int i = 0; i < RUN / 4; ++i) {
                                const int j = hh * (RUN / 2) + 2 * i, col = 128 * hh + RUN * g + 4 * i;
                                const float4 v = make_float4(acc[j][nt][c] * inv, acc[j][nt][c + 2] * inv,
                                                             acc[j + 1][nt][c] * inv, acc[j + 1][nt][c + 2] * inv);
                                if (whole)
                                    store_out4(a, sq.start + t, hq, col, v);
                                else
                                    *reinterpret_cast<float4*>(kept + r * C::KD + 128 * hh + 32 * i + 4 * g) = v;
                            }
                        if (g == 0) {
                            if (whole) {
                                store_lse(a, sq.start + t, hq, m[nt][c], sum);
                            } else {
                                kept[C::ROWS * C::KD + r] = m[nt][c];
                                kept[C::ROWS * (C::KD + 1) + r] = sum;
                            }
                        }
                    }
                if (!whole && lane == 0) {
                    const int i = 2 * wid + (x + 1 == x1 ? 1 : 0);
                    s_unit[i] = ustart;
                    s_end[i] = uend;
                    s_sq[i] = sq;
                    s_head[i] = head;
                    s_row[i] = row0;
                }
                if (o == sq.tiles && x + 1 < x1) {
                    next_unit<C::ROWS>(a, b, h, sq);
                    o = 0;
                    fresh = true;
                }
            }
        }
        if (!ok)  // given up: let what is in flight land before the shared memory goes
            for (int i = 0; i < C::STAGES; ++i)
                if (live >> i & 1) umma::drain_bar(bars + 8 * i, phase >> i & 1, &g_kv_stream_error);
    }
    __syncthreads();
    if (s_abort) return;

    // ---- the CTA's incomplete units: the slots in use are the parts, those of one unit in a row
    if (wid == 0) {
        const int u = lane < 2 * C::WARPS ? s_unit[lane] : -1;
        const unsigned used = __ballot_sync(0xffffffffu, u >= 0), before = used & ((1u << lane) - 1);
        const int prev = __shfl_sync(0xffffffffu, u, before ? 31 - __clz(before) : 0);
        const bool first = u >= 0 && (before == 0 || prev != u);
        const unsigned starts = __ballot_sync(0xffffffffu, first);
        const int j = __popc(before);
        if (u >= 0) s_part[j] = kept_at<C, D>(lane & 1 ? smem + (lane >> 1) * C::STAGES * C::REC : nullptr, a, lane >> 1);
        if (first) {
            const int run = __popc(starts & ((1u << lane) - 1));
            s_slot[run] = lane;
            s_run[run] = j;
        }
        if (lane == 0) {
            s_runs = __popc(starts);
            s_run[__popc(starts)] = __popc(used);
            s_out[0] = s_out[1] = -1;
        }
    }
    __syncthreads();
    const int cta0 = s_x[0], cta1 = s_x[min(W - w0, C::WARPS)];
    const int each = min(C::ROWS, a.bt.max_new * a.group) * (D / 4), items = s_runs * each;
    // a unit's last part may be the one in the workspace: three of them at a time are on their way
    constexpr int U = 3;
    for (int base = tid; base < items; base += U * C::THREADS) {
        float4 y[U];
        float my[U], ly[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int idx = base + k * C::THREADS, run = idx / each, x = idx - run * each, r = x / (D / 4);
            if (idx >= items) break;
            const float* part = s_part[s_run[run + 1] - 1];
            y[k] = *reinterpret_cast<const float4*>(part + r * C::KD + 4 * (x % (D / 4)));
            my[k] = part[C::ROWS * C::KD + r];
            ly[k] = part[C::ROWS * (C::KD + 1) + r];
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int idx = base + k * C::THREADS, run = idx / each, x = idx - run * each, r = x / (D / 4), piece = x % (D / 4);
            if (idx >= items) break;
            const int i = s_slot[run], u = s_unit[i], rs = s_row[i] + r;
            if (rs >= s_sq[i].n * a.group) continue;
            Joined j;
            j.add(y[k], my[k], ly[k]);
#pragma unroll 1
            for (int p = s_run[run]; p < s_run[run + 1] - 1; ++p) {
                const float* part = s_part[p];
                j.add(*reinterpret_cast<const float4*>(part + r * C::KD + 4 * piece), part[C::ROWS * C::KD + r],
                      part[C::ROWS * (C::KD + 1) + r]);
            }
            if (u >= cta0 && s_end[i] <= cta1) {
                const int t = rs / a.group, hq = s_head[i] * a.group + rs - t * a.group;
                store_out4(a, s_sq[i].start + t, hq, C::column(piece), j.out());
                if (piece == 0) store_lse(a, s_sq[i].start + t, hq, j.m, j.l);
            } else {
                const int side = u >= cta0 ? 1 : 0;
                float* part = part_slot(a, blockIdx.x, side);
                *reinterpret_cast<float4*>(part + r * D + 4 * piece) = j.o;
                if (piece == 0) {
                    part[WS_ROWS * D + r] = j.m;
                    part[WS_ROWS * (D + 1) + r] = j.l;
                    s_out[side] = i;
                }
            }
        }
    }
    __syncthreads();  // with the release of the thread that counts below, the CTA's parts are there first
    // ---- the units that other CTAs have parts of: the last to arrive joins them, in CTA order
    if (tid < 2 && s_out[tid] >= 0) {
        const int u = s_unit[s_out[tid]], c0 = work_owner(T, u, W) / C::WARPS,
                  c1 = work_owner(T, s_end[s_out[tid]] - 1, W) / C::WARPS;
        unsigned* counter = reinterpret_cast<unsigned*>(a.ws) + c0;
        // one step for the parts of this CTA before and those of the others behind it
        if (ptx::atom_inc_acq_rel(counter) == (unsigned)(c1 - c0)) {
            *counter = 0;
            s_first[tid] = c0;
            s_final[tid] = c1;
        } else {
            s_out[tid] = -1;
        }
    }
    __syncthreads();
    for (int side = 0; side < 2; ++side) {
        if (s_out[side] < 0) continue;
        const Seq& sq = s_sq[s_out[side]];
        const int row0 = s_row[s_out[side]], rows = min(C::ROWS, sq.n * a.group - row0), c0 = s_first[side], c1 = s_final[side];
        for (int idx = tid; idx < rows * (D / 4); idx += C::THREADS) {
            const int r = idx / (D / 4), piece = idx % (D / 4), col = C::column(piece);
            Joined j;
            // (code that runs once costs its own fetching: two parts are not worth the steps of eight)
            for (int c = c0; c <= c1; c += 8)
                if (c1 - c < 4)
                    add_parts<4, D>(a, j, r, piece, c, c0, c1);
                else
                    add_parts<8, D>(a, j, r, piece, c, c0, c1);
            const int rs = row0 + r, t = rs / a.group, hq = s_head[s_out[side]] * a.group + rs - t * a.group;
            store_out4(a, sq.start + t, hq, col, j.out());
            if (col == 0) store_lse(a, sq.start + t, hq, j.m, j.l);
        }
    }
}

template <int D, int NT, bool SPLIT>
int launch(const Attend& a, cudaStream_t s) {
    using C = Stream<D, NT>;
    static SmemAttr attr;
    const char* fn = "mmq_kv_attend";
    const void* func = reinterpret_cast<const void*>(&k_kv_attend_stream<D, NT, SPLIT>);
    const int st = ensure_smem(func, C::SMEM, attr);
    if (st != MMQ_OK) {
        report(fn, st, "the attention stream's shared memory was refused");
        return st;
    }
    // no more warps than records can be in reach
    const long long groups = ((long long)a.bt.max_new * a.group + C::ROWS - 1) / C::ROWS;
    const long long most = (long long)a.bt.seqs * a.c.heads * a.bt.table_pages * a.c.blocks * groups;
    if (most > 0x7fffffff) {
        report(fn, MMQ_ERR_SHAPE, "seqs * heads * table_pages * page / 32 * rows / 8 must be below 2^31");
        return MMQ_ERR_SHAPE;
    }
    const long long ctas = (most + C::WARPS - 1) / C::WARPS, sms = device_shape().sms < 341 ? device_shape().sms : 341;
    const dim3 grid((unsigned)(ctas < 1 ? 1 : ctas < sms ? ctas : sms));
    ProfScope ps("k_kv_attend_stream", s);
    return pdl_status(launch_pdl(&k_kv_attend_stream<D, NT, SPLIT>, grid, dim3(C::THREADS), C::SMEM, s, a), fn);
}

// Rows a unit holds: as many as its warps' registers do.
template <bool SPLIT>
int launch_rows(const Attend& a, int rows, cudaStream_t s) {
    if (a.c.dim == 256) return launch<256, 1, SPLIT>(a, s);
    if (a.c.dim == 64)
        return rows <= 8 ? launch<64, 1, SPLIT>(a, s) : rows <= 16 ? launch<64, 2, SPLIT>(a, s) : launch<64, 3, SPLIT>(a, s);
    if (rows <= 8) return launch<128, 1, SPLIT>(a, s);
    return SPLIT || rows <= 16 ? launch<128, 2, SPLIT>(a, s) : launch<128, SPLIT ? 2 : 3, SPLIT>(a, s);
}

}  // namespace

// The most query rows of one sequence and head, by the longest sequence, that go to the stream: past it the
// tiles' time, which hardly changes from 8 to 128 rows, is shorter.  Measured, stream / tiles in us, 8 heads,
// as sequences x tokens, all sequences with the same rows:
//                      50 x 150      8 x 2000     200 x 200     1 x 65536    50 x 12000
//   128, 16-bit, 24   31.7 / 41.9   28.3 / 42.2   84.5 / 138   56.3 / 87      322 / 584
//                48   48.1 / 42.2   42.1 / 43.8    123 / 140   86.7 / 94      618 / 584
//                64   50.0 / 42.4   49.0 / 43.6    149 / 142    120 / 93      912 / 584
//   128, f32,    48   42.8 / 52.8   44.2 / 61.1    128 / 249    120 / 165     954 / 1204
//                64   52.3 / 54.1   52.1 / 61.0    160 / 251    152 / 165    1249 / 1205
//    64, 16-bit, 48   31.1 / 35.4   30.1 / 35.1   74.2 / 107   59.4 / 74      428 / 508
//                64   33.2 / 35.4   35.1 / 34.9   91.7 / 108   81.2 / 74      633 / 508
//   256, 16-bit, 16   39.0 / 42.5   37.9 / 46.5   99.7 / 166   94.0 / 130     754 / 962
//                24   46.5 / 43.8   47.1 / 47.0    131 / 174    131 / 131    1111 / 965
//    64, f32,    48   33.2 / 36.1   34.1 / 41.6   87.2 / 140   73.7 / 108     555 / 823
//                64   35.9 / 36.4   39.3 / 41.6    109 / 144    103 / 108     826 / 823
//   256, f32,    32   62.3 / 64.2   71.3 / 79.9    201 / 285    219 / 244    1878 / 2025
//                48   78.6 / 68.5   98.4 / 83.6    293 / 299    320 / 253    2767 / 2031
// Where most sequences have fewer rows than the longest one the stream gains, the tiles do not: 8 sequences
// of 517 to 3001 tokens with 14 to 35 rows of 128 take 30.1 us there, 32.2 in the tiles.
int kv_stream_rows(int dim, int dtype) {
    if (dim == 256) return dtype == MMQ_F32 ? 32 : 16;
    return 48;
}

int kv_stream_launch(const Attend& a, int rows, cudaStream_t s) {
    return a.dtype == MMQ_F32 ? launch_rows<true>(a, rows, s) : launch_rows<false>(a, rows, s);
}

unsigned kv_stream_take_error() {
    unsigned v = 0;
    if (cudaMemcpyFromSymbol(&v, g_kv_stream_error, sizeof(v)) != cudaSuccess) return 0;
    if (v) {
        const unsigned zero = 0;
        cudaMemcpyToSymbol(g_kv_stream_error, &zero, sizeof(zero));
    }
    return v;
}

}  // namespace mmq
