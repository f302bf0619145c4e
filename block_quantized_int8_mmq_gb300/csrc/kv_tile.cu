// Attention of many query rows per sequence and key/value head (prompts, chunks of prompts, many
// drafted tokens) over the 8-bit cache: k_kv_attend_tile.
//
// Bound: the tensor cores (4 D operations per row and key). A CTA takes units (kv_attend.cuh) of two
// tiles of 128 rows (heads of 256: one); a row is a (token, query head) pair of one key/value head's group, so that
// the heads that share keys fill a tile together and a tile of keys and values, once converted,
// serves all of them.  Roles:
//   converter warps (4)  records by bulk copies into a staging of their own, one tile ahead; codes to
//                        exact f16 in shared memory, in the core-matrix order of tcgen05 (8 x 16
//                        bytes): keys as the K-major B operand of S = Q K^T, values in the same
//                        physical order as the MN-major B operand of O += P V (no transpose);
//   softmax warps (4 per row tile), a thread per row: S from TMEM, the running maximum, P as f16
//                        back into S's own columns as the A operand of the second product, the
//                        (rare) rescaling of O in TMEM, and at the end of a unit its output;
//   one elected thread of each row tile's first warp issues that tile's MMAs: the two row tiles
//                        alternate, one's products run while the other's softmax does.
// S of a tile and its P share columns: the products of one row tile run in issue order, and a
// row's thread has read its S before it writes its P.  f32 rows (SPLIT): queries and weights as
// two f16 terms each, twice the products.
//
// Measured (GB300): 1024 new of 32768 tokens, 32 heads of 128 over 8: 463 us, 1.17 PFLOP/s, 0.61 of
// the library's rate for a plain product; tensor pipe 0.47 of the cycles, issue slots 0.45.  Two row tiles of
// 128 x 128 keys take about 4050 cycles, 1024 of them the products' own at the tensor rate: the
// products' operands, the staged codes and the converted tiles move 320 KB through shared memory (2560
// cycles), and S, maximum, weights and P are a chain that the other tile's products cover in part.  Short
// prompts pay their units' ends (queries to f16 tiles, an empty pipeline, the output), five tiles' time
// each: 2048 tokens, 28 heads over 4, 53.4 us where the same work inside a long one would be 26.
// Registers: the launch's 168 a thread are the compiler's limit, whatever the split gives later; every instance
// spills, 140 to 268 bytes a thread stored, f32 rows of 128 640 (their flushed output alone is 128 registers
// beside 64 of S).
#include "kv_attend.cuh"
#include "umma.cuh"

namespace mmq {
namespace {

using namespace kv;

__device__ unsigned g_kv_tile_error;

template <int D, bool SPLIT>
struct Tile {
    // D = 256: the two groups of softmax warps share one tile of rows and take half of the value
    // columns each (S is formed twice; a group's TMEM and registers are those of D = 128)
    static constexpr bool HALF = D == 256;
    static constexpr int OD = HALF ? D / 2 : D;                  // value columns of a group
    static constexpr int KT = !SPLIT ? (HALF ? 64 : 128) : (HALF ? 32 : 64);  // keys per tile
    static constexpr int ST = 2;                                 // converted tiles in shared memory
    static constexpr int TERMS = SPLIT ? 2 : 1;
    static constexpr int SOFT = 8, CONV = 4, WARPS = SOFT + CONV, THREADS = 32 * WARPS;
    static constexpr int ROWS = HALF ? 128 : 256;
    static constexpr int KV = KT * D * 2, Q = 128 * D * 2;       // bytes of a converted tile, of a row tile's term
    static constexpr int RAW_HALF = KT / 4 * D, RAW = 2 * RAW_HALF + 16;  // a converter warp's codes of a tile, their scales
    static constexpr int OFF_V = ST * KV, OFF_Q = 2 * ST * KV, OFF_RAW = OFF_Q + (HALF ? 1 : 2) * TERMS * Q;
    static constexpr int OFF_BAR = OFF_RAW + CONV * RAW;
    static constexpr int NBAR = 4 * ST + 2 * 5 + 2 + 2 * CONV;
    static constexpr int USED = OFF_BAR + NBAR * 8;
    static constexpr int SMEM = USED > 120 * 1024 ? USED : 120 * 1024;  // one CTA an SM: it takes all of TMEM
    static constexpr int COL_O = 2 * KT;                         // TMEM columns: S of each group, then O
    static constexpr int BLK = KT / BT;                          // records per key tile
    // SPLIT: O leaves TMEM for f32 registers every 256 keys: the tensor core's accumulation rounds
    // towards zero, and its error grows with the number of products added (f32 rows of 1500 tokens:
    // 2.3e-6 off in all without it)
    static constexpr int FLUSH = 256 / KT;
    // registers: the softmax warps' and the converters' shares of the launch's 384 x 168
    static constexpr int R_SOFT = 216, R_CONV = 72;
    static_assert(2 * (KT + OD) <= 512 && SMEM <= 232448 - 2176, "tile sizes");
    static_assert(256 * R_SOFT + 128 * R_CONV <= 384 * 168, "register shares");
};

// A unit: a run of ROWS rows of one sequence and head, and the key tiles that they see.
struct Unit {
    int b, u, h;              // sequence, row run, head
    int start, n, len, rows;  // of the sequence; rows: n * group
    int lo, hi, kt0, tiles;   // keys that some row sees, first key tile, key tiles (0: no such unit)
};
template <int ROWS, int KT>
__device__ __forceinline__ void unit_span(const Attend& a, Unit& w) {
    const int r0 = w.u * ROWS;
    if (r0 >= w.rows) {
        w.tiles = 0;
        return;
    }
    const int first = w.len - w.n, t0 = r0 / a.group, t1 = min(w.n - 1, (r0 + ROWS - 1) / a.group);
    w.hi = first + t1 + 1;
    w.lo = w.hi > 0 ? first_key(a, first + t0) : 0;
    w.kt0 = w.lo / KT;
    w.tiles = max(1, (w.hi + KT - 1) / KT - w.kt0);  // a unit of padding rows alone: one tile, all of it masked
}
template <int ROWS, int KT>
__device__ __forceinline__ void unit_load(const Attend& a, Unit& w, int b, int u) {
    seq_range(a.c, a.bt, b, w.start, w.n, w.len, &g_kv_tile_error);
    w.rows = w.n * a.group;
    w.b = b;
    w.u = u;
    w.h = 0;
    unit_span<ROWS, KT>(a, w);
}

// What a unit costs beside its key tiles (queries in, output out, an empty pipeline), in key tiles: a unit
// takes OVERHEAD + tiles places in the list of work, and the first OVERHEAD of them hold nothing.
// Fitted to the CTAs' clocks: a tile 4050 cycles, a piece of a unit 20000 beside its tiles, a join 8000.
// Measured at 4 / 5 / 6, all units cut: a 2048-token bf16 prompt 68.5 / 68.4 / 68.7 us, 8192 tokens 551 / 524 /
// 509, 1024 tokens 43.0 / 36.5 / 37.4.
constexpr int OVERHEAD = 6;
constexpr int JOIN = 8;  // parts joined at a time (three levels: up to 512 CTAs)

// Units that are short beside a CTA's share are dealt whole instead: the longest first, round after round in
// turning order (0 .. W - 1, W - 1 .. 0, ..), where the longest of the shares that come of it is at most
// CUT key tiles above the even share.  What cutting costs, a second piece of a unit and a join, is seven of the tiles
// that OVERHEAD was fitted to (128 keys, 16 bits); CUT is fitted too, at 5 / 7 / 9: a 1024-token bf16 prompt 40.3 / 33.0 /
// 33.0 us, the f32 prompts below 88.0 / 88.2 / 79.9.  Both count tiles of 64 and 32 keys (f32, heads of 256), which
// take less time, the same; a figure for each was not measured.
// Measured dealt / cut, us: one prompt of 1024 tokens 33.0 / 39.3, 2048 54.4 / 70.9, 4096 157 / 189, 8192 465 / 507; sixteen
// of 100 to 900 on 900 to 1200 196 / 236; f32 79.4 / 87.7; where it would leave SMs idle (700 of 3000 with 16 heads of
// 64: 48 units) 55.8 / 38.7.  Its price where units are cut all the same, with / without the code for it: 1 to 4 us of
// ranking, and long chunks of f32 and of heads of 256, whose registers it takes: 1024 of 32768, 16 heads, f32 561 / 540,
// 256 829 / 778, 128 in 16 bits 247 / 247; dealt prompts of 2048 with heads of 256 78 / 92, six of 600 72 / 86, f32 60 / 70.
constexpr int CUT = 9;
__device__ __forceinline__ int dealt_unit(int round, int cta, int W) { return round * W + (round & 1 ? W - 1 - cta : cta); }

// How many CTAs share T places in U units: all, but for few units no more than 2 sqrt(T / U) a unit, where
// fewer tiles a CTA and more parts to join balance. Measured at 1.4, 2 and without the limit: 26 tokens x 8
// heads of 256 on 3838 tokens (two units) 49.8 / 47.5 / 63.6 us, 8 tokens on 65536 (four units) 69 / 65 / 65.
__device__ __forceinline__ int workers(int T, int U) {
    return min(min((int)gridDim.x, T), max(U, (int)(2.f * sqrtf((float)T * (float)U))));
}

template <int D, bool SPLIT>
__global__ void __launch_bounds__(Tile<D, SPLIT>::THREADS, 1)
k_kv_attend_tile(const Attend a) {
    using C = Tile<D, SPLIT>;
    constexpr int KT = C::KT, ST = C::ST, OD = C::OD, SBO = D * 16;
    constexpr bool HALF = C::HALF;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_scan[C::WARPS], s_at[3], s_last[2];
    __shared__ __align__(16) int s_pref[C::THREADS];
    __shared__ int s_work[3];  // T, W, U (below): not in registers throughout
    __shared__ float4 s_sc[4][C::BLK];  // dk, log2 dv, 1 / dv of the blocks of four consecutive tiles
    const int tid = threadIdx.x, lane = tid & 31, wid = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform
    const uint32_t base = ptx::smem_u32(smem), bars = base + C::OFF_BAR;
    const uint32_t k_full = bars, k_empty = bars + 8 * ST, v_full = bars + 16 * ST, v_empty = bars + 24 * ST;
    const uint32_t s_full = bars + 32 * ST, o_full = s_full + 16, p_ready = o_full + 16, joined = p_ready + 16;
    const uint32_t turn = joined + 16;  // the groups issue their products in turn
    const uint32_t q_ready = turn + 16, q_free = q_ready + 8;  // HALF: of the queries that both groups use
    const uint32_t raw_full = q_free + 8;                      // a converter warp's keys, values
    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            ptx::mbar_init(k_full + 8 * i, C::CONV);
            ptx::mbar_init(v_full + 8 * i, C::CONV);
            ptx::mbar_init(k_empty + 8 * i, 2);
            ptx::mbar_init(v_empty + 8 * i, 2);
        }
        for (int i = 0; i < 2 * C::CONV; ++i) ptx::mbar_init(raw_full + 8 * i, 1);
        ptx::mbar_init(q_ready, C::SOFT);
        ptx::mbar_init(q_free, C::SOFT);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(s_full + 8 * i, 1);
            ptx::mbar_init(o_full + 8 * i, 1);
            ptx::mbar_init(p_ready + 8 * i, 4);
            ptx::mbar_init(joined + 8 * i, 1);
            ptx::mbar_init(turn + 8 * i, 1);
        }
        ptx::fence_barrier_init();
        s_abort = 0;
    }
    ptx::grid_dep_wait();
    ptx::grid_dep_launch_dependents();

    // ---- this CTA's range of the work: sequences THREADS at a time, their row runs spread over the threads
    int T = 0, U = 0, W = 0, x0 = 0, x1 = 0;
    int my_tiles = 0, my_run = 0;  // the thread's row run, where every run has a thread
    bool located = false, dealt = false;
    for (int pass = 0; pass < 2 && !located; ++pass) {
        int carry = 0;
        for (int b0 = 0, units = 0; b0 < a.bt.seqs; b0 += C::THREADS) {
            int runs = 0, total;
            if (b0 + tid < a.bt.seqs) {
                int start, n, len;
                seq_range(a.c, a.bt, b0 + tid, start, n, len, &g_kv_tile_error);
                runs = (n * a.group + C::ROWS - 1) / C::ROWS;
            }
            s_pref[tid] = scan_cta<C::WARPS>(runs, total, s_scan);
            __syncthreads();
            U = (units += total) * a.c.heads;
            for (int i0 = 0; i0 < total; i0 += C::THREADS) {
                const int i = i0 + tid;
                Unit q;
                q.tiles = 0;
                if (i < total) {
                    int lo = 0, hi = C::THREADS - 1;  // the last sequence that begins at or before run i
                    while (lo < hi) {
                        const int mid = (lo + hi + 1) / 2;
                        if (s_pref[mid] <= i)
                            lo = mid;
                        else
                            hi = mid - 1;
                    }
                    unit_load<C::ROWS, KT>(a, q, b0 + lo, i - s_pref[lo]);
                }
                int sum;
                const int v = q.tiles ? (q.tiles + OVERHEAD) * a.c.heads : 0;
                const int e = carry + scan_cta<C::WARPS>(v, sum, s_scan);
                carry += sum;
                if (pass == 0 && a.bt.seqs <= C::THREADS && total <= C::THREADS) {  // that was all of it
                    located = true;
                    T = carry;
                    W = workers(T, total * a.c.heads);
                    x0 = work_start(T, min((int)blockIdx.x, W), W);
                    my_tiles = q.tiles;
                    my_run = q.b << 16 | q.u;
                }
                if ((pass == 1 || located) && x0 >= e && x0 < e + v) {
                    s_at[0] = q.b;
                    s_at[1] = q.u;
                    s_at[2] = x0 - e;
                }
            }
            __syncthreads();
        }
        if (pass == 0) {
            T = carry;
            W = workers(T, U);
            if (located) {  // the runs by falling tiles, and the longest share when they are dealt
                s_pref[tid] = my_tiles;
                __syncthreads();
                int rank = 0, share = 0;
                for (int i = 0; i < U / a.c.heads; i += 4) {
                    const int4 v = *reinterpret_cast<const int4*>(s_pref + i);
                    rank += (v.x > my_tiles || (v.x == my_tiles && i < tid)) + (v.y > my_tiles || (v.y == my_tiles && i + 1 < tid)) +
                            (v.z > my_tiles || (v.z == my_tiles && i + 2 < tid)) + (v.w > my_tiles || (v.w == my_tiles && i + 3 < tid));
                }
                __syncthreads();
                if (my_tiles > 0) s_pref[rank] = my_tiles;
                __syncthreads();
                const int all = min((int)gridDim.x, U);
                if (tid < all)
                    for (int r, k = 0; (r = dealt_unit(k, tid, all)) < U; ++k) share += s_pref[r / a.c.heads] + OVERHEAD;
                share = __reduce_max_sync(0xffffffffu, share);
                if (lane == 0) s_scan[wid] = share;
                __syncthreads();
#pragma unroll
                for (int i = 0; i < C::WARPS; ++i) share = max(share, s_scan[i]);
                dealt = (long long)(share - CUT) * W <= T;
                if (dealt) {
                    W = all;
                    if (my_tiles > 0) s_pref[rank] = my_run;
                }
            }
            if ((int)blockIdx.x >= W) return;
            x0 = work_start(T, blockIdx.x, W);
            x1 = dealt ? -1 : work_start(T, blockIdx.x + 1, W);
            if (tid == 0) {
                s_work[0] = T;
                s_work[1] = W;
                s_work[2] = U;
            }
        }
    }
    if (wid == 0) {
        ptx::tmem_alloc(ptx::smem_u32(&s_tmem), 512);
        ptx::tmem_relinquish();
    }
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
    volatile int* abort = &s_abort;
    unsigned* err = &g_kv_tile_error;

    Unit w;
    unit_load<C::ROWS, KT>(a, w, s_at[0], s_at[1]);
    w.h = s_at[2] / (w.tiles + OVERHEAD);
    int place = s_at[2] - w.h * (w.tiles + OVERHEAD), x = x0, o0 = 0, o1 = 0;  // place in the unit, key tiles of the piece
    if (place == w.tiles + OVERHEAD - 1) ++place, ++x;  // the CTA before has taken it
    if (x1 < 0) x = 0;  // dealt: its round
    // The next run of key tiles [o0, o1) of this CTA: a dealt unit, or what its places x .. x1 - 1 hold of the next
    // one in order (row runs of a sequence, the heads of each).  A unit's last tile is not parted from the one
    // before: the range that ends there takes it, the next one begins behind it (with / without, all units cut:
    // 1024 tokens 37.4 / 41.4 us, 2048 68.7 / 70.0, 700 of 3000 with heads of 64 36.9 / 35.3).
    auto next = [&]() -> bool {
        for (;;) {
            int b = w.b, u = w.u, h = w.h;
            bool other = x1 < 0;
            if (x1 < 0) {
                const int r = dealt_unit(x, blockIdx.x, s_work[1]);
                if (r >= s_work[2]) return false;
                const int run = r / a.c.heads, at = s_pref[run];
                b = at >> 16;
                u = at & 0xffff;
                h = r - run * a.c.heads;
            } else {
                if (x >= x1) return false;
                if (place == w.tiles + OVERHEAD) {
                    place = 0;
                    if (++h == a.c.heads) {
                        h = 0;
                        ++u;
                        other = true;
                    }
                }
            }
            if (other)
                for (; unit_load<C::ROWS, KT>(a, w, b, u), w.tiles == 0 && ++b < a.bt.seqs;) u = 0;
            w.h = h;
            if (x1 < 0) {
                o0 = 0;
                o1 = w.tiles;
                ++x;
                return true;
            }
            int span = min(w.tiles + OVERHEAD - place, x1 - x);
            if (w.tiles + OVERHEAD - place - span == 1) ++span;
            o0 = max(0, place - OVERHEAD);
            o1 = max(0, place + span - OVERHEAD);
            place += span;
            x += span;
            if (o1 > o0) return true;
        }
    };

    if (wid >= C::SOFT) {
        // ------------------------------------------------ converters: warp cw takes tokens KT/4 cw ..
        // Its codes come by bulk copies into its own staging, keys and values by turns, each requested
        // as soon as the tile before has been read. Lanes read and write diagonally (row l, chunk
        // l + s): eight lanes then touch eight bank groups of the codes' rows and of the core matrices.
        ptx::regs_dec<C::R_CONV>();
        constexpr int GROUPS = KT / 32, PER = D / 64;  // groups of eight rows, 16-byte chunks a lane and group
        const int cw = wid - C::SOFT, l8 = lane & 7, cq = lane >> 3;
        const int tok0 = cw * (KT / 4), bi = tok0 / BT, sub = tok0 % BT;
        uint8_t* raw = smem + C::OFF_RAW + cw * C::RAW;
        const uint32_t raw_k = raw_full + 16 * cw, raw_v = raw_k + 8;
        bool more[3];           // whether tiles n, n + 1, n + 2 of this CTA exist
        const uint8_t* rec[2];  // this warp's record in tiles n, n + 1 (nullptr: nothing in reach there)
        int o = 0, in = 0, id = -1;  // of tile n + 2: its place in its record's page, its page number (on its way)
        bool begun = false, reach = false;  // reach: some row of the tile sees keys of this warp's
        auto advance = [&]() -> bool {  // the cursor to the next tile
            if (!begun || ++o == o1) {
                begun = true;
                if (!next()) return false;
                o = o0;
            }
            const int blk = (w.kt0 + o) * C::BLK + bi;
            reach = false;
            if (blk * BT < w.hi && blk * BT + BT > w.lo) {
                const int pg = blk / a.c.blocks;
                in = blk - pg * a.c.blocks;
                id = a.bt.table[(long long)w.b * a.bt.table_stride + pg];
                reach = true;
            }
            return true;
        };
        auto resolve = [&]() -> const uint8_t* {
            if (!reach) return nullptr;
            if (id < 0 || id >= a.c.pages) {
                if (lane == 0) atomicOr(err, ERR_RANGE);
                return nullptr;
            }
            return a.c.data + (((long long)id * a.c.heads + w.h) * a.c.blocks + in) * rec_bytes(D);
        };
        uint32_t k_asked = 0, k_had = 0, v_asked = 0, v_had = 0;  // copies requested and waited for
        auto fetch_k = [&](const uint8_t* p) {
            __syncwarp();
            if (!p) return;
            ++k_asked;
            if (ptx::elect_one()) {
                ptx::mbar_arrive_expect_tx(raw_k, C::RAW_HALF + 16);
                ptx::bulk_load(ptx::smem_u32(raw), p + sub * D, C::RAW_HALF, raw_k);
                ptx::bulk_load(ptx::smem_u32(raw) + 2 * C::RAW_HALF, p + 2 * BT * D, 16, raw_k);
            }
        };
        auto fetch_v = [&](const uint8_t* p) {
            __syncwarp();
            if (!p) return;
            ++v_asked;
            if (ptx::elect_one()) {
                ptx::mbar_arrive_expect_tx(raw_v, C::RAW_HALF);
                ptx::bulk_load(ptx::smem_u32(raw) + C::RAW_HALF, p + (BT + sub) * D, C::RAW_HALF, raw_v);
            }
        };
        auto convert = [&](const uint8_t* src, uint8_t* dst, bool some) {
#pragma unroll
            for (int gr = 0; gr < GROUPS; ++gr)
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int ch = D == 64 ? ((l8 >> 1) + cq) & 3 : (l8 + cq + 4 * i) & (D / 16 - 1);
                    uint4 q = make_uint4(0u, 0u, 0u, 0u);
                    if (some) q = *reinterpret_cast<const uint4*>(src + (8 * gr + l8) * D + 16 * ch);
                    uint8_t* p = dst + ((tok0 >> 3) + gr) * SBO + 256 * ch + 16 * l8;
                    const uint2 c0 = umma::i8x4_to_f16x4(q.x), c1 = umma::i8x4_to_f16x4(q.y);
                    const uint2 c2 = umma::i8x4_to_f16x4(q.z), c3 = umma::i8x4_to_f16x4(q.w);
                    *reinterpret_cast<uint4*>(p) = make_uint4(c0.x, c0.y, c1.x, c1.y);
                    *reinterpret_cast<uint4*>(p + 128) = make_uint4(c2.x, c2.y, c3.x, c3.y);
                }
            ptx::fence_proxy_async_smem();
            __syncwarp();
        };
        more[0] = advance();
        rec[0] = more[0] ? resolve() : nullptr;
        fetch_k(rec[0]);
        fetch_v(rec[0]);
        more[1] = more[0] && advance();
        rec[1] = more[1] ? resolve() : nullptr;
        more[2] = more[1] && advance();
        for (int n = 0; more[0]; ++n) {
            const int st = n % ST;
            const uint32_t par = ((n / ST) & 1) ^ 1;
            const bool some = rec[0] != nullptr;
            if (!umma::warp_wait(k_empty + 8 * st, par, abort, err)) break;
            if (some && !umma::warp_wait(raw_k, k_had & 1, abort, err)) break;
            if (some) ++k_had;
            if (lane == 0 && sub == 0) {
                float dk = 0.f, lv = -INFINITY, rv = 0.f;
                if (some) {
                    const float2 sc = *reinterpret_cast<const float2*>(raw + 2 * C::RAW_HALF);
                    dk = sc.x;
                    value_scale(sc.y, lv, rv);
                }
                s_sc[n & 3][bi] = make_float4(dk, lv, rv, 0.f);
            }
            convert(raw, smem + st * C::KV, some);
            if (lane == 0) ptx::mbar_arrive(k_full + 8 * st);
            fetch_k(rec[1]);
            if (!umma::warp_wait(v_empty + 8 * st, par, abort, err)) break;
            if (some && !umma::warp_wait(raw_v, v_had & 1, abort, err)) break;
            if (some) ++v_had;
            convert(raw + C::RAW_HALF, smem + C::OFF_V + st * C::KV, some);
            if (lane == 0) ptx::mbar_arrive(v_full + 8 * st);
            fetch_v(rec[1]);
            more[0] = more[1];
            rec[0] = rec[1];
            more[1] = more[2];
            rec[1] = more[1] ? resolve() : nullptr;
            more[2] = more[1] && advance();
        }
        // given up: let the copies in flight land before the shared memory goes
        const uint64_t t0 = ptx::globaltimer_ns();
        while ((k_had != k_asked || v_had != v_asked) && ptx::globaltimer_ns() - t0 < umma::WAIT_LIMIT_NS) {
            if (k_had != k_asked && ptx::mbar_test_wait(raw_k, k_had & 1)) ++k_had;
            if (v_had != v_asked && ptx::mbar_test_wait(raw_v, v_had & 1)) ++v_had;
        }
    } else {
        // ------------------------------------------------ softmax: thread = row, and the MMA issue
        ptx::regs_inc<C::R_SOFT>();
        const int gt = wid >> 2, row = tid & 127, wrow = (wid & 3) * 32;  // group, row of its tile, the warp's first
        const int tile0 = HALF ? 0 : gt * 128, col0 = HALF ? gt * OD : 0;  // first row of the unit, first value column
        const bool lead = (wid & 3) == 0;  // the warp that issues the group's products
        const uint32_t lane_off = (uint32_t)wrow << 16;
        const uint32_t t_s = tmem + gt * KT, t_o = tmem + C::COL_O + gt * OD;
        const uint32_t sf = s_full + 8 * gt, of = o_full + 8 * gt, pr = p_ready + 8 * gt, jn = joined + 8 * gt;
        const uint32_t q_addr = base + C::OFF_Q + (HALF ? 0 : gt * C::TERMS * C::Q);
        uint8_t* q_smem = smem + C::OFF_Q + (HALF ? 0 : gt * C::TERMS * C::Q);
        constexpr uint32_t idesc_s = umma::make_idesc(128, KT), idesc_o = umma::make_idesc(128, OD) | (1u << 16);
        uint32_t n_pr = 0, n_sf = 0, n_of = 0, n_jn = 0, n_unit = 0;  // phases
        auto issue_s = [&](int stage) {  // S = Q K^T, the small terms first
            const int st = __shfl_sync(0xffffffffu, stage, 0);
            if (!ptx::elect_one()) return;
            const uint64_t bd = umma::sdesc(base + st * C::KV, SBO);
#pragma unroll
            for (int e = C::TERMS - 1; e >= 0; --e) {
                const uint64_t ad = umma::sdesc(q_addr + e * C::Q, SBO);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    ptx::umma_f16(t_s, ad + 16 * ks, bd + 16 * ks, idesc_s, e < C::TERMS - 1 || ks > 0);
            }
            ptx::umma_commit(k_empty + 8 * st);
            ptx::umma_commit(sf);
        };
        // values: 8-column groups 128 B apart (stride offset), 8-token groups SBO apart (leading offset)
        auto issue_o = [&](int stage, bool fresh, bool last) {
            const int st = __shfl_sync(0xffffffffu, stage, 0), first = __shfl_sync(0xffffffffu, (int)fresh, 0);
            if (!ptx::elect_one()) return;
            const uint32_t va = base + C::OFF_V + st * C::KV + col0 * 16;
            const uint64_t bd = (uint64_t)((va & 0x3FFFFu) >> 4) | ((uint64_t)(SBO >> 4) << 16) | ((uint64_t)(128 >> 4) << 32) |
                                (1ull << 46);
#pragma unroll
            for (int ks = 0; ks < KT / 16; ++ks)
#pragma unroll
                for (int e = 0; e < C::TERMS; ++e)
                    ptx::umma_f16_ts(t_o, t_s + 32 * (ks >> 1) + 16 * e + 8 * (ks & 1), bd + (uint64_t)(2 * SBO >> 4) * ks, idesc_o,
                                     !(first && ks + e == 0));
            ptx::umma_commit(v_empty + 8 * st);
            if (last) ptx::umma_commit(of);
        };
        // The groups alternate batch by batch (O += P V, then the next S): batches that ran side by
        // side would end together, and then both groups' softmaxes would run side by side too.
        uint32_t n_turn = gt == 0 ? 1 : 0;
        auto take_turn = [&]() { return umma::warp_wait(turn + 8 * gt, n_turn++ & 1, abort, err); };
        auto pass_turn = [&]() {
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(turn + 8 * (1 - gt));
        };
        auto signal = [&](uint32_t bar) {  // this warp's part is in place
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar);
        };
        bool ok = true;
        for (int n = 0; ok && next();) {
            const int tiles = o1 - o0;  // this unit's tiles here
            const int row0 = w.u * C::ROWS + tile0, r = row0 + row;
            if (row0 >= w.rows) {
                // no rows in this row tile: only pass the converted tiles on
                if (lead)
                    for (int i = 0; i <= tiles && ok; ++i) {
                        if (i > 0) {
                            ok = umma::warp_wait(v_full + 8 * ((n + i - 1) % ST), ((n + i - 1) / ST) & 1, abort, err);
                            if (ok && lane == 0) ptx::mbar_arrive(v_empty + 8 * ((n + i - 1) % ST));
                        }
                        if (i < tiles && ok) {
                            ok = umma::warp_wait(k_full + 8 * ((n + i) % ST), ((n + i) / ST) & 1, abort, err);
                            if (ok && lane == 0) ptx::mbar_arrive(k_empty + 8 * ((n + i) % ST));
                        }
                        ok = ok && take_turn();
                        if (ok) pass_turn();
                    }
            } else {
                const bool real = r < w.rows;
                const int t = r / a.group, hq = w.h * a.group + r - t * a.group, pos = w.len - w.n + t;
                // the warp's rows of queries, scaled into f16's range, in core-matrix order: eight rows at
                // a time, lane (row % 8, 16-byte chunk % 4); HALF: each group writes half of the columns
                if (HALF && n_unit > 0 && !umma::warp_wait(q_free, (n_unit - 1) & 1, abort, err)) {
                    ok = false;
                    break;
                }
                float up = 1.f;
                constexpr int NC = D / 32, GB = (SPLIT ? 2 : 4) / (HALF ? 2 : 1);  // chunks a lane, row groups in flight
#pragma unroll 1
                for (int g0 = 0; g0 < 4; g0 += GB) {
                    uint4 raw[GB][NC][SPLIT ? 2 : 1];
#pragma unroll
                    for (int gi = 0; gi < GB; ++gi) {
                        const int rr = row0 + wrow + 8 * (g0 + gi) + (lane & 7), tt = rr / a.group;
                        const long long at = (long long)(w.start + tt) * a.q.token_stride +
                                             (long long)(w.h * a.group + rr - tt * a.group) * a.q.head_stride + 8 * (lane >> 3);
                        const uint8_t* src = static_cast<const uint8_t*>(a.q.data) + at * (SPLIT ? 4 : 2);
#pragma unroll
                        for (int i = 0; i < NC; ++i)
#pragma unroll
                            for (int e = 0; e < (SPLIT ? 2 : 1); ++e)
                                raw[gi][i][e] = rr < w.rows ? *reinterpret_cast<const uint4*>(src + i * (SPLIT ? 128 : 64) + 16 * e)
                                                            : make_uint4(0u, 0u, 0u, 0u);
                    }
#pragma unroll
                    for (int gi = 0; gi < GB; ++gi) {
                        const int rl = wrow + 8 * (g0 + gi) + (lane & 7);
                        auto eight = [&](int i, float4& u, float4& v) {
                            const uint4 p = raw[gi][i][0], q = raw[gi][i][SPLIT ? 1 : 0];
                            if (SPLIT) {
                                u = make_float4(__uint_as_float(p.x), __uint_as_float(p.y), __uint_as_float(p.z), __uint_as_float(p.w));
                                v = make_float4(__uint_as_float(q.x), __uint_as_float(q.y), __uint_as_float(q.z), __uint_as_float(q.w));
                            } else {
                                u = Elem<__nv_bfloat16>::widen(make_uint2(p.x, p.y));
                                v = Elem<__nv_bfloat16>::widen(make_uint2(p.z, p.w));
                            }
                        };
                        float down = 1.f, upr = 1.f;
                        if (SPLIT || a.dtype == MMQ_BF16) {  // f16 rows are operands as they are
                            // magnitudes order as their bits do; bf16 pairs as two 16-bit numbers
                            uint32_t am = 0u;
#pragma unroll
                            for (int i = 0; i < NC; ++i)
#pragma unroll
                                for (int e = 0; e < (SPLIT ? 2 : 1); ++e) {
                                    const uint4 p = raw[gi][i][e];
                                    const uint32_t mask = SPLIT ? 0x7fffffffu : 0x7fff7fffu;
                                    const uint32_t p0 = p.x & mask, p1 = p.y & mask, p2 = p.z & mask, p3 = p.w & mask;
                                    am = SPLIT ? max(max(am, max(p0, p1)), max(p2, p3))
                                               : __vmaxu2(__vmaxu2(am, __vmaxu2(p0, p1)), __vmaxu2(p2, p3));
                                }
                            if (!SPLIT) am = max(am & 0xffffu, am >> 16) << 16;
                            am = max(am, __shfl_xor_sync(0xffffffffu, am, 8));
                            am = max(am, __shfl_xor_sync(0xffffffffu, am, 16));
                            row_scale(__uint_as_float(am), down, upr);
                        }
                        if (lane >> 3 == g0 + gi) up = upr;
                        uint8_t* dst = q_smem + (rl >> 3) * SBO + (lane >> 3) * 128 + (rl & 7) * 16;
#pragma unroll
                        for (int i = 0; i < NC; ++i) {
                            if (HALF && (i >= NC / 2) != (gt == 1)) continue;
                            if (!SPLIT && a.dtype == MMQ_F16) {
                                *reinterpret_cast<uint4*>(dst + 512 * i) = raw[gi][i][0];
                                continue;
                            }
                            float4 u, v;
                            eight(i, u, v);
                            uint4 hi4, lo4;
                            split_h2(u.x * down, u.y * down, hi4.x, lo4.x);
                            split_h2(u.z * down, u.w * down, hi4.y, lo4.y);
                            split_h2(v.x * down, v.y * down, hi4.z, lo4.z);
                            split_h2(v.z * down, v.w * down, hi4.w, lo4.w);
                            *reinterpret_cast<uint4*>(dst + 512 * i) = hi4;
                            if (SPLIT) *reinterpret_cast<uint4*>(dst + C::Q + 512 * i) = lo4;
                        }
                    }
                }
                ptx::fence_proxy_async_smem();
                const float fq = up * a.scale2;
                const int hi = real ? pos + 1 : 0x7fffffff, lo = real && a.window > 0 ? max(0, pos - a.window + 1) : 0;
                const int hi_min = __reduce_min_sync(0xffffffffu, hi), lo_max = __reduce_max_sync(0xffffffffu, lo);
                signal(HALF ? q_ready : pr);
                if (lead) {
                    ok = umma::warp_wait(HALF ? q_ready : pr, HALF ? n_unit & 1 : n_pr & 1, abort, err) &&
                         umma::warp_wait(k_full + 8 * (n % ST), (n / ST) & 1, abort, err) && take_turn();
                    if (ok) {
                        ptx::tc_fence_after();
                        issue_s(n % ST);
                        pass_turn();
                    }
                }
                if (!HALF) ++n_pr;
                ++n_unit;
                float m = M_NONE, l = 0.f;
                unsigned long long om[SPLIT ? OD / 2 : 1];  // SPLIT: O so far, pairs of columns
#pragma unroll
                for (int k = 0; k < (SPLIT ? OD / 2 : 1); ++k) om[k] = 0ull;
#pragma unroll 1
                for (int i = 0; i < tiles; ++i) {
                    const int nn = n + i, j0 = (w.kt0 + o0 + i) * KT;
                    if (!umma::warp_wait(sf, n_sf++ & 1, abort, err)) {
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    if (HALF && i + 1 == tiles) signal(q_free);
                    uint32_t sr[C::BLK][32];
#pragma unroll
                    for (int c = 0; c < C::BLK; ++c) ptx::tmem_ld32(t_s + lane_off + 32 * c, sr[c]);
                    const float4* scv = s_sc[nn & 3];
                    const bool edge = j0 + KT > hi_min || j0 < lo_max;
                    float af[C::BLK], lv[C::BLK], rv[C::BLK];
#pragma unroll
                    for (int c = 0; c < C::BLK; ++c) {
                        const float4 s4 = scv[c];
                        af[c] = fq * s4.x;
                        lv[c] = s4.y;
                        rv[c] = s4.z;
                    }
                    float tm = -INFINITY;
#pragma unroll
                    for (int c = 0; c < C::BLK; ++c) ptx::tmem_ld_wait(sr[c]);
                    if (!edge) {
#pragma unroll
                        for (int c = 0; c < C::BLK; ++c) {
                            float mx = __uint_as_float(sr[c][0]), my = __uint_as_float(sr[c][1]);
#pragma unroll
                            for (int k = 2; k < 32; k += 4) {
                                mx = fmaxf(fmaxf(mx, __uint_as_float(sr[c][k])), __uint_as_float(sr[c][k + 1]));
                                if (k + 3 < 32)
                                    my = fmaxf(fmaxf(my, __uint_as_float(sr[c][k + 2])), __uint_as_float(sr[c][k + 3]));
                            }
                            tm = fmaxf(tm, fmaf(fmaxf(mx, my), af[c], lv[c]));
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < C::BLK; ++c)
#pragma unroll
                            for (int k = 0; k < 32; ++k) {
                                const int j = j0 + 32 * c + k;
                                const float tk = j >= lo && j < hi ? fmaf(__uint_as_float(sr[c][k]), af[c], lv[c]) : -INFINITY;
                                tm = fmaxf(tm, tk);
                                sr[c][k] = __float_as_uint(tk);
                            }
                    }
                    // the products so far are done: S came after them
                    const bool flush = SPLIT && i > 0 && i % C::FLUSH == 0;
                    if (SPLIT && flush) {
#pragma unroll
                        for (int c = 0; c < OD / 16; ++c) {
                            uint32_t ov[16];
                            ptx::tmem_ld16(t_o + lane_off + 16 * c, ov);
                            ptx::tmem_ld_wait(ov);
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                om[SPLIT ? 8 * c + k : 0] = ptx::add_f32x2(
                                    om[SPLIT ? 8 * c + k : 0], ptx::f2_bits(__uint_as_float(ov[2 * k]), __uint_as_float(ov[2 * k + 1])));
                        }
                    }
                    if (__any_sync(0xffffffffu, tm > m + LIMIT)) {
                        const float mn = fmaxf(m, tm - SHIFT), f = exp2_approx(m - mn);
                        m = mn;
                        l *= f;
                        if (SPLIT) {
                            const unsigned long long f2 = ptx::f2_bits(f, f);
#pragma unroll
                            for (int k = 0; k < (SPLIT ? OD / 2 : 1); ++k) om[k] = ptx::mul_f32x2(om[k], f2);
                        }
                        if (i > 0 && !flush) {
#pragma unroll 1
                            for (int c = 0; c < OD / 16; ++c) {
                                uint32_t ov[16];
                                ptx::tmem_ld16(t_o + lane_off + 16 * c, ov);
                                ptx::tmem_ld_wait(ov);
#pragma unroll
                                for (int k = 0; k < 16; ++k) ov[k] = __float_as_uint(__uint_as_float(ov[k]) * f);
                                ptx::tmem_st16(t_o + lane_off + 16 * c, ov);
                            }
                        }
                    }
#pragma unroll
                    for (int c = 0; c < C::BLK; ++c) {
                        if (edge) {
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                sr[c][k] = __float_as_uint(exp2_approx(__uint_as_float(sr[c][k]) - m));
                        } else {
                            const float bf = lv[c] - m;
                            const unsigned long long a2 = ptx::f2_bits(af[c], af[c]), b2 = ptx::f2_bits(bf, bf);
#pragma unroll
                            for (int k = 0; k < 32; k += 2) {
                                const unsigned long long t2 = ptx::fma_f32x2(
                                    ptx::f2_bits(__uint_as_float(sr[c][k]), __uint_as_float(sr[c][k + 1])), a2, b2);
                                sr[c][k] = __float_as_uint(exp2_approx(__uint_as_float((uint32_t)t2)));
                                sr[c][k + 1] = __float_as_uint(exp2_approx(__uint_as_float((uint32_t)(t2 >> 32))));
                            }
                        }
                        unsigned long long sum2 = 0ull, sum3 = 0ull;
#pragma unroll
                        for (int k = 0; k < 32; k += 4) {
                            sum2 = ptx::add_f32x2(sum2, ptx::f2_bits(__uint_as_float(sr[c][k]), __uint_as_float(sr[c][k + 1])));
                            sum3 = ptx::add_f32x2(sum3,
                                                  ptx::f2_bits(__uint_as_float(sr[c][k + 2]), __uint_as_float(sr[c][k + 3])));
                        }
                        sum2 = ptx::add_f32x2(sum2, sum3);
                        l = fmaf(__uint_as_float((uint32_t)sum2) + __uint_as_float((uint32_t)(sum2 >> 32)), rv[c], l);
                        uint32_t pw[16];
                        if (SPLIT) {
                            uint32_t pl[16];
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                split_h2(__uint_as_float(sr[c][2 * k]), __uint_as_float(sr[c][2 * k + 1]), pw[k], pl[k]);
                            ptx::tmem_st16(t_s + lane_off + 32 * c + 16, pl);
                        } else {
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                pw[k] = pack_h2(__uint_as_float(sr[c][2 * k]), __uint_as_float(sr[c][2 * k + 1]));
                        }
                        ptx::tmem_st16(t_s + lane_off + 32 * c, pw);
                    }
                    ptx::tmem_st_wait();
                    signal(pr);
                    if (lead) {
                        // the next tile's keys are converted after this one's values: one wait for both
                        const int st = nn % ST, par = (nn / ST) & 1, s2 = (nn + 1) % ST, par2 = ((nn + 1) / ST) & 1;
                        ok = umma::warp_wait(pr, n_pr & 1, abort, err) &&
                             (i + 1 == tiles ? umma::warp_wait(v_full + 8 * st, par, abort, err)
                                             : umma::warp_wait(k_full + 8 * s2, par2, abort, err)) &&
                             take_turn();
                        if (ok) {
                            ptx::tc_fence_after();
                            issue_o(st, i == 0 || flush, i + 1 == tiles);
                            if (i + 1 < tiles) issue_s(s2);
                            pass_turn();
                        }
                    }
                    ++n_pr;
                }
                ok = ok && umma::warp_wait(of, n_of++ & 1, abort, err);
                if (!ok) break;
                ptx::tc_fence_after();
                // ---- the unit's output, or this CTA's part of it
                const int ufirst = x - place + OVERHEAD;  // place of the unit's first key tile
                const bool whole = o0 == 0 && tiles == w.tiles;
                // a part's layout: [OD / 4][128 rows] float4, then m, l of the rows, for each level of joining
                auto part = [&](int cta, int slot) { return part_slot(a, cta, slot) + gt * 128 * (OD + WS_ROW_STATS); };
                float* mine = part(blockIdx.x, o0 == 0 ? 1 : 0);
                const float inv = whole ? (l > 0.f ? __frcp_rn(l) : 0.f) : 1.f;
#pragma unroll
                for (int c = 0; c < OD / 16; ++c) {
                    uint32_t ov[16];
                    ptx::tmem_ld16(t_o + lane_off + 16 * c, ov);
                    ptx::tmem_ld_wait(ov);
                    if (real) {
                        float f[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const unsigned long long o2 = om[SPLIT ? 8 * c + k / 2 : 0];
                            f[k] = (__uint_as_float(ov[k]) + (SPLIT ? __uint_as_float((uint32_t)(k & 1 ? o2 >> 32 : o2)) : 0.f)) * inv;
                        }
#pragma unroll
                        for (int k = 0; k < 16; k += 8) {
                            const float4 f0 = make_float4(f[k], f[k + 1], f[k + 2], f[k + 3]);
                            const float4 f1 = make_float4(f[k + 4], f[k + 5], f[k + 6], f[k + 7]);
                            if (whole) {
                                store_out8(a, w.start + t, hq, col0 + 16 * c + k, f0, f1);
                            } else {
                                *reinterpret_cast<float4*>(mine + ((4 * c + k / 4) * 128 + row) * 4) = f0;
                                *reinterpret_cast<float4*>(mine + ((4 * c + k / 4 + 1) * 128 + row) * 4) = f1;
                            }
                        }
                    }
                }
                ptx::tc_fence_before();
                if (whole) {
                    if (real && col0 == 0) store_lse(a, w.start + t, hq, m, l);
                } else {
                    if (real) {
                        mine[128 * OD + row] = m;
                        mine[128 * (OD + 1) + row] = l;
                    }
                    const int c0 = work_owner(s_work[0], ufirst, s_work[1]), c1 = work_owner(s_work[0], ufirst + w.tiles - 2, s_work[1]);
                    // few rows: several threads a row, a share of the columns each
                    const int nr = min(128, w.rows - row0), lg = nr > 64 ? 7 : nr > 32 ? 6 : 5;
                    const int jr = row & ((1 << lg) - 1), seg = row >> lg, span = (OD / 4) >> (7 - lg);
                    int at = blockIdx.x - c0, step = 1;  // this part among the level's, their distance in CTAs
                    for (int level = 0;; ++level) {
                        const int all = (c1 - c0 + step) / step, begin = at / JOIN * JOIN, count = min(JOIN, all - begin);
                        const int first = c0 + begin * step;
                        signal(pr);  // with the counter's release and acquire: the rows' parts are there first
                        if (lead) {
                            ok = umma::warp_wait(pr, n_pr & 1, abort, err);
                            if (lane == 0) {
                                unsigned* counter = reinterpret_cast<unsigned*>(a.ws) +
                                                    ((level * (int)gridDim.x + first) * 2 + (first == c0)) * 2 + gt;
                                s_last[gt] = 0;
                                if (ok && ptx::atom_inc_acq_rel(counter) == (unsigned)(count - 1)) {
                                    *counter = 0;
                                    s_last[gt] = 1;
                                }
                                ptx::mbar_arrive(jn);
                            }
                        }
                        ++n_pr;
                        ok = ok && umma::warp_wait(jn, n_jn++ & 1, abort, err);
                        if (!ok || !s_last[gt]) break;
                        const bool final = count == all;
                        if (jr < nr) {
                            const int rj = row0 + jr, tj = rj / a.group, hj = w.h * a.group + rj - tj * a.group;
                            float M = M_NONE, L = 0.f, f[JOIN], lp[JOIN];
#pragma unroll
                            for (int i = 0; i < JOIN; ++i) {
                                f[i] = M_NONE;
                                lp[i] = 0.f;
                                if (i < count) {
                                    const int c = first + i * step;
                                    const float* p = part(c, c == c0) + 128 * OD + level * 256 + jr;
                                    f[i] = __ldcg(p);
                                    lp[i] = __ldcg(p + 128);
                                }
                            }
#pragma unroll
                            for (int i = 0; i < JOIN; ++i) M = fmaxf(M, f[i]);
#pragma unroll
                            for (int i = 0; i < JOIN; ++i) {
                                f[i] = exp2_approx(f[i] - M);
                                L += lp[i] * f[i];
                            }
                            const float sc = final ? (L > 0.f ? __frcp_rn(L) : 0.f) : 1.f;
                            float* to = part(first, first == c0);
                            auto put = [&](int k, float4 x, float4 y) {  // float4 k and k + 1 of the row
                                x = make_float4(x.x * sc, x.y * sc, x.z * sc, x.w * sc);
                                y = make_float4(y.x * sc, y.y * sc, y.z * sc, y.w * sc);
                                if (final) {
                                    store_out8(a, w.start + tj, hj, col0 + 4 * k, x, y);
                                } else {
                                    *reinterpret_cast<float4*>(to + (k * 128 + jr) * 4) = x;
                                    *reinterpret_cast<float4*>(to + ((k + 1) * 128 + jr) * 4) = y;
                                }
                            };
                            if (count == 2 && lg == 7) {  // the usual end: a long run of both parts' columns in flight
                                const float4* p = reinterpret_cast<const float4*>(to) + jr;
                                const float4* q = reinterpret_cast<const float4*>(part(first + step, 0)) + jr;
                                const float fp = f[0], fq2 = f[1];
#pragma unroll 1
                                for (int k = 0; k < OD / 4; k += 16) {
                                    float4 y[16], z[16];
#pragma unroll
                                    for (int e = 0; e < 16; ++e) {
                                        y[e] = __ldcg(p + (k + e) * 128);
                                        z[e] = __ldcg(q + (k + e) * 128);
                                    }
#pragma unroll
                                    for (int e = 0; e < 16; ++e)
                                        y[e] = make_float4(y[e].x * fp + z[e].x * fq2, y[e].y * fp + z[e].y * fq2,
                                                           y[e].z * fp + z[e].z * fq2, y[e].w * fp + z[e].w * fq2);
#pragma unroll
                                    for (int e = 0; e < 16; e += 2) put(k + e, y[e], y[e + 1]);
                                }
                            } else {
#pragma unroll 1
                                for (int k = seg * span; k < (seg + 1) * span; k += 4) {
                                    float4 v[4];
#pragma unroll
                                    for (int e = 0; e < 4; ++e) v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                                    for (int i = 0; i < JOIN; ++i) {
                                        if (i >= count) break;
                                        const int c = first + i * step;
                                        const float4* p = reinterpret_cast<const float4*>(part(c, c == c0)) + k * 128 + jr;
#pragma unroll
                                        for (int e = 0; e < 4; ++e) {
                                            const float4 y = __ldcg(p + e * 128);
                                            v[e] = make_float4(v[e].x + y.x * f[i], v[e].y + y.y * f[i], v[e].z + y.z * f[i],
                                                               v[e].w + y.w * f[i]);
                                        }
                                    }
                                    put(k, v[0], v[1]);
                                    put(k + 2, v[2], v[3]);
                                }
                            }
                            if (seg == 0) {
                                if (!final) {
                                    to[128 * OD + (level + 1) * 256 + jr] = M;
                                    to[128 * OD + (level + 1) * 256 + 128 + jr] = L;
                                } else if (col0 == 0) {
                                    store_lse(a, w.start + tj, hj, M, L);
                                }
                            }
                        }
                        if (final) break;
                        at /= JOIN;
                        step *= JOIN;
                    }
                    if (!ok) break;
                }
            }
            n += tiles;
        }
        // given up: the products in flight end before TMEM and the shared memory go
        if (lead && *abort && ptx::elect_one()) {
            ptx::umma_commit(jn);
            umma::drain_bar(jn, n_jn & 1, err);
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (wid == 0) ptx::tmem_dealloc(tmem, 512);
}

template <int D, bool SPLIT>
int launch(const Attend& a, cudaStream_t s) {
    using C = Tile<D, SPLIT>;
    static SmemAttr attr;
    const char* fn = "mmq_kv_attend";
    const long long runs = (long long)a.bt.tokens * a.group / C::ROWS + a.bt.seqs;
    const long long tiles = runs * a.c.heads * ((long long)a.bt.table_pages * a.c.page / C::KT + 1 + OVERHEAD);
    if (tiles > 0x7fffffff || (long long)a.bt.max_new * a.group > 0x7fffffff - C::ROWS) {
        report(fn, MMQ_ERR_SHAPE, "too many row and key tiles (rows / 128 * heads * keys / 64 above 2^31)");
        return MMQ_ERR_SHAPE;
    }
    const int st = ensure_smem(reinterpret_cast<const void*>(&k_kv_attend_tile<D, SPLIT>), C::SMEM, attr);
    if (st != MMQ_OK) {
        report(fn, st, "the attention tiles' shared memory was refused");
        return st;
    }
    const long long sms = device_shape().sms < 341 ? device_shape().sms : 341;  // the counters' room
    ProfScope ps("k_kv_attend_tile", s);
    return pdl_status(launch_pdl(&k_kv_attend_tile<D, SPLIT>, dim3((unsigned)(tiles < sms ? tiles : sms)), dim3(C::THREADS),
                                 C::SMEM, s, a),
                      fn);
}

}  // namespace

int kv_tile_launch(const Attend& a, cudaStream_t s) {
    const bool split = a.dtype == MMQ_F32;
    if (a.c.dim == 64) return split ? launch<64, true>(a, s) : launch<64, false>(a, s);
    if (a.c.dim == 128) return split ? launch<128, true>(a, s) : launch<128, false>(a, s);
    return split ? launch<256, true>(a, s) : launch<256, false>(a, s);
}

unsigned kv_tile_take_error() {
    unsigned v = 0;
    if (cudaMemcpyFromSymbol(&v, g_kv_tile_error, sizeof(v)) != cudaSuccess) return 0;
    if (v) {
        const unsigned zero = 0;
        cudaMemcpyToSymbol(g_kv_tile_error, &zero, sizeof(zero));
    }
    return v;
}

}  // namespace mmq
