// How a feed-forward call is laid out on the GPU (row tiles, rounds, cuts, rings, scratch memory), and its two
// launches: the rows as operands, then the products.
#include "ffn_weights.cuh"

namespace mmq {
namespace {

using namespace ffn;

constexpr long long up_to(long long n, long long unit) { return (n + unit - 1) / unit * unit; }
constexpr long long ceil_div(long long n, long long d) { return (n + d - 1) / d; }

// How the products of many rows are dealt out: rows of a tile; rounds of whole units, then `rest` units laid end to end
// and cut into `ctas` equal runs of chunks.
struct Deal {
    int nt = 0, mtiles = 0, units = 0, rounds = 0, rest = 0, ctas = 0;
    double us = 0;
};

// The cheapest deal by times measured on GB300 (us).  A chunk: its products at the tensor rate, or its weights' way to f16
// where that takes longer (a 64-value step of 256 weight rows: 16-bit rows 0.55, backward 0.4, of Q6_K 0.9, f32 rows
// 1.1).  A unit's output 1.5 and 0.02 for each row of x.  What cutting costs: a counter's trip, 3, and a part written and
// `parts` read back by the last to arrive, 0.02 for each row and part (525 x 469 x 9472 in 25 parts a unit: 85 of 106 us).
// Smaller tiles are more units, which share fewer parts each but turn the same weights to f16 on more SMs.  (Q5_K counts as Q4_K and
// f16 rows as bf16, a little too cheap.)
Deal deal(long long M, long long pairs, int chunks, double pieces, int nt_most, int fmt, bool split, bool back, int sms) {
    Deal best;
    const double weights = split ? 1.1 : fmt == FMT_Q6_K ? 0.9 : back ? 0.4 : 0.55;
    const long long least = ceil_div(M, nt_most);
    for (long long k = least; k < least + 12 && k <= ceil_div(M, 16); ++k) {
        Deal d;
        d.nt = (int)up_to(ceil_div(M, k), 16);
        d.mtiles = (int)ceil_div(M, d.nt);
        if (d.mtiles != k) continue;  // (another tile's size again)
        const long long units = d.mtiles * pairs;
        d.units = (int)units;
        const double products = 8 * (split ? 3 : 1) * (d.nt < 64 ? 64 : d.nt) / 2 / 1900.0;
        const double chunk = pieces * (weights > products ? weights : products), output = 1.5 + 0.02 * d.nt;
        auto take = [&](long long rounds, long long rest, long long ctas, double us) {
            if (best.ctas && us >= best.us) return;
            d.rounds = (int)rounds;
            d.rest = (int)rest;
            d.ctas = (int)ctas;
            d.us = us;
            best = d;
        };
        const long long whole = ceil_div(units, sms);
        take(whole, 0, units < sms ? units : sms, whole * (chunks * chunk + output));
        if (units % sms == 0) continue;
        // what does not fill the SMs, with the round before it, is cut
        const long long full = units < sms ? 0 : units / sms - 1, rest = units - full * sms;
        for (int p = 1; p <= 24; ++p) {
            long long ctas = units > sms || rest * p > sms ? sms : rest * p;
            if (ctas > rest * chunks) ctas = rest * chunks;
            const double parts = 1.0 + (double)ctas / (double)rest;
            const double us = full * (chunks * chunk + output) + (double)ceil_div(rest * chunks, ctas) * chunk + output + 3.0 +
                              0.02 * d.nt * (1.0 + parts);
            if (ctas != rest) take(full, rest, ctas, us);
            if (ctas == sms || ctas == rest * chunks) break;
        }
    }
    return best;
}

// scratch_alloc, but under capture the graph's own memory without the library's pool, which cannot be made there: so a
// program's first call may be a captured one.
int scratch_of(size_t bytes, cudaStream_t s, void** p, const char* fn) {
    cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(s, &status) != cudaSuccess || status == cudaStreamCaptureStatusNone) {
        cudaGetLastError();
        return scratch_alloc(bytes, s, p, fn);
    }
    if (cudaMallocAsync(p, bytes, s) == cudaSuccess) return MMQ_OK;
    cudaGetLastError();
    *p = nullptr;
    report(fn, MMQ_ERR_NOMEM, "scratch allocation failed");
    return MMQ_ERR_NOMEM;
}

// The row kernel's side of a call.
Rows rows_of(const Call& c, int groups) {
    Rows r{};
    r.x = c.x;
    r.stride = c.x_stride;
    r.dtype = c.dtype;
    r.act = c.act;
    r.mats = c.mats;
    r.rows = (int)c.M;
    r.width = (int)(c.backward ? c.N : c.K);
    r.groups = groups;
    for (int g = 0; g < 2; ++g) {
        r.pre[g] = c.backward ? c.pre[g] : nullptr;
        r.dz[g] = c.dz[g];
    }
    return r;
}

bool weight_maps(const Call& c, CUtensorMap* map, long long row_bytes, int box_rows) {
    for (int g = 0; g < c.mats; ++g)
        if (!make_byte_map(&map[g], c.w[g], (uint64_t)row_bytes, (uint64_t)c.N, (uint32_t)chunk_bytes(c.fmt), box_rows, 2)) {
            report(c.fn, MMQ_ERR_CUDA, "the weights' tensor map was refused");
            return false;
        }
    return true;
}

// Few rows, forward: the weights as a stream.
int stream(const Call& c, cudaStream_t s) {
    const int terms = c.dtype == MMQ_F32 ? 2 : 1;
    Stream a{};
    a.row_bytes = c.fmt == FMT_Q8_0 ? c.K / QK * Q8_0_BYTES : c.K / QK_K * kq_bytes(c.fmt);
    a.mats = c.mats;
    a.M = (int)c.M;
    a.N = (int)c.N;
    a.K = (int)c.K;
    a.chunks = (int)ceil_div(c.K, CHUNK);
    a.xgroups = (int)ceil_div(c.M, 8);
    a.aligned = c.fmt != FMT_Q6_K && a.row_bytes % 16 == 0;  // (whose chunks of 210 bytes are not, wherever rows begin)
    a.slot = slot_bytes(c.fmt, a.aligned);
    a.dtype = c.dtype;
    a.act = c.act;
    for (int g = 0; g < 2; ++g) {
        a.w[g] = static_cast<const uint8_t*>(c.w[g]);
        a.bias[g] = c.bias[g];
        a.pre[g] = c.pre[g];
    }
    a.residual = c.residual;
    a.residual_stride = c.residual_stride;
    a.out = c.out;
    // Column runs of a CTA, shares of the reduction in it, CTAs that share one: the fewest chunks in a row, a wave's start
    // counted as two and the cluster's meeting as one.  (Clusters of four and eight leave some of a GPC's SMs out.)
    const long long runs = ceil_div(c.N, STREAM_SLAB), sms = device_shape().sms;
    long long best = 0, ctas = 0;
    for (int cluster = 1; cluster <= 8; cluster *= 2)
        for (int per = 1; per * c.mats <= STREAM_WARPS; ++per) {
            const int splits = STREAM_WARPS / (per * c.mats);
            const long long n = ceil_div(runs, per) * cluster, fit = cluster > 2 ? sms * 5 / 6 : sms;
            const long long time = ceil_div(n, fit) * (ceil_div(a.chunks, splits * cluster) + 2 + (cluster > 1));
            if (best && time >= best) continue;
            best = time;
            ctas = n;
            a.groups = per * c.mats;
            a.splits = splits;
            a.cluster = cluster;
        }
    // shared memory: all of x where two places of every ring are left beside it (else the SM's cache has the rest)
    const int place = STREAM_WARPS * STREAM_SLAB * a.slot;
    const long long term = ceil_div(c.K, STEP) * a.xgroups * 1024, sums = is_kquant(c.fmt) ? (long long)a.chunks * a.xgroups * 256 : 0;
    const long long x_bytes = ceil_div(c.K, STEP) * c.M * 128 * terms + sums;  // held: the rows that there are
    a.held = x_bytes <= SMEM_MOST - 2 * place;
    a.rs = (int)((a.held ? SMEM_MOST - x_bytes : 200 * 1024) / place);
    a.rs = a.rs > R_MOST ? R_MOST : a.rs;
    const int smem = place * a.rs + (a.held ? (int)x_bytes : 0);
    if (a.aligned && !weight_maps(c, a.map, a.row_bytes, STREAM_SLAB)) return MMQ_ERR_CUDA;

    a.rows = c.x;
    a.rows_stride = c.x_stride;
    if (a.held) return ffn_stream_launch(c.fmt, a, smem, (int)ctas, true, c.fn, s);
    Rows r = rows_of(c, a.xgroups);
    int st = ffn_stream_launch(c.fmt, a, smem, (int)ctas, false, c.fn, s);
    void* scratch = nullptr;
    if (!st) st = scratch_of((size_t)(256 + term * terms + sums), s, &scratch, c.fn);
    if (st != MMQ_OK) return st;
    uint8_t* at = static_cast<uint8_t*>(scratch);
    r.up = reinterpret_cast<float*>(at);
    a.up = r.up;
    r.tiles = at + 256;
    a.x = r.tiles;
    r.term = a.x_term = term;
    if (sums) a.sums = r.sums = r.tiles + term * terms;
    st = ffn_rows_launch(r, false, true, c.fn, s);
    if (st == MMQ_OK) st = ffn_stream_launch(c.fmt, a, smem, (int)ctas, true, c.fn, s);
    scratch_free(scratch, s);  // stream-ordered: after the kernels above
    return st;
}

}  // namespace

int ffn_launch(const Call& c, cudaStream_t s) {
    // Up to 16 rows, forward, as a stream.  Measured at 1 / 8 / 16 rows against these tiles (us): project 3584 x 18944 of Q6_K 22 / 25 /
    // 29 against 37 / 37 / 38, 512 x 3584 of Q8_0 in f32 4.8 / 6.6 / 7.7 against 19, gated 18944 x 3584 of Q6_K in f16 32 / 36 / 56
    // against 58, in f32 of Q4_K 26 / 36 / 55 against 57, of Q4_K in bf16 22 / 30 / 45 against 38: there alone the tiles would be
    // faster from 13 rows on, but round the weights.  17 rows take the tiles' time.  Backward all rows take tiles: the stream's order of
    // the reduction is along a weight row.
    if (!c.backward && c.M <= STREAM_ROWS) return stream(c, s);
    const bool split = c.dtype == MMQ_F32;
    const int terms = split ? 2 : 1;
    Tile a{};
    a.w[0] = static_cast<const uint8_t*>(c.w[0]);
    a.w[1] = static_cast<const uint8_t*>(c.w[1]);
    a.row_bytes = c.fmt == FMT_Q8_0 ? c.K / QK * Q8_0_BYTES : c.K / QK_K * kq_bytes(c.fmt);
    a.mats = c.mats;
    a.M = (int)c.M;
    a.N = (int)c.N;
    a.K = (int)c.K;
    a.width = c.backward ? a.K : a.N;
    a.groups = (int)ceil_div(c.M, 8);
    a.aligned = c.fmt != FMT_Q6_K && a.row_bytes % 16 == 0;  // (whose chunks of 210 bytes are not, wherever rows begin)
    a.slot = slot_bytes(c.fmt, a.aligned);
    // rows of a tile: the most, but for two steps of them in shared memory beside two places of the rings
    const int w_bytes = rings(c.backward) * 32 * a.slot;
    const int left = SMEM_MOST - (c.backward ? 2 * terms * Shape<true, true>::A_BYTES : 0);
    int nt_most = split ? Shape<true, false>::NT : Shape<false, false>::NT;
    while ((left - 2 * w_bytes) / (nt_most * 128 * terms) < 2) nt_most -= 16;
    const int pieces = (int)(c.backward ? c.mats * ceil_div(c.N, STEP) : ceil_div(c.K, STEP));  // of 64 values
    a.chunks = c.backward ? pieces : (int)ceil_div(c.K, CHUNK);
    const Deal d = deal(c.M, ceil_div(a.width, !c.backward && c.mats == 2 ? 128 : 256), a.chunks, c.backward ? 1 : CHUNK / STEP,
                        nt_most, c.fmt, split, c.backward, device_shape().sms);
    a.nt = d.nt;
    a.mtiles = d.mtiles;
    a.units = d.units;
    a.rounds = d.rounds;
    a.rest = d.rest;
    const int ctas = d.ctas;
    a.sub = !c.backward && !split && a.nt <= Shape<false, false, 2>::NT && c.K % (2 * STEP) == 0 ? 2 : 1;
    a.steps = pieces / a.sub;
    a.dtype = c.dtype;
    a.act = c.act;
    for (int g = 0; g < 2; ++g) {
        a.bias[g] = c.bias[g];
        a.pre[g] = c.backward ? nullptr : c.pre[g];
    }
    a.residual = c.residual;
    a.residual_stride = c.residual_stride;
    a.out = c.out;
    // shared memory: two chunks' places and two steps of rows at least, then four places, four steps, more places
    const int x_bytes = a.nt * 128 * terms * a.sub;
    auto steps_left = [&](int places) { return (left - places * w_bytes) / x_bytes; };
    a.rs = steps_left(4) >= 2 ? 4 : steps_left(3) >= 2 ? 3 : 2;
    a.xs = steps_left(a.rs) < 4 ? steps_left(a.rs) : 4;
    a.rs = (left - a.xs * x_bytes) / w_bytes;
    a.rs = a.rs > R_MOST ? R_MOST : a.rs;
    if (a.xs < 1 || a.rs < 2) {
        report(c.fn, MMQ_ERR_SMEM, "the rings do not fit in shared memory");
        return MMQ_ERR_SMEM;
    }
    const int smem = SMEM_MOST - left + a.xs * x_bytes + a.rs * w_bytes;

    if (a.aligned && !weight_maps(c, a.map, a.row_bytes, 32)) return MMQ_ERR_CUDA;
    const long long term = (long long)pieces * a.groups * 1024;
    const long long counters = up_to(4ll * a.rest, 256), ups = up_to(4 * c.M, 256);
    const long long parts = a.rest ? 2ll * ctas * 2 * a.nt * 128 * 4 : 0;
    Rows r = rows_of(c, a.groups);
    auto products = c.backward ? ffn_backward_launch : ffn_forward_launch;
    int st = products(c.fmt, a, smem, ctas, false, c.fn, s);
    if (!st) st = ffn_rows_launch(r, c.backward, false, c.fn, s);
    void* scratch = nullptr;
    if (!st) st = scratch_of((size_t)(counters + ups + term * terms + parts), s, &scratch, c.fn);
    if (st != MMQ_OK) return st;
    uint8_t* at = static_cast<uint8_t*>(scratch);
    r.counters = a.counters = reinterpret_cast<unsigned*>(at);
    r.n_counters = a.rest;
    r.up = reinterpret_cast<float*>(at + counters);
    a.up = r.up;
    r.tiles = at + counters + ups;
    r.term = a.x_term = term;
    a.x = r.tiles;
    a.parts = reinterpret_cast<float*>(r.tiles + term * terms);
    st = ffn_rows_launch(r, c.backward, true, c.fn, s);
    if (st == MMQ_OK) st = products(c.fmt, a, smem, ctas, true, c.fn, s);
    scratch_free(scratch, s);  // stream-ordered: after the kernels above
    return st;
}

}  // namespace mmq
