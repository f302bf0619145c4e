// How a feed-forward call is laid out on the GPU (row tiles, rounds, cuts, rings, scratch memory), and its two
// launches: the rows as operands, then the products.
#include "ffn_weights.cuh"

namespace mmq {
namespace {

using namespace ffn;

constexpr long long up_to(long long n, long long unit) { return (n + unit - 1) / unit * unit; }
constexpr long long ceil_div(long long n, long long d) { return (n + d - 1) / d; }

// Times in us, for the choice between whole and cut units.  A chunk: its products at the tensor rate, or its weights'
// way to f16 where that takes longer (measured a 64-value step of 256 weight rows: 16-bit rows 0.55, backward 0.4, of Q6_K 0.9, f32
// rows 1.1).  What cutting costs: parts of nt x 256 sums written and read back, and a counter's trip (measured at 192 rows 14).
struct Cost {
    double chunk, join;
};
Cost cost(const Tile& a, int fmt, bool split, bool back) {
    const double pieces = back ? 1 : CHUNK / STEP;
    const double weights = split ? 1.1 : fmt == FMT_Q6_K ? 0.9 : back ? 0.4 : 0.55;
    const double products = 8 * (split ? 3 : 1) * (a.nt < 64 ? 64 : a.nt) / 2 / 1900.0;
    return {pieces * (weights > products ? weights : products), 3.0 + a.nt * 0.06};
}

// Rounds of whole units; or, where the last round leaves too much undone, it and the one before it cut evenly.
int deal(Tile& a, const Cost& t, int sms) {
    const long long whole = ceil_div(a.units, sms) * a.chunks;
    const long long full = a.units % sms == 0 ? a.units / sms : a.units < sms ? 0 : a.units / sms - 1;
    const long long rest = a.units - full * sms;
    if (rest > 0) {
        const double cut = full * a.chunks + (double)ceil_div(rest * a.chunks, sms);
        if (cut * t.chunk + t.join < 0.93 * whole * t.chunk) {
            a.rounds = (int)full;
            a.rest = (int)rest;
            return (int)(rest * a.chunks < sms ? rest * a.chunks : sms);
        }
    }
    a.rounds = (int)ceil_div(a.units, sms);
    a.rest = 0;
    return (int)(a.units < sms ? a.units : sms);
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
    // Column runs of a CTA and shares of the reduction: the fewest chunks in a row, a wave's start counted as two.
    const long long runs = ceil_div(c.N, STREAM_SLAB), sms = device_shape().sms;
    long long best = 0, ctas = 0;
    for (int per = 1; per * c.mats <= STREAM_WARPS; ++per) {
        const int splits = STREAM_WARPS / (per * c.mats);
        const long long n = ceil_div(runs, per), time = ceil_div(n, sms) * (ceil_div(a.chunks, splits) + 2);
        if (best && time >= best) continue;
        best = time;
        ctas = n;
        a.groups = per * c.mats;
        a.splits = splits;
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
    a.nt = (int)up_to(ceil_div(c.M, ceil_div(c.M, nt_most)), 16);
    a.mtiles = (int)ceil_div(c.M, a.nt);
    a.units = (int)(a.mtiles * ceil_div(a.width, !c.backward && c.mats == 2 ? 128 : 256));
    a.sub = !c.backward && !split && a.nt <= Shape<false, false, 2>::NT && c.K % (2 * STEP) == 0 ? 2 : 1;
    const int pieces = (int)(c.backward ? c.mats * ceil_div(c.N, STEP) : ceil_div(c.K, STEP));  // of 64 values
    a.steps = pieces / a.sub;
    a.chunks = c.backward ? a.steps : (int)ceil_div(c.K, CHUNK);
    a.dtype = c.dtype;
    a.act = c.act;
    for (int g = 0; g < 2; ++g) {
        a.bias[g] = c.bias[g];
        a.pre[g] = c.backward ? nullptr : c.pre[g];
    }
    a.residual = c.residual;
    a.residual_stride = c.residual_stride;
    a.out = c.out;
    const int ctas = deal(a, cost(a, c.fmt, split, c.backward), device_shape().sms);
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
