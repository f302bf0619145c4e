// C entry points of the 8-bit key/value cache: argument checks, then the launchers
// (kv_cache.cu; kv_stream.cu or kv_tile.cu).  The error protocol is that of the whole library: a refused
// call launches nothing, writes nothing and prints one line.
#include <math.h>

#include "kv_attend.cuh"

namespace mmq {
namespace {

using namespace kv;

constexpr int64_t LIMIT = (int64_t)1 << 40;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool dim_ok(int64_t dim) { return dim == 64 || dim == 128 || dim == 256; }

int refuse(const char* fn, int status, const char* why) {
    report(fn, status, why);
    return status;
}

int check_cache(const char* fn, const mmq_kv_cache* c, Cache& o) {
    if (!c || !c->data) return refuse(fn, MMQ_ERR_NULL, "the cache and its data must be non-NULL");
    if (!dim_ok(c->dim)) return refuse(fn, MMQ_ERR_SHAPE, "dim must be 64, 128 or 256");
    if (c->page < BT || c->page % BT != 0) return refuse(fn, MMQ_ERR_SHAPE, "page must be a positive multiple of 32");
    if (c->heads < 1 || c->heads > 32767) return refuse(fn, MMQ_ERR_SHAPE, "heads must be in 1 .. 32767");
    if (c->pages < 1 || c->pages > 0x7fffffff || c->pages > LIMIT / c->heads / (c->page / BT))
        return refuse(fn, MMQ_ERR_SHAPE, "pages must be in 1 .. 2^31 - 1 and the records below 2^40");
    if (!aligned(c->data, 16)) return refuse(fn, MMQ_ERR_ALIGN, "the cache must be 16-byte aligned");
    o = Cache{static_cast<uint8_t*>(c->data), (long long)c->pages, c->page, c->heads, c->dim, c->page / BT};
    return MMQ_OK;
}

int check_batch(const char* fn, const mmq_kv_cache* c, const mmq_kv_batch* b, Batch& o) {
    if (!b) return refuse(fn, MMQ_ERR_NULL, "the batch must be non-NULL");
    if (b->seqs < 0 || b->tokens < 0 || b->max_new < 0 || b->table_pages < 0 || b->table_stride < b->table_pages)
        return refuse(fn, MMQ_ERR_SHAPE, "seqs, tokens, max_new and table_pages must be >= 0, table_stride >= table_pages");
    if (b->seqs > 0 && (!b->starts || !b->lens || (b->table_pages > 0 && !b->table)))
        return refuse(fn, MMQ_ERR_NULL, "starts, lens and table must be non-NULL");
    // the block numbering of a batch and a sequence's tokens stay below 2^31
    if (b->seqs > 1 << 24 || b->tokens > 1 << 30 || (int64_t)b->table_pages * c->page > 1 << 30)
        return refuse(fn, MMQ_ERR_SHAPE, "seqs above 2^24, or tokens or table_pages * page above 2^30");
    if (!aligned(b->starts, 4) || !aligned(b->lens, 4) || !aligned(b->table, 4))
        return refuse(fn, MMQ_ERR_ALIGN, "starts, lens and table must be 4-byte aligned");
    o = Batch{b->starts, b->lens, b->table, (long long)b->table_stride, b->seqs, b->tokens, b->max_new, b->table_pages};
    return MMQ_OK;
}

int check_dtype(const char* fn, int dtype) {
    return dtype == MMQ_F32 || dtype == MMQ_BF16 || dtype == MMQ_F16
               ? MMQ_OK
               : refuse(fn, MMQ_ERR_ARG, "dtype must be MMQ_F32, MMQ_BF16 or MMQ_F16");
}

int check_rows(const char* fn, int dtype, int tokens, const mmq_kv_rows* r, Rows& o) {
    if (!r || (!r->data && tokens)) return refuse(fn, MMQ_ERR_NULL, "row arrays must be non-NULL");
    const int64_t per16 = dtype == MMQ_F32 ? 4 : 8;
    if (!aligned(r->data, 16) || r->token_stride % per16 != 0 || r->head_stride % per16 != 0)
        return refuse(fn, MMQ_ERR_ALIGN, "every row must be 16-byte aligned (base and strides)");
    o = Rows{r->data, (long long)r->token_stride, (long long)r->head_stride};
    return MMQ_OK;
}

int check_q_heads(const char* fn, const mmq_kv_cache* c, int64_t q_heads) {
    return q_heads >= c->heads && q_heads <= 32767 && q_heads % c->heads == 0
               ? MMQ_OK
               : refuse(fn, MMQ_ERR_SHAPE, "q_heads must be a multiple of the cache's heads, at most 32767");
}

}  // namespace
}  // namespace mmq

using namespace mmq;
using namespace mmq::kv;

extern "C" {

size_t mmq_kv_block_bytes(int64_t dim) { return dim_ok(dim) ? (size_t)rec_bytes((int)dim) : 0; }

// the arrival counters, then two partial results for every SM
size_t mmq_kv_workspace_bytes(int64_t dim) {
    return dim_ok(dim) ? WS_COUNTERS + (size_t)device_shape().sms * 2 * WS_ROWS * (dim + WS_ROW_STATS) * 4 : 0;
}

int mmq_kv_append(const mmq_kv_cache* cache, const mmq_kv_batch* batch, int dtype, const mmq_kv_rows* k,
                  const mmq_kv_rows* v, const mmq_kv_rows* q, int64_t q_heads, const mmq_kv_rope* rope, void* q_out,
                  void* stream) {
    const char* fn = "mmq_kv_append";
    Cache c;
    Batch b;
    Rows kr, vr, qr{nullptr, 0, 0};
    Rope rp{nullptr, nullptr, 0, 0, 0};
    int st = check_cache(fn, cache, c);
    if (!st) st = check_batch(fn, cache, batch, b);
    if (!st) st = check_dtype(fn, dtype);
    if (!st) st = check_rows(fn, dtype, b.tokens, k, kr);
    if (!st) st = check_rows(fn, dtype, b.tokens, v, vr);
    if (!st && q) {
        st = check_q_heads(fn, cache, q_heads);
        if (!st) st = check_rows(fn, dtype, b.tokens, q, qr);
        if (!st && !q_out && b.tokens) st = refuse(fn, MMQ_ERR_NULL, "q_out must be non-NULL where q is");
        if (!st && !aligned(q_out, 16)) st = refuse(fn, MMQ_ERR_ALIGN, "q_out must be 16-byte aligned");
    }
    if (!st && rope) {
        if (rope->rotary < 0 || rope->rotary > c.dim || rope->rotary % 8 != 0 || rope->rows < 0)
            st = refuse(fn, MMQ_ERR_SHAPE, "rotary must be a multiple of 8, at most dim");
        else if (rope->rotary && (!rope->cos || !rope->sin))
            st = refuse(fn, MMQ_ERR_NULL, "the rotation tables must be non-NULL");
        else if (!aligned(rope->cos, 16) || !aligned(rope->sin, 16))
            st = refuse(fn, MMQ_ERR_ALIGN, "the rotation tables must be 16-byte aligned");
        else
            rp = Rope{rope->cos, rope->sin, (long long)rope->rows, rope->rotary, rope->interleaved != 0};
    }
    if (st) return st;
    if (b.seqs == 0 || b.tokens == 0 || b.max_new == 0) return MMQ_OK;
    return kv_append_launch(c, b, dtype, kr, vr, qr, (int)q_heads, rp, q_out, static_cast<cudaStream_t>(stream));
}

int mmq_kv_read(const mmq_kv_cache* cache, const mmq_kv_batch* batch, int dtype, void* k_out, void* v_out,
                void* stream) {
    const char* fn = "mmq_kv_read";
    Cache c;
    Batch b;
    int st = check_cache(fn, cache, c);
    if (!st) st = check_batch(fn, cache, batch, b);
    if (!st) st = check_dtype(fn, dtype);
    if (!st && b.tokens && (!k_out || !v_out)) st = refuse(fn, MMQ_ERR_NULL, "k_out and v_out must be non-NULL");
    if (!st && (!aligned(k_out, 16) || !aligned(v_out, 16)))
        st = refuse(fn, MMQ_ERR_ALIGN, "k_out and v_out must be 16-byte aligned");
    if (st) return st;
    if (b.seqs == 0 || b.tokens == 0 || b.max_new == 0) return MMQ_OK;
    return kv_read_launch(c, b, dtype, k_out, v_out, static_cast<cudaStream_t>(stream));
}

int mmq_kv_attend(const mmq_kv_cache* cache, const mmq_kv_batch* batch, int dtype, const mmq_kv_rows* q,
                  int64_t q_heads, float scale, int64_t window, void* out, float* lse, void* workspace,
                  size_t workspace_bytes, void* stream) {
    const char* fn = "mmq_kv_attend";
    Cache c;
    Batch b;
    Rows qr;
    int st = check_cache(fn, cache, c);
    if (!st) st = check_batch(fn, cache, batch, b);
    if (!st) st = check_dtype(fn, dtype);
    if (!st) st = check_q_heads(fn, cache, q_heads);
    if (!st) st = check_rows(fn, dtype, b.tokens, q, qr);
    if (!st && ((!out && b.tokens) || !workspace)) st = refuse(fn, MMQ_ERR_NULL, "out and workspace must be non-NULL");
    if (!st && (!aligned(out, 16) || !aligned(lse, 4) || !aligned(workspace, 256)))
        st = refuse(fn, MMQ_ERR_ALIGN, "out must be 16-byte, lse 4-byte and workspace 256-byte aligned");
    if (!st && !(scale > 0.f && isfinite(scale))) st = refuse(fn, MMQ_ERR_ARG, "scale must be finite and > 0");
    // (the four factors together can pass 2^64)
    if (!st && b.table_pages > 0 && (int64_t)b.seqs * c.heads > 0x7fffffff / ((int64_t)b.table_pages * c.blocks))
        st = refuse(fn, MMQ_ERR_SHAPE, "seqs * heads * table_pages * page / 32 must be below 2^31");
    if (!st && window < 0) st = refuse(fn, MMQ_ERR_ARG, "window must be >= 0");
    if (!st && workspace_bytes < mmq_kv_workspace_bytes(c.dim))
        st = refuse(fn, MMQ_ERR_SHAPE, "the workspace is smaller than mmq_kv_workspace_bytes(dim)");
    if (st) return st;
    if (b.seqs == 0 || b.tokens == 0 || b.max_new == 0) return MMQ_OK;
    // a window past every length is none
    const int w = window >= (int64_t)b.table_pages * c.page ? 0 : (int)window;
    const int group = (int)(q_heads / c.heads);
    const Attend a{c, b, qr, (int)q_heads, group, dtype, w, scale * 1.44269504088896341f, out, lse,
                   static_cast<uint8_t*>(workspace)};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t rows = (int64_t)b.max_new * group;
    return rows <= kv_stream_rows(c.dim, dtype) ? kv_stream_launch(a, (int)rows, s) : kv_tile_launch(a, s);
}

}  // extern "C"
