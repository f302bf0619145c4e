// Writing and reading the 8-bit key/value cache: k_kv_append (rotation, the joint scale of a
// block's older and new tokens, codes) and k_kv_read (codes back to values).
//
// Both are bandwidth-bound passes whose unit is one block of 32 tokens of one head, so that a
// block's scale is one CTA's business: no atomics, no second pass, the same bits whatever the
// order.  The grid is laid out without knowing the lengths: the blocks that sequence b's new
// tokens touch are numbered from starts[b] / 32 + 2b (at most n / 32 + 2 blocks, so the ranges
// of consecutive sequences never overlap), or from b where every sequence has at most one new
// token; a CTA looks for the sequence whose range holds its own number, and leaves when there is
// none or its block does not exist.
//
// Measured (GB300), k_kv_append alone: a prompt of 8192 tokens, 4 + 28 heads of 128 of bf16, 147 MB
// moved: 28 us, 5.2 TB/s, 0.77 of the copy rate; five ragged f32 sequences, 33 to 997 tokens, 16 heads of
// 64, 15.3 us (1404 CTAs with work, four an SM: 2.3 waves, each behind a look for its sequence); single tokens of 64 sequences 4.4 us: a read of the older codes behind
// a read of the table.  k_kv_read of the same tokens: 6.9, 5.7 and 4.7 us.
#include "kv.cuh"

namespace mmq {
namespace {

using namespace kv;

constexpr int THREADS = 256;

__device__ unsigned g_kv_cache_error;

// The CTA's block of its sequence: rows [i0, i1) of block blk are new (row r of the block is
// row `row` + r of the row arrays); false: no such block.
struct Where {
    int b, blk, i0, i1, row, pos0;
};
__device__ __forceinline__ bool find_block(const Cache& c, const Batch& bt, Where& w) {
    const int x = blockIdx.x;
    int start = 0, n = 0, len = 0, nth = 0;
    if (bt.max_new <= 1) {
        w.b = x;
        if (!seq_range(c, bt, x, start, n, len, &g_kv_cache_error)) return false;
    } else {
        // one round of loads: a thread whose sequence's range holds x says so (in a disordered list more
        // than one may, and any of them is as good: what it names is read again, from the L1)
        __shared__ int found;
        if (threadIdx.x == 0) found = -1;
        __syncthreads();
        for (int i = threadIdx.x; i < bt.seqs; i += THREADS) {
            int si, ni, li;
            if (seq_range(c, bt, i, si, ni, li, &g_kv_cache_error) && x >= si / BT + 2 * i && x < (si + ni) / BT + 2 * (i + 1))
                found = i;
        }
        __syncthreads();
        w.b = found;
        if (w.b < 0 || !seq_range(c, bt, w.b, start, n, len, &g_kv_cache_error)) return false;
        nth = x - (start / BT + 2 * w.b);
    }
    if (n == 0) return false;
    const int first = len - n;  // negative: the first rows are padding
    w.blk = max(first, 0) / BT + nth;
    w.pos0 = w.blk * BT;
    if (w.pos0 >= len) return false;
    w.i0 = max(0, first - w.pos0);
    w.i1 = min(BT, len - w.pos0);
    w.row = start + w.pos0 - first;
    return true;
}

// One unit of a row: 2V values as two runs of V, `a` and `b` elements into the row, that turn
// together (halves: a pair's members lie in different runs; interleaved: side by side).  V is what
// one 16-byte load brings, or 4 of a 16-bit type where the rotation ends inside a run of 8.
struct Unit {
    int a, b, pair;  // pair: first column of the tables, or -1
};
template <int V>
__device__ __forceinline__ Unit unit(int o, const Rope& r) {
    if (2 * V * o < r.rotary)
        return r.interleaved ? Unit{2 * V * o, 2 * V * o + V, V * o} : Unit{V * o, V * o + r.rotary / 2, V * o};
    return Unit{2 * V * o, 2 * V * o + V, -1};
}
// each product and sum rounded on its own
__device__ __forceinline__ void turn1(float& x, float& y, float c, float s) {
    const float a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
    y = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
    x = a;
}
// a unit's columns of the tables at a position; false: not rotated
template <int V>
__device__ __forceinline__ bool table(const Unit& o, const Rope& r, int pos, float (&c)[V], float (&s)[V]) {
    if (o.pair < 0) return false;
    const long long at = (long long)pos * (r.rotary / 2) + o.pair;
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        const float4 c4 = *reinterpret_cast<const float4*>(r.cos + at + i);
        const float4 s4 = *reinterpret_cast<const float4*>(r.sin + at + i);
        c[i] = c4.x, c[i + 1] = c4.y, c[i + 2] = c4.z, c[i + 3] = c4.w;
        s[i] = s4.x, s[i + 1] = s4.y, s[i + 2] = s4.z, s[i + 3] = s4.w;
    }
    return true;
}
template <int V>
__device__ __forceinline__ void turn(float (&a)[V], float (&b)[V], const Rope& r, const float (&c)[V], const float (&s)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (r.interleaved) {
            if (i & 1) continue;
            turn1(a[i], a[i + 1], c[i / 2], s[i / 2]);
            turn1(b[i], b[i + 1], c[V / 2 + i / 2], s[V / 2 + i / 2]);
        } else {
            turn1(a[i], b[i], c[i], s[i]);
        }
    }
}
template <int V>
__device__ __forceinline__ float amax(const float (&x)[V]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, fabsf(x[i]));
    return m;
}

__device__ __forceinline__ uint32_t code(float q) { return (uint32_t)(max(-127, min(127, __float2int_rn(q))) & 0xff); }
template <int V>
__device__ __forceinline__ void put_codes(uint8_t* p, const float (&x)[V], float d) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        uint32_t w = 0u;
        if (d != 0.f)
            w = code(__fdiv_rn(x[i], d)) | code(__fdiv_rn(x[i + 1], d)) << 8 | code(__fdiv_rn(x[i + 2], d)) << 16 |
                code(__fdiv_rn(x[i + 3], d)) << 24;
        *reinterpret_cast<uint32_t*>(p + i) = w;
    }
}
// older codes under the new scale: rint(c * r), r = d / d'
template <int V>
__device__ __forceinline__ void rescale_codes(uint8_t* p, float r) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(p + i);
        uint32_t o = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) o |= code(__fmul_rn((float)(int8_t)(w >> (8 * k)), r)) << (8 * k);
        *reinterpret_cast<uint32_t*>(p + i) = o;
    }
}

constexpr int QH = 8;  // query heads of a CTA that rotates queries

// grid (blocks, kv heads [+ eighths of the query heads]).  A CTA of the first kind holds its
// block's keys and values in registers (D / 4 values a thread), so the rows are read once; the
// second kind turns the block's rows of up to eight query heads, a few rows' loads in flight at a
// time.
template <typename T, int D, int V>
__global__ void __launch_bounds__(THREADS, D == 256 ? 2 : 4)
k_kv_append(Cache c, Batch bt, Rows kr, Rows vr, Rows qr, int q_heads, Rope rope, T* __restrict__ q_out) {
    constexpr int O = D / (2 * V), RP = THREADS / O, PASSES = BT > RP ? BT / RP : 1;  // units a row, rows a pass
    __shared__ float part[2][THREADS / 32];
    ptx::grid_dep_wait();
    ptx::grid_dep_launch_dependents();
    Where w;
    if (!find_block(c, bt, w)) return;
    if (rope.rotary > 0 && w.pos0 + w.i1 > rope.rows) {  // positions past the tables are skipped
        if (threadIdx.x == 0) atomicOr(&g_kv_cache_error, ERR_RANGE);
        w.i1 = (int)(max(rope.rows, (long long)w.pos0) - w.pos0);
        if (w.i1 <= w.i0) return;
    }
    const int tid = threadIdx.x;
    const Unit o = unit<V>(tid % O, rope);
    if (blockIdx.y >= c.heads) {
        constexpr int B = 16 / V;
        const int h0 = (blockIdx.y - c.heads) * QH, group = min(QH, q_heads - h0), tokens = w.i1 - w.i0;
        const T* q = static_cast<const T*>(qr.data) + (long long)w.row * qr.token_stride + h0 * qr.head_stride;
        T* to = q_out + ((long long)w.row * q_heads + h0) * D;
        float ct[V], st[V], a[B][V], b[B][V];
        if (2 * tokens > RP) {  // a token per thread: its columns of the tables serve all heads
            for (int i = w.i0 + tid / O; i < w.i1; i += RP) {
                const bool on = table<V>(o, rope, w.pos0 + i, ct, st);
                for (int h = 0; h < group; h += B) {
#pragma unroll
                    for (int u = 0; u < B; ++u) {
                        const T* src = q + i * qr.token_stride + min(h + u, group - 1) * qr.head_stride;
                        load_run<T, V>(src + o.a, a[u]);
                        load_run<T, V>(src + o.b, b[u]);
                    }
#pragma unroll
                    for (int u = 0; u < B; ++u) {
                        if (h + u >= group) break;
                        if (on) turn<V>(a[u], b[u], rope, ct, st);
                        T* dst = to + ((long long)i * q_heads + h + u) * D;
                        store_run<T, V>(dst + o.a, a[u]);
                        store_run<T, V>(dst + o.b, b[u]);
                    }
                }
            }
        } else {  // few tokens: a row per thread
            for (int r0 = tid / O; r0 < tokens * group; r0 += B * RP) {
#pragma unroll
                for (int u = 0; u < B; ++u) {
                    const int r = min(r0 + u * RP, tokens * group - 1), i = w.i0 + r / group;
                    const T* src = q + i * qr.token_stride + (r % group) * qr.head_stride;
                    load_run<T, V>(src + o.a, a[u]);
                    load_run<T, V>(src + o.b, b[u]);
                }
#pragma unroll
                for (int u = 0; u < B; ++u) {
                    const int r = r0 + u * RP, i = w.i0 + r / group;
                    if (r >= tokens * group) break;
                    if (table<V>(o, rope, w.pos0 + i, ct, st)) turn<V>(a[u], b[u], rope, ct, st);
                    T* dst = to + ((long long)i * q_heads + r % group) * D;
                    store_run<T, V>(dst + o.a, a[u]);
                    store_run<T, V>(dst + o.b, b[u]);
                }
            }
        }
        return;
    }
    const int h = blockIdx.y;
    float ka[PASSES][V], kb[PASSES][V], va[PASSES][V], vb[PASSES][V];
#pragma unroll
    for (int u = 0; u < PASSES; ++u) {
        const int i = u * RP + tid / O;
#pragma unroll
        for (int e = 0; e < V; ++e) ka[u][e] = kb[u][e] = va[u][e] = vb[u][e] = 0.f;
        if (i >= w.i0 && i < w.i1) {
            const T* ks = static_cast<const T*>(kr.data) + (long long)(w.row + i) * kr.token_stride + h * kr.head_stride;
            const T* vs = static_cast<const T*>(vr.data) + (long long)(w.row + i) * vr.token_stride + h * vr.head_stride;
            load_run<T, V>(ks + o.a, ka[u]);
            load_run<T, V>(ks + o.b, kb[u]);
            load_run<T, V>(vs + o.a, va[u]);
            load_run<T, V>(vs + o.b, vb[u]);
        }
    }
    uint8_t* rec = record(c, bt, w.b, w.blk, h, &g_kv_cache_error);  // while the rows are on their way
    if (!rec) return;
    const float2 d_old = *reinterpret_cast<const float2*>(rec + 2 * BT * D);
    float mk = 0.f, mv = 0.f;
#pragma unroll
    for (int u = 0; u < PASSES; ++u) {
        const int i = u * RP + tid / O;
        float ct[V], st[V];
        if (i >= w.i0 && i < w.i1 && table<V>(o, rope, w.pos0 + i, ct, st)) turn<V>(ka[u], kb[u], rope, ct, st);
        mk = fmaxf(mk, fmaxf(amax<V>(ka[u]), amax<V>(kb[u])));
        mv = fmaxf(mv, fmaxf(amax<V>(va[u]), amax<V>(vb[u])));
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) {
        mk = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, off));
        mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, off));
    }
    if ((tid & 31) == 0) {
        part[0][tid >> 5] = mk;
        part[1][tid >> 5] = mv;
    }
    __syncthreads();  // also: every thread has read the record's old scales
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
        mk = fmaxf(mk, part[0][i]);
        mv = fmaxf(mv, part[1][i]);
    }
    // the scale of a block that keeps older tokens never shrinks
    const bool kept = w.i0 > 0;
    float dk = __fdiv_rn(mk, 127.0f), dv = __fdiv_rn(mv, 127.0f);
    if (kept) {
        dk = fmaxf(dk, d_old.x);
        dv = fmaxf(dv, d_old.y);
    }
    if (dk < MIN_SCALE) dk = 0.f;
    if (dv < MIN_SCALE) dv = 0.f;
    const bool grew_k = kept && dk != d_old.x, grew_v = kept && dv != d_old.y;
    const float rk = grew_k && dk != 0.f ? __fdiv_rn(d_old.x, dk) : 0.f;
    const float rv = grew_v && dv != 0.f ? __fdiv_rn(d_old.y, dv) : 0.f;
#pragma unroll
    for (int u = 0; u < PASSES; ++u) {
        const int i = u * RP + tid / O;
        uint8_t* kc = rec + i * D;
        uint8_t* vc = kc + BT * D;
        if (i < w.i0) {
            if (grew_k) {
                rescale_codes<V>(kc + o.a, rk);
                rescale_codes<V>(kc + o.b, rk);
            }
            if (grew_v) {
                rescale_codes<V>(vc + o.a, rv);
                rescale_codes<V>(vc + o.b, rv);
            }
        } else if (i < w.i1) {
            put_codes<V>(kc + o.a, ka[u], dk);
            put_codes<V>(kc + o.b, kb[u], dk);
            put_codes<V>(vc + o.a, va[u], dv);
            put_codes<V>(vc + o.b, vb[u], dv);
        }
    }
    if (tid == 0) *reinterpret_cast<float2*>(rec + 2 * BT * D) = make_float2(dk, dv);
}

// grid (blocks, kv heads); a thread turns 16 bytes' worth of output at a time
template <typename T, int D>
__global__ void __launch_bounds__(THREADS)
k_kv_read(Cache c, Batch bt, T* __restrict__ k_out, T* __restrict__ v_out) {
    constexpr int CH = 16 / (int)sizeof(T), CR = D / CH;  // codes a chunk, chunks a row
    ptx::grid_dep_wait();
    ptx::grid_dep_launch_dependents();
    Where w;
    if (!find_block(c, bt, w)) return;
    const int h = blockIdx.y;
    const uint8_t* rec = record(c, bt, w.b, w.blk, h, &g_kv_cache_error);
    if (!rec) return;
    const float2 d = *reinterpret_cast<const float2*>(rec + 2 * BT * D);
    const int chunks = (w.i1 - w.i0) * CR;
    for (int x = threadIdx.x; x < 2 * chunks; x += THREADS) {
        const bool val = x >= chunks;
        const int y = val ? x - chunks : x, i = w.i0 + y / CR, e = y % CR * CH;
        const uint8_t* src = rec + (val ? BT * D : 0) + i * D + e;
        const float sc = val ? d.y : d.x;
        T* dst = (val ? v_out : k_out) + ((long long)(w.row + i) * c.heads + h) * D + e;
#pragma unroll
        for (int u = 0; u < CH; u += 4) {
            const uint32_t q = *reinterpret_cast<const uint32_t*>(src + u);
            Elem<T>::store4(dst + u, make_float4(__fmul_rn((float)(int8_t)q, sc), __fmul_rn((float)(int8_t)(q >> 8), sc),
                                                 __fmul_rn((float)(int8_t)(q >> 16), sc),
                                                 __fmul_rn((float)(int8_t)(q >> 24), sc)));
        }
    }
}

// CTAs for the blocks that the new tokens may touch (see the numbering above)
unsigned block_grid(const Batch& b) {
    return b.max_new <= 1 ? (unsigned)b.seqs : (unsigned)(b.tokens / BT + 2 * b.seqs);
}

template <typename T>
int append_t(const Cache& c, const Batch& b, const Rows& k, const Rows& v, const Rows& q, int q_heads, const Rope& rope,
             void* q_out, cudaStream_t s) {
    const dim3 grid(block_grid(b), c.heads + (q.data ? (q_heads + QH - 1) / QH : 0));
    ProfScope ps("k_kv_append", s);
    auto go = [&](auto kernel) {
        return pdl_status(launch_pdl(kernel, grid, dim3(THREADS), 0, s, c, b, k, v, q, q_heads, rope, static_cast<T*>(q_out)),
                          "mmq_kv_append");
    };
    constexpr int W = sizeof(T) == 2 ? 8 : 4;
    if (rope.rotary % (2 * W) == 0)
        return c.dim == 64    ? go(k_kv_append<T, 64, W>)
               : c.dim == 128 ? go(k_kv_append<T, 128, W>)
                              : go(k_kv_append<T, 256, W>);
    return c.dim == 64    ? go(k_kv_append<T, 64, 4>)
           : c.dim == 128 ? go(k_kv_append<T, 128, 4>)
                          : go(k_kv_append<T, 256, 4>);
}

template <typename T>
int read_t(const Cache& c, const Batch& b, void* k_out, void* v_out, cudaStream_t s) {
    const dim3 grid(block_grid(b), c.heads);
    ProfScope ps("k_kv_read", s);
    auto go = [&](auto kernel) {
        return pdl_status(launch_pdl(kernel, grid, dim3(THREADS), 0, s, c, b, static_cast<T*>(k_out), static_cast<T*>(v_out)),
                          "mmq_kv_read");
    };
    return c.dim == 64 ? go(k_kv_read<T, 64>) : c.dim == 128 ? go(k_kv_read<T, 128>) : go(k_kv_read<T, 256>);
}

}  // namespace

int kv_append_launch(const Cache& c, const Batch& b, int dtype, const Rows& k, const Rows& v, const Rows& q, int q_heads,
                     const Rope& rope, void* q_out, cudaStream_t s) {
    return dtype == MMQ_F32    ? append_t<float>(c, b, k, v, q, q_heads, rope, q_out, s)
           : dtype == MMQ_BF16 ? append_t<__nv_bfloat16>(c, b, k, v, q, q_heads, rope, q_out, s)
                               : append_t<__half>(c, b, k, v, q, q_heads, rope, q_out, s);
}

int kv_read_launch(const Cache& c, const Batch& b, int dtype, void* k_out, void* v_out, cudaStream_t s) {
    return dtype == MMQ_F32    ? read_t<float>(c, b, k_out, v_out, s)
           : dtype == MMQ_BF16 ? read_t<__nv_bfloat16>(c, b, k_out, v_out, s)
                               : read_t<__half>(c, b, k_out, v_out, s);
}

unsigned kv_cache_take_error() {
    unsigned v = 0;
    if (cudaMemcpyFromSymbol(&v, g_kv_cache_error, sizeof(v)) != cudaSuccess) return 0;
    if (v) {
        const unsigned zero = 0;
        cudaMemcpyToSymbol(g_kv_cache_error, &zero, sizeof(zero));
    }
    return v;
}

}  // namespace mmq
