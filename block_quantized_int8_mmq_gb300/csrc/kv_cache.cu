// Writing and reading the 8-bit key/value cache: k_kv_append (rotation, the joint scale of a
// block's older and new tokens, codes) and k_kv_read (codes back to values).
//
// Both are bandwidth-bound passes whose unit is one block of 32 tokens of one head, so that a
// block's scale is one CTA's business: no atomics, no second pass, the same bits whatever the
// order.  The grid is laid out without knowing the lengths: the blocks that sequence b's new
// tokens touch are numbered from starts[b] / 32 + 2b (at most n / 32 + 2 blocks, so the ranges
// of consecutive sequences never overlap), or from b where every sequence has at most one new
// token; a CTA finds its sequence by counting the sequences whose range begins at or before
// its own number, and leaves when its block does not exist.
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
    if (bt.max_new <= 1) {
        w.b = x;
    } else {
        int cnt = 0;
        for (int i0 = 0; i0 < bt.seqs; i0 += THREADS) {
            const int i = i0 + threadIdx.x;
            cnt += __syncthreads_count(i < bt.seqs && bt.starts[min(i, bt.seqs - 1)] / BT + 2 * i <= x);
        }
        w.b = cnt - 1;
        // every sequence is checked once, also those that no CTA finds in a disordered list
        if (x == 0 && blockIdx.y == 0)
            for (int i = threadIdx.x; i < bt.seqs; i += THREADS) {
                int s, n, l;
                seq_range(c, bt, i, s, n, l, &g_kv_cache_error);
            }
        if (w.b < 0) return false;
    }
    int start, n, len;
    if (!seq_range(c, bt, w.b, start, n, len, &g_kv_cache_error) || n == 0) return false;
    const int first = len - n;  // negative: the first rows are padding
    w.blk = max(first, 0) / BT + (bt.max_new <= 1 ? 0 : x - (start / BT + 2 * w.b));
    w.pos0 = w.blk * BT;
    if (w.pos0 >= len) return false;
    w.i0 = max(0, first - w.pos0);
    w.i1 = min(BT, len - w.pos0);
    w.row = start + w.pos0 - first;
    return true;
}

// One octet of a row: eight values as two groups of four, `a` and `b` elements into the row,
// that turn together (halves: a pair's members lie in different groups; interleaved: side by
// side).  Each product and sum rounded on its own.
struct Octet {
    int a, b, pair;  // pair: first column of the tables, or -1
};
__device__ __forceinline__ Octet octet(int o, const Rope& r) {
    if (8 * o < r.rotary) return r.interleaved ? Octet{8 * o, 8 * o + 4, 4 * o} : Octet{4 * o, 4 * o + r.rotary / 2, 4 * o};
    return Octet{8 * o, 8 * o + 4, -1};
}
__device__ __forceinline__ void turn1(float& x, float& y, float c, float s) {
    const float a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
    y = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
    x = a;
}
__device__ __forceinline__ void turn(float4& a, float4& b, const Octet& o, const Rope& r, int pos) {
    if (o.pair < 0) return;
    if (pos >= r.rows) {
        atomicOr(&g_kv_cache_error, ERR_RANGE);
        return;
    }
    const long long at = (long long)pos * (r.rotary / 2) + o.pair;
    const float4 c = *reinterpret_cast<const float4*>(r.cos + at);
    const float4 s = *reinterpret_cast<const float4*>(r.sin + at);
    if (r.interleaved) {
        turn1(a.x, a.y, c.x, s.x);
        turn1(a.z, a.w, c.y, s.y);
        turn1(b.x, b.y, c.z, s.z);
        turn1(b.z, b.w, c.w, s.w);
    } else {
        turn1(a.x, b.x, c.x, s.x);
        turn1(a.y, b.y, c.y, s.y);
        turn1(a.z, b.z, c.z, s.z);
        turn1(a.w, b.w, c.w, s.w);
    }
}
__device__ __forceinline__ float amax4(float4 v) { return fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))); }

__device__ __forceinline__ uint32_t code(float q) { return (uint32_t)(max(-127, min(127, __float2int_rn(q))) & 0xff); }
__device__ __forceinline__ uint32_t codes4(float4 v, float d) {
    if (d == 0.f) return 0u;
    return code(__fdiv_rn(v.x, d)) | code(__fdiv_rn(v.y, d)) << 8 | code(__fdiv_rn(v.z, d)) << 16 |
           code(__fdiv_rn(v.w, d)) << 24;
}
// older codes under the new scale: rint(c * r), r = d / d'
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float r) {
    uint32_t o = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) o |= code(__fmul_rn((float)(int8_t)(w >> (8 * i)), r)) << (8 * i);
    return o;
}

// grid (blocks, kv heads [+ kv heads for the queries' rotation]).  A CTA of the first kind
// holds its block's keys and values in registers (D / 4 values a thread), so the rows are read
// once; the second kind turns the block's rows of one group of query heads.
template <typename T, int D>
__global__ void __launch_bounds__(THREADS)
k_kv_append(Cache c, Batch bt, Rows kr, Rows vr, Rows qr, int group, Rope rope, T* __restrict__ q_out) {
    constexpr int O = D / 8, RP = THREADS / O, PASSES = BT / RP;  // octets a row, rows a pass
    __shared__ float part[2][THREADS / 32];
    ptx::grid_dep_wait();
    ptx::grid_dep_launch_dependents();
    Where w;
    if (!find_block(c, bt, w)) return;
    const int tid = threadIdx.x;
    const Octet o = octet(tid % O, rope);
    if (blockIdx.y >= c.heads) {
        const int h0 = (blockIdx.y - c.heads) * group, q_heads = c.heads * group;
        const int rows = (w.i1 - w.i0) * group;
        for (int r = tid / O; r < rows; r += RP) {
            const int i = w.i0 + r / group, h = h0 + r % group;
            const T* src = static_cast<const T*>(qr.data) + (long long)(w.row + i) * qr.token_stride + h * qr.head_stride;
            float4 a = Elem<T>::load4(src + o.a), b = Elem<T>::load4(src + o.b);
            turn(a, b, o, rope, w.pos0 + i);
            T* dst = q_out + ((long long)(w.row + i) * q_heads + h) * D;
            Elem<T>::store4(dst + o.a, a);
            Elem<T>::store4(dst + o.b, b);
        }
        return;
    }
    const int h = blockIdx.y;
    uint8_t* rec = record(c, bt, w.b, w.blk, h, &g_kv_cache_error);
    if (!rec) return;
    const float dk_old = *reinterpret_cast<const float*>(rec + 2 * BT * D);
    const float dv_old = *reinterpret_cast<const float*>(rec + 2 * BT * D + 4);
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    float4 ka[PASSES], kb[PASSES], va[PASSES], vb[PASSES];
#pragma unroll
    for (int u = 0; u < PASSES; ++u) {
        const int i = u * RP + tid / O;
        ka[u] = kb[u] = va[u] = vb[u] = zero;
        if (i >= w.i0 && i < w.i1) {
            const T* ks = static_cast<const T*>(kr.data) + (long long)(w.row + i) * kr.token_stride + h * kr.head_stride;
            const T* vs = static_cast<const T*>(vr.data) + (long long)(w.row + i) * vr.token_stride + h * vr.head_stride;
            ka[u] = Elem<T>::load4(ks + o.a);
            kb[u] = Elem<T>::load4(ks + o.b);
            va[u] = Elem<T>::load4(vs + o.a);
            vb[u] = Elem<T>::load4(vs + o.b);
        }
    }
    float mk = 0.f, mv = 0.f;
#pragma unroll
    for (int u = 0; u < PASSES; ++u) {
        const int i = u * RP + tid / O;
        if (i >= w.i0 && i < w.i1) turn(ka[u], kb[u], o, rope, w.pos0 + i);
        mk = fmaxf(mk, fmaxf(amax4(ka[u]), amax4(kb[u])));
        mv = fmaxf(mv, fmaxf(amax4(va[u]), amax4(vb[u])));
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
        dk = fmaxf(dk, dk_old);
        dv = fmaxf(dv, dv_old);
    }
    if (dk < MIN_SCALE) dk = 0.f;
    if (dv < MIN_SCALE) dv = 0.f;
    const bool grew_k = kept && dk != dk_old, grew_v = kept && dv != dv_old;
    const float rk = grew_k && dk != 0.f ? __fdiv_rn(dk_old, dk) : 0.f;
    const float rv = grew_v && dv != 0.f ? __fdiv_rn(dv_old, dv) : 0.f;
#pragma unroll
    for (int u = 0; u < PASSES; ++u) {
        const int i = u * RP + tid / O;
        uint8_t* kc = rec + i * D;
        uint8_t* vc = kc + BT * D;
        uint32_t *k0 = reinterpret_cast<uint32_t*>(kc + o.a), *k1 = reinterpret_cast<uint32_t*>(kc + o.b);
        uint32_t *v0 = reinterpret_cast<uint32_t*>(vc + o.a), *v1 = reinterpret_cast<uint32_t*>(vc + o.b);
        if (i < w.i0) {
            if (grew_k) {
                *k0 = rescale4(*k0, rk);
                *k1 = rescale4(*k1, rk);
            }
            if (grew_v) {
                *v0 = rescale4(*v0, rv);
                *v1 = rescale4(*v1, rv);
            }
        } else if (i < w.i1) {
            *k0 = codes4(ka[u], dk);
            *k1 = codes4(kb[u], dk);
            *v0 = codes4(va[u], dv);
            *v1 = codes4(vb[u], dv);
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
int append_t(const Cache& c, const Batch& b, const Rows& k, const Rows& v, const Rows& q, int group, const Rope& rope,
             void* q_out, cudaStream_t s) {
    const dim3 grid(block_grid(b), q.data ? 2 * c.heads : c.heads);
    ProfScope ps("k_kv_append", s);
    auto go = [&](auto kernel) {
        return pdl_status(launch_pdl(kernel, grid, dim3(THREADS), 0, s, c, b, k, v, q, group, rope, static_cast<T*>(q_out)),
                          "mmq_kv_append");
    };
    return c.dim == 64 ? go(k_kv_append<T, 64>) : c.dim == 128 ? go(k_kv_append<T, 128>) : go(k_kv_append<T, 256>);
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
    const int group = q.data ? q_heads / c.heads : 0;
    return dtype == MMQ_F32    ? append_t<float>(c, b, k, v, q, group, rope, q_out, s)
           : dtype == MMQ_BF16 ? append_t<__nv_bfloat16>(c, b, k, v, q, group, rope, q_out, s)
                               : append_t<__half>(c, b, k, v, q, group, rope, q_out, s);
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
