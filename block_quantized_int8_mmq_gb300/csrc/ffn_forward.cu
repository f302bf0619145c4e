// The products of the forward pass: the instances of k_ffn_tile (ffn_tile.cuh) for each format and type.
#include "ffn_tile.cuh"

namespace mmq {
namespace {

// (Q8_0's scales are f16 values: nothing but its weights is rounded as it is)
template <int FMT, int SUB>
int launch16(const ffn::Tile& a, int smem, int ctas, bool go, const char* fn, cudaStream_t s) {
    return a.dtype == MMQ_F16 ? ffn::launch_tile<FMT, false, false, SUB, FMT != FMT_Q8_0>(a, smem, ctas, go, fn, s)
                              : ffn::launch_tile<FMT, false, false, SUB, false>(a, smem, ctas, go, fn, s);
}
template <int FMT>
int launch(const ffn::Tile& a, int smem, int ctas, bool go, const char* fn, cudaStream_t s) {
    if (a.dtype == MMQ_F32) return ffn::launch_tile<FMT, true, false, 1, false>(a, smem, ctas, go, fn, s);
    return a.sub == 2 ? launch16<FMT, 2>(a, smem, ctas, go, fn, s) : launch16<FMT, 1>(a, smem, ctas, go, fn, s);
}

}  // namespace

int ffn_forward_launch(int fmt, const ffn::Tile& a, int smem, int ctas, bool go, const char* fn, cudaStream_t s) {
    if (fmt == FMT_Q8_0) return launch<FMT_Q8_0>(a, smem, ctas, go, fn, s);
    if (fmt == FMT_Q4_K) return launch<FMT_Q4_K>(a, smem, ctas, go, fn, s);
    if (fmt == FMT_Q5_K) return launch<FMT_Q5_K>(a, smem, ctas, go, fn, s);
    return launch<FMT_Q6_K>(a, smem, ctas, go, fn, s);
}

unsigned ffn_forward_take_error() { return ffn::take_tile_error(); }
int ffn_forward_set_wait_limit(unsigned long long ns) { return ffn::set_tile_wait_limit(ns); }

}  // namespace mmq
