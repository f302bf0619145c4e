// The way back through the weights: the instances of k_ffn_tile (ffn_tile.cuh) for each format and type.
#include "ffn_tile.cuh"

namespace mmq {
namespace {

// (Q8_0's scales are f16 values: nothing but its weights is rounded as it is)
template <int FMT>
int launch(const ffn::Tile& a, int smem, int ctas, bool go, const char* fn, cudaStream_t s) {
    if (a.dtype == MMQ_F32) return ffn::launch_tile<FMT, true, true, 1, false>(a, smem, ctas, go, fn, s);
    return a.dtype == MMQ_F16 ? ffn::launch_tile<FMT, false, true, 1, FMT != FMT_Q8_0>(a, smem, ctas, go, fn, s)
                              : ffn::launch_tile<FMT, false, true, 1, false>(a, smem, ctas, go, fn, s);
}

}  // namespace

int ffn_backward_launch(int fmt, const ffn::Tile& a, int smem, int ctas, bool go, const char* fn, cudaStream_t s) {
    if (fmt == FMT_Q8_0) return launch<FMT_Q8_0>(a, smem, ctas, go, fn, s);
    if (fmt == FMT_Q4_K) return launch<FMT_Q4_K>(a, smem, ctas, go, fn, s);
    if (fmt == FMT_Q5_K) return launch<FMT_Q5_K>(a, smem, ctas, go, fn, s);
    return launch<FMT_Q6_K>(a, smem, ctas, go, fn, s);
}

unsigned ffn_backward_take_error() { return ffn::take_tile_error(); }
int ffn_backward_set_wait_limit(unsigned long long ns) { return ffn::set_tile_wait_limit(ns); }

}  // namespace mmq
