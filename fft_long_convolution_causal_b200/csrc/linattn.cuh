// linattn.cuh -- what the linear-attention kernels share: the argument block of
// a call and the length of a row.
#pragma once

#include "mixer.h"

namespace fftc {
namespace la {

struct Args {
    LaPass p[kLaMaxPasses];
    int H, nseg;
    int64_t N, seg;             // tokens, tokens a segment
    const int32_t* lengths;
    const float* pw;            // [H][kLaPowers]
    float* work;                // [pass][bh][nseg][dk * dv]: segment states
    size_t pass_floats, state_floats;
};

__device__ __forceinline__ int64_t live_tokens(const Args& a, int b) {
    if (!a.lengths) return a.N;
    const int64_t n = a.lengths[b];
    return n < 0 ? 0 : n > a.N ? a.N : n;
}

// tcgen05 kernels (bf16): the segments' own states, and the outputs.
cudaError_t launch_tc_states(const Args& a, int dx, int dz, int bh, int passes, const fftconv_linattn_s& p, cudaStream_t s);
cudaError_t launch_tc_main(const Args& a, int dx, int dz, int bh, int passes, const fftconv_linattn_s& p, cudaStream_t s);

}  // namespace la
}  // namespace fftc
