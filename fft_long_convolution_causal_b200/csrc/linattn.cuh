// linattn.cuh -- what the linear-attention kernels share (the argument block of a
// call, the length of a row, a block's place), and the launches that the mixers' kernels use.
#pragma once

#include <atomic>

#include "mixer.h"

namespace fftc {
namespace la {

struct Args {
    LaPass p[kLaMaxPasses];
    int H, passes;
    int whole, nseg;            // rows (b, h) in front that run unsplit, segments of each of the others
    int first;                  // index of the launch's block 0 among all blocks
    int64_t N, seg;             // tokens, tokens a segment
    const int32_t* lengths;
    const float* pw;            // [H][kLaPowers]
    const float2* decay;        // the same in two parts
    float* work;                // [pass][split row][nseg][dk * dv]: segment states
    size_t pass_floats, state_floats;
};

// What a block works on.  Blocks run over the unsplit rows, then over the segments of the others, the passes of one
// row side by side: they find each other's tensors in L2.
struct Place {
    int pass, bh, sg;
    bool split;
    int64_t first, tokens;  // of the segment
    size_t state;           // offset of its state in the workspace, in floats
    __device__ __forceinline__ explicit Place(const Args& a) {
        const int i = (int)blockIdx.x + a.first, r = i / a.passes;
        pass = i - r * a.passes;
        split = r >= a.whole;
        const int s = r - a.whole;
        bh = split ? a.whole + s / a.nseg : r;
        sg = split ? s % a.nseg : 0;
        first = sg * a.seg;
        tokens = split ? min(a.seg, a.N - first) : a.N;
        state = pass * a.pass_floats + (split ? (size_t)s * a.state_floats : 0);
    }
    // the pass's last segment, whose own state only a final state needs
    __device__ __forceinline__ bool ends(const Args& a) const { return sg == (a.p[pass].reverse ? 0 : a.nseg - 1); }
};

__device__ __forceinline__ int64_t live_tokens(const Args& a, int b) {
    if (!a.lengths) return a.N;
    const int64_t n = a.lengths[b];
    return n < 0 ? 0 : n > a.N ? a.N : n;
}

// a s + u for a decay a in two parts.  Rounded to fp32, a is off by up to 2^-25, always to the same side, and a state
// that lives for n steps would drift by n times that (a decay nearer to one than that would not decay at all).
__device__ __forceinline__ float decayed(float2 a, float s, float u) { return fmaf(a.x, s, fmaf(a.y, s, u)); }

// The shared-memory limit of a kernel, set once a device (again at worst).
template <auto kKernel>
cudaError_t allow(int bytes) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load() & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done |= bit;
    return e;
}

// Launches that may begin while the kernel before them in the stream still runs (`early`): it calls let_next_start,
// they call after_previous before they touch what it writes.
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
template <auto kKernel, typename... A>
cudaError_t launch(dim3 grid, int threads, size_t bytes, cudaStream_t s, bool early, const A&... args) {
    cudaLaunchConfig_t c = {};
    c.gridDim = grid;
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = bytes;
    c.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    c.attrs = &attr;
    c.numAttrs = early ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&c, kKernel, args...);
    if (e != cudaSuccess) cudaGetLastError();
    return e;
}

// Joins the segments' own states.
cudaError_t launch_carry(const Args& a, int rows, int passes, const double* lg, cudaStream_t s);
// The whole call on tcgen05 (bf16); ends: a pass returns its final states.
cudaError_t launch_tc(const Args& a, int dx, int dz, int B, int passes, bool ends, const fftconv_linattn_s& p,
                      cudaStream_t s);

}  // namespace la
}  // namespace fftc
