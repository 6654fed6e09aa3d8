// mixer.h -- plan objects and kernel launchers of the sequence-mixer operators
// (linear attention with a decay per head, rotary positions, layer norm).
// Not part of the ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "fftconv.h"

struct fftconv_linattn_s {
    int B = 0, H = 0, dk = 0, dv = 0, dtype = 0, device = 0, sms = 1;
    int64_t N = 0;
    void* block = nullptr;            // one allocation: the tables below and the status word
    const double* d_log = nullptr;    // [H] natural logarithm of the decay
    const float* d_pow = nullptr;     // [H][kLaPowers] a^n, n = 0, 1, ...
    const float2* d_decay = nullptr;  // [H][kLaPowers] a^n in two parts, for what a state is multiplied by again and again
    int* d_err = nullptr;             // device status word
    uint32_t wait_limit = FFTCONV_DEFAULT_WAIT_PROBES;
};

struct fftconv_rotary_s {
    int dim = 0, rot = 0, interleaved = 0, dtype = 0, device = 0, sms = 1;
    float magnitude = 1.f;
    uint64_t* d_turns = nullptr;  // [rot / 2] turns per position, in units of 2^-64 turn
};

struct fftconv_norm_s {
    int64_t rows = 0;
    int C = 0, groups = 1, dtype = 0, device = 0, sms = 1;
    float eps = 0.f;
};

namespace fftc {

// One pass of decayed linear attention over [B, H, N] tokens:
//   out_t = s_p sum a^|t-s| (x_t . y_s) z_s + s_i a^(..) x_t S
// over s <= t (forward) or s >= t (reverse), with the state S [dx][dz] fp32
//   forward  S_t = a S_{t-1} + s_u y_t^T z_t   (S_{-1} = s_in;  out_t reads S_t)
//   reverse  R_t = a R_{t+1} + s_u y_t^T z_t   (R_{len-1} = s_in + ...; s_out = a R_0)
// Rows at or behind a sequence's length are not read; out there is zero.
struct LaPass {
    const void *x, *y, *z;
    void* out;
    fftconv_strides sx, sy, sz, so;   // in elements; the head dimension is contiguous
    int dx, dz;
    int reverse;
    const float* s_in;                // [B][H] states or NULL (zero)
    float* s_out;                     // or NULL
    int in_trans;                     // s_in holds [dz][dx]
    float s_p, s_i, s_u;
};

constexpr int kLaChunk = 64;      // tokens a step of the fp32 kernel
constexpr int kLaChunkTc = 128;   // and of the tensor-core kernel
constexpr int kLaPowers = 132;    // table length per head (exponents 0 .. 128, padded)
constexpr int kLaMaxSegments = 64;
constexpr int kLaMaxWaves = 4;    // segments times CTAs, over what the GPU holds at once
constexpr int kLaMaxPasses = 3;

struct LaCall {
    LaPass pass[kLaMaxPasses];
    int passes;
    int B, H;
    int64_t N;
    const int32_t* lengths;           // [B] or NULL
    float* work;                      // segment states
};

// Workspace of a call of that many passes, in floats.
size_t la_workspace_floats(const fftconv_linattn_s& p, int passes);
cudaError_t launch_la(const fftconv_linattn_s& p, const LaCall& c, cudaStream_t s);

struct LaStep {
    const void *q, *k, *v;
    void* o;
    int64_t qb, qh, kb, kh, vb, vh, ob, oh;  // strides in elements
    float* state;
    const int32_t* slots;
    int B, slots_n;
    float scale;
};
cudaError_t launch_la_step(const fftconv_linattn_s& p, const LaStep& c, cudaStream_t s);

struct RotaryView {
    const void* x;
    void* y;
    int H;
    int64_t xb, xh, xn, yb, yh, yn;
};
cudaError_t launch_rotary(const fftconv_rotary_s& p, const RotaryView* v, int views, int B, int64_t N,
                          const int64_t* pos, int64_t pos_stride, int inverse, cudaStream_t s);

cudaError_t launch_norm_fwd(const fftconv_norm_s& p, int64_t rows, const void* x, const float* w, const float* b,
                            void* y, float* mean, float* rstd, cudaStream_t s);
size_t norm_workspace_bytes(const fftconv_norm_s& p);
cudaError_t launch_norm_bwd(const fftconv_norm_s& p, int64_t rows, const void* dy, const void* x, const float* w,
                            const float* mean, const float* rstd, void* dx, float* dw, float* db, float* work,
                            cudaStream_t s);

}  // namespace fftc
