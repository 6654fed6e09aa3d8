// rotary.cu -- rotary positions: pair i of a head turns by pos * f_i,
//   y_1 = m (x_1 cos - x_2 sin),  y_2 = m (x_2 cos + x_1 sin),
// (inverse: sin negated, the gradient of the rotation), the rest of the head copied.
//
// The angle is held in turns as a 64-bit fixed-point fraction: pos * f_i is an
// integer product that wraps modulo one turn exactly, so a position of millions
// costs no accuracy (the table's rounding, 2^-65 turn, times the position) and
// no 64-bit floating-point arithmetic.  Its upper 32 bits give the sine and
// cosine in fp32.
//
// Bound by memory (each element read and written once).  A thread owns some
// pairs of one token, computes their sines once and walks a range of heads, the
// next heads' loads in flight: 4 x 4096 tokens x 32 heads x 128 in bf16 take
// 48.5 us, 5.5 TB/s (75 us without loads ahead and packed arithmetic).
#include <cuda_bf16.h>

#include "mixer.h"
#include "pairs.cuh"

namespace fftc {
namespace rot {

constexpr int kThreads = 256;
constexpr int kAhead = 2;  // heads whose loads are in flight together

struct Args {
    RotaryView v[2];
    int H, rot, dim, per_token, heads_per, inverse;
    int64_t tokens, N, pos_stride;
    const int64_t* pos;
    const uint64_t* turns;
    float m;
};

// V = elements of a 16-byte piece, or 1: an unaligned shape
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kThreads, 4) rotary(const __grid_constant__ Args a) {
    using P = Piece<T, V>;
    constexpr int NP = INTER && V > 1 ? V / 2 : V;  // pairs of an item
    const int64_t idx = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t token = idx / a.per_token;
    if (token >= a.tokens) return;
    const int item = (int)(idx - token * a.per_token);
    const int64_t b = token / a.N, n = token - b * a.N;
    const int h0 = blockIdx.y * a.heads_per, h1 = min(a.H, h0 + a.heads_per);
    const int items = a.rot / 2 / NP;
    auto from = [&](int h) -> const T* {
        const RotaryView& w = a.v[h >= a.v[0].H];
        return (const T*)w.x + b * w.xb + (h >= a.v[0].H ? h - a.v[0].H : h) * w.xh + n * w.xn;
    };
    auto to = [&](int h) -> T* {
        const RotaryView& w = a.v[h >= a.v[0].H];
        return (T*)w.y + b * w.yb + (h >= a.v[0].H ? h - a.v[0].H : h) * w.yh + n * w.yn;
    };
    if (item >= items) {  // behind the rotated part
        const int e = a.rot + (item - items) * V;
        for (int h = h0; h < h1; ++h) *reinterpret_cast<P*>(to(h) + e) = *reinterpret_cast<const P*>(from(h) + e);
        return;
    }
    // offsets of the two pieces of an item; one piece when the pairs are neighbours
    constexpr bool kOne = INTER && V > 1;
    const int e0 = INTER ? 2 * NP * item : NP * item, e1 = INTER ? e0 + 1 : e0 + a.rot / 2;
    // the first heads' loads are in flight while the sines are computed
    P u[kAhead], w[kAhead];
    auto fetch = [&](int h) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (h + k < h1) {
                const T* x = from(h + k);
                u[k] = *reinterpret_cast<const P*>(x + e0);
                if (!kOne) w[k] = *reinterpret_cast<const P*>(x + e1);
            }
    };
    fetch(h0);
    // pairs of neighbours: cosines twice each, the sine negated for the first; pairs apart: by two
    constexpr int NQ = kOne ? P::kPairs : (NP + 1) / 2;
    float2 cs[NQ], sn[NQ];
    const uint64_t pos = (uint64_t)a.pos[b * a.pos_stride + n];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const uint64_t ph = pos * a.turns[item * NP + i];  // turns modulo 1, exactly
        float s, c;
        sincospif((float)(int32_t)(ph >> 32) * 0x1p-31f, &s, &c);
        c *= a.m;
        s *= a.inverse ? -a.m : a.m;
        if (kOne) {
            cs[i] = both(c);
            sn[i] = make_float2(-s, s);
        } else if (i & 1) {
            cs[i / 2].y = c;
            sn[i / 2].y = s;
        } else {
            cs[i / 2] = make_float2(c, 0.f);
            sn[i / 2] = make_float2(s, 0.f);
        }
    }
    for (int h = h0;;) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (h + k < h1) {
                T* y = to(h + k);
                P r, t;
#pragma unroll
                for (int i = 0; i < NQ; ++i) {
                    const float2 x1 = u[k].get(i);
                    if (kOne) {
                        r.set(i, fma2(x1, cs[i], mul2(make_float2(x1.y, x1.x), sn[i])));
                    } else {
                        const float2 x2 = w[k].get(i);
                        r.set(i, fma2(x1, cs[i], mul2(x2, make_float2(-sn[i].x, -sn[i].y))));
                        t.set(i, fma2(x2, cs[i], mul2(x1, sn[i])));
                    }
                }
                *reinterpret_cast<P*>(y + e0) = r;
                if (!kOne) *reinterpret_cast<P*>(y + e1) = t;
            }
        h += kAhead;
        if (h >= h1) break;
        fetch(h);
    }
}

template <typename T, int V, bool INTER>
cudaError_t run(Args a, int sms, bool copy_rest, cudaStream_t s) {
    constexpr int NP = INTER && V > 1 ? V / 2 : V;
    a.per_token = a.rot / 2 / NP + (copy_rest ? (a.dim - a.rot) / V : 0);
    const int64_t threads = a.tokens * a.per_token;
    // Heads a thread walks: 8 share their sines; one each where few threads are there to fill the SMs.
    const int64_t most = threads * a.H;
    a.heads_per = most >= (int64_t)sms * 8192 ? 8 : most >= (int64_t)sms * 4096 ? 4 : 1;
    const int groups = (a.H + a.heads_per - 1) / a.heads_per;
    rotary<T, V, INTER><<<dim3((unsigned)((threads + kThreads - 1) / kThreads), groups), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t pick(const fftconv_rotary_s& p, Args& a, int views, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    bool vec = a.dim % V == 0 && (p.interleaved ? a.rot % V == 0 : (a.rot / 2) % V == 0), rest = a.dim > a.rot;
    bool same = true;
    for (int i = 0; i < views; ++i) {
        const RotaryView& v = a.v[i];
        vec = vec && (((uintptr_t)v.x | (uintptr_t)v.y) & 15u) == 0 &&
              ((v.xb | v.xh | v.xn | v.yb | v.yh | v.yn) % V) == 0;
        same = same && v.x == v.y;
    }
    rest = rest && !same;
    if (p.interleaved) return vec ? run<T, V, true>(a, p.sms, rest, s) : run<T, 1, true>(a, p.sms, rest, s);
    return vec ? run<T, V, false>(a, p.sms, rest, s) : run<T, 1, false>(a, p.sms, rest, s);
}

}  // namespace rot

cudaError_t launch_rotary(const fftconv_rotary_s& p, const RotaryView* v, int views, int B, int64_t N,
                          const int64_t* pos, int64_t pos_stride, int inverse, cudaStream_t s) {
    rot::Args a;
    a.v[0] = v[0];
    a.v[1] = views > 1 ? v[1] : v[0];
    a.H = v[0].H + (views > 1 ? v[1].H : 0);
    a.rot = p.rot;
    a.dim = p.dim;
    a.inverse = inverse;
    a.tokens = (int64_t)B * N;
    a.N = N;
    a.pos = pos;
    a.pos_stride = pos_stride;
    a.turns = p.d_turns;
    a.m = p.magnitude;
    a.per_token = a.heads_per = 0;
    return p.dtype == FFTCONV_BF16 ? rot::pick<__nv_bfloat16>(p, a, views, s) : rot::pick<float>(p, a, views, s);
}

}  // namespace fftc
