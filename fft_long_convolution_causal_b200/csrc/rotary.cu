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
// 48 us, 5.6 TB/s (75 us without loads ahead and packed arithmetic); neighbouring
// pairs 56 us with any even part rotated (230 us by elements).
#include <cuda_bf16.h>

#include <string.h>

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

// the same piece of heads h0 .. h1 - 1, four in flight
template <typename P, typename From, typename To>
__device__ __forceinline__ void copy(int h0, int h1, From from, To to) {
    for (int h = h0; h < h1; h += 4) {
        P p[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (h + k < h1) p[k] = *from(h + k);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (h + k < h1) *to(h + k) = p[k];
    }
}

// V = elements of a 16-byte piece, or 1: an unaligned shape
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kThreads, 4) rotary(const __grid_constant__ Args a) {
    using P = Piece<T, V>;
    constexpr int NP = INTER && V > 1 ? V / 2 : V;  // pairs of an item
    constexpr bool kWhole = INTER && V > 1;          // items go on behind the rotated part, which may end inside one
    const int64_t idx = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t token = idx / a.per_token;
    if (token >= a.tokens) return;
    const int item = (int)(idx - token * a.per_token);
    const int64_t b = token / a.N, n = token - b * a.N;
    const int h0 = blockIdx.y * a.heads_per, h1 = min(a.H, h0 + a.heads_per);
    const int pairs = a.rot / 2, items = (pairs + NP - 1) / NP;
    auto from = [&](int h) -> const T* {
        const RotaryView& w = a.v[h >= a.v[0].H];
        return (const T*)w.x + b * w.xb + (h >= a.v[0].H ? h - a.v[0].H : h) * w.xh + n * w.xn;
    };
    auto to = [&](int h) -> T* {
        const RotaryView& w = a.v[h >= a.v[0].H];
        return (T*)w.y + b * w.yb + (h >= a.v[0].H ? h - a.v[0].H : h) * w.yh + n * w.yn;
    };
    if (!kWhole && item >= items) {  // behind the rotated part
        const int e = a.rot + (item - items) * V;
        copy<P>(h0, h1, [&](int h) { return reinterpret_cast<const P*>(from(h) + e); },
                [&](int h) { return reinterpret_cast<P*>(to(h) + e); });
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
        const uint64_t ph = pos * a.turns[kWhole ? min(item * NP + i, pairs - 1) : item * NP + i];  // turns modulo 1, exactly
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
                P r = u[k], t;
#pragma unroll
                for (int i = 0; i < NQ; ++i) {
                    const float2 x1 = u[k].get(i);
                    if (kOne) {
                        if (item * NP + i >= pairs) continue;  // copied
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

// Pairs half a rotated part apart where that is no multiple of a piece, out of place: a thread has one aligned piece of
// the result.  Its partners start anywhere in a piece: two aligned pieces are loaded and shifted together; where the
// first half ends inside the thread's piece, the second half's partners likewise.
template <typename T>
__device__ __forceinline__ void shifted(uint32_t (&o)[4], const uint4& lo, const uint4& hi, int bytes) {
    uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int i = 0; i < 7; ++i) w[i] = bytes & 4 ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = bytes & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = sizeof(T) == 4 ? w[i] : __funnelshift_r(w[i], w[i + 1], bytes & 2 ? 16 : 0);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 3) rotary_shifted(const __grid_constant__ Args a) {
    constexpr int V = 16 / sizeof(T), NP = V / 2;
    using P = Piece<T, V>;
    const int64_t idx = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t token = idx / a.per_token;
    if (token >= a.tokens) return;
    const int e = (int)(idx - token * a.per_token) * V, half = a.rot / 2, last = a.dim - V;
    const int64_t b = token / a.N, n = token - b * a.N;
    const int h0 = blockIdx.y * a.heads_per, h1 = min(a.H, h0 + a.heads_per);
    auto from = [&](int h) -> const T* {
        const RotaryView& w = a.v[h >= a.v[0].H];
        return (const T*)w.x + b * w.xb + (h >= a.v[0].H ? h - a.v[0].H : h) * w.xh + n * w.xn;
    };
    auto to = [&](int h) -> T* {
        const RotaryView& w = a.v[h >= a.v[0].H];
        return (T*)w.y + b * w.yb + (h >= a.v[0].H ? h - a.v[0].H : h) * w.yh + n * w.yn + e;
    };
    // where the partners start, in the first half's terms (+ half) or the second's (- half); behind the rotated part
    // nothing is done with them (a branch of its own for those pieces took as long again)
    const bool first = e < half, two = first && e + V > half;
    const int s1 = first ? e + half : e < a.rot ? e - half : e, p1 = s1 / V * V, q1 = min(p1 + V, last), m1 = (s1 - p1) * (int)sizeof(T);
    const int s2 = e - half + V, q2 = s2 / V * V, m2 = (s2 - q2) * (int)sizeof(T);  // two: from the piece before q2 on
    const int p2 = max(q2 - V, 0);
    struct Head {
        P x;
        uint4 lo, hi, lo2, hi2;
    } u[kAhead];
    auto piece = [](const T* p) { return *reinterpret_cast<const uint4*>(p); };
    auto fetch = [&](int h) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (h + k < h1) {
                const T* x = from(h + k);
                u[k].x = *reinterpret_cast<const P*>(x + e);
                u[k].lo = piece(x + p1);
                u[k].hi = piece(x + q1);
                if (two) {
                    u[k].lo2 = piece(x + p2);
                    u[k].hi2 = piece(x + q2);
                }
            }
    };
    fetch(h0);
    float2 cs[NP], sn[NP];
    uint32_t of1[4] = {0u, 0u, 0u, 0u};  // two: which bits of the partners are the first half's
    const uint64_t pos = (uint64_t)a.pos[b * a.pos_stride + n];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = min(e + i, a.rot - 1);
        float s, k;
        const uint64_t ph = pos * a.turns[c < half ? c : c - half];  // turns modulo 1, exactly
        sincospif((float)(int32_t)(ph >> 32) * 0x1p-31f, &s, &k);
        k *= a.m;
        s *= (c < half) != (a.inverse != 0) ? -a.m : a.m;
        if (c < half) of1[i * sizeof(T) / 4] |= sizeof(T) == 4 ? 0xffffffffu : 0xffffu << (i & 1) * 16;
        (i & 1 ? cs[i / 2].y : cs[i / 2].x) = k;
        (i & 1 ? sn[i / 2].y : sn[i / 2].x) = s;
    }
    for (int h = h0;;) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (h + k < h1) {
                uint32_t w[4];
                shifted<T>(w, u[k].lo, u[k].hi, m1);
                if (two) {
                    uint32_t w2[4];
                    shifted<T>(w2, u[k].lo2, u[k].hi2, m2);
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = (w[i] & of1[i]) | (w2[i] & ~of1[i]);
                }
                P p, r = u[k].x;
                memcpy(&p, w, 16);
#pragma unroll
                for (int i = 0; i < NP; ++i)
                    if (e + 2 * i < a.rot) r.set(i, fma2(u[k].x.get(i), cs[i], mul2(p.get(i), sn[i])));
                *reinterpret_cast<P*>(to(h + k)) = r;
            }
        h += kAhead;
        if (h >= h1) break;
        fetch(h);
    }
}

template <typename K>
cudaError_t start(K kernel, Args& a, int sms, cudaStream_t s) {
    const int64_t threads = a.tokens * a.per_token;
    // Heads a thread walks: 8 share their sines; one each where few threads are there to fill the SMs.
    const int64_t most = threads * a.H;
    a.heads_per = most >= (int64_t)sms * 8192 ? 8 : most >= (int64_t)sms * 4096 ? 4 : 1;
    const int groups = (a.H + a.heads_per - 1) / a.heads_per;
    kernel<<<dim3((unsigned)((threads + kThreads - 1) / kThreads), groups), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int V, bool INTER>
cudaError_t run(Args a, int sms, bool copy_rest, cudaStream_t s) {
    constexpr int NP = INTER && V > 1 ? V / 2 : V;
    const int items = (a.rot / 2 + NP - 1) / NP;
    a.per_token = items + (copy_rest ? (a.dim - (INTER && V > 1 ? items * V : a.rot)) / V : 0);
    return start(rotary<T, V, INTER>, a, sms, s);
}

template <typename T>
cudaError_t pick(const fftconv_rotary_s& p, Args& a, int views, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    bool vec = a.dim % V == 0, same = true, apart = true;
    const bool rest = a.dim > a.rot;
    for (int i = 0; i < views; ++i) {
        const RotaryView& v = a.v[i];
        vec = vec && (((uintptr_t)v.x | (uintptr_t)v.y) & 15u) == 0 &&
              ((v.xb | v.xh | v.xn | v.yb | v.yh | v.yn) % V) == 0;
        same = same && v.x == v.y;
        apart = apart && v.x != v.y;
    }
    const bool copy_rest = rest && !same;
    if (!p.interleaved && vec && (a.rot / 2) % V) {
        // By elements 235 us at 4 x 4096 x 32 heads x 128 with 90 rotated (bf16), 89 us with the partners shifted
        // together; in place another thread's result would be in the way.
        if (apart) {
            a.per_token = a.dim / V;
            return start(rotary_shifted<T>, a, p.sms, s);
        }
        vec = false;
    }
    if (p.interleaved) return vec ? run<T, V, true>(a, p.sms, copy_rest, s) : run<T, 1, true>(a, p.sms, copy_rest, s);
    return vec ? run<T, V, false>(a, p.sms, copy_rest, s) : run<T, 1, false>(a, p.sms, copy_rest, s);
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
