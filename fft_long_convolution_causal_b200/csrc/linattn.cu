// linattn.cu -- linear attention with a decay per head, chunk by chunk.
//
// Within a chunk of C tokens (local index i, j; L of them live)
//   out_i = s_p sum_{j <= i} a^(i-j) (x_i . y_j) z_j + s_i a^(i+1) x_i S
//   S    <- a^L S + s_u sum_j a^(L-1-j) y_j^T z_j
// and mirrored (j >= i, exponents L-1-i and j+1) where the tokens run backwards:
// the gradients are the same operator on other operands,
//   dq = pass(do, v, k) forward, dk = pass(v, do, q) and dv = pass(k, q, do) in reverse.
// Every exponent is >= 0, so nothing overflows however strong the decay is.
//
// bf16 runs on tcgen05 (linattn_tc.cu), fp32 here.  The token axis is cut into segments where one CTA per (row, head) would leave
// SMs idle: a first kernel sums each segment's own contribution to the state, a
// second carries the states over the segments, the third computes the outputs.
#include <cuda_bf16.h>
#include <math.h>

#include <type_traits>

#include "linattn.cuh"

namespace fftc {
namespace la {

constexpr int kC = kLaChunk;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }

// ---- fp32 on the tensor cores: every operand as a sum of two tf32 values (the
// second exact to 2^-23 of the first's), three products, the largest last.  The
// product of the two small parts, below 2^-22, is left out.  Below 2^-114 the second
// part is a subnormal number and loses bits; within 2^-12 of the largest number the
// first is an infinity (kept finite by one instruction more a value, 24 x 4096 x 64
// took 121 us instead of 115).
struct Two {
    uint32_t hi, lo;
};
__device__ __forceinline__ Two split(float x) {
    Two r;
    r.hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;  // to nearest, ties away (a NaN stays one in the second part)
    r.lo = __float_as_uint(x - __uint_as_float(r.hi));
    return r;
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// The products of one A and N B fragments, FIRST: into u, else added to it.  Two steps of 8 go into one u before it is
// added to the sum in fp32: the tensor core truncates when it accumulates, and over the dozens of steps of a sum that
// bias reached 4e-6.
template <bool FIRST, int N>
__device__ __forceinline__ void mma3(float (&u)[N][4], const Two (&a)[4], const Two (&b)[N][2], uint32_t tiles) {
#pragma unroll
    for (int q = 0; q < N; ++q) {
        if (!(tiles >> q & 1u)) continue;
        if (FIRST)
            mma_tf32_zero(u[q], a[0].lo, a[1].lo, a[2].lo, a[3].lo, b[q][0].hi, b[q][1].hi);
        else
            mma_tf32(u[q], a[0].lo, a[1].lo, a[2].lo, a[3].lo, b[q][0].hi, b[q][1].hi);
    }
#pragma unroll
    for (int q = 0; q < N; ++q)
        if (tiles >> q & 1u) mma_tf32(u[q], a[0].hi, a[1].hi, a[2].hi, a[3].hi, b[q][0].lo, b[q][1].lo);
#pragma unroll
    for (int q = 0; q < N; ++q)
        if (tiles >> q & 1u) mma_tf32(u[q], a[0].hi, a[1].hi, a[2].hi, a[3].hi, b[q][0].hi, b[q][1].hi);
}
template <int N>
__device__ __forceinline__ void add(float (&acc)[N][4], const float (&u)[N][4], uint32_t tiles) {
#pragma unroll
    for (int q = 0; q < N; ++q)
        if (tiles >> q & 1u)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[q][e] += u[q][e];
}
// fragments of rows i0.., columns k0.. of a row-major matrix (A), and of its transpose (B: columns are rows)
template <int P>
__device__ __forceinline__ void frag_a(Two (&a)[4], const float* m, int i0, int k0, int g, int t) {
    const float* p = m + (i0 + g) * P + k0 + t;
    a[0] = split(p[0]), a[1] = split(p[8 * P]), a[2] = split(p[4]), a[3] = split(p[8 * P + 4]);
}
template <int P>
__device__ __forceinline__ void frag_bt(Two (&b)[2], const float* m, int n0, int k0, int g, int t) {
    const float* p = m + (n0 + g) * P + k0 + t;
    b[0] = split(p[0]), b[1] = split(p[4]);
}
template <int P>
__device__ __forceinline__ void frag_b(Two (&b)[2], const float* m, int k0, int n0, int g, int t) {
    const float* p = m + (k0 + t) * P + n0 + g;
    b[0] = split(p[0]), b[1] = split(p[4 * P]);
}

// Row pitches (floats): 4 or 8 more than a multiple of 32, so that the 8 rows x 4 columns (or 4 x 8) of a
// fragment lie in 32 different banks.
template <int DX, int DZ>
struct Shape {
    static constexpr int PX = DX + 4, PZ = DZ + 8, PP = kC + 4;
    static constexpr int kFloats = 2 * kC * PX + kC * PZ + kC * PP + DX * PZ + kLaPowers;
    static constexpr int kCtas = DX == 64 && DZ == 64 ? 2 : 1;
    static constexpr int kThreads = DX == 64 && DZ == 64 ? 256 : 512, kGroups = kThreads / 128;  // 4 warps down, kGroups across
};

// rows of a tensor into shared memory, zeros behind row `live` and column d
template <int D, int P, int kThreads>
__device__ __forceinline__ void load_tile(float* dst, const float* src, int64_t stride, int live, int d) {
    for (int e = threadIdx.x; e < kC * (D / 4); e += kThreads) {
        const int r = e / (D / 4), c = 4 * (e % (D / 4));
        const bool on = r < live && c < d;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(
                         (uint32_t)__cvta_generic_to_shared(dst + r * P + c)),
                     "l"(on ? src + r * stride + c : src), "r"(on ? 16 : 0)
                     : "memory");
    }
}

// One block a Place; STATES: only the segments' own states.
// Warp w has rows 16 (w & 3) of scores and outputs, and every kGroups-th 8-column
// tile of theirs from w >> 2 on (tiles behind dz are left out); the state lives
// in registers as accumulators (m-tiles w & 3, + 4), with a copy in shared
// memory for the outputs.  Two CTAs of 8 warps an SM at 64 x 64, one of 16 above.
// Bound by the chain of a chunk's steps, with one or two CTAs an SM to hide it:
// its copies are waited for, four barriers part the steps, and every product loads
// and splits its operands anew (ten instructions a 16 x 8 x 8).  Neither the issue
// slots (52% used) nor the tensor pipe (42%) are full; warps wait for fixed
// latencies (1.7 an issue), the math pipe (1.1) and barriers (0.7).  Dims off 64 at
// 128 x 128 spill 430 bytes as well.  24 rows x 4096 at 64 x 64 take 115 us
// (0.9 TB/s), 3 x 5 x 1023 at 40 x 104 with gradients 120 to 145 us (as its lengths
// fall); fp32 multiplications without the tensor cores took 242 and 363.
template <int DX, int DZ, bool STATES, bool FULL>
__global__ void __launch_bounds__((Shape<DX, DZ>::kThreads), (Shape<DX, DZ>::kCtas)) la_f32(const __grid_constant__ Args a) {
    using S = Shape<DX, DZ>;
    constexpr int kThreads = S::kThreads, NG = S::kGroups;
    constexpr int MT = DX / 64, NT = DZ / 8 / NG, NS = kC / 8 / NG;  // tiles of a warp: state MT x NT, scores NS
    extern __shared__ __align__(16) float sm[];
    float *xs = sm, *ys = xs + kC * S::PX, *zs = ys + kC * S::PX, *ps = zs + kC * S::PZ, *ss = ps + kC * S::PP,
          *pw = ss + DX * S::PZ;
    const Place at(a);
    const LaPass& p = a.p[at.pass];
    if (STATES && !p.s_out && at.ends(a)) return;
    const int tid = threadIdx.x, bh = at.bh, b = bh / a.H, h = bh % a.H;
    const int lane = tid & 31, g = lane >> 2, t = lane & 3, warp = tid >> 5, mi = warp & 3, nj = warp >> 2;
    const bool rev = p.reverse;
    const int64_t first = at.first, len = live_tokens(a, b);
    const int64_t rows = at.tokens;                                 // output rows of this segment
    const int64_t live = max((int64_t)0, min(rows, len - first));   // of which read
    const float* x = (const float*)p.x + b * p.sx.batch + h * p.sx.head + first * p.sx.token;
    const float* y = (const float*)p.y + b * p.sy.batch + h * p.sy.head + first * p.sy.token;
    const float* z = (const float*)p.z + b * p.sz.batch + h * p.sz.head + first * p.sz.token;
    float* out = (float*)p.out + b * p.so.batch + h * p.so.head + first * p.so.token;
    float* wseg = a.work + at.state;
    for (int i = tid; i < kLaPowers; i += kThreads) pw[i] = a.pw[h * kLaPowers + i];
    // the state entering the segment
    if (STATES)
        let_next_start();
    else
        after_previous();
    const uint32_t tiles = FULL ? ~0u : (1u << max(0, min(NT, (p.dz / 8 - nj + NG - 1) / NG))) - 1u;  // this warp's, those in front of dz
    const float* s0 = STATES ? nullptr : at.split ? wseg : p.s_in ? p.s_in + (size_t)bh * p.dx * p.dz : nullptr;
    const bool trans = !at.split && p.in_trans;
    float st[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int q = 0; q < NT; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int d = 16 * (mi + 4 * m) + g + 8 * (e >> 1), n = 8 * (nj + NG * q) + 2 * t + (e & 1);
                st[m][q][e] = s0 && d < p.dx && n < p.dz ? s0[trans ? n * p.dx + d : d * p.dz + n] : 0.f;
            }
    const int nch = (int)((live + kC - 1) / kC);
#pragma unroll 1
    for (int ch = 0; ch < nch; ++ch) {
        const int64_t t0 = (int64_t)(rev ? nch - 1 - ch : ch) * kC;
        const int L = (int)min((int64_t)kC, live - t0);
        __syncthreads();
        if (!STATES) load_tile<DX, S::PX, S::kThreads>(xs, x + t0 * p.sx.token, p.sx.token, L, p.dx);
        load_tile<DX, S::PX, S::kThreads>(ys, y + t0 * p.sy.token, p.sy.token, L, p.dx);
        load_tile<DZ, S::PZ, S::kThreads>(zs, z + t0 * p.sz.token, p.sz.token, L, p.dz);
        if (!STATES) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int q = 0; q < NT; ++q)
#pragma unroll
                    for (int e = 0; e < 4; e += 2)
                        *reinterpret_cast<float2*>(ss + (16 * (mi + 4 * m) + g + 4 * e) * S::PZ + 8 * (nj + NG * q) + 2 * t) =
                            make_float2(st[m][q][e], st[m][q][e + 1]);
        }
        asm volatile("cp.async.commit_group;\ncp.async.wait_group 0;\n" ::: "memory");
        __syncthreads();
        if (!STATES) {
            // scores: 16 x 32 a warp, 8-column tiles on the far side of the diagonal left out
            {
                float acc[NS][4] = {};
                // tiles on the far side of the diagonal are left out
                uint32_t near = 0;
#pragma unroll
                for (int q = 0; q < NS; ++q) {
                    const int n0 = 8 * (nj + NG * q);
                    near |= (rev ? n0 + 7 >= 16 * mi : n0 <= 16 * mi + 15) ? 1u << q : 0u;
                }
                if (near)
#pragma unroll 1
                    for (int k = 0; k < p.dx; k += 16) {
                        float u[NS][4];
                        Two fa[4], fb[NS][2];
                        frag_a<S::PX>(fa, xs, 16 * mi, k, g, t);
#pragma unroll
                        for (int q = 0; q < NS; ++q) frag_bt<S::PX>(fb[q], ys, 8 * (nj + NG * q), k, g, t);
                        mma3<true>(u, fa, fb, near);
                        frag_a<S::PX>(fa, xs, 16 * mi, k + 8, g, t);
#pragma unroll
                        for (int q = 0; q < NS; ++q) frag_bt<S::PX>(fb[q], ys, 8 * (nj + NG * q), k + 8, g, t);
                        mma3<false>(u, fa, fb, near);
                        add(acc, u, near);
                    }
#pragma unroll
                for (int q = 0; q < NS; ++q)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int i = 16 * mi + g + 8 * r, j = 8 * (nj + NG * q) + 2 * t, e = rev ? j - i : i - j;
                        const float u = e >= 0 ? p.s_p * pw[e] * acc[q][2 * r] : 0.f;
                        const int f = rev ? e + 1 : e - 1;
                        const float v = f >= 0 ? p.s_p * pw[f] * acc[q][2 * r + 1] : 0.f;
                        *reinterpret_cast<float2*>(ps + i * S::PP + j) = make_float2(u, v);
                    }
            }
            __syncthreads();
            // outputs
            float acc[NT][4] = {};
#pragma unroll 1
            for (int k = 0; k < p.dx; k += 16) {
                float u[NT][4];
                Two fa[4], fb[NT][2];
                frag_a<S::PX>(fa, xs, 16 * mi, k, g, t);
#pragma unroll
                for (int q = 0; q < NT; ++q) frag_b<S::PZ>(fb[q], ss, k, 8 * (nj + NG * q), g, t);
                mma3<true>(u, fa, fb, tiles);
                frag_a<S::PX>(fa, xs, 16 * mi, k + 8, g, t);
#pragma unroll
                for (int q = 0; q < NT; ++q) frag_b<S::PZ>(fb[q], ss, k + 8, 8 * (nj + NG * q), g, t);
                mma3<false>(u, fa, fb, tiles);
                add(acc, u, tiles);
            }
            const int i0 = 16 * mi + g;
            const float f0 = p.s_i * (rev ? pw[max(L - 1 - i0, 0)] : pw[i0 + 1]),
                        f1 = p.s_i * (rev ? pw[max(L - 9 - i0, 0)] : pw[i0 + 9]);
#pragma unroll
            for (int q = 0; q < NT; ++q) acc[q][0] *= f0, acc[q][1] *= f0, acc[q][2] *= f1, acc[q][3] *= f1;
            const int from = rev ? 16 * mi : 0, to = rev ? kC : 16 * mi + 16;
#pragma unroll 1
            for (int k = from; k < to; k += 16) {
                float u[NT][4];
                Two fa[4], fb[NT][2];
                frag_a<S::PP>(fa, ps, 16 * mi, k, g, t);
#pragma unroll
                for (int q = 0; q < NT; ++q) frag_b<S::PZ>(fb[q], zs, k, 8 * (nj + NG * q), g, t);
                mma3<true>(u, fa, fb, tiles);
                frag_a<S::PP>(fa, ps, 16 * mi, k + 8, g, t);
#pragma unroll
                for (int q = 0; q < NT; ++q) frag_b<S::PZ>(fb[q], zs, k + 8, 8 * (nj + NG * q), g, t);
                mma3<false>(u, fa, fb, tiles);
                add(acc, u, tiles);
            }
#pragma unroll
            for (int q = 0; q < NT; ++q)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int i = i0 + 8 * r, n = 8 * (nj + NG * q) + 2 * t;
                    if (i < L && n < p.dz)
                        *reinterpret_cast<float2*>(out + (t0 + i) * p.so.token + n) =
                            make_float2(acc[q][2 * r], acc[q][2 * r + 1]);
                }
        }
        if (STATES || ch + 1 < nch || (!at.split && p.s_out)) {
            // S <- a^L S + s_u sum_j a^(..) y_j^T z_j
            constexpr int kSteps = FULL ? 2 : 1;  // into one u; with the conditions on tiles beside it, two spill more (496 bytes, one 428)
            const float2 fl = a.decay[h * kLaPowers + L];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int q = 0; q < NT; ++q)
#pragma unroll
                    for (int e = 0; e < 4; ++e) st[m][q][e] = decayed(fl, st[m][q][e], 0.f);
#pragma unroll 1
            for (int k = 0; k < L; k += 8 * kSteps) {  // rows behind the length are zeros
                float u[MT][NT][4];
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
                    const int j = k + 8 * s + t;
                    const float w0 = p.s_u * pw[rev ? j + 1 : max(L - 1 - j, 0)],
                                w1 = p.s_u * pw[rev ? j + 5 : max(L - 5 - j, 0)];
                    Two fb[NT][2];
#pragma unroll
                    for (int q = 0; q < NT; ++q) frag_b<S::PZ>(fb[q], zs, k + 8 * s, 8 * (nj + NG * q), g, t);
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        if (!FULL && 16 * (mi + 4 * m) >= p.dx) break;
                        const float* v = ys + j * S::PX + 16 * (mi + 4 * m) + g;
                        Two fa[4];
                        fa[0] = split(w0 * v[0]), fa[1] = split(w0 * v[8]);
                        fa[2] = split(w1 * v[4 * S::PX]), fa[3] = split(w1 * v[4 * S::PX + 8]);
                        if (s == 0)
                            mma3<true>(u[m], fa, fb, tiles);
                        else
                            mma3<false>(u[m], fa, fb, tiles);
                        if (s + 1 == kSteps) add(st[m], u[m], tiles);
                    }
                }
            }
        }
    }
    float* so = STATES ? wseg : !at.split && p.s_out ? p.s_out + (size_t)bh * p.dx * p.dz : nullptr;
    if (so)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int q = 0; q < NT; ++q)
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const int d = 16 * (mi + 4 * m) + g + 4 * e, n = 8 * (nj + NG * q) + 2 * t;
                    if (d < p.dx && n < p.dz)
                        *reinterpret_cast<float2*>(so + (size_t)d * p.dz + n) = make_float2(st[m][q][e], st[m][q][e + 1]);
                }
    if (!STATES)  // rows behind the sequence
        for (int64_t e = tid; e < (rows - live) * (p.dz / 4); e += kThreads)
            store4(out + (live + e / (p.dz / 4)) * p.so.token + 4 * (e % (p.dz / 4)), make_float4(0.f, 0.f, 0.f, 0.f));
}

// Replaces each segment's own state by the state entering it, in the order the
// pass runs, and writes the last one out; a thread per four elements, the loads
// of eight segments in flight together.
constexpr int kCarryThreads = 128;
__global__ void __launch_bounds__(kCarryThreads) la_carry(const __grid_constant__ Args a, const double* __restrict__ lg) {
    const LaPass& p = a.p[blockIdx.z];
    let_next_start();
    __shared__ float2 decay[kLaMaxSegments];  // over a segment, in two parts; below zero: an empty one
    const int bh = a.whole + blockIdx.y, b = bh / a.H, h = bh % a.H, n = p.dx * p.dz;
    const int64_t len = live_tokens(a, b);
    for (int k = threadIdx.x; k < a.nseg; k += kCarryThreads) {
        const int sg = p.reverse ? a.nseg - 1 - k : k;
        const int64_t live = min(a.seg, len - sg * a.seg);
        // an empty segment passes the state on (also where the decay is zero)
        const double d = live > 0 ? exp(lg[h] * (double)live) : -1.0;
        const float hi = __double2float_rd(d), lo = (float)(d - hi);
        decay[k] = make_float2(hi, hi >= 0x1p-100f ? fmaxf(lo, 0x1p-149f) : lo);  // as the plan's table
    }
    __syncthreads();
    after_previous();
    const int e = 4 * (blockIdx.x * kCarryThreads + threadIdx.x);
    if (e >= n) return;
    float* w = a.work + blockIdx.z * a.pass_floats + (size_t)blockIdx.y * a.nseg * a.state_floats + e;
    const int64_t step = (p.reverse ? -1 : 1) * (int64_t)a.state_floats;
    if (p.reverse) w += (a.nseg - 1) * a.state_floats;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.s_in) {
        const float* q = p.s_in + (size_t)bh * n;
        if (p.in_trans) {
            const int d = e / p.dz, c = e % p.dz;
            s = make_float4(q[c * p.dx + d], q[(c + 1) * p.dx + d], q[(c + 2) * p.dx + d], q[(c + 3) * p.dx + d]);
        } else {
            s = load4(q + e);
        }
    }
    for (int k0 = 0; k0 < a.nseg; k0 += 8) {
        float4 own[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (k0 + i < a.nseg) own[i] = load4(w + (k0 + i) * step);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (k0 + i < a.nseg) {
                const float2 f = decay[k0 + i];
                store4(w + (k0 + i) * step, s);
                if (f.x >= 0.f) {
                    s.x = decayed(f, s.x, own[i].x), s.y = decayed(f, s.y, own[i].y);
                    s.z = decayed(f, s.z, own[i].z), s.w = decayed(f, s.w, own[i].w);
                }
            }
    }
    if (p.s_out) store4(p.s_out + (size_t)bh * n + e, s);
}

cudaError_t launch_carry(const Args& a, int rows, int passes, const double* lg, cudaStream_t s) {
    const unsigned blocks = (unsigned)((a.state_floats / 4 + kCarryThreads - 1) / kCarryThreads);
    return launch<la_carry>(dim3(blocks, rows, passes), kCarryThreads, 0, s, true, a, lg);
}

template <int DX, int DZ, bool FULL>
cudaError_t run(const Args& a, int bh, int passes, bool states, cudaStream_t s) {
    using S = Shape<DX, DZ>;
    constexpr int bytes = S::kFloats * (int)sizeof(float);
    cudaError_t e = states ? allow<la_f32<DX, DZ, true, FULL>>(bytes) : allow<la_f32<DX, DZ, false, FULL>>(bytes);
    if (e != cudaSuccess) return e;
    const int split = (bh - a.whole) * a.nseg * passes;
    Args g = a;
    g.first = states ? a.whole * passes : 0;
    return states ? launch<la_f32<DX, DZ, true, FULL>>(split, S::kThreads, bytes, s, false, g)
                  : launch<la_f32<DX, DZ, false, FULL>>(a.whole * passes + split, S::kThreads, bytes, s, split > 0, g);
}

cudaError_t launch_f32(const Args& a, int dx, int dz, int bh, int passes, bool states, cudaStream_t s) {
    // Tiles behind dx and dz are skipped where there are any: 164 -> 118 us at 40 and 104 (padded to 128), but the
    // conditions cost a fifth where there are none.
    bool full = true;
    for (int i = 0; i < passes; ++i) full = full && a.p[i].dx % 64 == 0 && a.p[i].dz % 64 == 0 && a.p[i].dx == a.p[0].dx;
    auto pick = [&](auto f) {
        constexpr bool F = decltype(f)::value;
        if (dx <= 64)
            return dz <= 64 ? run<64, 64, F>(a, bh, passes, states, s) : run<64, 128, F>(a, bh, passes, states, s);
        return dz <= 64 ? run<128, 64, F>(a, bh, passes, states, s) : run<128, 128, F>(a, bh, passes, states, s);
    };
    return full ? pick(std::true_type{}) : pick(std::false_type{});
}

// one CTA per (row, head), its state in registers between the read and the write
constexpr int kStepThreads = 256;
template <typename T>
__global__ void __launch_bounds__(kStepThreads)
la_step(const LaStep c, int H, int dk, int dv, const float2* __restrict__ decay) {
    __shared__ float sq[128], sk[128], sv[128];
    __shared__ float4 part[kStepThreads];
    const int h = blockIdx.x, tid = threadIdx.x;
    const int b0 = blockIdx.y;
    const int slot = c.slots ? c.slots[b0] : b0;
    const int nv = dv / 4, groups = kStepThreads / nv, col = tid % nv, grp = tid / nv;
    if (slot < 0 || slot >= c.slots_n) {  // idle row
        for (int j = tid; j < dv; j += kStepThreads) ((T*)c.o)[b0 * c.ob + h * c.oh + j] = T(0.f);
        return;
    }
    float4* st = reinterpret_cast<float4*>(c.state + ((size_t)slot * H + h) * dk * dv);
    constexpr int kRows = 16;  // state rows a thread holds at most: dk <= 128 in at least 8 groups (dv <= 128)
    float4 s[kRows];
    if (grp < groups) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int d = grp + i * groups;
            if (d < dk) s[i] = st[d * nv + col];
        }
    }
    // rows that share a slot are taken in row order, by the first of them (the others may have loaded its state while it
    // was being stored, and drop it)
    bool more = false;
    if (c.slots) {
        int before = 0, after = 0;
        for (int b = tid; b < c.B; b += kStepThreads)
            if (b != b0 && c.slots[b] == slot) (b < b0 ? before : after) = 1;
        if (__syncthreads_or(before)) return;
        more = __syncthreads_or(after);
    }
    const float2 a = decay[h * kLaPowers + 1];
    for (int b = b0; b < c.B; ++b) {
        if (b != b0 && c.slots[b] != slot) continue;
        __syncthreads();
        for (int j = tid; j < dk; j += kStepThreads) {
            sq[j] = to_f(((const T*)c.q)[b * c.qb + h * c.qh + j]);
            sk[j] = to_f(((const T*)c.k)[b * c.kb + h * c.kh + j]);
        }
        for (int j = tid; j < dv; j += kStepThreads) sv[j] = to_f(((const T*)c.v)[b * c.vb + h * c.vh + j]);
        __syncthreads();
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        if (grp < groups) {
            const float4 v = *reinterpret_cast<float4*>(sv + 4 * col);
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int d = grp + i * groups;
                if (d < dk) {
                    const float k = sk[d], q = sq[d];
                    s[i].x = decayed(a, s[i].x, k * v.x), s[i].y = decayed(a, s[i].y, k * v.y);
                    s[i].z = decayed(a, s[i].z, k * v.z), s[i].w = decayed(a, s[i].w, k * v.w);
                    o.x = fmaf(q, s[i].x, o.x), o.y = fmaf(q, s[i].y, o.y);
                    o.z = fmaf(q, s[i].z, o.z), o.w = fmaf(q, s[i].w, o.w);
                }
            }
        }
        part[tid] = o;
        __syncthreads();
        if (tid < nv) {
            float4 t = part[tid];
            for (int g = 1; g < groups; ++g) {
                const float4 u = part[g * nv + tid];
                t.x += u.x, t.y += u.y, t.z += u.z, t.w += u.w;
            }
            T* o_ = (T*)c.o + b * c.ob + h * c.oh + 4 * tid;
            o_[0] = T(c.scale * t.x), o_[1] = T(c.scale * t.y), o_[2] = T(c.scale * t.z), o_[3] = T(c.scale * t.w);
        }
        if (!more) break;
    }
    if (grp < groups) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int d = grp + i * groups;
            if (d < dk) st[d * nv + col] = s[i];
        }
    }
}

}  // namespace la

namespace {

// dk and dv padded to one shape for every pass of the call
void padded(const fftconv_linattn_s& p, int passes, int* dx, int* dz) {
    *dx = passes == 1 ? p.dk : (p.dk > p.dv ? p.dk : p.dv);
    *dz = passes == 1 ? p.dv : *dx;
}

int chunk_of(const fftconv_linattn_s& p) { return p.dtype == FFTCONV_BF16 ? kLaChunkTc : kLaChunk; }

// CTAs the GPU holds at once: two an SM where both dims fit 64
int64_t slots_of(const fftconv_linattn_s& p, int passes) {
    int dx, dz;
    padded(p, passes, &dx, &dz);
    return (int64_t)p.sms * (dx <= 64 && dz <= 64 ? 2 : 1);
}

// How a call is cut: rows (b, h) in front that run whole, and the segments that
// the token axis of the others is cut into.  In units of one chunk's time, a CTA
// costs its chunks and about 1.5 to start; segments add the pass over their own
// states (two tensors of four: about 0.6 a chunk) and the launch that joins them.
// Rows run whole as long as they fill the GPU; segments spread what is left over
// it, or everything where there are few rows.  Of a padded fp32 batch some 9/16 of
// the segments have tokens (lengths spread evenly, one of them full): shorter ones
// fill the SMs that the others leave (3 x 5 x 1023 at 40 and 104: 179 us with 3
// segments, 121 with 4; in bf16, where a segment's start weighs more, 8 x 12 x 4096
// took 91 us with 5 segments and 79 with 3).
struct Cut {
    int whole, nseg;
};
Cut cut_of(const fftconv_linattn_s& p, int B, int64_t N, int passes, bool padded) {
    const int64_t chunks = (N + chunk_of(p) - 1) / chunk_of(p), rows = (int64_t)B * p.H, slots = slots_of(p, passes);
    const int64_t full = rows * passes / slots * slots / passes;  // rows in whole waves
    auto waves = [&](int64_t ctas) { return (double)((ctas + slots - 1) / slots); };
    Cut best{(int)rows, 1};
    double least = waves(rows * passes) * (chunks + 1.5);
    for (int64_t n = 2; n <= kLaMaxSegments && n <= chunks; ++n) {
        const int64_t per = (chunks + n - 1) / n;
        if ((chunks + per - 1) / per != n) continue;  // an empty segment
        for (int64_t whole : {(int64_t)0, full}) {
            const int64_t ctas = (rows - whole) * passes * n;
            if (ctas == 0 || ctas > kLaMaxWaves * slots) continue;
            const int64_t busy = padded && p.dtype == FFTCONV_F32 ? (ctas * 9 + 15) / 16 : ctas;
            const double cost = waves(whole * passes) * (chunks + 1.5) + waves(busy) * (per + 1.5 + 0.6 * per + 1.0) + 3.0;
            if (cost < least) {
                best = {(int)whole, (int)n};
                least = cost;
            }
        }
    }
    return best;
}

}  // namespace

size_t la_workspace_floats(const fftconv_linattn_s& p, int passes) {
    // enough for every B and N up to the plan's: segments times CTAs is bounded above, one segment needs none
    const int64_t chunks = (p.N + chunk_of(p) - 1) / chunk_of(p), cap = kLaMaxWaves * slots_of(p, passes);
    if (chunks == 1) return 0;
    const int64_t most = (int64_t)p.B * p.H * passes * (chunks < kLaMaxSegments ? chunks : kLaMaxSegments);
    return (size_t)(most < cap ? most : cap) * p.dk * p.dv;
}

cudaError_t launch_la(const fftconv_linattn_s& p, const LaCall& c, cudaStream_t s) {
    const int64_t chunk = chunk_of(p), chunks = (c.N + chunk - 1) / chunk;
    const bool tc = p.dtype == FFTCONV_BF16;
    la::Args a;
    a.H = p.H;
    a.passes = c.passes;
    const int bh = c.B * p.H;
    const Cut cut = cut_of(p, c.B, c.N, c.passes, c.lengths != nullptr);
    a.whole = cut.whole;
    a.nseg = cut.nseg;
    a.first = 0;
    a.seg = (chunks + a.nseg - 1) / a.nseg * chunk;
    a.N = c.N;
    a.lengths = c.lengths;
    a.pw = p.d_pow;
    a.decay = p.d_decay;
    a.work = c.work;
    a.state_floats = (size_t)p.dk * p.dv;
    a.pass_floats = (size_t)(bh - a.whole) * a.nseg * a.state_floats;
    bool ends = false;
    for (int i = 0; i < c.passes; ++i) {
        a.p[i] = c.pass[i];
        ends = ends || a.p[i].s_out;
    }
    int dx, dz;
    padded(p, c.passes, &dx, &dz);
    if (tc) return la::launch_tc(a, dx, dz, c.B, c.passes, ends, p, s);
    cudaError_t e = cudaSuccess;
    if (bh > a.whole) {
        e = la::launch_f32(a, dx, dz, bh, c.passes, true, s);
        if (e == cudaSuccess) e = la::launch_carry(a, bh - a.whole, c.passes, p.d_log, s);
    }
    return e == cudaSuccess ? la::launch_f32(a, dx, dz, bh, c.passes, false, s) : e;
}

cudaError_t launch_la_step(const fftconv_linattn_s& p, const LaStep& c, cudaStream_t s) {
    const dim3 grid(p.H, c.B);
    if (p.dtype == FFTCONV_BF16)
        la::la_step<__nv_bfloat16><<<grid, la::kStepThreads, 0, s>>>(c, p.H, p.dk, p.dv, p.d_decay);
    else
        la::la_step<float><<<grid, la::kStepThreads, 0, s>>>(c, p.H, p.dk, p.dv, p.d_decay);
    return cudaGetLastError();
}

}  // namespace fftc
