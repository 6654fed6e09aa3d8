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
// bf16 runs on the tensor cores (linattn_tc.cu), fp32 here.  The token axis is cut into segments where one CTA per (row, head) would leave
// SMs idle: a first kernel sums each segment's own contribution to the state, a
// second carries the states over the segments, the third computes the outputs.
#include <cuda_bf16.h>
#include <math.h>

#include "linattn.cuh"

namespace fftc {
namespace la {

constexpr int kC = kLaChunk;
constexpr int kThreads = 256;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }

template <int DX, int DZ>
struct Shape {
    static constexpr int PX = DX + 4, PZ = DZ + 4, PP = kC + 4;  // row pitches (floats)
    static constexpr int kFloats = 2 * kC * PX + kC * PZ + kC * PP + DX * PZ + 132;
};

// rows [t0, t0 + kC) of a tensor into shared memory as fp32, zeros behind row `live` and column d
template <int D, int P>
__device__ __forceinline__ void load_tile(float* dst, const float* src, int64_t stride, int live, int d) {
    for (int e = threadIdx.x; e < kC * (D / 4); e += kThreads) {
        const int r = e / (D / 4), c = 4 * (e % (D / 4));
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < live && c < d) v = load4(src + r * stride + c);
        *reinterpret_cast<float4*>(dst + r * P + c) = v;
    }
}

// grid (segments, rows x heads, passes); STATES: only the segments' own states
template <int DX, int DZ, bool STATES>
__global__ void __launch_bounds__(kThreads) la_simt(const __grid_constant__ Args a) {
    using S = Shape<DX, DZ>;
    extern __shared__ __align__(16) float sm[];
    float *xs = sm, *ys = xs + kC * S::PX, *zs = ys + kC * S::PX, *ps = zs + kC * S::PZ, *ss = ps + kC * S::PP,
          *pw = ss + DX * S::PZ;
    const LaPass& p = a.p[blockIdx.z];
    const int tid = threadIdx.x, sg = blockIdx.x, bh = blockIdx.y, b = bh / a.H, h = bh % a.H;
    const int ti = tid / 16, tj = tid % 16;
    const int64_t first = sg * a.seg, len = live_tokens(a, b);
    const int64_t rows = min(a.seg, a.N - first);                   // output rows of this segment
    const int64_t live = max((int64_t)0, min(rows, len - first));   // of which read
    const float* x = (const float*)p.x + b * p.sx.batch + h * p.sx.head + first * p.sx.token;
    const float* y = (const float*)p.y + b * p.sy.batch + h * p.sy.head + first * p.sy.token;
    const float* z = (const float*)p.z + b * p.sz.batch + h * p.sz.head + first * p.sz.token;
    float* out = (float*)p.out + b * p.so.batch + h * p.so.head + first * p.so.token;
    float* wseg = a.work + blockIdx.z * a.pass_floats + ((size_t)bh * a.nseg + sg) * a.state_floats;
    for (int i = tid; i < kLaPowers; i += kThreads) pw[i] = a.pw[h * kLaPowers + i];
    // the state entering the segment
    const float* s0 = STATES ? nullptr : p.carried ? wseg : p.s_in ? p.s_in + (size_t)bh * p.dx * p.dz : nullptr;
    const bool trans = !p.carried && p.in_trans;
    for (int e = tid; e < DX * DZ; e += kThreads) {
        const int d = e / DZ, n = e % DZ;
        ss[d * S::PZ + n] = s0 && d < p.dx && n < p.dz ? s0[trans ? n * p.dx + d : d * p.dz + n] : 0.f;
    }
    const int nch = (int)((live + kC - 1) / kC);
    for (int ch = 0; ch < nch; ++ch) {
        const int64_t t0 = (int64_t)(p.reverse ? nch - 1 - ch : ch) * kC;
        const int L = (int)min((int64_t)kC, live - t0);
        __syncthreads();
        if (!STATES) load_tile<DX, S::PX>(xs, x + t0 * p.sx.token, p.sx.token, L, p.dx);
        load_tile<DX, S::PX>(ys, y + t0 * p.sy.token, p.sy.token, L, p.dx);
        load_tile<DZ, S::PZ>(zs, z + t0 * p.sz.token, p.sz.token, L, p.dz);
        __syncthreads();
        if (!STATES) {
            float acc[4][4] = {};
            for (int d = 0; d < DX; d += 4) {
                float4 u[4], v[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    u[r] = *reinterpret_cast<float4*>(xs + (ti + 16 * r) * S::PX + d);
                    v[r] = *reinterpret_cast<float4*>(ys + (tj + 16 * r) * S::PX + d);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        acc[r][c] += u[r].x * v[c].x + u[r].y * v[c].y + u[r].z * v[c].z + u[r].w * v[c].w;
            }
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int i = ti + 16 * r, j = tj + 16 * c, e = p.reverse ? j - i : i - j;
                    ps[i * S::PP + j] = e >= 0 ? p.s_p * pw[e] * acc[r][c] : 0.f;
                }
            __syncthreads();
#pragma unroll
            for (int m = 0; m < DZ / 64; ++m) {
                const int n = 4 * tj + 64 * m;
                float4 o[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) o[r] = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int d = 0; d < DX; d += 4) {
                    float4 sv[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) sv[q] = *reinterpret_cast<float4*>(ss + (d + q) * S::PZ + n);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float4 u = *reinterpret_cast<float4*>(xs + (ti + 16 * r) * S::PX + d);
                        o[r].x += u.x * sv[0].x + u.y * sv[1].x + u.z * sv[2].x + u.w * sv[3].x;
                        o[r].y += u.x * sv[0].y + u.y * sv[1].y + u.z * sv[2].y + u.w * sv[3].y;
                        o[r].z += u.x * sv[0].z + u.y * sv[1].z + u.z * sv[2].z + u.w * sv[3].z;
                        o[r].w += u.x * sv[0].w + u.y * sv[1].w + u.z * sv[2].w + u.w * sv[3].w;
                    }
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i = ti + 16 * r;
                    const float f = p.s_i * (p.reverse ? pw[max(L - 1 - i, 0)] : pw[i + 1]);
                    o[r].x *= f, o[r].y *= f, o[r].z *= f, o[r].w *= f;
                }
                for (int j = 0; j < kC; j += 4) {
                    float4 zv[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) zv[q] = *reinterpret_cast<float4*>(zs + (j + q) * S::PZ + n);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float4 u = *reinterpret_cast<float4*>(ps + (ti + 16 * r) * S::PP + j);
                        o[r].x += u.x * zv[0].x + u.y * zv[1].x + u.z * zv[2].x + u.w * zv[3].x;
                        o[r].y += u.x * zv[0].y + u.y * zv[1].y + u.z * zv[2].y + u.w * zv[3].y;
                        o[r].z += u.x * zv[0].z + u.y * zv[1].z + u.z * zv[2].z + u.w * zv[3].z;
                        o[r].w += u.x * zv[0].w + u.y * zv[1].w + u.z * zv[2].w + u.w * zv[3].w;
                    }
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i = ti + 16 * r;
                    if (i < L && n < p.dz) store4(out + (t0 + i) * p.so.token + n, o[r]);
                }
            }
            __syncthreads();
        }
        // S <- a^L S + s_u sum_j a^(..) y_j^T z_j
        const float fl = pw[L];
#pragma unroll
        for (int m = 0; m < DZ / 64; ++m) {
            const int n = 4 * tj + 64 * m;
            float4 acc[DX / 16];
#pragma unroll
            for (int r = 0; r < DX / 16; ++r) {
                acc[r] = *reinterpret_cast<float4*>(ss + (ti + 16 * r) * S::PZ + n);
                acc[r].x *= fl, acc[r].y *= fl, acc[r].z *= fl, acc[r].w *= fl;
            }
            for (int j = 0; j < L; ++j) {
                const float w = p.s_u * pw[p.reverse ? j + 1 : L - 1 - j];
                const float4 zv = *reinterpret_cast<float4*>(zs + j * S::PZ + n);
#pragma unroll
                for (int r = 0; r < DX / 16; ++r) {
                    const float u = w * ys[j * S::PX + ti + 16 * r];
                    acc[r].x += u * zv.x, acc[r].y += u * zv.y, acc[r].z += u * zv.z, acc[r].w += u * zv.w;
                }
            }
#pragma unroll
            for (int r = 0; r < DX / 16; ++r) *reinterpret_cast<float4*>(ss + (ti + 16 * r) * S::PZ + n) = acc[r];
        }
    }
    __syncthreads();
    float* so = STATES ? wseg : !p.carried && p.s_out ? p.s_out + (size_t)bh * p.dx * p.dz : nullptr;
    if (so)
        for (int e = tid; e < p.dx * p.dz; e += kThreads) so[e] = ss[(e / p.dz) * S::PZ + e % p.dz];
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
    if (!p.carried) return;
    __shared__ float decay[kLaMaxSegments];  // over a segment; below zero: an empty one
    const int bh = blockIdx.y, b = bh / a.H, h = bh % a.H, n = p.dx * p.dz;
    const int64_t len = live_tokens(a, b);
    for (int k = threadIdx.x; k < a.nseg; k += kCarryThreads) {
        const int sg = p.reverse ? a.nseg - 1 - k : k;
        const int64_t live = min(a.seg, len - sg * a.seg);
        // an empty segment passes the state on (also where the decay is zero)
        decay[k] = live > 0 ? (float)exp(lg[h] * (double)live) : -1.f;
    }
    __syncthreads();
    const int e = 4 * (blockIdx.x * kCarryThreads + threadIdx.x);
    if (e >= n) return;
    float* w = a.work + blockIdx.z * a.pass_floats + (size_t)bh * a.nseg * a.state_floats + e;
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
                const float f = decay[k0 + i];
                store4(w + (k0 + i) * step, s);
                if (f >= 0.f) {
                    s.x = fmaf(f, s.x, own[i].x), s.y = fmaf(f, s.y, own[i].y);
                    s.z = fmaf(f, s.z, own[i].z), s.w = fmaf(f, s.w, own[i].w);
                }
            }
    }
    if (p.s_out) store4(p.s_out + (size_t)bh * n + e, s);
}

template <int DX, int DZ>
cudaError_t run(const Args& a, int bh, int passes, bool states, cudaStream_t s) {
    constexpr int bytes = Shape<DX, DZ>::kFloats * (int)sizeof(float);
    const cudaError_t e = states ? allow<la_simt<DX, DZ, true>>(bytes) : allow<la_simt<DX, DZ, false>>(bytes);
    if (e != cudaSuccess) return e;
    const dim3 grid(a.nseg, bh, passes);
    if (states)
        la_simt<DX, DZ, true><<<grid, kThreads, bytes, s>>>(a);
    else
        la_simt<DX, DZ, false><<<grid, kThreads, bytes, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_simt(const Args& a, int dx, int dz, int bh, int passes, bool states, cudaStream_t s) {
    if (dx <= 64)
        return dz <= 64 ? run<64, 64>(a, bh, passes, states, s) : run<64, 128>(a, bh, passes, states, s);
    return dz <= 64 ? run<128, 64>(a, bh, passes, states, s) : run<128, 128>(a, bh, passes, states, s);
}

// one CTA per (row, head), its state in registers between the read and the write
constexpr int kStepThreads = 256;
template <typename T>
__global__ void __launch_bounds__(kStepThreads)
la_step(const LaStep c, int H, int dk, int dv, const float* __restrict__ pw) {
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
    // rows that share a slot are taken in row order, by the first of them
    bool more = false;
    if (c.slots) {
        int before = 0, after = 0;
        for (int b = tid; b < c.B; b += kStepThreads)
            if (b != b0 && c.slots[b] == slot) (b < b0 ? before : after) = 1;
        if (__syncthreads_or(before)) return;
        more = __syncthreads_or(after);
    }
    const float a = pw[h * kLaPowers + 1];
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
                    s[i].x = fmaf(a, s[i].x, k * v.x), s[i].y = fmaf(a, s[i].y, k * v.y);
                    s[i].z = fmaf(a, s[i].z, k * v.z), s[i].w = fmaf(a, s[i].w, k * v.w);
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

// Segments the token axis is cut into.  In units of one chunk's time, a CTA
// costs its chunks and about 1.5 to start; more than one segment adds the pass
// over the segments' own states (two tensors of four: about 0.6 a chunk) and
// the launch that joins them.
int segments(const fftconv_linattn_s& p, int B, int64_t N, int passes) {
    const int64_t chunks = (N + chunk_of(p) - 1) / chunk_of(p), ctas = (int64_t)B * p.H * passes;
    const int64_t slots = slots_of(p, passes);
    int best = 1;
    double least = 0.0;
    for (int n = 1; n <= kLaMaxSegments && n <= chunks && (n == 1 || ctas * n <= kLaMaxWaves * slots); ++n) {
        const int64_t per = (chunks + n - 1) / n, waves = (ctas * n + slots - 1) / slots;
        if (n > 1 && (chunks + per - 1) / per != n) continue;  // an empty segment
        const double cost = waves * (per + 1.5) + (n > 1 ? waves * (0.6 * per + 1.0) + 3.0 : 0.0);
        if (n == 1 || cost < least) {
            best = n;
            least = cost;
        }
    }
    return best;
}

}  // namespace

size_t la_workspace_floats(const fftconv_linattn_s& p, int passes) {
    // enough for every B and N up to the plan's: one state a CTA, and the bound on segments times CTAs
    const int64_t chunks = (p.N + chunk_of(p) - 1) / chunk_of(p), ctas = (int64_t)p.B * p.H * passes;
    const int64_t most = ctas * (chunks < kLaMaxSegments ? chunks : kLaMaxSegments), cap = kLaMaxWaves * slots_of(p, passes);
    const int64_t states = most < cap ? most : cap > ctas ? cap : ctas;
    return (size_t)states * p.dk * p.dv;
}

cudaError_t launch_la(const fftconv_linattn_s& p, const LaCall& c, cudaStream_t s) {
    const int64_t chunk = chunk_of(p), chunks = (c.N + chunk - 1) / chunk;
    const bool tc = p.dtype == FFTCONV_BF16;
    la::Args a;
    a.H = p.H;
    a.nseg = segments(p, c.B, c.N, c.passes);
    a.seg = (chunks + a.nseg - 1) / a.nseg * chunk;
    a.N = c.N;
    a.lengths = c.lengths;
    a.pw = p.d_pow;
    a.work = c.work;
    a.state_floats = (size_t)p.dk * p.dv;
    a.pass_floats = (size_t)c.B * p.H * a.nseg * a.state_floats;
    bool carried = false;
    for (int i = 0; i < c.passes; ++i) {
        a.p[i] = c.pass[i];
        // the tensor-core outputs' kernel keeps its state for the outputs alone: states that a caller
        // asks for come from the states' kernel, which sums them in fp32
        a.p[i].carried = a.nseg > 1 || (tc && a.p[i].s_out);
        carried = carried || a.p[i].carried;
    }
    int dx, dz;
    padded(p, c.passes, &dx, &dz);
    const int bh = c.B * p.H;
    cudaError_t e;
    if (carried) {
        e = tc ? la::launch_tc(a, dx, dz, c.B, c.passes, true, p, s) : la::launch_simt(a, dx, dz, bh, c.passes, true, s);
        if (e != cudaSuccess) return e;
        const unsigned blocks = (unsigned)((a.state_floats / 4 + la::kCarryThreads - 1) / la::kCarryThreads);
        la::la_carry<<<dim3(blocks, bh, c.passes), la::kCarryThreads, 0, s>>>(a, p.d_log);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    return tc ? la::launch_tc(a, dx, dz, c.B, c.passes, false, p, s) : la::launch_simt(a, dx, dz, bh, c.passes, false, s);
}

cudaError_t launch_la_step(const fftconv_linattn_s& p, const LaStep& c, cudaStream_t s) {
    const dim3 grid(p.H, c.B);
    if (p.dtype == FFTCONV_BF16)
        la::la_step<__nv_bfloat16><<<grid, la::kStepThreads, 0, s>>>(c, p.H, p.dk, p.dv, p.d_pow);
    else
        la::la_step<float><<<grid, la::kStepThreads, 0, s>>>(c, p.H, p.dk, p.dv, p.d_pow);
    return cudaGetLastError();
}

}  // namespace fftc
