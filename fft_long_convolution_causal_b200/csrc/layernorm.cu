// layernorm.cu -- layer norm over the last dimension, forward and backward:
//   y = (x - mu) rstd w + b
//   dx = rstd (g - mean(g) - xh mean(g xh)),  g = dy w,  xh = (x - mu) rstd
//   dw = sum over rows of dy xh,  db = sum over rows of dy
// Row r uses weight row r mod G (G = 1: one weight for all; G = heads: the norm
// behind each head).
//
// Bound by memory.  A row is read once into registers (mean first, then the sum
// of centred squares: no cancellation) by TPR threads, each holding E pieces of
// 16 bytes (or single elements where rows are not 16-byte aligned).  The weight
// gradient is summed over the rows a block walks in registers, then over blocks
// by a second kernel in a fixed order: repeated calls agree bit for bit.
// 32768 x 768 bf16: forward 22.9 us (4.4 TB/s of x and y), backward 35.3 us
// (4.3 TB/s of dy, x and dx), the launches' ramps included; 49152 x 64 fp32
// forward 9.4 us, 17 x 2708 both ways 31 us, which is the host's time.
#include <cuda_bf16.h>

#include "linattn.cuh"
#include "mixer.h"
#include "pairs.cuh"

namespace fftc {
namespace ln {

// threads of a block: rows on several warps have one row a block
template <int TPR, int N>
__host__ __device__ constexpr int block_threads() {
    return TPR > 32 ? TPR : N;
}

// sum over the TPR threads of a row
template <int TPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (TPR > 32) {
        __shared__ float part[TPR / 32];
        __syncthreads();  // the previous sum has been read
        if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int i = 0; i < TPR / 32; ++i) v += part[i];
    }
    return v;
}

template <typename T, int V, int TPR, int E>
__global__ void __launch_bounds__((block_threads<TPR, 256>()))
norm_fwd(const T* x, const float* __restrict__ w, const float* __restrict__ bias, T* y, float* __restrict__ mean,
         float* __restrict__ rstd, int64_t rows, int C, int G, float eps) {
    using P = Piece<T, V>;
    using W = Piece<float, V>;
    constexpr int kRows = block_threads<TPR, 256>() / TPR;
    const int lane = threadIdx.x % TPR, items = C / V;
    const int64_t step = (int64_t)gridDim.x * kRows;
    constexpr int NP = P::kPairs;
    const float inv = 1.f / (float)C;
    P p[E];
    auto fetch = [&](int64_t r) {
        if (r >= rows) return;
        const P* xr = reinterpret_cast<const P*>(x + r * C);
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (lane + i * TPR < items) p[i] = xr[lane + i * TPR];
    };
    int64_t r = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
    fetch(r);
    for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < rows; r0 += step, r += step) {
        const bool on = r < rows;
        float2 v[E][NP], s = both(0.f);
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (lane + i * TPR < items && on) {
#pragma unroll
                for (int j = 0; j < NP; ++j) s = add2(s, v[i][j] = p[i].get(j));
            }
        fetch(r + step);  // in flight while this row is worked on
        const float mu = row_sum<TPR>(s.x + s.y) * inv;
        s = both(0.f);
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (lane + i * TPR < items && on) {
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    v[i][j] = add2(v[i][j], make_float2(-mu, V > 1 ? -mu : 0.f));
                    s = fma2(v[i][j], v[i][j], s);
                }
            }
        const float rs = 1.f / sqrtf(row_sum<TPR>(s.x + s.y) * inv + eps);
        if (on) {
            const int64_t g = G == 1 ? 0 : r % G;
            const W* wr = reinterpret_cast<const W*>(w + g * C);
            const W* br = reinterpret_cast<const W*>(bias + g * C);
            P* yr = reinterpret_cast<P*>(y + r * C);
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int c = lane + i * TPR;
                if (c < items) {
                    const W wv = wr[c], bv = br[c];
                    P o;
#pragma unroll
                    for (int j = 0; j < NP; ++j) o.set(j, fma2(mul2(v[i][j], both(rs)), wv.get(j), bv.get(j)));
                    yr[c] = o;
                }
            }
            if (lane == 0) {
                if (mean) mean[r] = mu;
                if (rstd) rstd[r] = rs;
            }
        }
    }
}

// The backward pass holds two rows of weight-gradient sums, a row and the next one's loads in registers: 12 warps of
// up to 170 registers an SM (at 128 registers and 16 warps it spilled, and 32768 x 768 took 98 us instead of 29).
constexpr int kBwdThreads = 384;

// Blocks blockIdx.x of group blockIdx.y walk the group's rows, the next row's loads in flight while a row is worked on;
// partial sums of the weight gradients to part[(group * blocks + block)][2][C].
template <typename T, int V, int TPR, int E>
__global__ void __launch_bounds__((block_threads<TPR, kBwdThreads>()), 1)
norm_bwd(const T* dy, const T* x, const float* __restrict__ w, const float* __restrict__ mean,
         const float* __restrict__ rstd, T* dx, float* __restrict__ part, int64_t rows, int C, int G) {
    using P = Piece<T, V>;
    using W = Piece<float, V>;
    constexpr int kThreads = block_threads<TPR, kBwdThreads>(), kRows = kThreads / TPR;
    const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR, items = C / V, g = blockIdx.y;
    const int64_t group_rows = rows / G, step = (int64_t)gridDim.x * kRows;
    const float inv = 1.f / (float)C;
    constexpr int NP = P::kPairs;
    float2 dw[E][NP], db[E][NP];
#pragma unroll
    for (int i = 0; i < E; ++i)
#pragma unroll
        for (int j = 0; j < NP; ++j) dw[i][j] = db[i][j] = both(0.f);
    const W* wr = reinterpret_cast<const W*>(w + (int64_t)g * C);
    struct Row {
        P x[E], d[E];
        float mu, rs;
    };
    auto fetch = [&](Row& q, int64_t k) {
        if (k >= group_rows) return;
        const int64_t r = k * G + g;
        const P* xr = reinterpret_cast<const P*>(x + r * C);
        const P* dr = reinterpret_cast<const P*>(dy + r * C);
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (lane + i * TPR < items) {
                q.x[i] = xr[lane + i * TPR];
                q.d[i] = dr[lane + i * TPR];
            }
        q.mu = mean[r];
        q.rs = rstd[r];
    };
    constexpr bool kAhead = E * V <= 24;  // where the registers allow it
    Row row;
    if (kAhead) fetch(row, (int64_t)blockIdx.x * kRows + sub);
    for (int64_t k0 = (int64_t)blockIdx.x * kRows; k0 < group_rows; k0 += step) {
        const int64_t k = k0 + sub;
        const bool on = k < group_rows;
        Row next;
        if (kAhead)
            fetch(next, k + step);
        else
            fetch(row, k);
        float2 s1 = both(0.f), s2 = both(0.f);
        const float2 rs = both(row.rs), shift = make_float2(-row.mu, V > 1 ? -row.mu : 0.f);
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (lane + i * TPR < items && on) {
                const W wv = wr[lane + i * TPR];
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    const float2 d = row.d[i].get(j), xh = mul2(add2(row.x[i].get(j), shift), rs), gv = mul2(d, wv.get(j));
                    dw[i][j] = fma2(d, xh, dw[i][j]);
                    db[i][j] = add2(db[i][j], d);
                    s1 = add2(s1, gv);
                    s2 = fma2(gv, xh, s2);
                }
            }
        const float m1 = row_sum<TPR>(s1.x + s1.y) * inv, m2 = row_sum<TPR>(s2.x + s2.y) * inv;
        if (on) {
            P* o = reinterpret_cast<P*>(dx + (k * G + g) * C);
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (lane + i * TPR < items) {
                    const W wv = wr[lane + i * TPR];
                    P q;
#pragma unroll
                    for (int j = 0; j < NP; ++j) {
                        const float2 xh = mul2(add2(row.x[i].get(j), shift), rs);
                        const float2 c = fma2(row.d[i].get(j), wv.get(j), both(-m1));
                        q.set(j, mul2(rs, fma2(xh, both(-m2), c)));
                    }
                    o[lane + i * TPR] = q;
                }
        }
        if (kAhead) row = next;
    }
    la::let_next_start();
    // over the block's rows, then out
    float* out = part + ((int64_t)g * gridDim.x + blockIdx.x) * 2 * C;
    if constexpr (kRows > 1) {
        __shared__ float red[kRows][TPR * E * V];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < E; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float2 u = q ? db[i][j / 2] : dw[i][j / 2];
                    red[sub][(i * V + j) * TPR + lane] = j & 1 ? u.y : u.x;
                }
            __syncthreads();
            for (int e = threadIdx.x; e < TPR * E * V; e += kThreads) {
                const int l = e % TPR, j = e / TPR % V, i = e / TPR / V, c = l + i * TPR;
                if (c < items) {
                    float v = 0.f;
#pragma unroll
                    for (int k = 0; k < kRows; ++k) v += red[k][e];
                    out[q * C + c * V + j] = v;
                }
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int c = lane + i * TPR;
            if (c < items)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    out[c * V + j] = j & 1 ? dw[i][j / 2].y : dw[i][j / 2].x;
                    out[C + c * V + j] = j & 1 ? db[i][j / 2].y : db[i][j / 2].x;
                }
        }
    }
}

// dw, db [G][C] from the blocks' partial sums: 32 columns x 32 threads a block, in a fixed order
__global__ void __launch_bounds__(1024) norm_reduce(const float* __restrict__ part, float* __restrict__ dw,
                                                    float* __restrict__ db, int blocks, int C) {
    __shared__ float2 red[32][32];
    const int l = threadIdx.x % 32, c = blockIdx.x * 32 + l, k0 = threadIdx.x / 32, g = blockIdx.y;
    float2 s = make_float2(0.f, 0.f);
    la::after_previous();
    if (c < C)
#pragma unroll 4
        for (int k = k0; k < blocks; k += 32) {
            const float* p = part + ((int64_t)g * blocks + k) * 2 * C + c;
            s.x += p[0];
            s.y += p[C];
        }
    red[k0][l] = s;
    __syncthreads();
    if (k0 == 0 && c < C) {
#pragma unroll 8
        for (int k = 1; k < 32; ++k) {
            s.x += red[k][l].x;
            s.y += red[k][l].y;
        }
        dw[(int64_t)g * C + c] = s.x;
        db[(int64_t)g * C + c] = s.y;
    }
}

struct FwdArgs {
    const void* x;
    const float *w, *b;
    void* y;
    float *mean, *rstd;
    int64_t rows;
    int C, G;
    float eps;
    int sms;
};
struct BwdArgs {
    const void *dy, *x;
    const float *w, *mean, *rstd;
    void* dx;
    float* part;
    int64_t rows;
    int C, G, blocks;
};

template <typename T, int V, int TPR, int E>
cudaError_t fwd(const FwdArgs& a, cudaStream_t s) {
    constexpr int kThreads = block_threads<TPR, 256>(), kRows = kThreads / TPR;
    // the blocks that the SMs hold at once, each walking rows
    static const int held = [] {
        int n = 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, norm_fwd<T, V, TPR, E>, kThreads, 0) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
        return n > 0 ? n : 1;
    }();
    const int64_t blocks = (a.rows + kRows - 1) / kRows, most = (int64_t)a.sms * held;
    norm_fwd<T, V, TPR, E><<<(unsigned)(blocks < most ? blocks : most), kThreads, 0, s>>>(
        (const T*)a.x, a.w, a.b, (T*)a.y, a.mean, a.rstd, a.rows, a.C, a.G, a.eps);
    return cudaGetLastError();
}
template <typename T, int V, int TPR, int E>
cudaError_t bwd(const BwdArgs& a, cudaStream_t s) {
    norm_bwd<T, V, TPR, E><<<dim3(a.blocks, a.G), block_threads<TPR, kBwdThreads>(), 0, s>>>(
        (const T*)a.dy, (const T*)a.x, a.w, a.mean, a.rstd, (T*)a.dx, a.part, a.rows, a.C, a.G);
    return cudaGetLastError();
}

// threads and pieces a row, by its pieces: the fewest threads that hold a row in few registers
template <typename T, int V, typename F>
cudaError_t by_items(int items, F f) {
    if constexpr (V > 1) {
        if (items <= 8) return f.template operator()<T, V, 8, 1>();
        if (items <= 16) return f.template operator()<T, V, 16, 1>();
        if (items <= 32) return f.template operator()<T, V, 32, 1>();
        if (items <= 64) return f.template operator()<T, V, 32, 2>();
        if (items <= 96) return f.template operator()<T, V, 32, 3>();
        if (items <= 128) return f.template operator()<T, V, 32, 4>();
        if (items <= 256) return f.template operator()<T, V, 128, 2>();
        if (items <= 512) return f.template operator()<T, V, 128, 4>();
        if (items <= 1024) return f.template operator()<T, V, 512, 2>();
        if (items <= 2048) return f.template operator()<T, V, 512, 4>();
        return f.template operator()<T, V, 512, 8>();
    } else {
        if (items <= 256) return f.template operator()<T, 1, 32, 8>();
        if (items <= 1024) return f.template operator()<T, 1, 128, 8>();
        if (items <= 4096) return f.template operator()<T, 1, 512, 8>();
        return f.template operator()<T, 1, 512, 32>();
    }
}
struct FwdPick {
    const FwdArgs& a;
    cudaStream_t s;
    template <typename T, int V, int TPR, int E>
    cudaError_t operator()() {
        return fwd<T, V, TPR, E>(a, s);
    }
};
struct BwdPick {
    const BwdArgs& a;
    cudaStream_t s;
    template <typename T, int V, int TPR, int E>
    cudaError_t operator()() {
        return bwd<T, V, TPR, E>(a, s);
    }
};
template <typename T, typename F>
cudaError_t pick(int C, F f) {
    constexpr int V = 16 / sizeof(T);
    return C % V == 0 ? by_items<T, V>(C / V, f) : by_items<T, 1>(C, f);
}

// blocks a group of the backward pass: one an SM in all, no more than rows
inline int bwd_blocks(const fftconv_norm_s& p, int64_t rows) {
    int64_t n = ((int64_t)p.sms + p.groups - 1) / p.groups;
    const int64_t most = rows / p.groups;
    n = n < most ? n : most;
    return (int)(n < 1 ? 1 : n);
}

}  // namespace ln

cudaError_t launch_norm_fwd(const fftconv_norm_s& p, int64_t rows, const void* x, const float* w, const float* b,
                            void* y, float* mean, float* rstd, cudaStream_t s) {
    const ln::FwdArgs a{x, w, b, y, mean, rstd, rows, p.C, p.groups, p.eps, p.sms};
    return p.dtype == FFTCONV_BF16 ? ln::pick<__nv_bfloat16>(p.C, ln::FwdPick{a, s})
                                   : ln::pick<float>(p.C, ln::FwdPick{a, s});
}

size_t norm_workspace_bytes(const fftconv_norm_s& p) {
    return (size_t)ln::bwd_blocks(p, p.rows) * p.groups * 2 * p.C * sizeof(float);
}

cudaError_t launch_norm_bwd(const fftconv_norm_s& p, int64_t rows, const void* dy, const void* x, const float* w,
                            const float* mean, const float* rstd, void* dx, float* dw, float* db, float* work,
                            cudaStream_t s) {
    const ln::BwdArgs a{dy, x, w, mean, rstd, dx, work, rows, p.C, p.groups, ln::bwd_blocks(p, rows)};
    cudaError_t e = p.dtype == FFTCONV_BF16 ? ln::pick<__nv_bfloat16>(p.C, ln::BwdPick{a, s})
                                            : ln::pick<float>(p.C, ln::BwdPick{a, s});
    if (e != cudaSuccess) return e;
    return la::launch<ln::norm_reduce>(dim3((p.C + 31) / 32, p.groups), 1024, 0, s, true, (const float*)work, dw, db,
                                       a.blocks, p.C);
}

}  // namespace fftc
