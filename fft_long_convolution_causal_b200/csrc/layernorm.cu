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
#include <cuda_bf16.h>

#include "mixer.h"

namespace fftc {
namespace ln {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T, int V>
struct alignas(V * sizeof(T) < 16 ? V * sizeof(T) : 16) Piece {
    T e[V];
};

template <int TPR>
__host__ __device__ constexpr int block_threads() {
    return TPR > 32 ? TPR : 256;  // rows on several warps: one row a block
}

// sums of two values over the TPR threads of a row
template <int TPR>
__device__ __forceinline__ float2 row_sum(float2 v) {
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    if constexpr (TPR > 32) {
        __shared__ float2 part[TPR / 32];
        __syncthreads();  // the previous sum has been read
        if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = v;
        __syncthreads();
        v = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < TPR / 32; ++i) {
            v.x += part[i].x;
            v.y += part[i].y;
        }
    }
    return v;
}

template <typename T, int V, int TPR, int E>
__global__ void __launch_bounds__(block_threads<TPR>())
norm_fwd(const T* x, const float* __restrict__ w, const float* __restrict__ bias, T* y,
         float* __restrict__ mean, float* __restrict__ rstd, int64_t rows, int C, int G, float eps) {
    using P = Piece<T, V>;
    using W = Piece<float, V>;
    constexpr int kRows = block_threads<TPR>() / TPR;
    const int lane = threadIdx.x % TPR, items = C / V;
    const int64_t r = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
    const bool on = r < rows;
    const P* xr = reinterpret_cast<const P*>(x + (on ? r : 0) * C);
    float v[E][V];
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int c = lane + i * TPR;
        if (c < items && on) {
            const P p = xr[c];
#pragma unroll
            for (int j = 0; j < V; ++j) s.x += v[i][j] = to_f(p.e[j]);
        }
    }
    const float inv = 1.f / (float)C, mu = row_sum<TPR>(s).x * inv;
    s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < E; ++i)
        if (lane + i * TPR < items && on) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                v[i][j] -= mu;
                s.x = fmaf(v[i][j], v[i][j], s.x);
            }
        }
    const float rs = 1.f / sqrtf(row_sum<TPR>(s).x * inv + eps);
    if (!on) return;
    const int64_t g = G == 1 ? 0 : r % G;
    const W* wr = reinterpret_cast<const W*>(w + g * C);
    const W* br = reinterpret_cast<const W*>(bias + g * C);
    P* yr = reinterpret_cast<P*>(y + r * C);
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int c = lane + i * TPR;
        if (c < items) {
            const W wv = wr[c], bv = br[c];
            P p;
#pragma unroll
            for (int j = 0; j < V; ++j) p.e[j] = T(fmaf(v[i][j] * rs, wv.e[j], bv.e[j]));
            yr[c] = p;
        }
    }
    if (lane == 0) {
        if (mean) mean[r] = mu;
        if (rstd) rstd[r] = rs;
    }
}

// Blocks blockIdx.x of group blockIdx.y walk the group's rows; partial sums of
// the weight gradients to part[(group * blocks + block)][2][C].
template <typename T, int V, int TPR, int E>
__global__ void __launch_bounds__(block_threads<TPR>())
norm_bwd(const T* dy, const T* x, const float* __restrict__ w,
         const float* __restrict__ mean, const float* __restrict__ rstd, T* dx,
         float* __restrict__ part, int64_t rows, int C, int G) {
    using P = Piece<T, V>;
    using W = Piece<float, V>;
    constexpr int kRows = block_threads<TPR>() / TPR;
    const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR, items = C / V, g = blockIdx.y;
    const int64_t group_rows = rows / G;
    const float inv = 1.f / (float)C;
    float dw[E][V] = {}, db[E][V] = {};
    const W* wr = reinterpret_cast<const W*>(w + (int64_t)g * C);
    for (int64_t k = (int64_t)blockIdx.x * kRows; k < group_rows; k += (int64_t)gridDim.x * kRows) {
        const bool on = k + sub < group_rows;
        const int64_t r = on ? (k + sub) * G + g : 0;
        const P* xr = reinterpret_cast<const P*>(x + r * C);
        const P* dr = reinterpret_cast<const P*>(dy + r * C);
        P xp[E], dp[E];
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int c = lane + i * TPR;
            if (c < items && on) {
                xp[i] = xr[c];
                dp[i] = dr[c];
            }
        }
        const float mu = on ? mean[r] : 0.f, rs = on ? rstd[r] : 0.f;
        float2 s = make_float2(0.f, 0.f);
        float gv[E][V], xh[E][V];
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int c = lane + i * TPR;
            if (c < items && on) {
                const W wv = wr[c];
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float d = to_f(dp[i].e[j]);
                    xh[i][j] = (to_f(xp[i].e[j]) - mu) * rs;
                    gv[i][j] = d * wv.e[j];
                    dw[i][j] = fmaf(d, xh[i][j], dw[i][j]);
                    db[i][j] += d;
                    s.x += gv[i][j];
                    s.y = fmaf(gv[i][j], xh[i][j], s.y);
                }
            }
        }
        s = row_sum<TPR>(s);
        const float m1 = s.x * inv, m2 = s.y * inv;
        if (on) {
            P* o = reinterpret_cast<P*>(dx + r * C);
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int c = lane + i * TPR;
                if (c < items) {
                    P p;
#pragma unroll
                    for (int j = 0; j < V; ++j) p.e[j] = T(rs * (gv[i][j] - m1 - xh[i][j] * m2));
                    o[c] = p;
                }
            }
        }
    }
    // over the block's rows, then out
    float* out = part + ((int64_t)g * gridDim.x + blockIdx.x) * 2 * C;
    if constexpr (kRows > 1) {
        __shared__ float red[block_threads<TPR>()];
#pragma unroll
        for (int i = 0; i < E; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    __syncthreads();
                    red[threadIdx.x] = q ? db[i][j] : dw[i][j];
                    __syncthreads();
                    const int c = lane + i * TPR;
                    if (sub == 0 && c < items) {
                        float t = 0.f;
                        for (int k = 0; k < kRows; ++k) t += red[k * TPR + lane];
                        out[q * C + c * V + j] = t;
                    }
                }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int c = lane + i * TPR;
            if (c < items)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    out[c * V + j] = dw[i][j];
                    out[C + c * V + j] = db[i][j];
                }
        }
    }
}

// dw, db [G][C] from the blocks' partial sums: 32 columns x 8 threads a block, in a fixed order
__global__ void __launch_bounds__(256) norm_reduce(const float* __restrict__ part, float* __restrict__ dw,
                                                   float* __restrict__ db, int blocks, int C) {
    __shared__ float2 red[8][32];
    const int c = blockIdx.x * 32 + threadIdx.x % 32, k0 = threadIdx.x / 32, g = blockIdx.y;
    float2 s = make_float2(0.f, 0.f);
    if (c < C)
        for (int k = k0; k < blocks; k += 8) {
            const float* p = part + ((int64_t)g * blocks + k) * 2 * C + c;
            s.x += p[0];
            s.y += p[C];
        }
    red[k0][threadIdx.x % 32] = s;
    __syncthreads();
    if (k0 == 0 && c < C) {
        for (int k = 1; k < 8; ++k) {
            s.x += red[k][threadIdx.x].x;
            s.y += red[k][threadIdx.x].y;
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
    constexpr int kRows = block_threads<TPR>() / TPR;
    norm_fwd<T, V, TPR, E><<<(unsigned)((a.rows + kRows - 1) / kRows), block_threads<TPR>(), 0, s>>>(
        (const T*)a.x, a.w, a.b, (T*)a.y, a.mean, a.rstd, a.rows, a.C, a.G, a.eps);
    return cudaGetLastError();
}
template <typename T, int V, int TPR, int E>
cudaError_t bwd(const BwdArgs& a, cudaStream_t s) {
    norm_bwd<T, V, TPR, E><<<dim3(a.blocks, a.G), block_threads<TPR>(), 0, s>>>(
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

// blocks a group of the backward pass: two an SM in all, no more than rows
inline int bwd_blocks(const fftconv_norm_s& p, int64_t rows) {
    int64_t n = (2 * (int64_t)p.sms + p.groups - 1) / p.groups;
    const int64_t most = rows / p.groups;
    n = n < most ? n : most;
    return (int)(n < 1 ? 1 : n);
}

}  // namespace ln

cudaError_t launch_norm_fwd(const fftconv_norm_s& p, int64_t rows, const void* x, const float* w, const float* b,
                            void* y, float* mean, float* rstd, cudaStream_t s) {
    const ln::FwdArgs a{x, w, b, y, mean, rstd, rows, p.C, p.groups, p.eps};
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
    ln::norm_reduce<<<dim3((p.C + 31) / 32, p.groups), 256, 0, s>>>(work, dw, db, a.blocks, p.C);
    return cudaGetLastError();
}

}  // namespace fftc
