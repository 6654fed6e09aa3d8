// layernorm.cu -- layer norm over the last dimension, forward and backward:
//   y = (x - mu) rstd w + b
//   dx = rstd (g - mean(g) - xh mean(g xh)),  g = dy w,  xh = (x - mu) rstd
//   dw = sum over rows of dy xh,  db = sum over rows of dy
// Row r uses weight row r mod G (G = 1: one weight for all; G = heads: the norm
// behind each head).
//
// Moves each tensor once (x twice, both ways together), at two thirds of the copy
// rate: what is left is the loads' latency (the backward pass has 12 warps an SM with
// one row of loads ahead; its issue slots are 53% used) and the launches' ramps.  A row is read once into registers (mean first, then the sum
// of centred squares: no cancellation) by TPR threads, each holding E pieces of
// 16 bytes.  Where C is not a multiple of a piece (OFF), a row starts up to a piece
// behind a 16-byte boundary: pieces lie on the boundaries all the same, the two
// at the row's ends are read and written by elements, and a thread walks rows in
// steps that keep its columns, with their weights in registers.  38668 x 557 bf16
// both ways: 318 us with one element a piece, 111 us so.  The weight
// gradient is summed over the rows a block walks in registers, then over blocks
// by a second kernel in a fixed order: repeated calls agree bit for bit.
// 32768 x 768 bf16: forward 23.1 us (4.4 TB/s of x and y), backward 35.9 us
// (4.2 TB/s of dy, x and dx), the launches' ramps included; 16384 x 768 fp32 19.0
// (5.3 TB/s) and 41.6 us (3.6 TB/s); 49152 x 64 fp32 forward 9.0 us, 17 x 2708 both
// ways 31 us, which is the host's time.
#include <cuda_bf16.h>

#include "linattn.cuh"
#include "mixer.h"
#include "norm_rows.h"
#include "pairs.cuh"

namespace fftc {
namespace ln {

// rows a block: as many as its threads hold; the backward pass has 384 threads (up to 170 registers, see there)
template <int TPR>
constexpr int kFwdRows = TPR > 32 ? 1 : 256 / TPR;
template <int TPR, int W>
constexpr int kBwdRows = TPR > 128 ? 1 : TPR == 128 ? (W > 24 ? 2 : 3) : 384 / TPR;

// Sums over the TPR threads of row `sub` of a block.  Rows on several warps meet in shared memory, in buffer `buf`:
// two in turn, so that a buffer is written again only behind the barrier of the other.
template <int TPR, int ROWS>
__device__ __forceinline__ float2 row_sums(float2 v, int sub, int buf) {
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    if constexpr (TPR > 32) {
        __shared__ float2 part[2][ROWS][TPR / 32];
        if ((threadIdx.x & 31) == 0) part[buf][sub][threadIdx.x % TPR / 32] = v;
        asm volatile("bar.sync %0, %1;" ::"r"(sub + 1), "r"(TPR) : "memory");
        v = both(0.f);
#pragma unroll
        for (int i = 0; i < TPR / 32; ++i) v = add2(v, part[buf][sub][i]);
    }
    return v;
}
template <int TPR, int ROWS>
__device__ __forceinline__ float row_sum(float v, int sub, int buf) {
    if constexpr (TPR > 32) {
        return row_sums<TPR, ROWS>(make_float2(v, 0.f), sub, buf).x;
    } else {
#pragma unroll
        for (int o = TPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
}

// two elements, stored together
template <typename T>
struct alignas(2 * sizeof(T)) Two {
    T x, y;
    __device__ __forceinline__ explicit Two(float2 v) : x(T(v.x)), y(T(v.y)) {}
};

// A thread's pieces of rows in memory.
template <typename T, int V, int TPR, bool OFF>
struct Columns : Pieces<V, TPR, OFF> {
    using P = Piece<T, V>;
    using Pieces<V, TPR, OFF>::first, Pieces<V, TPR, OFF>::inside, Pieces<V, TPR, OFF>::has, Pieces<V, TPR, OFF>::C;
    __device__ __forceinline__ Columns(int lane, int off, int C) : Pieces<V, TPR, OFF>{lane, off, C} {}
    // A piece at a row's end is loaded whole (its other elements are a neighbouring row's), but by elements at the
    // tensor's end; trim() puts zeros in place of what is not the row's.  In place, another block may be storing the
    // neighbour's elements of such a piece meanwhile: whichever bytes come back for them, trim() drops them, and the
    // row's own are written by this thread alone, later.
    __device__ __forceinline__ void load(P& q, const T* row, int i, int end) const {
        const int c = first(i);
        if (this->whole(i, end)) {
            q = *reinterpret_cast<const P*>(row + c);
        } else {
#pragma unroll
            for (int j = 0; j < P::kPairs; ++j)
                q.set(j, make_float2(has(c + 2 * j) ? (float)row[c + 2 * j] : 0.f,
                                     has(c + 2 * j + 1) ? (float)row[c + 2 * j + 1] : 0.f));
        }
    }
    __device__ __forceinline__ void trim(P& q, int i) const {
        if (inside(i)) return;
        const int c = first(i);
#pragma unroll
        for (int j = 0; j < P::kPairs; ++j) {
            const float2 v = q.get(j);
            q.set(j, make_float2(has(c + 2 * j) ? v.x : 0.f, has(c + 2 * j + 1) ? v.y : 0.f));
        }
    }
    // by pairs and elements at the row's ends
    __device__ __forceinline__ void store(const P& q, T* row, int i) const {
        const int c = first(i);
        if (inside(i)) {
            *reinterpret_cast<P*>(row + c) = q;
        } else {
#pragma unroll
            for (int j = 0; j < P::kPairs; ++j) {
                const int e = c + 2 * j;
                const Two<T> v(q.get(j));
                if (e >= 0 && e + 1 < C)
                    *reinterpret_cast<Two<T>*>(row + e) = v;
                else if (has(e))
                    row[e] = v.x;
                else if (has(e + 1))
                    row[e + 1] = v.y;
            }
        }
    }
    __device__ __forceinline__ float2 weight(const float* w, int i, int j) const {
        const int c = first(i) + 2 * j;
        return make_float2(has(c) ? w[c] : 0.f, has(c + 1) ? w[c + 1] : 0.f);
    }
};
template <typename T, int V, int TPR, int E, bool OFF>
__global__ void __launch_bounds__((TPR * kFwdRows<TPR>), (OFF && TPR <= 32 ? (E < 3 ? 3 : 2) : 0))
norm_fwd(const T* x, const float* __restrict__ w, const float* __restrict__ bias, T* y, float* __restrict__ mean,
         float* __restrict__ rstd, int64_t rows, int64_t step, int C, int G, float eps) {
    using P = Piece<T, V>;
    using W = Piece<float, V>;
    constexpr int kRows = kFwdRows<TPR>, NP = P::kPairs;
    const int sub = threadIdx.x / TPR;
    const float inv = 1.f / (float)C;
    int64_t r = (int64_t)blockIdx.x * kRows + sub;
    if (r >= step) r = rows;  // OFF: past the last of a step's rows
    const Columns<T, V, TPR, OFF> col((int)(threadIdx.x % TPR), offset<V, OFF>(r, C), C);
    P p[E];
    auto fetch = [&](int64_t r) {
        if (r >= rows) return;
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (col.any(i)) col.load(p[i], x + r * C, i, to_end(r, rows, C));
    };
    fetch(r);
    float2 hw[OFF ? E : 1][NP], hb[OFF ? E : 1][NP];
    if constexpr (OFF) {
        const int64_t g = r < rows ? r % G : 0;
#pragma unroll
        for (int i = 0; i < E; ++i)
#pragma unroll
            for (int j = 0; j < NP; ++j) hw[i][j] = col.weight(w + g * C, i, j), hb[i][j] = col.weight(bias + g * C, i, j);
    }
    for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < rows; r0 += step, r += step) {
        const bool on = r < rows;
        float2 v[E][NP], s = both(0.f);
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (col.any(i) && on) {
                col.trim(p[i], i);
#pragma unroll
                for (int j = 0; j < NP; ++j) s = add2(s, v[i][j] = p[i].get(j));
            }
        fetch(r + step);  // in flight while this row is worked on
        const float mu = row_sum<TPR, kRows>(s.x + s.y, sub, 0) * inv;
        s = both(0.f);
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (col.any(i) && on) {
#pragma unroll
                for (int j = 0; j < NP; ++j) v[i][j] = add2(v[i][j], both(-mu));
                if (!col.inside(i)) {
#pragma unroll
                    for (int j = 0; j < NP; ++j) {
                        if (!col.has(col.first(i) + 2 * j)) v[i][j].x = 0.f;
                        if (!col.has(col.first(i) + 2 * j + 1)) v[i][j].y = 0.f;
                    }
                }
#pragma unroll
                for (int j = 0; j < NP; ++j) s = fma2(v[i][j], v[i][j], s);
            }
        const float rs = 1.f / sqrtf(row_sum<TPR, kRows>(s.x + s.y, sub, 1) * inv + eps);
        if (on) {
            const int64_t g = OFF || G == 1 ? 0 : r % G;
            const W* wr = reinterpret_cast<const W*>(w + g * C);
            const W* br = reinterpret_cast<const W*>(bias + g * C);
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (col.any(i)) {
                    P o;
                    if constexpr (OFF) {
#pragma unroll
                        for (int j = 0; j < NP; ++j) o.set(j, fma2(mul2(v[i][j], both(rs)), hw[i][j], hb[i][j]));
                    } else {
                        const W wv = wr[col.lane + i * TPR], bv = br[col.lane + i * TPR];
#pragma unroll
                        for (int j = 0; j < NP; ++j) o.set(j, fma2(mul2(v[i][j], both(rs)), wv.get(j), bv.get(j)));
                    }
                    col.store(o, y + r * C, i);
                }
            if (col.lane == 0) {
                if (mean) mean[r] = mu;
                if (rstd) rstd[r] = rs;
            }
        }
    }
}

// The backward pass holds two rows of weight-gradient sums, a row and the next one's loads in registers: 12 warps of
// up to 170 registers an SM (at 128 registers and 16 warps it spilled, and 32768 x 768 took 98 us instead of 29).
// Blocks blockIdx.x of group blockIdx.y walk the group's rows, the next row's loads in flight while a row is worked on;
// partial sums of the weight gradients to part[(group * blocks + block)][2][C].
template <typename T, int V, int TPR, int E, bool OFF>
__global__ void __launch_bounds__((TPR * kBwdRows<TPR, E * V>), 1)
norm_bwd(const T* dy, const T* x, const float* __restrict__ w, const float* __restrict__ mean,
         const float* __restrict__ rstd, T* dx, float* __restrict__ part, int64_t rows, int64_t step, int C, int G) {
    using P = Piece<T, V>;
    using W = Piece<float, V>;
    constexpr int kRows = kBwdRows<TPR, E * V>, kThreads = TPR * kRows, NP = P::kPairs;
    const int sub = threadIdx.x / TPR, g = blockIdx.y;
    const int64_t group_rows = rows / G;
    const float inv = 1.f / (float)C;
    int64_t k = (int64_t)blockIdx.x * kRows + sub;
    if (k >= step) k = group_rows;  // OFF: past the last of a step's rows
    const Columns<T, V, TPR, OFF> col((int)(threadIdx.x % TPR), offset<V, OFF>(k * G + g, C), C);
    float2 dw[E][NP], db[E][NP];
#pragma unroll
    for (int i = 0; i < E; ++i)
#pragma unroll
        for (int j = 0; j < NP; ++j) dw[i][j] = db[i][j] = both(0.f);
    const W* wr = reinterpret_cast<const W*>(w + (int64_t)g * C);
    float2 hw[OFF ? E : 1][NP];
    if constexpr (OFF) {
#pragma unroll
        for (int i = 0; i < E; ++i)
#pragma unroll
            for (int j = 0; j < NP; ++j) hw[i][j] = col.weight(w + (int64_t)g * C, i, j);
    }
    struct Weights {
        float2 v[NP];
    };
    auto weights = [&](int i) {
        Weights q;
        if constexpr (OFF) {
#pragma unroll
            for (int j = 0; j < NP; ++j) q.v[j] = hw[i][j];
        } else {
            const W wv = wr[col.lane + i * TPR];
#pragma unroll
            for (int j = 0; j < NP; ++j) q.v[j] = wv.get(j);
        }
        return q;
    };
    struct Row {
        P x[E], d[E];
        float mu, rs;
    };
    auto fetch = [&](Row& q, int64_t k) {
        if (k >= group_rows) return;
        const int64_t r = k * G + g;
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (col.any(i)) {
                col.load(q.x[i], x + r * C, i, to_end(r, rows, C));
                col.load(q.d[i], dy + r * C, i, to_end(r, rows, C));
            }
        q.mu = mean[r];
        q.rs = rstd[r];
    };
    constexpr bool kAhead = E * V <= 24;  // where the registers allow it
    Row row;
    if (kAhead) fetch(row, k);
    int buf = 0;
    for (int64_t k0 = (int64_t)blockIdx.x * kRows; k0 < group_rows; k0 += step, k += step, buf ^= 1) {
        const bool on = k < group_rows;
        Row next;
        if (kAhead)
            fetch(next, k + step);
        else
            fetch(row, k);
        float2 s1 = both(0.f), s2 = both(0.f);
        const float2 rs = both(row.rs), shift = both(-row.mu);
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (col.any(i) && on) {
                col.trim(row.x[i], i);
                col.trim(row.d[i], i);
                const Weights wv = weights(i);
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    const float2 d = row.d[i].get(j), xh = mul2(add2(row.x[i].get(j), shift), rs), gv = mul2(d, wv.v[j]);
                    dw[i][j] = fma2(d, xh, dw[i][j]);
                    db[i][j] = add2(db[i][j], d);
                    s1 = add2(s1, gv);
                    s2 = fma2(gv, xh, s2);
                }
            }
        const float2 m = row_sums<TPR, kRows>(make_float2(s1.x + s1.y, s2.x + s2.y), sub, buf);
        const float m1 = m.x * inv, m2 = m.y * inv;
        if (on) {
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (col.any(i)) {
                    const Weights wv = weights(i);
                    P q;
#pragma unroll
                    for (int j = 0; j < NP; ++j) {
                        const float2 xh = mul2(add2(row.x[i].get(j), shift), rs);
                        const float2 c = fma2(row.d[i].get(j), wv.v[j], both(-m1));
                        q.set(j, mul2(rs, fma2(xh, both(-m2), c)));
                    }
                    col.store(q, dx + (k * G + g) * C, i);
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
                    const int c = col.first(i) + j;
                    if (!OFF || col.has(c)) red[sub][OFF ? c : (i * V + j) * TPR + col.lane] = j & 1 ? u.y : u.x;
                }
            __syncthreads();
            for (int e = threadIdx.x; e < (OFF ? C : TPR * E * V); e += kThreads) {
                const int c = OFF ? e : (e % TPR + e / TPR / V * TPR) * V + e / TPR % V;
                if (c < C) {
                    float v = 0.f;
#pragma unroll
                    for (int k = 0; k < kRows; ++k) v += red[k][e];
                    out[q * C + c] = v;
                }
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = col.first(i) + j;
                if (col.has(c)) {
                    out[c] = j & 1 ? dw[i][j / 2].y : dw[i][j / 2].x;
                    out[C + c] = j & 1 ? db[i][j / 2].y : db[i][j / 2].x;
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
    float *part, *dw, *db;
    int64_t rows;
    int C, G, blocks;
};

int64_t common_multiple(int64_t a, int64_t b) {
    int64_t x = a, y = b;
    while (y) {
        const int64_t t = x % y;
        x = y;
        y = t;
    }
    return a / x * b;
}

template <typename T, int V, int TPR, int E, bool OFF>
cudaError_t fwd(const FwdArgs& a, cudaStream_t s) {
    constexpr int kRows = kFwdRows<TPR>, kThreads = TPR * kRows;
    // the blocks that the SMs hold at once, each walking rows
    static const int held = [] {
        int n = 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, norm_fwd<T, V, TPR, E, OFF>, kThreads, 0) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
        return n > 0 ? n : 1;
    }();
    const int64_t all = (a.rows + kRows - 1) / kRows * kRows, most = (int64_t)a.sms * held * kRows;
    int64_t step = all < most ? all : most;
    if (OFF && step < a.rows) {  // a thread's rows have one offset and one weight row
        const int64_t unit = common_multiple(V, a.G);
        step = step > unit ? step / unit * unit : unit;
    }
    const int64_t units = step < all ? step : all;
    norm_fwd<T, V, TPR, E, OFF><<<(unsigned)((units + kRows - 1) / kRows), kThreads, 0, s>>>(
        (const T*)a.x, a.w, a.b, (T*)a.y, a.mean, a.rstd, a.rows, step, a.C, a.G, a.eps);
    return cudaGetLastError();
}
template <typename T, int V, int TPR, int E, bool OFF>
cudaError_t bwd(const BwdArgs& a, cudaStream_t s) {
    constexpr int kRows = kBwdRows<TPR, E * V>;
    const int64_t group_rows = a.rows / a.G, all = (group_rows + kRows - 1) / kRows;
    const int blocks = (int)(a.blocks < all ? a.blocks : all);
    int64_t step = (int64_t)blocks * kRows;
    if (OFF && step < group_rows) step = step / V * V;  // at least V: see bwd_blocks
    norm_bwd<T, V, TPR, E, OFF><<<dim3(blocks, a.G), TPR * kRows, 0, s>>>(
        (const T*)a.dy, (const T*)a.x, a.w, a.mean, a.rstd, (T*)a.dx, a.part, a.rows, step, a.C, a.G);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return la::launch<norm_reduce>(dim3((a.C + 31) / 32, a.G), 1024, 0, s, true, (const float*)a.part, a.dw, a.db, blocks,
                                   a.C);
}

// threads and pieces a row, by its pieces: the fewest threads that hold a row in few registers
template <typename T, typename F>
cudaError_t pick(int C, F f) {
    constexpr int V = 16 / sizeof(T);
    if (C % V == 0) {
        const int items = C / V;
        if (items <= 8) return f.template operator()<T, V, 8, 1, false>();
        if (items <= 16) return f.template operator()<T, V, 16, 1, false>();
        if (items <= 32) return f.template operator()<T, V, 32, 1, false>();
        if (items <= 64) return f.template operator()<T, V, 32, 2, false>();
        if (items <= 96) return f.template operator()<T, V, 32, 3, false>();
        if (items <= 128) return f.template operator()<T, V, 32, 4, false>();
        if (items <= 256) return f.template operator()<T, V, 128, 2, false>();
        if (items <= 512) return f.template operator()<T, V, 128, 4, false>();
        if (items <= 1024) return f.template operator()<T, V, 512, 2, false>();
        if (items <= 2048) return f.template operator()<T, V, 512, 4, false>();
        return f.template operator()<T, V, 512, 8, false>();
    }
    const int items = (C + 2 * V - 2) / V;  // of the largest offset; the weights are in registers too
    if (items <= 8) return f.template operator()<T, V, 8, 1, true>();
    if (items <= 16) return f.template operator()<T, V, 8, 2, true>();
    if (items <= 24) return f.template operator()<T, V, 8, 3, true>();
    if (items <= 32) return f.template operator()<T, V, 16, 2, true>();
    if (items <= 48) return f.template operator()<T, V, 16, 3, true>();
    if (items <= 64) return f.template operator()<T, V, 32, 2, true>();
    if constexpr (F::kThree)
        if (items <= 96) return f.template operator()<T, V, 32, 3, true>();
    if (items <= 128) return f.template operator()<T, V, 128, 1, true>();
    if (items <= 256) return f.template operator()<T, V, 128, 2, true>();
    if constexpr (F::kThree)
        if (items <= 384) return f.template operator()<T, V, 128, 3, true>();
    if (items <= 512) return f.template operator()<T, V, 512, 1, true>();
    if (items <= 1024) return f.template operator()<T, V, 512, 2, true>();
    if (items <= 1536) return f.template operator()<T, V, 512, 3, true>();
    return f.template operator()<T, V, 512, V == 8 ? 5 : 9, true>();  // 16383 columns and an offset
}
struct FwdPick {
    static constexpr bool kThree = false;  // registers for a third block an SM: 38668 x 557 bf16 54 -> 48 us
    const FwdArgs& a;
    cudaStream_t s;
    template <typename T, int V, int TPR, int E, bool OFF>
    cudaError_t operator()() {
        return fwd<T, V, TPR, E, OFF>(a, s);
    }
};
struct BwdPick {
    static constexpr bool kThree = true;  // a row on one warp: 60 us, on four 80
    const BwdArgs& a;
    cudaStream_t s;
    template <typename T, int V, int TPR, int E, bool OFF>
    cudaError_t operator()() {
        return bwd<T, V, TPR, E, OFF>(a, s);
    }
};

// Blocks a group of the backward pass: at most one an SM in all, no more than rows; eight where rows start at different offsets,
// so that a step of rows can be a multiple of the offsets' period.
inline int bwd_blocks(const fftconv_norm_s& p, int64_t rows) {
    int64_t n = p.sms / p.groups;
    if (n < 8 && p.C % (p.dtype == FFTCONV_BF16 ? 8 : 4)) n = 8;
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
    const ln::BwdArgs a{dy, x, w, mean, rstd, dx, work, dw, db, rows, p.C, p.groups, ln::bwd_blocks(p, rows)};
    return p.dtype == FFTCONV_BF16 ? ln::pick<__nv_bfloat16>(p.C, ln::BwdPick{a, s})
                                   : ln::pick<float>(p.C, ln::BwdPick{a, s});
}

}  // namespace fftc
