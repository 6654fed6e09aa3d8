// linattn_tc.cu -- decayed linear attention on the fifth-generation tensor cores
// (bf16 operands, fp32 accumulators in tensor memory), chunks of 128 tokens.
//
// la_main: a CTA walks the chunks of one (segment, row, head, pass) with the
// state S [dx][dz] resident in tensor memory.  Per chunk of L live tokens:
//   scores  P  = X Y^T                                   (128 x 128 x DX)
//   inter   OI = X bf16(S)                               (128 x DZ x DX)
//   intra   OA = bf16(s_p a^|i-j| P, masked) Z           (128 x DZ x 128)
//   out     o  = OA + s_i a^(i+1) OI                     (rows of bf16)
//   state   S  = a^L S + (s_u a^(L-1-j) y_j)^T Z         (DX x DZ x 128, two products)
// The decayed y would lose bits in one bf16, and with it the state that all later
// outputs read: it is split into a sum of two (off by 2^-17 at most).
//
// la_states: the state alone, of one (segment, row, head, pass), where it is an
// fp32 output or joins segments.  Three bf16 terms (exact to 2^-25), and each
// chunk's contribution is summed from zero and added to the state in fp32
// registers: the tensor core truncates when it accumulates, which over hundreds of
// chunks on top of a large state would cost the last six bits.
//
// Tiles come in by bulk tensor copies (TMA), as blocks of [token][64 elements] with
// the 128-byte swizzle; the same bytes serve as a K-major operand over elements
// and as an MN-major operand over tokens, so nothing is transposed.  The copies
// were cp.async at first: their traffic through the load/store unit slowed every
// shared-memory access of the other warps by three to five times (a chunk took
// 12300 cycles at 128 x 128, of which 7400 without the copies).  A chunk that a
// row's length cuts short is still copied that way, zero-filling rows behind the
// length (their memory may hold anything, NaN included).
//
// Every role is kept to a few rolled loops: fully unrolled, the kernel was 136 KB
// of code and ran at the rate of its instruction misses.
#include <cuda.h>
#include <cuda_bf16.h>

#include "linattn.cuh"
#include "umma.cuh"

namespace fftc {
namespace latc {

constexpr int kC = 128;                  // tokens a chunk
constexpr uint32_t kBlock = kC * 128u;   // bytes of a tile's block of 64 elements

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float lo_f(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
__device__ __forceinline__ float as_f(uint32_t u) { return __uint_as_float(u); }
__device__ __forceinline__ uint32_t as_u(float f) { return __float_as_uint(f); }
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int src_bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.commit_group;\ncp.async.wait_group 0;\n" ::: "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* map, int c0, int c1, int c2, int c3, uint32_t mbar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(mbar)
        : "memory");
}
// byte offset of 16-byte column c of token t in a tile (128-byte swizzle: column xor row)
__device__ __forceinline__ uint32_t tile_off(int t, int c) {
    return (uint32_t)(c >> 3) * kBlock + (uint32_t)t * 128u + (uint32_t)((c ^ t) & 7) * 16u;
}
// descriptors of a tile: rows = tokens, K = elements (16 a step: 32 bytes, a block after 4 steps), and
// rows = elements, K = tokens (16 a step: 2048 bytes; blocks of 64 rows)
constexpr uint64_t kSwizzle128 = 2ull << 61;
__device__ __forceinline__ uint64_t kmajor(uint32_t tile) { return um::sdesc(tile, 16, 1024) | kSwizzle128; }
__device__ __forceinline__ uint64_t mnmajor(uint32_t tile) { return um::sdesc(tile, kBlock, 1024) | kSwizzle128; }
__device__ __forceinline__ constexpr uint64_t kstep(int k) { return (uint64_t)(((k / 4) * kBlock + (k % 4) * 32u) >> 4); }
__device__ __forceinline__ constexpr uint64_t mnstep(int k) { return (uint64_t)((k * 2048u) >> 4); }

// a token tensor's map: dimensions (elements, then tokens, heads and rows in the order of their strides)
struct Source {
    CUtensorMap map;
    int at_token, at_head, at_row;  // dimension 1 .. 3 of each, 0: not a dimension (stride zero or one element)
    int by_hand;                    // no map: copied with plain loads
};
constexpr int kMaxSources = 4;
struct Args {
    la::Args a;
    Source src[kMaxSources];
    int x[kLaMaxPasses], y[kLaMaxPasses], z[kLaMaxPasses];  // sources of each pass
    int* err;
    uint32_t limit;
};

// waits of a CTA: bounded, given up together
struct Waiter {
    volatile int* abort;
    uint32_t limit;
    __device__ __forceinline__ bool operator()(const uint64_t& x, uint32_t parity) const {
        const uint32_t ad = smem_u32(&x);
#pragma unroll 1
        for (uint32_t i = 0; i < limit && !*abort; ++i)
            if (um::mbar_try_wait(ad, parity)) return true;
        *abort = 1;
        return false;
    }
    // one answer for a warp
    __device__ __forceinline__ bool all(const uint64_t& x, uint32_t parity) const {
        return __all_sync(0xffffffffu, (*this)(x, parity)) != 0;
    }
};

// a warp's tensor-memory and shared-memory accesses are done
__device__ __forceinline__ void arrive(const uint64_t& x) {
    um::fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) um::mbar_arrive(smem_u32(&x));
}

// the work of a CTA
struct Span {
    int64_t first, rows, live;  // first token of the segment, its tokens, of which live
    int nch;
    bool rev;
    __device__ __forceinline__ Span(const la::Args& a, const LaPass& p, int sg, int b) {
        first = sg * a.seg;
        rows = min(a.seg, a.N - first);
        live = max((int64_t)0, min(rows, la::live_tokens(a, b) - first));
        nch = (int)((live + kC - 1) / kC);
        rev = p.reverse;
    }
    // first token (in the segment) and live tokens of the n-th chunk of the walk
    __device__ __forceinline__ int64_t start(int n) const { return (int64_t)(rev ? nch - 1 - n : n) * kC; }
    __device__ __forceinline__ int tokens(int n) const { return (int)min((int64_t)kC, live - start(n)); }
};

// One warp copies the tiles of every chunk into a ring: y, x, z (or y, z) by turns.
template <int DX, int DZ, int kItems, int kSlots, uint32_t kSlot>
__device__ __forceinline__ void copy_tiles(const Args& g, const LaPass& p, const Span& sp, int b, int h, uint32_t ring,
                                           uint64_t* full, uint64_t* empty, const Waiter& wait) {
    const int lane = threadIdx.x & 31, pass = blockIdx.z;
    int made = 0;
    bool ok = true;
#pragma unroll 1
    for (int n = 0; n < sp.nch && ok; ++n) {
        const int64_t t0 = sp.start(n);
        const int L = sp.tokens(n);
#pragma unroll 1
        for (int it = 0; it < kItems; ++it, ++made) {
            const bool is_z = it == kItems - 1;
            const Source& s = g.src[is_z ? g.z[pass] : it == 0 ? g.y[pass] : g.x[pass]];
            const int sl = made % kSlots, blocks = (is_z ? DZ : DX) / 64;
            const uint32_t dst = ring + (uint32_t)sl * kSlot, bar = smem_u32(&full[sl]);
            if (made >= kSlots && !wait.all(empty[sl], (uint32_t)(made / kSlots - 1) & 1u)) {
                ok = false;
                break;
            }
            if (s.by_hand || (L < kC && sp.first + t0 + L < g.a.N)) {
                // rows behind the length are zeros whatever memory holds
                const fftconv_strides& st = is_z ? p.sz : it == 0 ? p.sy : p.sx;
                const __nv_bfloat16* base = (const __nv_bfloat16*)(is_z ? p.z : it == 0 ? p.y : p.x) + b * st.batch +
                                            h * st.head + (sp.first + t0) * st.token;
                const int d = is_z ? p.dz : p.dx;
#pragma unroll 1
                for (int e = lane; e < kC * blocks * 8; e += 32) {
                    const int c = e % (blocks * 8), t = e / (blocks * 8);
                    const bool on = t < L && c * 8 < d;
                    cp_async16(dst + tile_off(t, c), on ? base + t * st.token + c * 8 : base, on ? 16 : 0);
                }
                cp_wait();
                um::fence_proxy_async();
                __syncwarp();
                if (lane == 0) um::mbar_arrive(bar);
            } else if (lane == 0) {
                const int t = (int)(sp.first + t0);
                auto at = [&](int dim) { return s.at_token == dim ? t : s.at_head == dim ? h : s.at_row == dim ? b : 0; };
                um::mbar_arrive_expect_tx(bar, (uint32_t)blocks * kBlock);
#pragma unroll 1
                for (int k = 0; k < blocks; ++k)
                    tma_load_4d(dst + (uint32_t)k * kBlock, &s.map, 64 * k, at(1), at(2), at(3), bar);
            }
            __syncwarp();
        }
    }
    // copies still in flight after a wait gave up land before the CTA ends
    if (!ok || *wait.abort) {
#pragma unroll 1
        for (int i = made > kSlots ? made - kSlots : 0; i < made; ++i)
            um::mbar_wait(smem_u32(&full[i % kSlots]), (uint32_t)(i / kSlots) & 1u);
    }
}

// y decayed to the chunk's end, as a sum of NS bf16 terms: the first in place, the others `lo` apart.
// Thread (token t, part q of Q) takes every Q-th 16-byte column.
template <int DX, int NS, int Q>
__device__ __forceinline__ void split_y(uint32_t tile, uint32_t lo, uint32_t lo_step, int t, int q, float w) {
#pragma unroll 2
    for (int c = q; c < DX / 8; c += Q) {
        const uint32_t off = tile_off(t, c);
        const uint4 u = lds128(tile + off);
        const uint32_t in[4] = {u.x, u.y, u.z, u.w};
        uint32_t o[NS][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x = w * lo_f(in[i]), y = w * hi_f(in[i]);
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                o[s][i] = pack2(x, y);
                x -= lo_f(o[s][i]);
                y -= hi_f(o[s][i]);
            }
        }
        sts128(tile + off, o[0][0], o[0][1], o[0][2], o[0][3]);
#pragma unroll
        for (int s = 1; s < NS; ++s) sts128(lo + (uint32_t)(s - 1) * lo_step + off, o[s][0], o[s][1], o[s][2], o[s][3]);
    }
}

// Every product issued is complete before tensor memory is freed.
__device__ __forceinline__ void drain(uint64_t& bar, volatile int* abort) {
    um::mma_commit(smem_u32(&bar));
    if (!um::mbar_wait(smem_u32(&bar), 0)) *abort = 1;
}

// ---------------------------------------------------------------- outputs
template <int DX, int DZ>
struct Main {
    static constexpr bool kTwo = DX == 64 && DZ == 64;  // two CTAs an SM
    static constexpr uint32_t kSlot = (uint32_t)(DX > DZ ? DX : DZ) * 256u;
    static constexpr uint32_t kS = (uint32_t)DX * DZ * 2u, kLo = (uint32_t)DX * 256u;
    static constexpr int kSlots = 5;
    // The state's product has 128 rows whatever DX is: with DX = 64 its descriptor reads 16 KiB behind
    // a term of y (rows nobody looks at), which has to be this CTA's memory.
    static constexpr uint32_t kOffLo = kSlots * kSlot, kOffS = kOffLo + kLo, kOffTail = kOffS + kS;
    static constexpr uint32_t kTail = DX == 64 && kS < 16384u ? 16384u - kS : 2048u;
    static constexpr uint32_t kBytes = kOffTail + kTail;
    // tensor-memory columns
    static constexpr uint32_t kP = 0;                     // scores, then P' in the first 64
    static constexpr uint32_t kOA = DZ == 64 ? 64 : 128;  // DZ = 64: the scores' upper half, free by then
    static constexpr uint32_t kOI = DZ == 64 ? 128 : 256;
    static constexpr uint32_t kST = DZ == 64 ? 192 : 384;
    static constexpr uint32_t kCols = DZ == 64 ? 256 : 512;
    static constexpr int kThreads = 3 * 128 + 64;
};
struct MainTail {
    uint64_t full[5], empty[5], pfull, pready, ofull, ofree, sfull, yfull, sdone, drain;
    float pw[kLaPowers], ct[32], dt[64];
    uint32_t tmem;
    int abort;
};

template <int DX, int DZ>
__global__ void __launch_bounds__((Main<DX, DZ>::kThreads), (Main<DX, DZ>::kTwo ? 2 : 1))
la_main(const __grid_constant__ Args g) {
    using K = Main<DX, DZ>;
    static_assert(sizeof(MainTail) <= K::kTail, "the tail holds the barriers and tables");
    extern __shared__ __align__(1024) uint8_t smem[];
    MainTail& m = *reinterpret_cast<MainTail*>(smem + K::kOffTail);
    const la::Args& a = g.a;
    const LaPass& p = a.p[blockIdx.z];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int sg = blockIdx.x, bh = blockIdx.y, b = bh / a.H, h = bh % a.H;
    const Span sp(a, p, sg, b);
    const bool rev = sp.rev;
    const int nch = sp.nch;
    const uint32_t sb = smem_u32(smem);
    const Waiter wait{&m.abort, g.limit};
    constexpr int kMmaWarp = 12, kCopyWarp = 13;

    if (tid == 0) {
        for (int i = 0; i < K::kSlots; ++i) {
            um::mbar_init(smem_u32(&m.full[i]), 1);
            um::mbar_init(smem_u32(&m.empty[i]), 1);
        }
        um::mbar_init(smem_u32(&m.pfull), 1);
        um::mbar_init(smem_u32(&m.pready), 4);
        um::mbar_init(smem_u32(&m.ofull), 1);
        um::mbar_init(smem_u32(&m.ofree), 4);
        um::mbar_init(smem_u32(&m.sfull), 4);
        um::mbar_init(smem_u32(&m.yfull), 4);
        um::mbar_init(smem_u32(&m.sdone), 1);
        um::mbar_init(smem_u32(&m.drain), 1);
        m.abort = 0;
    }
    const float* pow_h = a.pw + (size_t)h * kLaPowers;
    for (int i = tid; i < kLaPowers; i += K::kThreads) m.pw[i] = pow_h[i];
    // weights on the diagonal block by column - row + 31, and on the others by column
    if (tid < 63) m.dt[tid] = (rev ? tid < 31 : tid > 31) ? 0.f : p.s_p * pow_h[rev ? tid - 31 : 31 - tid];
    if (tid < 32) m.ct[tid] = pow_h[rev ? tid : 31 - tid];
    if (warp == kMmaWarp) {
        um::tmem_alloc(smem_u32(&m.tmem), K::kCols);
        um::tmem_relinquish();
    }
    um::fence_before();
    __syncthreads();
    um::fence_after();
    const uint32_t tmem = m.tmem;
    const int quarter = warp & 3;
    const uint32_t tl = tmem + ((uint32_t)(32 * quarter) << 16);
    auto slot = [](int n, int item) { return (3 * n + item) % K::kSlots; };
    auto phase = [](int n, int item) { return (uint32_t)((3 * n + item) / K::kSlots) & 1u; };
    auto tile = [&](int n, int item) { return sb + (uint32_t)slot(n, item) * K::kSlot; };

    if (warp == kMmaWarp) {
        if (lane == 0) {
            constexpr uint32_t id_scores = um::idesc_bf16(128, 128), id_inter = um::idesc_bf16(128, DZ) | um::kBmn,
                               id_state = id_inter | um::kAmn;
            const uint64_t ds = um::sdesc(sb + K::kOffS, 128, DX * 16);
#pragma unroll 1
            for (int n = 0; n < nch; ++n) {
                const uint32_t par = (uint32_t)n & 1u, prev = par ^ 1u;
                const uint64_t ky = kmajor(tile(n, 0)), kx = kmajor(tile(n, 1)), zz = mnmajor(tile(n, 2));
                if (!wait(m.full[slot(n, 0)], phase(n, 0))) break;
                if (!wait(m.full[slot(n, 1)], phase(n, 1))) break;
                if (DZ == 64 && n && !wait(m.ofree, prev)) break;
                um::fence_after();
#pragma unroll
                for (int k = 0; k < DX / 16; ++k)
                    um::mma_ss(tmem + K::kP, kx + kstep(k), ky + kstep(k), id_scores, k > 0);
                um::mma_commit(smem_u32(&m.pfull));
                if (!wait(m.sfull, par)) break;
                if (DZ != 64 && n && !wait(m.ofree, prev)) break;
                um::fence_after();
#pragma unroll
                for (int k = 0; k < DX / 16; ++k)
                    um::mma_ss(tmem + K::kOI, kx + kstep(k), ds + (uint64_t)(k * 16), id_inter, k > 0);
                um::mma_commit(smem_u32(&m.empty[slot(n, 1)]));
                if (!wait(m.full[slot(n, 2)], phase(n, 2))) break;
                if (!wait(m.pready, par)) break;
                um::fence_after();
#pragma unroll
                for (int k = 0; k < kC / 16; ++k)
                    um::mma_ts(tmem + K::kOA, tmem + K::kP + 8u * k, zz + mnstep(k), id_inter, k > 0);
                um::mma_commit(smem_u32(&m.ofull));
                if (!wait(m.yfull, par)) break;
                um::fence_after();
                const uint64_t yh = mnmajor(tile(n, 0)), yl = mnmajor(sb + K::kOffLo);
#pragma unroll
                for (int k = 0; k < kC / 16; ++k) um::mma_ss(tmem + K::kST, yl + mnstep(k), zz + mnstep(k), id_state, 1);
#pragma unroll
                for (int k = 0; k < kC / 16; ++k) um::mma_ss(tmem + K::kST, yh + mnstep(k), zz + mnstep(k), id_state, 1);
                um::mma_commit(smem_u32(&m.sdone));
                um::mma_commit(smem_u32(&m.empty[slot(n, 0)]));
                um::mma_commit(smem_u32(&m.empty[slot(n, 2)]));
            }
            drain(m.drain, &m.abort);
        }
        __syncwarp();
    } else if (warp == kCopyWarp) {
        copy_tiles<DX, DZ, 3, K::kSlots, K::kSlot>(g, p, sp, b, h, sb, m.full, m.empty, wait);
    } else if (warp >= 8) {
        // ================================================ the split of y
        const int t = 32 * quarter + lane;
#pragma unroll 1
        for (int n = 0; n < nch; ++n) {
            const int L = sp.tokens(n);
            const float w = p.s_u * (rev ? m.pw[t + 1] : m.pw[max(L - 1 - t, 0)]);
            if (!wait.all(m.full[slot(n, 0)], phase(n, 0))) break;
            if (!wait.all(m.pfull, (uint32_t)n & 1u)) break;                  // the scores have read y
            if (n && !wait.all(m.sdone, (uint32_t)(n - 1) & 1u)) break;       // the state has read the other term
            split_y<DX, 2, 1>(tile(n, 0), sb + K::kOffLo, 0, t, 0, w);
            um::fence_proxy_async();
            arrive(m.yfull);
        }
    } else if (warp >= 4) {
        // ================================================ the state's decay and its bf16 copy
        const int d = 32 * quarter + lane;
        const bool mine = 32 * quarter < DX;  // this warp's lanes hold rows of the state
        const uint32_t ts = tl + K::kST;
        const float* s0 = p.carried ? a.work + blockIdx.z * a.pass_floats + ((size_t)bh * a.nseg + sg) * a.state_floats
                          : p.s_in    ? p.s_in + (size_t)bh * p.dx * p.dz
                                      : nullptr;
        const bool trans = !p.carried && p.in_trans, on = s0 && d < p.dx;
        if (mine) {
#pragma unroll 1
            for (int n0 = 0; n0 < DZ; n0 += 16) {
                uint32_t r[16];
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (on && n0 + i < p.dz) {
                        if (trans) {
                            const float* q = s0 + (size_t)(n0 + i) * p.dx + d;
                            v = make_float4(q[0], q[p.dx], q[2 * p.dx], q[3 * p.dx]);
                        } else {
                            v = *reinterpret_cast<const float4*>(s0 + (size_t)d * p.dz + n0 + i);
                        }
                    }
                    r[i] = as_u(v.x), r[i + 1] = as_u(v.y), r[i + 2] = as_u(v.z), r[i + 3] = as_u(v.w);
                }
                um::st32x32_x16(ts + n0, r);
            }
            um::wait_st();
        }
#pragma unroll 1
        for (int n = 0; n < nch; ++n) {
            const float f = m.pw[sp.tokens(n)];
            if (n && !wait.all(m.sdone, (uint32_t)(n - 1) & 1u)) break;
            um::fence_after();
            if (mine) {
                const uint32_t dst = sb + K::kOffS + (uint32_t)d * 16u;
#pragma unroll 1
                for (int n0 = 0; n0 < DZ; n0 += 32) {
                    uint32_t r[32];
                    um::ld32x32_x32(ts + n0, r);
                    um::wait_ld<32>(r);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        sts128(dst + (uint32_t)(n0 / 8 + q) * (DX * 16u), pack2(as_f(r[8 * q]), as_f(r[8 * q + 1])),
                               pack2(as_f(r[8 * q + 2]), as_f(r[8 * q + 3])), pack2(as_f(r[8 * q + 4]), as_f(r[8 * q + 5])),
                               pack2(as_f(r[8 * q + 6]), as_f(r[8 * q + 7])));
#pragma unroll
                    for (int i = 0; i < 32; ++i) r[i] = as_u(f * as_f(r[i]));
                    um::st32x32_x16(ts + n0, r);
                    um::st32x32_x16(ts + n0 + 16, r + 16);
                }
                um::wait_st();
            }
            um::fence_proxy_async();
            arrive(m.sfull);
        }
    } else {
        // ================================================ scores -> P', outputs
        const int i = 32 * quarter + lane;
        __nv_bfloat16* out = (__nv_bfloat16*)p.out + b * p.so.batch + h * p.so.head + sp.first * p.so.token;
        const bool wide = ((reinterpret_cast<uintptr_t>(p.out) & 31u) == 0) &&
                          ((p.so.batch | p.so.head | p.so.token) % 16 == 0);
        const uint32_t keep = rev ? 0xffffffffu << lane : 0xffffffffu >> (31 - lane);
        const float* diag = m.dt + 31 - lane;
#pragma unroll 1
        for (int n = 0; n < nch; ++n) {
            const uint32_t par = (uint32_t)n & 1u;
            const int L = sp.tokens(n);
            if (!wait.all(m.pfull, par)) break;
            um::fence_after();
#pragma unroll 1
            for (int jb = 0; jb < 4; ++jb) {
                uint32_t o[16];
                if (rev ? jb >= quarter : jb <= quarter) {
                    uint32_t r[32];
                    um::ld32x32_x32(tl + K::kP + 32u * jb, r);
                    um::wait_ld<32>(r);
                    if (jb == quarter) {
#pragma unroll
                        for (int c = 0; c < 32; ++c) r[c] = keep >> c & 1u ? as_u(as_f(r[c]) * diag[c]) : 0u;
                    } else {
                        // a^|i-j| = a^(distance to the block's near column) a^(from there)
                        const float f = p.s_p * m.pw[rev ? 32 * jb - i : i - 32 * jb - 31];
#pragma unroll
                        for (int c = 0; c < 32; c += 4) {
                            const float4 k = *reinterpret_cast<const float4*>(m.ct + c);
                            r[c] = as_u(as_f(r[c]) * (f * k.x));
                            r[c + 1] = as_u(as_f(r[c + 1]) * (f * k.y));
                            r[c + 2] = as_u(as_f(r[c + 2]) * (f * k.z));
                            r[c + 3] = as_u(as_f(r[c + 3]) * (f * k.w));
                        }
                    }
#pragma unroll
                    for (int c = 0; c < 16; ++c) o[c] = pack2(as_f(r[2 * c]), as_f(r[2 * c + 1]));
                } else {
#pragma unroll
                    for (int c = 0; c < 16; ++c) o[c] = 0u;
                }
                um::st32x32_x16(tl + K::kP + 16u * jb, o);
            }
            um::wait_st();
            arrive(m.pready);
            const float f = p.s_i * (rev ? m.pw[max(L - 1 - i, 0)] : m.pw[i + 1]);
            __nv_bfloat16* row = out + (sp.start(n) + i) * p.so.token;
            if (!wait.all(m.ofull, par)) break;
            um::fence_after();
#pragma unroll 1
            for (int n0 = 0; n0 < DZ; n0 += 16) {
                uint32_t ra[16], ri[16], o[8];
                um::ld32x32_x16(tl + K::kOA + n0, ra);
                um::ld32x32_x16(tl + K::kOI + n0, ri);
                um::wait_ld<16>(ra);
                um::wait_ld<16>(ri);
                if (n0 + 16 >= DZ) arrive(m.ofree);
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    o[c] = pack2(fmaf(f, as_f(ri[2 * c]), as_f(ra[2 * c])), fmaf(f, as_f(ri[2 * c + 1]), as_f(ra[2 * c + 1])));
                if (i < L) {
                    if (wide && n0 + 16 <= p.dz) {
                        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(row + n0), "r"(o[0]),
                                     "r"(o[1]), "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                                     : "memory");
                    } else {
                        if (n0 < p.dz) *reinterpret_cast<uint4*>(row + n0) = make_uint4(o[0], o[1], o[2], o[3]);
                        if (n0 + 8 < p.dz) *reinterpret_cast<uint4*>(row + n0 + 8) = make_uint4(o[4], o[5], o[6], o[7]);
                    }
                }
            }
        }
        // rows behind the sequence
        for (int64_t e = tid; e < (sp.rows - sp.live) * (p.dz / 8); e += 128)
            *reinterpret_cast<uint4*>(out + (sp.live + e / (p.dz / 8)) * p.so.token + 8 * (e % (p.dz / 8))) =
                make_uint4(0u, 0u, 0u, 0u);
    }
    um::fence_before();
    __syncthreads();
    um::fence_after();
    if (warp == kMmaWarp) um::tmem_dealloc(tmem, K::kCols);
    if (tid == 0 && m.abort) atomicExch(g.err, 1);
}

// ---------------------------------------------------------------- the segments' own states
template <int DX, int DZ>
struct States {
    static constexpr bool kTwo = DX == 64 && DZ == 64;
    static constexpr uint32_t kSlot = (uint32_t)(DX > DZ ? DX : DZ) * 256u;
    static constexpr uint32_t kLo = (uint32_t)DX * 256u;
    static constexpr int kSlots = kTwo ? 4 : 5;
    static constexpr uint32_t kOffLo = kSlots * kSlot, kOffTail = kOffLo + 2 * kLo;
    static constexpr uint32_t kTail = DX == 64 ? 16384u : 2048u;  // as in Main: rows 64 .. 127 of the last term
    static constexpr uint32_t kBytes = kOffTail + kTail;
    static constexpr uint32_t kU = 0, kST = 2 * DZ;                // two buffers of a chunk's contribution, the state
    static constexpr uint32_t kCols = DZ == 64 ? 256 : 512;
    static constexpr int kThreads = 3 * 128 + 64;
};
struct StatesTail {
    uint64_t full[5], empty[5], yfull, lofree, ufull[2], ufree[2], drain;
    float pw[kLaPowers];
    uint32_t tmem;
    int abort;
};

template <int DX, int DZ>
__global__ void __launch_bounds__((States<DX, DZ>::kThreads), (States<DX, DZ>::kTwo ? 2 : 1))
la_states(const __grid_constant__ Args g) {
    using K = States<DX, DZ>;
    static_assert(sizeof(StatesTail) <= K::kTail, "the tail holds the barriers and tables");
    extern __shared__ __align__(1024) uint8_t smem[];
    StatesTail& m = *reinterpret_cast<StatesTail*>(smem + K::kOffTail);
    const la::Args& a = g.a;
    const LaPass& p = a.p[blockIdx.z];
    if (!p.carried) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int sg = blockIdx.x, bh = blockIdx.y, b = bh / a.H, h = bh % a.H;
    const Span sp(a, p, sg, b);
    const int nch = sp.nch;
    const uint32_t sb = smem_u32(smem);
    const Waiter wait{&m.abort, g.limit};
    constexpr int kMmaWarp = 12, kCopyWarp = 13;

    if (tid == 0) {
        for (int i = 0; i < K::kSlots; ++i) {
            um::mbar_init(smem_u32(&m.full[i]), 1);
            um::mbar_init(smem_u32(&m.empty[i]), 1);
        }
        um::mbar_init(smem_u32(&m.yfull), 8);
        um::mbar_init(smem_u32(&m.lofree), 1);
        for (int i = 0; i < 2; ++i) {
            um::mbar_init(smem_u32(&m.ufull[i]), 1);
            um::mbar_init(smem_u32(&m.ufree[i]), 4);
        }
        um::mbar_init(smem_u32(&m.drain), 1);
        m.abort = 0;
    }
    for (int i = tid; i < kLaPowers; i += K::kThreads) m.pw[i] = a.pw[(size_t)h * kLaPowers + i];
    if (warp == kMmaWarp) {
        um::tmem_alloc(smem_u32(&m.tmem), K::kCols);
        um::tmem_relinquish();
    }
    um::fence_before();
    __syncthreads();
    um::fence_after();
    const uint32_t tmem = m.tmem;
    const int quarter = warp & 3;
    auto slot = [](int n, int item) { return (2 * n + item) % K::kSlots; };
    auto phase = [](int n, int item) { return (uint32_t)((2 * n + item) / K::kSlots) & 1u; };
    auto tile = [&](int n, int item) { return sb + (uint32_t)slot(n, item) * K::kSlot; };

    if (warp == kMmaWarp) {
        if (lane == 0) {
            constexpr uint32_t id = um::idesc_bf16(128, DZ) | um::kAmn | um::kBmn;
#pragma unroll 1
            for (int n = 0; n < nch; ++n) {
                const uint32_t u = tmem + K::kU + (uint32_t)(n & 1) * DZ;
                const uint64_t zz = mnmajor(tile(n, 1)), yh = mnmajor(tile(n, 0)), y1 = mnmajor(sb + K::kOffLo),
                               y2 = mnmajor(sb + K::kOffLo + K::kLo);
                if (!wait(m.full[slot(n, 1)], phase(n, 1))) break;
                if (n > 1 && !wait(m.ufree[n & 1], (uint32_t)(n / 2 - 1) & 1u)) break;
                if (!wait(m.yfull, (uint32_t)n & 1u)) break;
                um::fence_after();
                // the smallest terms first: fewer truncations next to a large sum
#pragma unroll
                for (int k = 0; k < kC / 16; ++k) um::mma_ss(u, y2 + mnstep(k), zz + mnstep(k), id, k > 0);
#pragma unroll
                for (int k = 0; k < kC / 16; ++k) um::mma_ss(u, y1 + mnstep(k), zz + mnstep(k), id, 1);
                um::mma_commit(smem_u32(&m.lofree));
#pragma unroll
                for (int k = 0; k < kC / 16; ++k) um::mma_ss(u, yh + mnstep(k), zz + mnstep(k), id, 1);
                um::mma_commit(smem_u32(&m.ufull[n & 1]));
                um::mma_commit(smem_u32(&m.empty[slot(n, 0)]));
                um::mma_commit(smem_u32(&m.empty[slot(n, 1)]));
            }
            drain(m.drain, &m.abort);
        }
        __syncwarp();
    } else if (warp == kCopyWarp) {
        copy_tiles<DX, DZ, 2, K::kSlots, K::kSlot>(g, p, sp, b, h, sb, m.full, m.empty, wait);
    } else if (warp >= 4) {
        // ================================================ the split of y: 8 warps
        const int t = 32 * quarter + lane, q = (warp - 4) / 4;
#pragma unroll 1
        for (int n = 0; n < nch; ++n) {
            const int L = sp.tokens(n);
            const float w = p.s_u * (sp.rev ? m.pw[t + 1] : m.pw[max(L - 1 - t, 0)]);
            if (!wait.all(m.full[slot(n, 0)], phase(n, 0))) break;
            if (n && !wait.all(m.lofree, (uint32_t)(n - 1) & 1u)) break;
            split_y<DX, 3, 2>(tile(n, 0), sb + K::kOffLo, K::kLo, t, q, w);
            um::fence_proxy_async();
            arrive(m.yfull);
        }
    } else {
        // ================================================ S <- a^L S + U
        const int d = 32 * quarter + lane;
        const bool mine = 32 * quarter < DX;
        const uint32_t tl = tmem + ((uint32_t)(32 * quarter) << 16), ts = tl + K::kST;
        float* out = a.work + blockIdx.z * a.pass_floats + ((size_t)bh * a.nseg + sg) * a.state_floats + (size_t)d * p.dz;
        bool ok = true;
#pragma unroll 1
        for (int n = 0; n < nch; ++n) {
            const float f = m.pw[sp.tokens(n)];
            if (!(ok = wait.all(m.ufull[n & 1], (uint32_t)(n / 2) & 1u))) break;
            um::fence_after();
            const uint32_t tu = tl + K::kU + (uint32_t)(n & 1) * DZ;
            if (mine) {
#pragma unroll 1
                for (int n0 = 0; n0 < DZ; n0 += 16) {
                    uint32_t u[16], s[16];
                    um::ld32x32_x16(tu + n0, u);
                    if (n) um::ld32x32_x16(ts + n0, s);
                    um::wait_ld<16>(u);
                    um::wait_ld<16>(s);
#pragma unroll
                    for (int i = 0; i < 16; ++i) u[i] = n ? as_u(fmaf(f, as_f(s[i]), as_f(u[i]))) : u[i];
                    um::st32x32_x16(ts + n0, u);
                }
                um::wait_st();
            }
            arrive(m.ufree[n & 1]);
        }
        if (ok && mine) {
#pragma unroll 1
            for (int n0 = 0; n0 < DZ; n0 += 16) {
                uint32_t r[16];
                if (nch) {
                    um::ld32x32_x16(ts + n0, r);
                    um::wait_ld<16>(r);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) r[i] = 0u;
                }
                if (d < p.dx) {
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        if (n0 + i < p.dz)
                            *reinterpret_cast<float4*>(out + n0 + i) =
                                make_float4(as_f(r[i]), as_f(r[i + 1]), as_f(r[i + 2]), as_f(r[i + 3]));
                }
            }
        }
    }
    um::fence_before();
    __syncthreads();
    um::fence_after();
    if (warp == kMmaWarp) um::tmem_dealloc(tmem, K::kCols);
    if (tid == 0 && m.abort) atomicExch(g.err, 1);
}

// ---------------------------------------------------------------- host
typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
    static const EncodeFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        if (!ok) cudaGetLastError();
        return ok ? (EncodeFn)f : nullptr;
    }();
    return fn;
}

// The map of a tensor [B][H][N][d]: dimensions in the order of their strides, those that do not move left out.
void describe(Source* s, const void* ptr, const fftconv_strides& st, int B, int H, int64_t N, int d) {
    struct Dim {
        int64_t extent, stride;
        int* at;
    } dim[3] = {{N, st.token, &s->at_token}, {H, st.head, &s->at_head}, {B, st.batch, &s->at_row}};
    s->at_token = s->at_head = s->at_row = 0;
    s->by_hand = 1;
    const EncodeFn enc = encoder();
    if (!enc || (N > 1 && st.token == 0) || N > 0x7fffffff) return;
    int n = 0;
    Dim use[3];
    for (const Dim& x : dim)
        if (x.extent > 1 && x.stride != 0) use[n++] = x;
    for (int i = 1; i < n; ++i)
        for (int j = i; j > 0 && use[j].stride < use[j - 1].stride; --j) {
            const Dim t = use[j];
            use[j] = use[j - 1];
            use[j - 1] = t;
        }
    cuuint64_t dims[4] = {(cuuint64_t)d, 1, 1, 1}, strides[3];
    cuuint32_t box[4] = {64, 1, 1, 1}, one[4] = {1, 1, 1, 1};
    cuuint64_t last = (cuuint64_t)d * 2;
    for (int i = 0; i < 3; ++i) {
        if (i < n) {
            dims[i + 1] = (cuuint64_t)use[i].extent;
            last = (cuuint64_t)use[i].stride * 2;
            *use[i].at = i + 1;
            if (use[i].at == &s->at_token) box[i + 1] = kC;
        }
        strides[i] = last;
    }
    if (N == 1) {  // one token: the box still has 128 rows, the others out of range
        for (int i = 0; i < 3; ++i)
            if (i == n) {
                s->at_token = i + 1;
                box[i + 1] = kC;
            }
    }
    if (enc(&s->map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS)
        s->by_hand = 0;
}

template <int DX, int DZ>
cudaError_t run(const Args& g, int bh, int passes, bool states, cudaStream_t s) {
    const dim3 grid(g.a.nseg, bh, passes);
    cudaError_t e;
    if (states) {
        using K = States<DX, DZ>;
        if ((e = la::allow<la_states<DX, DZ>>((int)K::kBytes)) != cudaSuccess) return e;
        la_states<DX, DZ><<<grid, K::kThreads, K::kBytes, s>>>(g);
    } else {
        using K = Main<DX, DZ>;
        if ((e = la::allow<la_main<DX, DZ>>((int)K::kBytes)) != cudaSuccess) return e;
        la_main<DX, DZ><<<grid, K::kThreads, K::kBytes, s>>>(g);
    }
    return cudaGetLastError();
}

}  // namespace latc

namespace la {

cudaError_t launch_tc(const Args& a, int dx, int dz, int B, int passes, bool states, const fftconv_linattn_s& p,
                      cudaStream_t s) {
    latc::Args g;
    g.a = a;
    g.err = p.d_err;
    g.limit = p.wait_limit;
    // the passes share their tensors: q, k, v (and do)
    struct {
        const void* ptr;
        fftconv_strides st;
        int d;
    } seen[latc::kMaxSources];
    int n = 0;
    auto source = [&](const void* q, const fftconv_strides& st, int d) {
        for (int i = 0; i < n; ++i)
            if (seen[i].ptr == q && seen[i].d == d && seen[i].st.batch == st.batch && seen[i].st.head == st.head &&
                seen[i].st.token == st.token)
                return i;
        latc::describe(&g.src[n], q, st, B, a.H, a.N, d);
        seen[n] = {q, st, d};
        return n++;
    };
    for (int i = 0; i < passes; ++i) {
        const LaPass& q = a.p[i];
        g.x[i] = source(q.x, q.sx, q.dx);
        g.y[i] = source(q.y, q.sy, q.dx);
        g.z[i] = source(q.z, q.sz, q.dz);
    }
    const int bh = B * a.H;
    if (dx <= 64)
        return dz <= 64 ? latc::run<64, 64>(g, bh, passes, states, s) : latc::run<64, 128>(g, bh, passes, states, s);
    return dz <= 64 ? latc::run<128, 64>(g, bh, passes, states, s) : latc::run<128, 128>(g, bh, passes, states, s);
}

}  // namespace la
}  // namespace fftc
