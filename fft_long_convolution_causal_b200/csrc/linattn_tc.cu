// linattn_tc.cu -- decayed linear attention on the fifth-generation tensor cores
// (bf16 operands, fp32 accumulators in tensor memory), chunks of 128 tokens.
//
// la_main: a CTA walks the chunks of one (segment, row, head, pass) with the
// state S [dx][dz] resident in tensor memory.  Per chunk of L live tokens:
//   scores  P = X Y^T                                    (128 x 128 x DX)
//   inter   O = X bf16(S), its rows times s_i a^(i+1)    (128 x DZ x DX)
//   intra   O += bf16(s_p a^|i-j| P, masked) Z           (128 x DZ x 128)
//   state   S = a^L S + (s_u a^(L-1-j) y_j)^T Z          (DX x DZ x 128, two products)
// Eight warps turn scores into P' and then split y; four do the state's decay and
// bf16 copy, the scaling of O's rows and the outputs.  One warp issues products,
// in the order inter, intra, state, next scores, so that a chunk's scores are
// weighed and its y split while the state and the next copies are under way; one
// warp issues copies.  Probing a barrier costs about 100 cycles and handing over
// through one 116, so each step waits for one barrier that several arrive at.
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
//
// Rounded to bf16 once each: P' and the copy of S that inter reads (each off by
// up to 2^-8 of a value), and the outputs: 2.4e-3 in the 2-norm, 1.7e-3 of it theirs.  la_main's
// own S stays in the accumulator: what its truncation (7e-6 over 256 chunks) and a
// decay rounded to fp32 (2^-25 a chunk) cost is far below that.
//
// Bound by shared memory (operands of the products, tiles in and out, P' and the
// split: 4500 cycles of it a chunk of 128 x 128, which takes 5900) and, in long
// runs, by power.  16 heads x 32768 tokens x 128: la_states 71 us (3.8 TB/s),
// la_main 114 us (4.7 TB/s), each alone; the call 182 us, 218 at the 1.56 GHz
// that the power limit leaves.
#include <cuda.h>
#include <cuda_bf16.h>

#include <numeric>

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
// (x, y) times a plus (u, v), two a time
__device__ __forceinline__ void fma2(float a, uint32_t x, uint32_t y, uint32_t& u, uint32_t& v) {
    asm("{\n.reg .b64 p, q, r;\nmov.b64 p, {%2, %3};\nmov.b64 q, {%4, %4};\nmov.b64 r, {%0, %1};\nfma.rn.f32x2 r, p, q, r;\n"
        "mov.b64 {%0, %1}, r;\n}\n"
        : "+r"(u), "+r"(v)
        : "r"(x), "r"(y), "f"(a));
}
// (x, y) times (a, b), two products an instruction
__device__ __forceinline__ void mul2(float& x, float& y, float a, float b) {
    asm("{\n.reg .b64 p, q;\nmov.b64 p, {%0, %1};\nmov.b64 q, {%2, %3};\nmul.rn.f32x2 p, p, q;\nmov.b64 {%0, %1}, p;\n}\n"
        : "+f"(x), "+f"(y)
        : "f"(a), "f"(b));
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
// a block of a tile out to global memory; rows and elements out of range are not written
__device__ __forceinline__ void tma_store_4d(const void* map, uint32_t src, int c0, int c1, int c2, int c3) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
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
    int head_step, row_step;        // coordinates from one to the next
    int by_hand;                    // no map: copied with plain loads
    __device__ __forceinline__ int at(int dim, int t, int h, int b) const {
        return (at_token == dim ? t : 0) + (at_head == dim ? h * head_step : 0) + (at_row == dim ? b * row_step : 0);
    }
};
constexpr int kMaxSources = 4 + kLaMaxPasses;
struct Args {
    la::Args a;
    Source src[kMaxSources];
    int x[kLaMaxPasses], y[kLaMaxPasses], z[kLaMaxPasses], out[kLaMaxPasses];  // maps of each pass
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
        for (uint32_t i = 0; !um::mbar_try_wait(ad, parity); ++i)
            if (*abort || i >= limit) {
                *abort = 1;
                return false;
            }
        return true;
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
    __device__ __forceinline__ Span(const la::Args& a, const LaPass& p, const la::Place& at, int b) {
        first = at.first;
        rows = at.tokens;
        live = max((int64_t)0, min(rows, la::live_tokens(a, b) - first));
        nch = (int)((live + kC - 1) / kC);
        rev = p.reverse;
    }
    // first token (in the segment) and live tokens of the n-th chunk of the walk
    __device__ __forceinline__ int64_t start(int n) const { return (int64_t)(rev ? nch - 1 - n : n) * kC; }
    __device__ __forceinline__ int tokens(int n) const { return (int)min((int64_t)kC, live - start(n)); }
};

// The copying warp's view: which tile is copied where.
struct Copier {
    const Args& g;
    const LaPass& p;
    const Span& sp;
    int pass, b, h;
    const Waiter& wait;
    // Tile `what` (0 y, 1 x, 2 z) of chunk n to dst, the use-th copy there, once the one before was left; false: a wait
    // gave up.
    __device__ __forceinline__ bool operator()(int what, int blocks, int n, uint32_t dst, const uint64_t& full,
                                               const uint64_t& empty, int use) const {
        const int lane = threadIdx.x & 31;
        if (use > 0 && !wait.all(empty, (uint32_t)(use - 1) & 1u)) return false;
        const int64_t t0 = sp.start(n);
        const int L = sp.tokens(n);
        const Source& src = g.src[what == 2 ? g.z[pass] : what == 1 ? g.x[pass] : g.y[pass]];
        const uint32_t bar = smem_u32(&full);
        if (src.by_hand || (L < kC && sp.first + t0 + L < g.a.N)) {
            // rows behind the length are zeros whatever memory holds
            const fftconv_strides& st = what == 2 ? p.sz : what == 1 ? p.sx : p.sy;
            const __nv_bfloat16* base = (const __nv_bfloat16*)(what == 2 ? p.z : what == 1 ? p.x : p.y) + b * st.batch +
                                        h * st.head + (sp.first + t0) * st.token;
            const int d = what == 2 ? p.dz : p.dx;
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
            const int c1 = src.at(1, t, h, b), c2 = src.at(2, t, h, b), c3 = src.at(3, t, h, b);
            um::mbar_arrive_expect_tx(bar, (uint32_t)blocks * kBlock);
#pragma unroll 1
            for (int k = 0; k < blocks; ++k)
                tma_load_4d(dst + (uint32_t)k * kBlock, &src.map, 64 * k, c1, c2, c3, bar);
        }
        __syncwarp();
        return true;
    }
};
// Probes for a copy in flight when a wait elsewhere gave up: it lands before the CTA ends.
constexpr uint32_t kLanding = 64;

// y decayed to the chunk's end, as a sum of NS bf16 terms: the first in place, the others `lo` apart.
// Thread (token t, part q of Q) takes every Q-th 16-byte column.
template <int DX, int NS, int Q>
__device__ __forceinline__ void split_y(uint32_t tile, uint32_t lo, uint32_t lo_step, int t, int q, float w) {
#pragma unroll 4
    for (int c = q; c < DX / 8; c += Q) {
        const uint32_t off = tile_off(t, c);
        const uint4 u = lds128(tile + off);
        const uint32_t in[4] = {u.x, u.y, u.z, u.w};
        uint32_t o[NS][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x = lo_f(in[i]), y = hi_f(in[i]);
            mul2(x, y, w, w);
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                o[s][i] = pack2(x, y);
                x -= lo_f(o[s][i]), y -= hi_f(o[s][i]);
            }
        }
        sts128(tile + off, o[0][0], o[0][1], o[0][2], o[0][3]);
#pragma unroll
        for (int s = 1; s < NS; ++s) sts128(lo + (uint32_t)(s - 1) * lo_step + off, o[s][0], o[s][1], o[s][2], o[s][3]);
    }
}

// One thread of a converged warp.  The issuing warp runs its loop as a whole, so that descriptors stay in uniform
// registers, and only the products themselves are elected (gradients of 4 x 16 x 4096 x 128: 210 -> 203 us).
__device__ __forceinline__ bool elect() {
    uint32_t r;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r != 0;
}

// 32 columns of row d of a state (zero: none) into tensor memory, all loads in flight together; trans: stored [dz][dx]
__device__ __forceinline__ void state_in(uint32_t ts, const float* s0, bool trans, const LaPass& p, int d, int n0) {
    uint32_t r[32];
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (s0 && d < p.dx && n0 + i < p.dz) {
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
    um::st32x32_x16(ts + n0 + 16, r + 16);
}

// Every product issued is complete before tensor memory is freed.
__device__ __forceinline__ void drain(uint64_t& bar, volatile int* abort) {
    if (elect()) um::mma_commit(smem_u32(&bar));
    __syncwarp();
    if (!um::mbar_wait(smem_u32(&bar), 0)) *abort = 1;
}

// ---------------------------------------------------------------- outputs
template <int DX, int DZ>
struct Main {
    static constexpr bool kTwo = DX == 64 && DZ == 64;  // two CTAs an SM
    static constexpr uint32_t kTX = (uint32_t)DX * 256u, kTZ = (uint32_t)DZ * 256u;  // bytes of a tile
    static constexpr uint32_t kS = (uint32_t)DX * DZ * 2u, kLo = kTX;
    // Five tiles: two of y, one of x, two of z.  x is done with after inter, y after the state's product, z after the
    // output staged in it has left: the next x, the next z and the y after next are requested in that order.
    // The state's product has 128 rows whatever DX is: with DX = 64 its descriptor reads 16 KiB behind
    // a term of y (rows nobody looks at), which has to be this CTA's memory.
    static constexpr uint32_t kOffLo = 3 * kTX + 2 * kTZ, kOffS = kOffLo + kLo, kOffTail = kOffS + kS;
    static constexpr uint32_t kTail = DX == 64 && kS < 16384u ? 16384u - kS : 2048u;
    static constexpr uint32_t kBytes = kOffTail + kTail;
    // tensor-memory columns: scores, O, the state.  P' (bf16) replaces the first quarter of each half of the scores:
    // the two warps of a row each overwrite only what they have read.
    // Where it has room, inter and intra have accumulators of their own and meet in the output's registers; where it
    // has not (two CTAs an SM), intra adds to inter's, whose rows are scaled in place first.
    static constexpr bool kApart = !kTwo;
    static constexpr uint32_t kP = 0, kO = 128, kOI = kApart ? kO + DZ : kO, kST = kOI + DZ, kCols = kTwo ? 256 : 512;
    static constexpr int kThreads = 3 * 128 + 64;
};
struct MainTail {
    uint64_t xy[2], zfull[2], empty[3], pfull, pored, iready, ifull, ofull, staged[2], yfull, sdone, drain;
    alignas(16) float ct[32];  // read four at a time
    float pw[kLaPowers], dt[64];
    uint32_t tmem;
    int abort;
};

template <int DX, int DZ>
__global__ void __launch_bounds__((Main<DX, DZ>::kThreads), (Main<DX, DZ>::kTwo ? 2 : 1))
la_main(const __grid_constant__ Args g) {
    using K = Main<DX, DZ>;
    static_assert(sizeof(MainTail) <= K::kTail && K::kOffTail % 16 == 0, "the tail holds the barriers and tables");
    extern __shared__ __align__(1024) uint8_t smem[];
    MainTail& m = *reinterpret_cast<MainTail*>(smem + K::kOffTail);
    const la::Args& a = g.a;
    const la::Place at(a);
    const LaPass& p = a.p[at.pass];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bh = at.bh, b = bh / a.H, h = bh % a.H;
    const Span sp(a, p, at, b);
    const bool rev = sp.rev;
    const int nch = sp.nch;
    const uint32_t sb = smem_u32(smem);
    const Waiter wait{&m.abort, g.limit};
    constexpr int kMmaWarp = 12, kCopyWarp = 13;
    // tile `item` (0 y, 1 x, 2 z) of chunk n: its barrier, how often its place was used before, and where that is
    auto slot = [](int n, int item) { return item == 1 ? 2 : n & 1; };
    auto use = [](int n, int item) { return item == 1 ? n : n >> 1; };
    auto tile = [&](int n, int item) {
        return sb + (item == 1 ? 2 * K::kTX : item == 0 ? (uint32_t)(n & 1) * K::kTX : 3 * K::kTX + (uint32_t)(n & 1) * K::kTZ);
    };
    const Copier copy{g, p, sp, at.pass, b, h, wait};
    auto load = [&](int n, int item) {
        if (n >= nch) return true;
        // z's place is free once the outputs staged there have left (this warp's own bulk copy)
        if (item == 2) {
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            __syncwarp();
        }
        return copy(item, (item == 2 ? DZ : DX) / 64, n, tile(n, item), item == 2 ? m.zfull[n & 1] : m.xy[n & 1],
                    m.empty[item == 2 ? 0 : slot(n, item)], item == 2 ? 0 : use(n, item));
    };
    // the outputs of chunk n, staged in z's tile, go out as a bulk copy
    auto store = [&](int n) {
        if (!wait.all(m.staged[n & 1], (uint32_t)(n >> 1) & 1u)) return false;
        if (lane == 0) {
            const Source& so = g.src[g.out[at.pass]];
            const int tk = (int)(sp.first + sp.start(n));
            const int c1 = so.at(1, tk, h, b), c2 = so.at(2, tk, h, b), c3 = so.at(3, tk, h, b);
#pragma unroll 1
            for (int k = 0; k < DZ / 64; ++k)
                if (64 * k < p.dz) tma_store_4d(&so.map, tile(n, 2) + (uint32_t)k * kBlock, 64 * k, c1, c2, c3);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
        __syncwarp();
        return true;
    };
    // the order of the copies: y0, then x, z of chunk k, y of chunk k + 1 and the outputs of chunk k - 1
    auto load_next = [&](int i) {
        const int k = i ? (i - 1) / 3 : -1, r = i ? (i - 1) % 3 : 2;
        return r == 2 ? load(k + 1, 0) && (k < 1 || store(k - 1)) : load(k, r + 1);
    };

    if (tid == 32 * kCopyWarp) {
        for (int i = 0; i < 2; ++i) {
            um::mbar_init(smem_u32(&m.xy[i]), 2);
            um::mbar_init(smem_u32(&m.zfull[i]), 1);
            um::mbar_init(smem_u32(&m.staged[i]), 4);  // two: a chunk may be staged before the last one is seen
        }
        for (int i = 0; i < 3; ++i) um::mbar_init(smem_u32(&m.empty[i]), 1);
        um::mbar_init(smem_u32(&m.pfull), 1);
        um::mbar_init(smem_u32(&m.pored), K::kApart ? 8 : 12);  // P' in place, O's rows scaled
        um::mbar_init(smem_u32(&m.iready), 4);  // the state decayed and copied, O read
        um::mbar_init(smem_u32(&m.ifull), 1);
        um::mbar_init(smem_u32(&m.ofull), 1);
        um::mbar_init(smem_u32(&m.yfull), 8);
        um::mbar_init(smem_u32(&m.sdone), 1);
        um::mbar_init(smem_u32(&m.drain), 1);
        m.abort = g.limit == 0;  // no wait at all: the first that would gives up
    }
    constexpr int kFirst = 4;  // the first copies need not wait for the other warps
    if (warp == kCopyWarp) {
        __syncwarp();
#pragma unroll 1
        for (int i = 0; i < kFirst; ++i) load_next(i);
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
    la::let_next_start();
    const uint32_t tmem = m.tmem;
    const int quarter = warp & 3;
    const uint32_t tl = tmem + ((uint32_t)(32 * quarter) << 16);
    if (warp == kMmaWarp) {
        constexpr uint32_t id_scores = um::idesc_bf16(128, 128), id_inter = um::idesc_bf16(128, DZ) | um::kBmn,
                           id_state = id_inter | um::kAmn;
        const uint64_t ds = um::sdesc(sb + K::kOffS, 128, DX * 16), kx = kmajor(tile(0, 1)), yl = mnmajor(sb + K::kOffLo);
        // chunk n of the walk, -1: the first chunk's scores
#pragma unroll 1
        for (int n = -1; n < nch; ++n) {
            const uint32_t par = (uint32_t)n & 1u, half = (uint32_t)(n >> 1) & 1u;
            if (n >= 0) {
                const uint64_t zz = mnmajor(tile(n, 2)), yh = mnmajor(tile(n, 0));
                if (!wait.all(m.iready, par)) break;
                um::fence_after();
                if (elect()) {
#pragma unroll
                    for (int k = 0; k < DX / 16; ++k)
                        um::mma_ss(tmem + K::kOI, kx + kstep(k), ds + (uint64_t)(k * 16), id_inter, k > 0);
                    if (!K::kApart) um::mma_commit(smem_u32(&m.ifull));
                    um::mma_commit(smem_u32(&m.empty[2]));
                }
                __syncwarp();
                if (!wait.all(m.zfull[n & 1], half) || !wait.all(m.pored, par)) break;
                um::fence_after();
                if (elect()) {
#pragma unroll
                    for (int k = 0; k < kC / 16; ++k)
                        um::mma_ts(tmem + K::kO, tmem + K::kP + (k / 4) * 64u + (k % 4) * 8u, zz + mnstep(k), id_inter, !K::kApart || k > 0);
                    um::mma_commit(smem_u32(&m.ofull));
                }
                __syncwarp();
                if (n + 1 < nch) {  // nobody reads the state behind the last chunk
                    if (!wait.all(m.yfull, par)) break;
                    um::fence_after();
                    if (elect()) {
#pragma unroll
                        for (int k = 0; k < kC / 16; ++k)
                            um::mma_ss(tmem + K::kST, yl + mnstep(k), zz + mnstep(k), id_state, 1);
#pragma unroll
                        for (int k = 0; k < kC / 16; ++k)
                            um::mma_ss(tmem + K::kST, yh + mnstep(k), zz + mnstep(k), id_state, 1);
                        um::mma_commit(smem_u32(&m.sdone));
                        um::mma_commit(smem_u32(&m.empty[n & 1]));
                    }
                    __syncwarp();
                }
            }
            if (n + 1 < nch) {
                const int c = n + 1;
                const uint64_t ky = kmajor(tile(c, 0));
                if (!wait.all(m.xy[c & 1], (uint32_t)(c >> 1) & 1u)) break;
                um::fence_after();
                if (elect()) {
#pragma unroll
                    for (int k = 0; k < DX / 16; ++k)
                        um::mma_ss(tmem + K::kP, kx + kstep(k), ky + kstep(k), id_scores, k > 0);
                    um::mma_commit(smem_u32(&m.pfull));
                }
                __syncwarp();
            }
        }
        drain(m.drain, &m.abort);
    } else if (warp == kCopyWarp) {
        bool ok = !*wait.abort;
        int i = kFirst;
#pragma unroll 1
        for (; i <= 3 * nch && ok; ++i) ok = load_next(i);
        if (ok && nch) ok = store(nch - 1);
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        if (!ok || *wait.abort) {  // copies of the last chunks may be in flight
            const int n = (i - 1) / 3;
            for (int c = n > 1 ? n - 1 : 0; c <= n + 1 && c < nch; ++c) {
                um::mbar_wait(smem_u32(&m.zfull[c & 1]), (uint32_t)(c >> 1) & 1u, kLanding);
                um::mbar_wait(smem_u32(&m.xy[c & 1]), (uint32_t)(c >> 1) & 1u, kLanding);
            }
        }
    } else if (warp >= 4 && warp < 8) {
        // ================================================ the state's decay and bf16 copy, O's rows, outputs
        const int d = 32 * quarter + lane;
        const bool mine = 32 * quarter < DX;  // this warp's lanes hold rows of the state
        const uint32_t ts = tl + K::kST;
        const float* s0 = at.split ? a.work + at.state : p.s_in ? p.s_in + (size_t)bh * p.dx * p.dz : nullptr;
        la::after_previous();  // the states entering the segments
        if (mine) {
#pragma unroll 1
            for (int n0 = 0; n0 < DZ; n0 += 32) state_in(ts, s0, !at.split && p.in_trans, p, d, n0);
            um::wait_st();
        }
        uint32_t o[DZ / 2];  // a row of O in bf16
        // through z's tile (all products have read it), then out as a bulk copy
        auto stage = [&](int n) {
            const uint32_t tz = tile(n, 2);
#pragma unroll
            for (int c = 0; c < DZ / 8; ++c) sts128(tz + tile_off(d, c), o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
            um::fence_proxy_async();
            arrive(m.staged[n & 1]);
        };
        bool ok = true;
#pragma unroll 1
        for (int n = 0; n < nch && ok; ++n) {
            const int L = sp.tokens(n);
            const float f = m.pw[L];
            if (mine) {
                const uint32_t dst = sb + K::kOffS + (uint32_t)d * 16u;
#pragma unroll 1
                for (int n0 = 0; n0 < DZ; n0 += 16) {
                    uint32_t r[16];
                    um::ld32x32_x16(ts + n0, r);
                    um::wait_ld<16>(r);
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        sts128(dst + (uint32_t)(n0 / 8 + q) * (DX * 16u), pack2(as_f(r[8 * q]), as_f(r[8 * q + 1])),
                               pack2(as_f(r[8 * q + 2]), as_f(r[8 * q + 3])), pack2(as_f(r[8 * q + 4]), as_f(r[8 * q + 5])),
                               pack2(as_f(r[8 * q + 6]), as_f(r[8 * q + 7])));
#pragma unroll
                    for (int i = 0; i < 16; ++i) r[i] = as_u(f * as_f(r[i]));
                    um::st32x32_x16(ts + n0, r);
                }
                um::wait_st();
            }
            um::fence_proxy_async();
            arrive(m.iready);
            if (n) stage(n - 1);
            const float fo = p.s_i * (rev ? m.pw[max(L - 1 - d, 0)] : m.pw[d + 1]);
            if (!K::kApart) {
                if (!(ok = wait.all(m.ifull, (uint32_t)n & 1u))) break;
                um::fence_after();
#pragma unroll 1
                for (int n0 = 0; n0 < DZ; n0 += 16) {
                    uint32_t r[16];
                    um::ld32x32_x16(tl + K::kO + n0, r);
                    um::wait_ld<16>(r);
#pragma unroll
                    for (int i = 0; i < 16; ++i) r[i] = as_u(fo * as_f(r[i]));
                    um::st32x32_x16(tl + K::kO + n0, r);
                }
                um::wait_st();
                arrive(m.pored);
            }
            if (!(ok = wait.all(m.ofull, (uint32_t)n & 1u))) break;
            um::fence_after();
#pragma unroll
            for (int n0 = 0; n0 < DZ; n0 += 16) {
                uint32_t r[16];
                um::ld32x32_x16(tl + K::kO + n0, r);
                if (K::kApart) {
                    uint32_t ri[16];
                    um::ld32x32_x16(tl + K::kOI + n0, ri);
                    um::wait_ld<16>(r);
                    um::wait_ld<16>(ri);
#pragma unroll
                    for (int i = 0; i < 16; ++i) r[i] = as_u(fmaf(fo, as_f(ri[i]), as_f(r[i])));
                } else {
                    um::wait_ld<16>(r);
                }
                // rows behind the length are zeros
#pragma unroll
                for (int c = 0; c < 8; ++c) o[n0 / 2 + c] = d < L ? pack2(as_f(r[2 * c]), as_f(r[2 * c + 1])) : 0u;
            }
            if (n + 1 < nch) ok = wait.all(m.sdone, (uint32_t)n & 1u);
            um::fence_after();
        }
        if (ok && nch) stage(nch - 1);
    } else {
        // ================================================ scores -> P', and the split of y
        const int i = 32 * quarter + lane, part = warp >> 3;  // row (then token), half of its columns
        const uint32_t keep = rev ? 0xffffffffu << lane : 0xffffffffu >> (31 - lane);
        const float* diag = m.dt + 31 - lane;
        const uint32_t tp = tl + K::kP;
#pragma unroll 1
        for (int n = 0; n < nch; ++n) {
            if (!wait.all(m.pfull, (uint32_t)n & 1u)) break;
            um::fence_after();
#pragma unroll 1
            for (int jb = 2 * part; jb < 2 * part + 2; ++jb) {
                uint32_t o[16];
                if (rev ? jb >= quarter : jb <= quarter) {
                    uint32_t r[32];
                    um::ld32x32_x32(tp + 32u * jb, r);
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
                            float x[4] = {as_f(r[c]), as_f(r[c + 1]), as_f(r[c + 2]), as_f(r[c + 3])};
                            mul2(x[0], x[1], k.x, k.y);
                            mul2(x[2], x[3], k.z, k.w);
                            mul2(x[0], x[1], f, f);
                            mul2(x[2], x[3], f, f);
#pragma unroll
                            for (int e = 0; e < 4; ++e) r[c + e] = as_u(x[e]);
                        }
                    }
#pragma unroll
                    for (int c = 0; c < 16; ++c) o[c] = pack2(as_f(r[2 * c]), as_f(r[2 * c + 1]));
                } else {
#pragma unroll
                    for (int c = 0; c < 16; ++c) o[c] = 0u;
                }
                um::st32x32_x16(tp + 64u * part + 16u * (jb & 1), o);
            }
            um::wait_st();
            arrive(m.pored);
            if (n + 1 < nch) {
                // the scores have read y, and all products before them the other term
                const int L = sp.tokens(n);
                split_y<DX, 2, 2>(tile(n, 0), sb + K::kOffLo, 0, i, part, p.s_u * (rev ? m.pw[i + 1] : m.pw[max(L - 1 - i, 0)]));
                um::fence_proxy_async();
                arrive(m.yfull);
            }
        }
        // chunks behind the sequence
        const int64_t from = (int64_t)nch * kC;
        if (from < sp.rows) {
            __nv_bfloat16* out = (__nv_bfloat16*)p.out + b * p.so.batch + h * p.so.head + (sp.first + from) * p.so.token;
            for (int64_t r = 16 * part + i / 8; r < sp.rows - from; r += 32)
                for (int c = i % 8; c < p.dz / 8; c += 8)
                    *reinterpret_cast<uint4*>(out + r * p.so.token + 8 * c) = make_uint4(0u, 0u, 0u, 0u);
        }
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
    uint64_t full[5], empty[5], yfull[2], lofree[2], ufull[2], ufree[2], drain;
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
    const la::Place at(a);
    const LaPass& p = a.p[at.pass];
    if (!p.s_out && (!at.split || at.ends(a))) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bh = at.bh, b = bh / a.H, h = bh % a.H;
    const Span sp(a, p, at, b);
    const int nch = sp.nch;
    const uint32_t sb = smem_u32(smem);
    const Waiter wait{&m.abort, g.limit};
    constexpr int kMmaWarp = 12, kCopyWarp = 13;

    if (tid == 0) {
        for (int i = 0; i < K::kSlots; ++i) {
            um::mbar_init(smem_u32(&m.full[i]), 1);
            um::mbar_init(smem_u32(&m.empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            um::mbar_init(smem_u32(&m.yfull[i]), 8);
            um::mbar_init(smem_u32(&m.lofree[i]), 1);
            um::mbar_init(smem_u32(&m.ufull[i]), 1);
            um::mbar_init(smem_u32(&m.ufree[i]), 4);
        }
        um::mbar_init(smem_u32(&m.drain), 1);
        m.abort = g.limit == 0;  // no wait at all: the first that would gives up
    }
    for (int i = tid; i < kLaPowers; i += K::kThreads) m.pw[i] = a.pw[(size_t)h * kLaPowers + i];
    if (warp == kMmaWarp) {
        um::tmem_alloc(smem_u32(&m.tmem), K::kCols);
        um::tmem_relinquish();
    }
    um::fence_before();
    __syncthreads();
    um::fence_after();
    la::let_next_start();
    const uint32_t tmem = m.tmem;
    const int quarter = warp & 3;
    auto slot = [](int n, int item) { return (2 * n + item) % K::kSlots; };
    auto phase = [](int n, int item) { return (uint32_t)((2 * n + item) / K::kSlots) & 1u; };
    auto tile = [&](int n, int item) { return sb + (uint32_t)slot(n, item) * K::kSlot; };

    if (warp == kMmaWarp) {
        constexpr uint32_t id = um::idesc_bf16(128, DZ) | um::kAmn | um::kBmn;
#pragma unroll 1
        for (int n = 0; n < nch; ++n) {
            const uint32_t u = tmem + K::kU + (uint32_t)(n & 1) * DZ;
            const uint64_t zz = mnmajor(tile(n, 1)), yh = mnmajor(tile(n, 0)), y1 = mnmajor(sb + K::kOffLo),
                           y2 = mnmajor(sb + K::kOffLo + K::kLo);
            if (!wait.all(m.full[slot(n, 1)], phase(n, 1))) break;
            if (n > 1 && !wait.all(m.ufree[n & 1], (uint32_t)(n / 2 - 1) & 1u)) break;
            // half a chunk at a time, while the other half is split
            bool ok = true;
#pragma unroll 1
            for (int hf = 0; hf < 2; ++hf) {
                if (!(ok = wait.all(m.yfull[hf], (uint32_t)n & 1u))) break;
                um::fence_after();
                const uint64_t at = mnstep(4 * hf);
                if (elect()) {
                    // the smallest terms first: fewer truncations next to a large sum
#pragma unroll
                    for (int k = 0; k < kC / 32; ++k)
                        um::mma_ss(u, y2 + at + mnstep(k), zz + at + mnstep(k), id, hf > 0 || k > 0);
#pragma unroll
                    for (int k = 0; k < kC / 32; ++k) um::mma_ss(u, y1 + at + mnstep(k), zz + at + mnstep(k), id, 1);
                    um::mma_commit(smem_u32(&m.lofree[hf]));
#pragma unroll
                    for (int k = 0; k < kC / 32; ++k) um::mma_ss(u, yh + at + mnstep(k), zz + at + mnstep(k), id, 1);
                    if (hf) {
                        um::mma_commit(smem_u32(&m.ufull[n & 1]));
                        um::mma_commit(smem_u32(&m.empty[slot(n, 0)]));
                        um::mma_commit(smem_u32(&m.empty[slot(n, 1)]));
                    }
                }
                __syncwarp();
            }
            if (!ok) break;
        }
        drain(m.drain, &m.abort);
    } else if (warp == kCopyWarp) {
        const Copier copy{g, p, sp, at.pass, b, h, wait};
        int made = 0;
#pragma unroll 1
        for (; made < 2 * nch; ++made) {
            const int n = made >> 1, it = made & 1, s = made % K::kSlots;
            if (!copy(2 * it, (it ? DZ : DX) / 64, n, tile(n, it), m.full[s], m.empty[s], made / K::kSlots)) break;
        }
        if (*wait.abort)
            for (int j = made > K::kSlots ? made - K::kSlots : 0; j < made; ++j)
                um::mbar_wait(smem_u32(&m.full[j % K::kSlots]), (uint32_t)(j / K::kSlots) & 1u, kLanding);
    } else if (warp >= 4) {
        // ================================================ the split of y: 8 warps
        const int t0 = 32 * (warp & 1) + lane, q = (warp - 4) / 2;
#pragma unroll 1
        for (int n = 0; n < nch; ++n) {
            const int L = sp.tokens(n);
            if (!wait.all(m.full[slot(n, 0)], phase(n, 0))) break;
            bool ok = true;
#pragma unroll 1
            for (int hf = 0; hf < 2; ++hf) {
                const int t = 64 * hf + t0;
                const float w = p.s_u * (sp.rev ? m.pw[t + 1] : m.pw[max(L - 1 - t, 0)]);
                if (n && !(ok = wait.all(m.lofree[hf], (uint32_t)(n - 1) & 1u))) break;
                split_y<DX, 3, 4>(tile(n, 0), sb + K::kOffLo, K::kLo, t, q, w);
                um::fence_proxy_async();
                arrive(m.yfull[hf]);
            }
            if (!ok) break;
        }
    } else {
        // ================================================ S <- a^L S + U
        const int d = 32 * quarter + lane;
        const bool mine = 32 * quarter < DX;
        const uint32_t tl = tmem + ((uint32_t)(32 * quarter) << 16), ts = tl + K::kST;
        const bool last = !at.split;  // the whole row: its final state, from the initial one
        float* out = (last ? p.s_out + (size_t)bh * p.dx * p.dz : a.work + at.state) + (size_t)d * p.dz;
        const float* s0 = last && p.s_in ? p.s_in + (size_t)bh * p.dx * p.dz : nullptr;
        if (mine) {
#pragma unroll 1
            for (int n0 = 0; n0 < DZ; n0 += 32) state_in(ts, s0, p.in_trans, p, d, n0);
            um::wait_st();
        }
        bool ok = true;
#pragma unroll 1
        for (int n = 0; n < nch; ++n) {
            const float2 f = a.decay[(size_t)h * kLaPowers + sp.tokens(n)];
            if (!(ok = wait.all(m.ufull[n & 1], (uint32_t)(n / 2) & 1u))) break;
            um::fence_after();
            const uint32_t tu = tl + K::kU + (uint32_t)(n & 1) * DZ;
            if (mine) {
#pragma unroll 1
                for (int n0 = 0; n0 < DZ; n0 += 16) {
                    uint32_t u[16], s[16];
                    um::ld32x32_x16(tu + n0, u);
                    um::ld32x32_x16(ts + n0, s);
                    um::wait_ld<16>(u);
                    um::wait_ld<16>(s);
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {  // as la::decayed
                        fma2(f.y, s[i], s[i + 1], u[i], u[i + 1]);
                        fma2(f.x, s[i], s[i + 1], u[i], u[i + 1]);
                    }
                    um::st32x32_x16(ts + n0, u);
                }
                um::wait_st();
            }
            arrive(m.ufree[n & 1]);
        }
        if (last) la::after_previous();  // the outputs' kernel has read the state that this may replace
        if (ok && mine) {
#pragma unroll 1
            for (int n0 = 0; n0 < DZ; n0 += 16) {
                uint32_t r[16];
                um::ld32x32_x16(ts + n0, r);
                um::wait_ld<16>(r);
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

// The map of a tensor [B][H][N][d]: dimensions in the order of their strides, those that do not move left out.  A map's
// strides have to be multiples of one another; where a view's are not (heads of 64 in tokens of 3 x 224, say), heads and
// rows become one dimension in steps of the greatest common divisor of all strides, in front of the tokens.  (8 x 11 x
// 4096 of 64 and 96 in one projection: 92 us, dense 90; copied by hand 408.)  Where all tokens are one, or coordinates
// would pass 31 bits, there is no map.
void describe(Source* s, const void* ptr, const fftconv_strides& st, int B, int H, int64_t N, int d) {
    struct Dim {
        int64_t extent, stride;
        int* at;
    } dim[3] = {{N, st.token, &s->at_token}, {H, st.head, &s->at_head}, {B, st.batch, &s->at_row}};
    s->at_token = s->at_head = s->at_row = 0;
    s->head_step = s->row_step = 1;
    s->by_hand = 1;
    const EncodeFn enc = encoder();
    if (!enc || (N > 1 && st.token == 0) || N > 0x7fffffff) return;
    int n = 0;
    Dim use[3];
    for (const Dim& x : dim)
        if (x.extent > 1 && x.stride != 0) {
            if (x.stride < 0) return;
            use[n++] = x;
        }
    for (int i = 1; i < n; ++i)
        for (int j = i; j > 0 && use[j].stride < use[j - 1].stride; --j) {
            const Dim t = use[j];
            use[j] = use[j - 1];
            use[j - 1] = t;
        }
    bool chain = true;
    for (int i = 1; i < n; ++i) chain = chain && use[i].stride % use[i - 1].stride == 0;
    if (!chain) {
        int64_t unit = 0, most = 1;
        for (int i = 0; i < n; ++i) unit = std::gcd(unit, use[i].stride);
        for (int i = 0; i < n; ++i) {
            if (use[i].at == &s->at_token) continue;
            const int64_t step = use[i].stride / unit;
            if (step > 0x7fffffff || (use[i].extent - 1) > (0x7fffffff - most) / step) return;
            most += (use[i].extent - 1) * step;
            *use[i].at = 1;
            (use[i].at == &s->at_head ? s->head_step : s->row_step) = (int)step;
        }
        use[0] = {most, unit, nullptr};
        n = 1;
        if (N > 1) use[n++] = dim[0];
    }
    cuuint64_t dims[4] = {(cuuint64_t)d, 1, 1, 1}, strides[3];
    cuuint32_t box[4] = {64, 1, 1, 1}, one[4] = {1, 1, 1, 1};
    cuuint64_t last = (cuuint64_t)d * 2;
    for (int i = 0; i < 3; ++i) {
        if (i < n) {
            dims[i + 1] = (cuuint64_t)use[i].extent;
            last = (cuuint64_t)use[i].stride * 2;
            if (use[i].at) *use[i].at = i + 1;
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
cudaError_t run(Args& g, int bh, int passes, bool ends, const double* lg, cudaStream_t s) {
    using M = Main<DX, DZ>;
    using S = States<DX, DZ>;
    const int whole = g.a.whole * passes, split = (bh - g.a.whole) * g.a.nseg * passes;
    cudaError_t e = la::allow<la_main<DX, DZ>>((int)M::kBytes);
    if (e == cudaSuccess && (split || ends)) e = la::allow<la_states<DX, DZ>>((int)S::kBytes);
    if (e == cudaSuccess && split) {
        g.a.first = whole;
        e = la::launch<la_states<DX, DZ>>(split, S::kThreads, S::kBytes, s, false, g);
        if (e == cudaSuccess) e = la::launch_carry(g.a, bh - g.a.whole, passes, lg, s);
        g.a.first = 0;
    }
    if (e == cudaSuccess) e = la::launch<la_main<DX, DZ>>(whole + split, M::kThreads, M::kBytes, s, split > 0, g);
    // The outputs' kernel keeps its state for the outputs alone: final states that a caller asks for come from the
    // states' kernel, which sums them in fp32 (beside the outputs, but written after them: a caller may update its
    // states in place).
    if (e == cudaSuccess && whole && ends) e = la::launch<la_states<DX, DZ>>(whole, S::kThreads, S::kBytes, s, true, g);
    return e;
}

}  // namespace latc

namespace la {

cudaError_t launch_tc(const Args& a, int dx, int dz, int B, int passes, bool ends, const fftconv_linattn_s& p,
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
        g.out[i] = source(q.out, q.so, q.dz);
        if (g.src[g.out[i]].by_hand) return cudaErrorNotSupported;
    }
    const int bh = B * a.H;
    if (dx <= 64)
        return dz <= 64 ? latc::run<64, 64>(g, bh, passes, ends, p.d_log, s)
                        : latc::run<64, 128>(g, bh, passes, ends, p.d_log, s);
    return dz <= 64 ? latc::run<128, 64>(g, bh, passes, ends, p.d_log, s)
                    : latc::run<128, 128>(g, bh, passes, ends, p.d_log, s);
}

}  // namespace la
}  // namespace fftc
