// linattn_tc.cu -- decayed linear attention on the fifth-generation tensor cores
// (bf16 operands, fp32 accumulators in tensor memory), chunks of 128 tokens.
//
// A CTA walks the chunks of one (segment, row, head, pass) with the state S
// [dx][dz] resident in tensor memory.  Per chunk of L live tokens:
//   scores  P  = X Y^T                                   (128 x 128 x DX)
//   inter   OI = X bf16(S)                               (128 x DZ x DX)
//   intra   OA = bf16(s_p a^|i-j| P, masked) Z           (128 x DZ x 128)
//   out     o  = OA + s_i a^(i+1) OI                     (rows of bf16)
//   state   S  = a^L S + (s_u a^(L-1-j) y_j)^T Z         (DX x DZ x 128, 2 or 3 products)
// The decayed y would lose bits in one bf16, and with it the fp32 state: it is
// split into a sum of NS bf16 terms (2: off by 2^-17 at most, below the rounding
// of the outputs it feeds; 3: exact to 2^-25, where the state is an output).
//
// Roles: 4 warps for scores -> P' and the outputs, 4 for the state's copy and the
// split of y, 4 that copy tiles in (cp.async, zero-filling rows behind a length
// and elements behind dx), 1 that issues the products.  Tiles are core matrices
// of 8 tokens x 16 bytes ([d / 8][token]): the same bytes serve as a K-major
// operand over d and as an MN-major operand over tokens, so nothing is transposed.
#include <cuda_bf16.h>

#include "linattn.cuh"
#include "umma.cuh"

namespace fftc {
namespace latc {

constexpr int kC = 128;               // tokens a chunk
constexpr int kGroup = 128;           // threads of a role
constexpr int kThreads = 3 * kGroup + 32;
constexpr uint32_t kCol = kC * 16;    // bytes of one 16-byte column of a tile

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
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int src_bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// MAIN: outputs; else the segments' own states only
template <int DX, int DZ, int NS, bool MAIN>
struct Cfg {
    static constexpr uint32_t kSlot = (uint32_t)(DX > DZ ? DX : DZ) * 256u;
    static constexpr uint32_t kS = MAIN ? (uint32_t)DX * DZ * 2u : 0u;  // bf16 copy of the state
    static constexpr uint32_t kLo = (uint32_t)DX * 256u;                // one term of the split y
    static constexpr bool kTwo = DX == 64 && DZ == 64;                  // two CTAs an SM
    static constexpr uint32_t kRoom = kTwo ? 112u * 1024u : 224u * 1024u;
    // The state's product has 128 rows whatever DX is: with DX = 64 its descriptor reads 16 KiB
    // behind a term of y (rows nobody looks at), which has to be this CTA's memory.
    static constexpr uint32_t kPad = DX == 64 && kS < 16384u ? 16384u - kS : 0u;
    static constexpr int kFit = (int)((kRoom - kS - (NS - 1) * kLo - kPad) / kSlot);
    static constexpr int kSlots = kFit > 8 ? 8 : kFit;
    static constexpr uint32_t kOffRing = 0, kOffLo = kSlots * kSlot, kOffS = kOffLo + (NS - 1) * kLo;
    static constexpr uint32_t kBytes = kOffS + kS + kPad;
    static constexpr int kItems = MAIN ? 3 : 2;  // tiles a chunk
    // tensor-memory columns
    static constexpr uint32_t kP = 0;                          // scores, then P' in the first 64
    static constexpr uint32_t kOA = DZ == 64 ? 64 : 128;       // DZ = 64: the scores' upper half, free by then
    static constexpr uint32_t kOI = DZ == 64 ? 128 : 256;
    static constexpr uint32_t kST = DZ == 64 ? 192 : 384;
    static constexpr uint32_t kCols = DZ == 64 ? 256 : 512;
    static_assert(kSlots >= kItems, "a chunk's tiles fit the ring");
};

struct Bars {
    uint64_t full[8], empty[8], pfull, pready, ofull, ofree, sfull, yfull, sdone, drain;
};

template <int DX, int DZ, int NS, bool MAIN>
__global__ void __launch_bounds__(kThreads, (DX == 64 && DZ == 64) ? 2 : 1)
la_tc(const __grid_constant__ la::Args a, int* __restrict__ err, uint32_t limit) {
    using K = Cfg<DX, DZ, NS, MAIN>;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ __align__(8) Bars bars;
    __shared__ __align__(16) float pw[kLaPowers], ct[32];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    const LaPass& p = a.p[blockIdx.z];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int sg = blockIdx.x, bh = blockIdx.y, b = bh / a.H, h = bh % a.H;
    const bool rev = p.reverse;
    const int64_t first = sg * a.seg, len = la::live_tokens(a, b);
    const int64_t rows = min(a.seg, a.N - first);
    const int64_t live = max((int64_t)0, min(rows, len - first));
    const int nch = (int)((live + kC - 1) / kC);
    const uint32_t sb = smem_u32(smem);
    float* wseg = a.work + blockIdx.z * a.pass_floats + ((size_t)bh * a.nseg + sg) * a.state_floats;
    float* s_out = MAIN ? (a.nseg == 1 && p.s_out ? p.s_out + (size_t)bh * p.dx * p.dz : nullptr) : wseg;
    // chunk n of the walk: its first token and live tokens
    auto start = [&](int n) { return (int64_t)(rev ? nch - 1 - n : n) * kC; };
    auto bar = [&](const uint64_t& x) { return smem_u32(&x); };
    auto wait = [&](const uint64_t& x, uint32_t parity) {
        const uint32_t ad = smem_u32(&x);
        for (uint32_t i = 0; i < limit && !s_abort; ++i)
            if (um::mbar_try_wait(ad, parity)) return true;
        s_abort = 1;
        return false;
    };
    // the same for a whole warp, with one answer
    auto wait_all = [&](const uint64_t& x, uint32_t parity) { return __all_sync(0xffffffffu, wait(x, parity)) != 0; };

    if (tid == 0) {
        for (int i = 0; i < K::kSlots; ++i) {
            um::mbar_init(bar(bars.full[i]), 4);
            um::mbar_init(bar(bars.empty[i]), 1);
        }
        um::mbar_init(bar(bars.pfull), 1);
        um::mbar_init(bar(bars.pready), 4);
        um::mbar_init(bar(bars.ofull), 1);
        um::mbar_init(bar(bars.ofree), 4);
        um::mbar_init(bar(bars.sfull), 4);
        um::mbar_init(bar(bars.yfull), 4);
        um::mbar_init(bar(bars.sdone), 1);
        um::mbar_init(bar(bars.drain), 1);
        s_abort = 0;
    }
    for (int i = tid; i < kLaPowers; i += kThreads) pw[i] = a.pw[h * kLaPowers + i];
    if (tid < 32) ct[tid] = a.pw[h * kLaPowers + (rev ? tid : 31 - tid)];
    if (warp == 12) {
        um::tmem_alloc(smem_u32(&s_tmem), K::kCols);
        um::tmem_relinquish();
    }
    um::fence_before();
    __syncthreads();
    um::fence_after();
    const uint32_t tmem = s_tmem;
    const uint32_t quarter = (uint32_t)(warp & 3), tl = tmem + ((32u * quarter) << 16);
    // arrival of a warp whose tensor-memory and shared-memory accesses are done
    auto arrive = [&](const uint64_t& x) {
        um::fence_before();
        __syncwarp();
        if (lane == 0) um::mbar_arrive(smem_u32(&x));
    };
    // tiles in the order they are copied: y, x, z (y, z)
    auto slot_of = [&](int n, int item) { return (n * K::kItems + item) % K::kSlots; };
    auto phase_of = [&](int n, int item) { return (uint32_t)((n * K::kItems + item) / K::kSlots) & 1u; };
    auto ring = [&](int n, int item) { return sb + K::kOffRing + (uint32_t)slot_of(n, item) * K::kSlot; };
    constexpr int kItY = 0, kItX = 1, kItZ = K::kItems - 1;

    if (warp == 12) {
        // ================================================ products
        if (lane == 0) {
            const uint32_t id_scores = um::idesc_bf16(128, 128), id_inter = um::idesc_bf16(128, DZ) | um::kBmn,
                           id_intra = id_inter, id_state = id_inter | um::kAmn;
            auto kmajor = [&](uint32_t t) { return um::sdesc(t, kCol, 128); };       // rows = tokens, K = elements
            auto mnmajor = [&](uint32_t t) { return um::sdesc(t, 128, kCol); };      // rows = elements, K = tokens
            auto add = [](uint64_t d, uint32_t bytes) { return d + (uint64_t)(bytes >> 4); };
            for (int n = 0; n < nch; ++n) {
                const uint32_t par = (uint32_t)n & 1u, prev = par ^ 1u;
                const uint32_t ty = ring(n, kItY), tz = ring(n, kItZ);
                if (MAIN) {
                    const uint32_t tx = ring(n, kItX);
                    if (!wait(bars.full[slot_of(n, kItY)], phase_of(n, kItY))) break;
                    if (!wait(bars.full[slot_of(n, kItX)], phase_of(n, kItX))) break;
                    if (DZ == 64 && n && !wait(bars.ofree, prev)) break;
                    um::fence_after();
#pragma unroll
                    for (int k = 0; k < DX / 16; ++k)
                        um::mma_ss(tmem + K::kP, add(kmajor(tx), 2 * k * kCol), add(kmajor(ty), 2 * k * kCol), id_scores,
                                   k > 0);
                    um::mma_commit(bar(bars.pfull));
                    if (!wait(bars.sfull, par)) break;
                    if (DZ != 64 && n && !wait(bars.ofree, prev)) break;
                    um::fence_after();
                    const uint64_t ds = um::sdesc(sb + K::kOffS, 128, DX * 16);
#pragma unroll
                    for (int k = 0; k < DX / 16; ++k)
                        um::mma_ss(tmem + K::kOI, add(kmajor(tx), 2 * k * kCol), add(ds, k * 256), id_inter, k > 0);
                    um::mma_commit(bar(bars.empty[slot_of(n, kItX)]));
                    if (!wait(bars.pready, par)) break;
                    if (!wait(bars.full[slot_of(n, kItZ)], phase_of(n, kItZ))) break;
                    um::fence_after();
#pragma unroll
                    for (int k = 0; k < kC / 16; ++k)
                        um::mma_ts(tmem + K::kOA, tmem + K::kP + 8u * k, add(mnmajor(tz), k * 256), id_intra, k > 0);
                    um::mma_commit(bar(bars.ofull));
                } else {
                    if (!wait(bars.full[slot_of(n, kItZ)], phase_of(n, kItZ))) break;
                    if (!wait(bars.sfull, par)) break;
                }
                if (!wait(bars.yfull, par)) break;
                um::fence_after();
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    const uint64_t dy = mnmajor(s == 0 ? ty : sb + K::kOffLo + (s - 1) * K::kLo);
#pragma unroll
                    for (int k = 0; k < kC / 16; ++k)
                        um::mma_ss(tmem + K::kST, add(dy, k * 256), add(mnmajor(tz), k * 256), id_state, 1);
                }
                um::mma_commit(bar(bars.sdone));
                um::mma_commit(bar(bars.empty[slot_of(n, kItY)]));
                um::mma_commit(bar(bars.empty[slot_of(n, kItZ)]));
            }
            // every product issued is complete before tensor memory is freed
            um::mma_commit(bar(bars.drain));
            bool ok = false;
            for (uint32_t i = 0; i < um::kDefaultWaitProbes && !ok; ++i) ok = um::mbar_try_wait(bar(bars.drain), 0);
            if (!ok) s_abort = 1;
        }
        __syncwarp();
    } else if (warp >= 8) {
        // ================================================ copies
        const int w = warp - 8, tr = lane & 7, cq = lane >> 3;
        const __nv_bfloat16* src[3] = {(const __nv_bfloat16*)p.y + b * p.sy.batch + h * p.sy.head + first * p.sy.token,
                                       (const __nv_bfloat16*)p.x + b * p.sx.batch + h * p.sx.head + first * p.sx.token,
                                       (const __nv_bfloat16*)p.z + b * p.sz.batch + h * p.sz.head + first * p.sz.token};
        const int64_t stride[3] = {p.sy.token, p.sx.token, p.sz.token};
        int told = 0, made = 0;  // tiles announced, tiles requested
        auto tell = [&]() {
            um::fence_proxy_async();
            __syncwarp();
            if (lane == 0) um::mbar_arrive(bar(bars.full[told % K::kSlots]));
            ++told;
        };
        bool ok = true;
        for (int n = 0; n < nch && ok; ++n) {
            const int64_t t0 = start(n);
            const int L = (int)min((int64_t)kC, live - t0);
#pragma unroll
            for (int it = 0; it < K::kItems; ++it) {
                const int what = K::kItems == 2 && it == 1 ? 2 : it;  // 0 y, 1 x, 2 z
                const int d = what == 2 ? p.dz : p.dx;
                const int sl = made % K::kSlots;
                if (made >= K::kSlots) {
                    const uint32_t ph = (uint32_t)(made / K::kSlots - 1) & 1u;
                    // what has been requested is announced before this warp waits for room
                    if (told < made && !__all_sync(0xffffffffu, um::mbar_test_wait(bar(bars.empty[sl]), ph))) {
                        cp_wait<0>();
                        while (told < made) tell();
                    }
                    if (!wait_all(bars.empty[sl], ph)) {
                        ok = false;
                        break;
                    }
                }
                const uint32_t dst = sb + K::kOffRing + (uint32_t)sl * K::kSlot + (uint32_t)tr * 16u;
                constexpr int kD = DX > DZ ? DX : DZ;
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int tg = w + 4 * g, t = tg * 8 + tr;
                    const __nv_bfloat16* row = src[what] + (t < L ? t0 + t : 0) * stride[what];
#pragma unroll
                    for (int c = 0; c < kD / 32; ++c) {
                        const int col = 4 * c + cq;
                        const bool on = t < L && col * 8 < d;
                        if ((what == 2 ? DZ : DX) > c * 32)
                            cp_async16(dst + (uint32_t)tg * 128u + (uint32_t)col * kCol, on ? row + col * 8 : src[what],
                                       on ? 16 : 0);
                    }
                }
                cp_commit();
                ++made;
                if (made - told > 2) {  // two tiles in flight behind this one
                    cp_wait<2>();
                    tell();
                }
            }
        }
        cp_wait<0>();
        if (ok)
            while (told < made) tell();
    } else if (warp >= 4) {
        // ================================================ state and the split of y
        const int d = 32 * (int)quarter + lane, t = d;
        const bool mine = 32 * (int)quarter < DX;  // this warp's lanes hold rows of the state
        const uint32_t ts = tl + K::kST;
        // the state entering the segment
        {
            const float* s0 = !MAIN ? nullptr : a.nseg > 1 ? wseg : p.s_in ? p.s_in + (size_t)bh * p.dx * p.dz : nullptr;
            const bool trans = a.nseg == 1 && p.in_trans;
            if (mine) {
#pragma unroll
                for (int n0 = 0; n0 < DZ; n0 += 16) {
                    uint32_t r[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) r[i] = 0u;
                    if (s0 && d < p.dx) {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (n0 + i < p.dz)
                                r[i] = __float_as_uint(trans ? s0[(size_t)(n0 + i) * p.dx + d] : s0[(size_t)d * p.dz + n0 + i]);
                    }
                    um::st32x32_x16(ts + n0, r);
                }
                um::wait_st();
            }
        }
        bool ok = true;
        for (int n = 0; n < nch; ++n) {
            const uint32_t par = (uint32_t)n & 1u;
            const int L = (int)min((int64_t)kC, live - start(n));
            if (n && !(ok = wait_all(bars.sdone, par ^ 1u))) break;
            um::fence_after();
            if (mine) {
                const float f = pw[L];
                const uint32_t dst = sb + K::kOffS + (uint32_t)d * 16u;
#pragma unroll
                for (int n0 = 0; n0 < DZ; n0 += 32) {
                    uint32_t r[32];
                    um::ld32x32_x32(ts + n0, r);
                    um::wait_ld<32>(r);
                    if (MAIN) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint4 v;
                            v.x = pack2(__uint_as_float(r[8 * q]), __uint_as_float(r[8 * q + 1]));
                            v.y = pack2(__uint_as_float(r[8 * q + 2]), __uint_as_float(r[8 * q + 3]));
                            v.z = pack2(__uint_as_float(r[8 * q + 4]), __uint_as_float(r[8 * q + 5]));
                            v.w = pack2(__uint_as_float(r[8 * q + 6]), __uint_as_float(r[8 * q + 7]));
                            sts128(dst + (uint32_t)(n0 / 8 + q) * (DX * 16u), v);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(f * __uint_as_float(r[i]));
                    um::st32x32_x16(ts + n0, r);
                    um::st32x32_x16(ts + n0 + 16, r + 16);
                }
                um::wait_st();
            }
            um::fence_proxy_async();
            arrive(bars.sfull);
            // y: decayed to the chunk's end and split, once the scores have read it
            if (!(ok = wait_all(bars.full[slot_of(n, kItY)], phase_of(n, kItY)))) break;
            if (MAIN && !(ok = wait_all(bars.pfull, par))) break;
            const float w = p.s_u * (rev ? pw[t + 1] : pw[max(L - 1 - t, 0)]);
            const uint32_t ty = ring(n, kItY) + (uint32_t)t * 16u, tlo = sb + K::kOffLo + (uint32_t)t * 16u;
#pragma unroll 4
            for (int c = 0; c < DX / 8; ++c) {
                const uint4 u = lds128(ty + c * kCol);
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
                sts128(ty + c * kCol, make_uint4(o[0][0], o[0][1], o[0][2], o[0][3]));
#pragma unroll
                for (int s = 1; s < NS; ++s)
                    sts128(tlo + (s - 1) * K::kLo + c * kCol, make_uint4(o[s][0], o[s][1], o[s][2], o[s][3]));
            }
            um::fence_proxy_async();
            arrive(bars.yfull);
        }
        if (s_out && ok && (nch == 0 || wait_all(bars.sdone, (uint32_t)(nch - 1) & 1u)) && mine) {
            um::fence_after();
#pragma unroll
            for (int n0 = 0; n0 < DZ; n0 += 16) {
                uint32_t r[16];
                um::ld32x32_x16(ts + n0, r);
                um::wait_ld<16>(r);
                if (d < p.dx) {
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        if (n0 + i < p.dz)
                            *reinterpret_cast<float4*>(s_out + (size_t)d * p.dz + n0 + i) =
                                make_float4(__uint_as_float(r[i]), __uint_as_float(r[i + 1]), __uint_as_float(r[i + 2]),
                                            __uint_as_float(r[i + 3]));
                }
            }
        }
    } else if (MAIN) {
        // ================================================ scores -> P', outputs
        const int i = 32 * (int)quarter + lane;
        __nv_bfloat16* out = (__nv_bfloat16*)p.out + b * p.so.batch + h * p.so.head + first * p.so.token;
        const bool wide = ((reinterpret_cast<uintptr_t>(p.out) & 31u) == 0) &&
                          ((p.so.batch | p.so.head | p.so.token) % 16 == 0);
        for (int n = 0; n < nch; ++n) {
            const uint32_t par = (uint32_t)n & 1u;
            const int64_t t0 = start(n);
            const int L = (int)min((int64_t)kC, live - t0);
            if (!wait_all(bars.pfull, par)) break;
            um::fence_after();
#pragma unroll
            for (int jb = 0; jb < 4; ++jb) {
                uint32_t o[16];
                const bool on = rev ? jb >= (int)quarter : jb <= (int)quarter;
                if (on) {
                    uint32_t r[32];
                    um::ld32x32_x32(tl + K::kP + 32u * jb, r);
                    um::wait_ld<32>(r);
                    if (jb == (int)quarter) {
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            const int e = rev ? c - lane : lane - c;
                            r[c] = e >= 0 ? __float_as_uint(__uint_as_float(r[c]) * (p.s_p * pw[max(e, 0)])) : 0u;
                        }
                    } else {
                        // a^|i-j| = a^(distance to the block's near column) a^(from there)
                        const float f = p.s_p * pw[rev ? 32 * jb - i : i - 32 * jb - 31];
#pragma unroll
                        for (int c = 0; c < 32; c += 4) {
                            const float4 k = *reinterpret_cast<const float4*>(ct + c);
                            r[c] = __float_as_uint(__uint_as_float(r[c]) * (f * k.x));
                            r[c + 1] = __float_as_uint(__uint_as_float(r[c + 1]) * (f * k.y));
                            r[c + 2] = __float_as_uint(__uint_as_float(r[c + 2]) * (f * k.z));
                            r[c + 3] = __float_as_uint(__uint_as_float(r[c + 3]) * (f * k.w));
                        }
                    }
#pragma unroll
                    for (int c = 0; c < 16; ++c) o[c] = pack2(__uint_as_float(r[2 * c]), __uint_as_float(r[2 * c + 1]));
                } else {
#pragma unroll
                    for (int c = 0; c < 16; ++c) o[c] = 0u;
                }
                um::st32x32_x16(tl + K::kP + 16u * jb, o);
            }
            um::wait_st();
            arrive(bars.pready);
            const float f = p.s_i * (rev ? pw[max(L - 1 - i, 0)] : pw[i + 1]);
            if (!wait_all(bars.ofull, par)) break;
            um::fence_after();
            __nv_bfloat16* row = out + (t0 + i) * p.so.token;
#pragma unroll
            for (int n0 = 0; n0 < DZ; n0 += 16) {
                uint32_t ra[16], ri[16], o[8];
                um::ld32x32_x16(tl + K::kOA + n0, ra);
                um::ld32x32_x16(tl + K::kOI + n0, ri);
                um::wait_ld<16>(ra);
                um::wait_ld<16>(ri);
                if (n0 + 16 >= DZ) arrive(bars.ofree);
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    o[c] = pack2(fmaf(f, __uint_as_float(ri[2 * c]), __uint_as_float(ra[2 * c])),
                                 fmaf(f, __uint_as_float(ri[2 * c + 1]), __uint_as_float(ra[2 * c + 1])));
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
        for (int64_t e = tid; e < (rows - live) * (p.dz / 8); e += kGroup)
            *reinterpret_cast<uint4*>(out + (live + e / (p.dz / 8)) * p.so.token + 8 * (e % (p.dz / 8))) =
                make_uint4(0u, 0u, 0u, 0u);
    }
    um::fence_before();
    __syncthreads();
    um::fence_after();
    if (warp == 12) um::tmem_dealloc(tmem, K::kCols);
    if (tid == 0 && s_abort) atomicExch(err, 1);
}

template <int DX, int DZ, int NS, bool MAIN>
cudaError_t run(const la::Args& a, int bh, int passes, const fftconv_linattn_s& p, cudaStream_t s) {
    constexpr int bytes = (int)Cfg<DX, DZ, NS, MAIN>::kBytes;
    static bool once = false;
    if (!once) {
        const cudaError_t e = cudaFuncSetAttribute(la_tc<DX, DZ, NS, MAIN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   bytes);
        if (e != cudaSuccess) return e;
        once = true;
    }
    la_tc<DX, DZ, NS, MAIN><<<dim3(a.nseg, bh, passes), kThreads, bytes, s>>>(a, p.d_err, p.wait_limit);
    return cudaGetLastError();
}

template <int NS, bool MAIN>
cudaError_t pick(const la::Args& a, int dx, int dz, int bh, int passes, const fftconv_linattn_s& p, cudaStream_t s) {
    if (dx <= 64) return dz <= 64 ? run<64, 64, NS, MAIN>(a, bh, passes, p, s) : run<64, 128, NS, MAIN>(a, bh, passes, p, s);
    return dz <= 64 ? run<128, 64, NS, MAIN>(a, bh, passes, p, s) : run<128, 128, NS, MAIN>(a, bh, passes, p, s);
}

}  // namespace latc

namespace la {

cudaError_t launch_tc_states(const Args& a, int dx, int dz, int bh, int passes, const fftconv_linattn_s& p,
                             cudaStream_t s) {
    return latc::pick<3, false>(a, dx, dz, bh, passes, p, s);
}

cudaError_t launch_tc_main(const Args& a, int dx, int dz, int bh, int passes, const fftconv_linattn_s& p,
                           cudaStream_t s) {
    bool exact = false;  // the kernel's own state is an output
    for (int i = 0; i < passes; ++i) exact = exact || (a.nseg == 1 && a.p[i].s_out);
    return exact ? latc::pick<3, true>(a, dx, dz, bh, passes, p, s) : latc::pick<2, true>(a, dx, dz, bh, passes, p, s);
}

}  // namespace la
}  // namespace fftc
