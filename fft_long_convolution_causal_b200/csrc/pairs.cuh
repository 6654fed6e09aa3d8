// pairs.cuh -- rows in pieces of V elements held as pairs of fp32: packed
// two-at-a-time arithmetic, and bf16 pieces unpacked and packed a word at a time.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace fftc {

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n.reg .b64 a, b, c;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nmov.b64 c, {%6, %7};\n"
        "fma.rn.f32x2 a, a, b, c;\nmov.b64 {%0, %1}, a;\n}\n"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n.reg .b64 a, b;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nmul.rn.f32x2 a, a, b;\nmov.b64 {%0, %1}, a;\n}\n"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n.reg .b64 a, b;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nadd.rn.f32x2 a, a, b;\nmov.b64 {%0, %1}, a;\n}\n"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// A piece of V elements of T in memory, and its pairs (V = 1: one, its second half zero).
template <typename T, int V>
struct Piece;
template <>
struct Piece<__nv_bfloat16, 8> {
    static constexpr int kPairs = 4;
    uint4 u;
    __device__ __forceinline__ float2 get(int i) const {
        const uint32_t w = i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w;
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    __device__ __forceinline__ void set(int i, float2 v) {
        uint32_t w;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(v.y), "f"(v.x));
        (i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w) = w;
    }
};
template <>
struct Piece<float, 4> {
    static constexpr int kPairs = 2;
    float4 u;
    __device__ __forceinline__ float2 get(int i) const { return i == 0 ? make_float2(u.x, u.y) : make_float2(u.z, u.w); }
    __device__ __forceinline__ void set(int i, float2 v) {
        if (i == 0)
            u.x = v.x, u.y = v.y;
        else
            u.z = v.x, u.w = v.y;
    }
};
template <>
struct Piece<float, 8> {  // fp32 partners of eight bf16 elements
    static constexpr int kPairs = 4;
    float4 u, v;
    __device__ __forceinline__ float2 get(int i) const {
        return i == 0 ? make_float2(u.x, u.y) : i == 1 ? make_float2(u.z, u.w) : i == 2 ? make_float2(v.x, v.y) : make_float2(v.z, v.w);
    }
};
template <>
struct Piece<__nv_bfloat16, 1> {
    static constexpr int kPairs = 1;
    __nv_bfloat16 u;
    __device__ __forceinline__ float2 get(int) const { return make_float2(__bfloat162float(u), 0.f); }
    __device__ __forceinline__ void set(int, float2 v) { u = __float2bfloat16_rn(v.x); }
};
template <>
struct Piece<float, 1> {
    static constexpr int kPairs = 1;
    float u;
    __device__ __forceinline__ float2 get(int) const { return make_float2(u, 0.f); }
    __device__ __forceinline__ void set(int, float2 v) { u = v.x; }
};

}  // namespace fftc
