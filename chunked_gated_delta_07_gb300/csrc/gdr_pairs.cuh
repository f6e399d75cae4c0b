// gdr_pairs.cuh -- arithmetic on two fp32 numbers in one instruction (f32x2), and the same on one,
// so that code written for pairs takes single elements too.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace gdr {

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ uint64_t bits(float2 v) {
    uint64_t u;
    asm("mov.b64 %0, {%1, %2};" : "=l"(u) : "f"(v.x), "f"(v.y));
    return u;
}
__device__ __forceinline__ float2 unbits(uint64_t u) {
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(u));
    return v;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
    return unbits(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)));
    return unbits(d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)));
    return unbits(d);
}

__device__ __forceinline__ float fma2(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float mul2(float a, float b) { return a * b; }
__device__ __forceinline__ float add2(float a, float b) { return a + b; }

// N elements as pairs, or one by one.
template <int N, bool PAIRED = (N > 1)> struct Pairs {
    using type = float2;
    static constexpr int count = N / 2;
    __device__ static float2 of(float v) { return both(v); }
    __device__ static float2 at(const float *x, int i) { return make_float2(x[2 * i], x[2 * i + 1]); }
    __device__ static void put(float *x, int i, float2 v) {
        x[2 * i] = v.x;
        x[2 * i + 1] = v.y;
    }
    __device__ static float sum(float2 v) { return v.x + v.y; }
};
template <int N> struct Pairs<N, false> {
    using type = float;
    static constexpr int count = N;
    __device__ static float of(float v) { return v; }
    __device__ static float at(const float *x, int i) { return x[i]; }
    __device__ static void put(float *x, int i, float v) { x[i] = v; }
    __device__ static float sum(float v) { return v; }
};

}  // namespace gdr
