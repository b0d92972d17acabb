// vec_io.cuh -- loads and stores of V consecutive elements, kept raw (as
// loaded) until their fp32 values are wanted, so that several can be in flight.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "common.cuh"

namespace ssd {

template <typename T, int V>
struct alignas(sizeof(T) * V) Raw {      // one load of 2..16 bytes
    T v[V];
};

// Read-only data.  Volatile, so that a load that is issued early for later use is
// not moved down to its use.
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> raw_load(const T* p) {
    Raw<T, V> r;
    constexpr int kBytes = sizeof(T) * V;
    if constexpr (kBytes == 16) {
        uint4 q;
        asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "l"(p));
        r = *reinterpret_cast<const Raw<T, V>*>(&q);
    } else if constexpr (kBytes == 8) {
        uint2 q;
        asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(q.x), "=r"(q.y) : "l"(p));
        r = *reinterpret_cast<const Raw<T, V>*>(&q);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) r.v[i] = p[i];
    }
    return r;
}

template <typename T, int V>
__device__ __forceinline__ Raw<T, V> raw_zero() {
    Raw<T, V> r;
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = from_f32<T>(0.f);
    return r;
}

template <typename T, int V>
__device__ __forceinline__ void raw_to_f32(const Raw<T, V>& r, float (&f)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = to_f32(r.v[i]);
}

template <typename T, int V>
__device__ __forceinline__ Raw<T, V> raw_from_f32(const float (&f)[V]) {
    Raw<T, V> r;
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = from_f32<T>(f[i]);
    return r;
}

template <typename T, int V>
__device__ __forceinline__ void raw_store(T* p, const Raw<T, V>& r) {
    *reinterpret_cast<Raw<T, V>*>(p) = r;
}

// Copies sizeof(R) bytes (4, 8 or 16, both sides aligned) to shared memory
// without a register in between, or writes zeros where there is nothing to copy
// (p is then not read).  Complete after copies_pending<..> in the same thread.
template <typename R, typename T>
__device__ __forceinline__ void copy_async(R* to, const T* p, bool exists) {
    const uint32_t s = (uint32_t)__cvta_generic_to_shared(to);
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;"
                 :: "r"(s), "l"(p), "n"((int)sizeof(R)), "r"(exists ? (int)sizeof(R) : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most N of this thread's committed groups are still under way.
template <int N>
__device__ __forceinline__ void copies_pending() {
    asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory");
}

constexpr float kLog2E = 1.4426950408889634f;

// 2^v; results below 2^-126 are zero (a decay that small leaves nothing of a state).
__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Two fp32 values in one 64-bit register: add, multiply and fma work on both in
// one instruction.
using F2 = unsigned long long;
__device__ __forceinline__ F2 pack2(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpack2(F2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 ex2_2(F2 v) {
    const float2 f = unpack2(v);
    return pack2(ex2(f.x), ex2(f.y));
}

__device__ __forceinline__ float rcp_fast(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// sigmoid(v) = 1 / (1 + 2^(-v log2(e))); where the power overflows to infinity the
// reciprocal is the right 0.
__device__ __forceinline__ float sigmoid_fast(float v) { return rcp_fast(1.f + ex2(-v * kLog2E)); }
__device__ __forceinline__ F2 sigmoid_fast(F2 v) {
    const float2 e = unpack2(add2(ex2_2(mul2(v, pack2(-kLog2E, -kLog2E))), pack2(1.f, 1.f)));
    return pack2(rcp_fast(e.x), rcp_fast(e.y));
}

// The tokens of sequence b that are its own.
__device__ __forceinline__ int64_t own_length(const int32_t* lens, int64_t b, int64_t L) {
    if (!lens) return L;
    const int64_t n = lens[b];
    return n < 0 ? 0 : (n > L ? L : n);
}

}  // namespace ssd
