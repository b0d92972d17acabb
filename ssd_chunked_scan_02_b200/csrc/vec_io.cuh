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

template <typename T, int V>
__device__ __forceinline__ Raw<T, V> raw_load(const T* p) {
    Raw<T, V> r;
    constexpr int kBytes = sizeof(T) * V;
    if constexpr (kBytes == 16) {
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(p));
        r = *reinterpret_cast<const Raw<T, V>*>(&q);
    } else if constexpr (kBytes == 8) {
        const uint2 q = __ldg(reinterpret_cast<const uint2*>(p));
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

// sigmoid(v) = 1 / (1 + exp(-v)); exp overflows to +inf for v < -88, whose
// reciprocal is the right 0.
__device__ __forceinline__ float sigmoid_f32(float v) {
    return __fdividef(1.f, 1.f + __expf(-v));
}

}  // namespace ssd
