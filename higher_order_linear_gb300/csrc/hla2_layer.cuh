// hla2_layer.cuh -- what the operators around the attention layer share
// (hla2_gated.cu, hla2_norm.cu, hla2_rotary.cu): typed vector accesses and the
// host-side checks of their entry points.
#pragma once

#include <cmath>

#include "../../include/hla2.h"
#include "hla2_internal.h"

namespace hla2 {
namespace {

using bf16 = __nv_bfloat16;

// N consecutive elements as fp32, read or written in accesses of up to 16
// bytes; VEC = false makes N scalar accesses, of which the first `n` are made.
template <typename T, int N, bool VEC>
struct Lane;

template <int N>
struct Lane<bf16, N, true> {
    static_assert(N == 4 || N % 8 == 0, "whole accesses");
    static constexpr int W = N / 2;  // 32-bit words
    uint32_t w[W];
    __device__ __forceinline__ void load(const bf16* p, int) {
        if constexpr (N % 8 == 0) {
#pragma unroll
            for (int i = 0; i < N / 8; ++i)
                *reinterpret_cast<uint4*>(w + 4 * i) = __ldcs(reinterpret_cast<const uint4*>(p) + i);
        } else {
            *reinterpret_cast<uint2*>(w) = __ldcs(reinterpret_cast<const uint2*>(p));
        }
    }
    __device__ __forceinline__ float get(int i) const {
        return __uint_as_float((i & 1) ? (w[i >> 1] & 0xffff0000u) : (w[i >> 1] << 16));
    }
    __device__ __forceinline__ void set(const float (&v)[N]) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
    }
    __device__ __forceinline__ void store(bf16* p, int) const {
        if constexpr (N % 8 == 0) {
#pragma unroll
            for (int i = 0; i < N / 8; ++i)
                reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        } else {
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        }
    }
};

template <int N>
struct Lane<bf16, N, false> {
    bf16 v[N];
    __device__ __forceinline__ void load(const bf16* p, int n) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = i < n ? p[i] : __float2bfloat16(0.f);
    }
    __device__ __forceinline__ float get(int i) const { return __bfloat162float(v[i]); }
    __device__ __forceinline__ void set(const float (&f)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __float2bfloat16(f[i]);
    }
    __device__ __forceinline__ void store(bf16* p, int n) const {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) p[i] = v[i];
    }
};

template <int N>
struct Lane<float, N, true> {
    static_assert(N % 4 == 0, "whole accesses");
    float v[N];
    __device__ __forceinline__ void load(const float* p, int) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
            *reinterpret_cast<float4*>(v + 4 * i) = __ldcs(reinterpret_cast<const float4*>(p) + i);
    }
    __device__ __forceinline__ float get(int i) const { return v[i]; }
    __device__ __forceinline__ void set(const float (&f)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = f[i];
    }
    __device__ __forceinline__ void store(float* p, int) const {
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
            reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    }
};

template <int N>
struct Lane<float, N, false> {
    float v[N];
    __device__ __forceinline__ void load(const float* p, int n) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = i < n ? p[i] : 0.f;
    }
    __device__ __forceinline__ float get(int i) const { return v[i]; }
    __device__ __forceinline__ void set(const float (&f)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = f[i];
    }
    __device__ __forceinline__ void store(float* p, int n) const {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) p[i] = v[i];
    }
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(bf16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ bf16 from_f32<bf16>(float x) { return __float2bfloat16(x); }

// ------------------------------------------------------------ host side ----
inline bool known_dtype(int t) { return t == HLA2_DTYPE_F32 || t == HLA2_DTYPE_BF16; }
inline int dtype_size(int t) { return t == HLA2_DTYPE_F32 ? 4 : 2; }
// base and every stride (in elements) a multiple of `bytes`
inline bool aligned_to(const void* p, int esize, const long long* s, int n, int bytes) {
    if (!p) return true;
    if (reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes) return false;
    for (int i = 0; i < n; ++i)
        if ((s[i] * esize) % bytes) return false;
    return true;
}
inline bool aligned_elem(const void* p, int esize) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)esize == 0; }

}  // namespace
}  // namespace hla2
