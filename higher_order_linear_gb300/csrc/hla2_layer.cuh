// hla2_layer.cuh -- what the operators around the attention layer share
// (hla2_gated*.cu, hla2_norm.cu, hla2_rotary.cu, hla2_linear*.cu, hla2_gnorm.cu): typed
// vector accesses, launches in a row and the host-side checks of their entry points.
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

// ---------------------------------------------- a call's kernels in a row ----
// Each one's CTAs may start once all CTAs of the one before have passed follow(), and do there what needs only the
// caller's inputs.  Behind follow() the kernel before is complete, and since that one lets nobody start before its
// own follow(), so are all the others: what the call's kernels hand on (never by read-only loads, which would allow
// an old copy) and its outputs are touched only behind it.  Every kernel of the row has one; the first starts like
// any other, after all the stream was given, and so does whatever is launched behind the row in the usual way.  CTAs that find room where earlier ones have ended also fill the gap
// that a kernel's last CTAs leave.  (Plain launches and these.  Training of the linear attention, 4 x 4096 x 16 x 64:
// 227 and 198 us; 16384 x 16 x 128: 347 and 329; 2 x 1023 x 3 x 80 in fp32: 152 and 132.)
__device__ __forceinline__ void follow() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
// after: what the stream was given last is a kernel of the same call
template <typename... P, typename... A>
cudaError_t launch_following(void (*kernel)(P...), dim3 grid, int threads, size_t bytes, cudaStream_t s, bool after,
                             const A&... args) {
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cfg.attrs = &early;
    cfg.numAttrs = after ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e == cudaSuccess) note_launches(1);
    return e;
}

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

// n rows of `width` bytes, `step` bytes apart.
struct Rows {
    const void* p;
    long long n, step, width;
};
// Whether two sets of rows share a byte.  Rows of one step (slices of one tensor, or a single row on one side) are
// compared at once, others row by row where the spans meet.
inline bool rows_meet(Rows a, Rows b) {
    if (!a.p || !b.p) return false;
    auto first = [](Rows& r) {
        long long at = (long long)reinterpret_cast<uintptr_t>(r.p);
        if (r.step < 0) {
            at += (r.n - 1) * r.step;
            r.step = -r.step;
        }
        return at;
    };
    const long long pa = first(a), pb = first(b);
    if (pa + (a.n - 1) * a.step + a.width <= pb || pb + (b.n - 1) * b.step + b.width <= pa) return false;
    if (a.n == 1) a.step = b.step;
    if (b.n == 1) b.step = a.step;
    if (a.step == b.step) {
        // row j of b lies d + (j - i) step behind row i of a: the least such distance above -b.width
        const long long d = pb - pa, s = a.step;
        if (s == 0 || (a.n == 1 && b.n == 1)) return true;
        const long long least = -b.width - d, k = max((least < 0 ? -((-least + s - 1) / s) : least / s) + 1, 1 - a.n);
        return k < b.n && d + k * s < a.width;
    }
    for (long long i = 0, j = 0; i < a.n && j < b.n;) {
        const long long x = pa + i * a.step, y = pb + j * b.step;
        if (x + a.width <= y) ++i;
        else if (y + b.width <= x) ++j;
        else return true;
    }
    return false;
}

}  // namespace
}  // namespace hla2
