// hla2_norm.cu -- root-mean-square norm with the residual's addition, its
// 8-bit output with a scale for each row, and its gradient.
//
//   t = x + r,  y = t w / sqrt(mean(t^2) + eps);
//   8 bits: scale = max|y| / 448 (448: the largest e4m3 number), q = e4m3(y / scale).
//
// One pass over the data: a row stays in the registers of the threads that
// share it (8 elements to a thread and step, up to 4 steps), which sum its
// squares and, for 8 bits, take the maximum of |t w| in the same reduction
// (max|y| = max|t w| / sqrt(...)); y is formed from the registers.  x, r, t and
// y cross HBM once.  Short rows share a block, a row to a group of lanes.
//
// HBM bounds it.  16384 rows of 2048 with a residual, 16 bits (268 MB): 41.6 us,
// 0.95 of the copy bandwidth (6.8 TB/s); 2^20 rows of 128, fp32 to 16 bits (805 MB):
// 116 us, 1.02; 8 bits, 8191 rows of 8192 (470 MB): 74 us, 0.94, with 256 threads of
// 32 elements to a row (512 of 16 took 91 us, 1024 of 8 153 us, when this took 76: a barrier holds up more
// of the SM).  16 rows of 2048 take 2.4 us, a launch.
//
// The maximum is taken over the bit patterns of |t w| as whole numbers, which
// order like the values with NaN above inf, so a NaN reaches the scale.
#include <cuda_fp8.h>

#include "hla2_layer.cuh"

namespace hla2 {
namespace {

constexpr int kMaxC = 16384;
enum { kOutF32 = 0, kOutBF16 = 1, kOutE4M3 = 2 };

struct NormParams {
    const void *x, *r, *w;
    void *s, *y;
    float* scale;
    long long rows, ldx, ldr, lds, ldy;
    int C, wdtype;
    float eps, inv_c;
};

// Sum over the TPR threads of a row (TPR a power of two).  Threads of a row are
// consecutive; TPR <= 32: lanes of one warp.  Every thread gets the result.
template <int TPR>
__device__ __forceinline__ void row_reduce(float& a, uint32_t& m, bool with_max, float* sh_a, uint32_t* sh_m) {
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) >> 1; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        if (with_max) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    if constexpr (TPR > 32) {
        constexpr int NW = TPR / 32;
        const int warp = threadIdx.x >> 5, w0 = warp / NW * NW;
        if ((threadIdx.x & 31) == 0) {
            sh_a[warp] = a;
            if (with_max) sh_m[warp] = m;
        }
        __syncthreads();
        a = 0.f;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            a += sh_a[w0 + i];
            if (with_max) m = max(m, sh_m[w0 + i]);
        }
    }
}

// Eight consecutive elements of the weight (or ones) as fp32
template <bool VEC>
__device__ __forceinline__ void load_weight(const void* w, int wdtype, int c, int n, float (&out)[8]) {
    if (!w) {
#pragma unroll
        for (int j = 0; j < 8; ++j) out[j] = 1.f;
    } else if (wdtype == HLA2_DTYPE_F32) {
        const float* p = static_cast<const float*>(w) + c;
        if (VEC) {
            const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
            out[0] = a.x; out[1] = a.y; out[2] = a.z; out[3] = a.w;
            out[4] = b.x; out[5] = b.y; out[6] = b.z; out[7] = b.w;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) out[j] = j < n ? __ldg(p + j) : 0.f;
        }
    } else {
        const bf16* p = static_cast<const bf16*>(w) + c;
        if (VEC) {
            const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
            const uint32_t v[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                out[2 * j] = __uint_as_float(v[j] << 16);
                out[2 * j + 1] = __uint_as_float(v[j] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) out[j] = j < n ? __bfloat162float(p[j]) : 0.f;
        }
    }
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

constexpr int block_of(int tpr) { return tpr > 256 ? tpr : 256; }

// TPR threads share a row, NV steps of 8 elements each.  VEC: C, strides and
// pointers allow 16-byte accesses of 8 elements (8 bytes of the 8-bit output).
template <typename T, int OUT, int TPR, int NV, bool VEC>
__global__ void __launch_bounds__(block_of(TPR)) rmsnorm_kernel(const NormParams p) {
    constexpr int kThreads = block_of(TPR), kRows = kThreads / TPR;
    constexpr bool Q8 = OUT == kOutE4M3;
    __shared__ float sh_a[kThreads / 32];
    __shared__ uint32_t sh_m[kThreads / 32];
    const int lane = threadIdx.x % TPR;
    const long long row = (long long)blockIdx.x * kRows + threadIdx.x / TPR;
    const bool live = row < p.rows;
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    const T* r = p.r ? static_cast<const T*>(p.r) + row * p.ldr : nullptr;

    Lane<T, 8, VEC> xv[NV], rv[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (v * TPR + lane) * 8, n = p.C - c;
        if (live && n > 0) {
            xv[v].load(x + c, n);
            if (r) rv[v].load(r + c, n);
        }
    }
    float t[NV][8];
    float ss = 0.f;
    uint32_t m = 0u;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (v * TPR + lane) * 8, n = p.C - c;
        const bool in = live && n > 0;
        if (in) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                t[v][j] = (VEC || j < n) ? xv[v].get(j) + (r ? rv[v].get(j) : 0.f) : 0.f;
                ss = fmaf(t[v][j], t[v][j], ss);
            }
            if (p.s) {
                xv[v].set(t[v]);
                xv[v].store(static_cast<T*>(p.s) + row * p.lds + c, n);
            }
            float w[8];
            load_weight<VEC>(p.w, p.wdtype, c, n, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                t[v][j] *= w[j];
                if (Q8) m = max(m, __float_as_uint(t[v][j]) & 0x7fffffffu);
            }
        }
    }
    row_reduce<TPR>(ss, m, Q8, sh_a, sh_m);
    if (!live) return;
    const float rstd = rsqrtf(fmaf(ss, p.inv_c, p.eps));  // 2 ulp; a root and a quotient took 30 instructions a row
    if constexpr (Q8) {
        // The codes are those of y / scale = 448 t w / max|t w|: the root cancels, and where the
        // quotient stands between two codes (16-bit operands often give such) it is exact, which
        // fp32's y and scale lose.  The quotient is the product with the reciprocal, corrected by
        // its remainder (Markstein's division).  Rows beyond 2^+-100 are scaled by a power of two,
        // so that neither the reciprocal nor 448 t w leaves fp32's range.
        const float most = __uint_as_float(m);
        const float scale = most == 0.f ? 1.f : most * rstd / 448.f;
        if (lane == 0) p.scale[row] = scale;
        const float by = most > 0x1p100f ? 0x1p-64f : most < 0x1p-100f ? 0x1p64f : 1.f;
        const float den = most == 0.f ? 1.f : most * by, inv = 1.f / den;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + lane) * 8, n = p.C - c;
            if (n > 0) {
                float q[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float num = t[v][j] * (448.f * by), first = num * inv;
                    q[j] = fmaf(fmaf(-first, den, num), inv, first);
                }
                unsigned char* o = static_cast<unsigned char*>(p.y) + row * p.ldy + c;
                const uint32_t a = e4m3x4(q[0], q[1], q[2], q[3]), b = e4m3x4(q[4], q[5], q[6], q[7]);
                if (VEC) {
                    *reinterpret_cast<uint2*>(o) = make_uint2(a, b);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j < n) o[j] = (unsigned char)((j < 4 ? a : b) >> (8 * (j & 3)));
                }
            }
        }
    } else {
        using TO = typename std::conditional<OUT == kOutF32, float, bf16>::type;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + lane) * 8, n = p.C - c;
            if (n > 0) {
                float y[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = t[v][j] * rstd;
                Lane<TO, 8, VEC> yv;
                yv.set(y);
                yv.store(static_cast<TO*>(p.y) + row * p.ldy + c, n);
            }
        }
    }
}

template <typename T, int OUT, int TPR, int NV>
cudaError_t launch_norm(const NormParams& p, bool vec, cudaStream_t s) {
    constexpr int kRows = block_of(TPR) / TPR;
    const unsigned grid = (unsigned)((p.rows + kRows - 1) / kRows);
    if (vec) rmsnorm_kernel<T, OUT, TPR, NV, true><<<grid, block_of(TPR), 0, s>>>(p);
    else rmsnorm_kernel<T, OUT, TPR, NV, false><<<grid, block_of(TPR), 0, s>>>(p);
    note_launches(1);
    return cudaGetLastError();
}

// Threads to a row x steps of 8 elements, each against its neighbours on 0.5 GB of
// 16-bit rows with a residual (us; 79 for its bytes; C = 128: fp32 in, 118; 2048: 39.5):
//   C = 64:    8 x 1  79.5, 16 x 1 105 (half its lanes idle)
//   C = 128:  16 x 1 115.4, 8 x 2 120.8
//   C = 256:  32 x 1  79.4, 16 x 2 79.5, 8 x 4 80.1
//   C = 512:  32 x 2  80.2, 64 x 1 79.9, 16 x 4 81.1
//   C = 1024: 128 x 1 80.0, 64 x 2 80.0, 32 x 4 81.0
//   C = 2048: 256 x 1 41.6, 128 x 2 42.0, 64 x 4 42.9
//   C = 4096: 256 x 2 80.1, 512 x 1 80.9, 128 x 4 81.2
//   C = 16384: 512 x 4 82.4, 1024 x 2 94.4
// and C = 8192 above.  Up to 512 a row stays in one warp, whose sum needs no barrier.
template <typename T, int OUT>
cudaError_t pick_norm(const NormParams& p, bool vec, cudaStream_t s) {
    const int C = p.C;
    if (C <= 64) return launch_norm<T, OUT, 8, 1>(p, vec, s);
    if (C <= 128) return launch_norm<T, OUT, 16, 1>(p, vec, s);
    if (C <= 256) return launch_norm<T, OUT, 32, 1>(p, vec, s);
    if (C <= 512) return launch_norm<T, OUT, 32, 2>(p, vec, s);
    if (C <= 1024) return launch_norm<T, OUT, 128, 1>(p, vec, s);
    if (C <= 2048) return launch_norm<T, OUT, 256, 1>(p, vec, s);
    if (C <= 4096) return launch_norm<T, OUT, 256, 2>(p, vec, s);
    if (C <= 8192) return launch_norm<T, OUT, 256, 4>(p, vec, s);
    return launch_norm<T, OUT, 512, 4>(p, vec, s);
}

// ------------------------------------------------------------- gradient ----
//   n = t rstd;  dx = rstd (w dy - n mean(w dy n)) + ds;  dw = sum_rows dy n.
// The row stays in registers between its two sums (t^2 and w dy t) and dx.
// The column sums of dw are kept in registers over all the rows that a group of
// threads walks; a block adds those of its groups in order and leaves them in the
// workspace, and a second kernel adds the blocks' in order, so the result does
// not depend on timing.
//
// 16384 x 2048, 16 bits (268 MB, 39.5 us at the copy bandwidth): 54 us, of which the
// second kernel 5.5.  The first one's instructions bound it as much as HBM does
// (about 29 for each element, the reductions' among them): 8 elements to a thread
// with the next row's loads in flight take 47 us, 16 elements, whose sums and weights
// leave registers for half the threads, 54 us or more.  Rows beyond 8192 have to take 16
// all the same, 1024 threads to a row, and go to local memory: 2048 x 12288 82 us, its
// bytes 30.  The fp32 norm of heads, 2^18 rows of 64 with a 16-bit dy: 45 us, bytes 25.
struct NormBwdParams {
    const void *t, *dy, *w, *ds;
    void* dx;
    float *dw, *part;  // part: [groups][C]
    long long rows, ldt, lddy, ldds, lddx;
    int C, wdtype;
    float eps, inv_c;
};

// Threads of a block of the gradient, and blocks to an SM: 64 registers to a
// thread hold a row's 8 elements of t, dy and ds, the weights, the column sums
// and the next row's loads.
constexpr int bwd_block(int tpr) { return tpr > 256 ? tpr : 256; }
constexpr int bwd_blocks(int tpr) { return 1024 / bwd_block(tpr); }

template <int TPR>
__device__ __forceinline__ void row_sum2(float& a, float& b, float2* sh, int& phase) {
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) >> 1; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if constexpr (TPR > 32) {
        constexpr int NW = TPR / 32, kWarps = bwd_block(TPR) / 32;
        const int warp = threadIdx.x >> 5, w0 = warp / NW * NW;
        float2* buf = sh + phase * kWarps;  // two buffers: one barrier for each row
        phase ^= 1;
        if ((threadIdx.x & 31) == 0) buf[warp] = make_float2(a, b);
        // the row's own threads only: the rows of a block do not wait for one another
        asm volatile("bar.sync %0, %1;" ::"r"((int)threadIdx.x / TPR + 1), "n"(TPR) : "memory");
        a = b = 0.f;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            a += buf[w0 + i].x;
            b += buf[w0 + i].y;
        }
    }
}

template <typename T, typename TY, int TPR, int NV, bool VEC>
__global__ void __launch_bounds__(bwd_block(TPR), bwd_blocks(TPR)) rmsnorm_bwd_kernel(const NormBwdParams p) {
    constexpr int kThreads = bwd_block(TPR), kRows = kThreads / TPR;
    __shared__ float2 sh[2 * kThreads / 32];
    extern __shared__ __align__(16) float columns[];  // [C], where rows share the block
    int phase = 0;
    const int lane = threadIdx.x % TPR;
    const long long group = (long long)blockIdx.x * kRows + threadIdx.x / TPR;
    const long long groups = (long long)gridDim.x * kRows;
    // a thread's columns are the same in every row: so are its weights
    float w[NV][8], acc[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (v * TPR + lane) * 8, n = p.C - c;
#pragma unroll
        for (int j = 0; j < 8; ++j) w[v][j] = acc[v][j] = 0.f;
        if (n > 0) load_weight<VEC>(p.w, p.wdtype, c, n, w[v]);
    }
    Lane<T, 8, VEC> tv[NV], sv[NV];
    Lane<TY, 8, VEC> yv[NV];
    auto load = [&](long long row) {
        const T* t = static_cast<const T*>(p.t) + row * p.ldt;
        const TY* dy = static_cast<const TY*>(p.dy) + row * p.lddy;
        const T* ds = static_cast<const T*>(p.ds) + row * p.ldds;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + lane) * 8, n = p.C - c;
            if (n > 0) {
                tv[v].load(t + c, n);
                yv[v].load(dy + c, n);
                if (p.ds) sv[v].load(ds + c, n);
            }
        }
    };
    // lanes of one warp that hold different rows make the same trips (the sums are taken by whole warps)
    const int trips = (int)((p.rows + groups - 1) / groups);
    long long row = group;
    if (row < p.rows) load(row);
    for (int k = 0; k < trips; ++k, row += groups) {
        const bool live = row < p.rows;
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int n = p.C - (v * TPR + lane) * 8;
            if (live && n > 0) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float t = tv[v].get(j);
                    a = fmaf(t, t, a);
                    b = fmaf(w[v][j] * yv[v].get(j), t, b);
                }
            }
        }
        row_sum2<TPR>(a, b, sh, phase);
        if (!live) continue;
        const float rstd = rsqrtf(fmaf(a, p.inv_c, p.eps));
        // rstd mean(w dy n): of dx's own size, where a power of rstd alone leaves fp32's range
        const float back = rstd * (rstd * (b * p.inv_c));
        Lane<T, 8, VEC> out[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int n = p.C - (v * TPR + lane) * 8;
            if (n > 0) {
                float dx[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float t = tv[v].get(j), dy = rstd * yv[v].get(j);
                    dx[j] = fmaf(w[v][j], dy, -((t * rstd) * back));
                    acc[v][j] = fmaf(dy, t, acc[v][j]);
                }
                if (p.ds) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) dx[j] += sv[v].get(j);
                }
                out[v].set(dx);
            }
        }
        if (row + groups < p.rows) load(row + groups);  // on its way while this row is written
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + lane) * 8, n = p.C - c;
            if (n > 0) out[v].store(static_cast<T*>(p.dx) + row * p.lddx + c, n);
        }
    }
    if (!p.dw) return;
    // the block's sums, group after group, then one line of partial sums to a block
    float* const part = p.part + (long long)blockIdx.x * p.C;
    for (int g = 0; g < kRows; ++g) {
        if (threadIdx.x / TPR == g) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = (v * TPR + lane) * 8;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c + j < p.C) {
                        const float s = g > 0 ? columns[c + j] + acc[v][j] : acc[v][j];
                        if (g + 1 < kRows) columns[c + j] = s;
                        else part[c + j] = s;
                    }
            }
        }
        if (g + 1 < kRows) __syncthreads();
    }
}

// dw[c] = sum of the blocks' partial sums, in a fixed order: 16 columns to a
// block, each 64 threads' sums of every 64th line.
constexpr int kFoldColumns = 16, kFoldThreads = 1024, kFoldLines = kFoldThreads / kFoldColumns;
__global__ void __launch_bounds__(kFoldThreads) fold_columns_kernel(const float* __restrict__ part,
                                                                   float* __restrict__ dw, int lines, int C) {
    __shared__ float sh[kFoldThreads / 32][kFoldColumns];
    const int col = threadIdx.x % kFoldColumns, line = threadIdx.x / kFoldColumns;
    const int c = blockIdx.x * kFoldColumns + col;
    float a = 0.f;
    if (c < C) {
#pragma unroll 8
        for (int g = line; g < lines; g += kFoldLines) a += part[(size_t)g * C + c];
    }
    a += __shfl_down_sync(0xffffffffu, a, 16);  // the warp's second line of threads
    if ((threadIdx.x & 31) < kFoldColumns) sh[threadIdx.x >> 5][col] = a;
    __syncthreads();
    if (threadIdx.x < kFoldColumns && c < C) {
        a = 0.f;
#pragma unroll
        for (int i = 0; i < kFoldThreads / 32; ++i) a += sh[i][col];
        dw[c] = a;
    }
}

// Blocks of the gradient's grid: what the SMs hold, at most one for each run of rows.
struct BwdPlan {
    int tpr, nv, rows_per_block, blocks;
};
BwdPlan bwd_plan(long long rows, int C) {
    BwdPlan b;
    b.nv = C <= 8192 ? 1 : 2;
    b.tpr = 8;
    while (b.tpr * b.nv * 8 < C) b.tpr *= 2;
    b.rows_per_block = bwd_block(b.tpr) / b.tpr;
    const long long most = (long long)sm_count() * bwd_blocks(b.tpr);
    const long long need = (rows + b.rows_per_block - 1) / b.rows_per_block;
    b.blocks = (int)(need < most ? need : most);
    return b;
}

template <typename T, typename TY, int TPR, int NV>
cudaError_t launch_bwd(const NormBwdParams& p, int blocks, bool vec, cudaStream_t s) {
    const size_t smem = p.dw && TPR < bwd_block(TPR) ? (size_t)p.C * 4 : 0;
    if (vec) rmsnorm_bwd_kernel<T, TY, TPR, NV, true><<<blocks, bwd_block(TPR), smem, s>>>(p);
    else rmsnorm_bwd_kernel<T, TY, TPR, NV, false><<<blocks, bwd_block(TPR), smem, s>>>(p);
    note_launches(1);
    return cudaGetLastError();
}

template <typename T, typename TY>
cudaError_t pick_bwd(const NormBwdParams& p, const BwdPlan& b, bool vec, cudaStream_t s) {
    switch (b.tpr) {
        case 8: return launch_bwd<T, TY, 8, 1>(p, b.blocks, vec, s);
        case 16: return launch_bwd<T, TY, 16, 1>(p, b.blocks, vec, s);
        case 32: return launch_bwd<T, TY, 32, 1>(p, b.blocks, vec, s);
        case 64: return launch_bwd<T, TY, 64, 1>(p, b.blocks, vec, s);
        case 128: return launch_bwd<T, TY, 128, 1>(p, b.blocks, vec, s);
        case 256: return launch_bwd<T, TY, 256, 1>(p, b.blocks, vec, s);
        case 512: return launch_bwd<T, TY, 512, 1>(p, b.blocks, vec, s);
        default:
            return b.nv == 1 ? launch_bwd<T, TY, 1024, 1>(p, b.blocks, vec, s)
                             : launch_bwd<T, TY, 1024, 2>(p, b.blocks, vec, s);
    }
}

int check_rows(const char* what, long long rows, int C, int dtype, int wdtype, const void* W) {
    if (rows <= 0 || C <= 0) return set_error(HLA2_ERR_INVALID, "%s: sizes must be positive (rows=%lld C=%d)", what, rows, C);
    if (C > kMaxC) return set_error(HLA2_ERR_UNSUPPORTED, "%s: C=%d exceeds %d", what, C, kMaxC);
    if (rows > 0x7fffffffLL) return set_error(HLA2_ERR_UNSUPPORTED, "%s: rows=%lld exceeds 2^31 - 1", what, rows);
    if (!known_dtype(dtype)) return set_error(HLA2_ERR_UNSUPPORTED, "%s: unknown dtype %d", what, dtype);
    if (W && !known_dtype(wdtype)) return set_error(HLA2_ERR_UNSUPPORTED, "%s: unknown weight dtype %d", what, wdtype);
    return HLA2_OK;
}
bool row_ok(const void* p, long long ld, int C, int es) { return !p || (ld >= C && aligned_elem(p, es)); }
bool row_vec(const void* p, long long ld, int es, int bytes) { return aligned_to(p, es, &ld, 1, bytes); }

int norm_common(const char* what, const void* X, const void* R, const void* W, void* S, void* Y, float* scale,
                long long rows, int C, long long ldx, long long ldr, long long lds, long long ldy, float eps, int dtype,
                int wdtype, int out, hla2_stream_t stream) {
    if (int rc = check_rows(what, rows, C, dtype, wdtype, W)) return rc;
    if (!X || !Y || (out == kOutE4M3 && !scale)) return set_error(HLA2_ERR_INVALID, "%s: null pointer", what);
    if (!(eps >= 0.f)) return set_error(HLA2_ERR_INVALID, "%s: eps must not be negative", what);
    const int es = dtype_size(dtype), os = out == kOutE4M3 ? 1 : out == kOutF32 ? 4 : 2;
    const int wsz = W ? dtype_size(wdtype) : 4;
    if (!row_ok(X, ldx, C, es) || !row_ok(R, ldr, C, es) || !row_ok(S, lds, C, es) || !row_ok(Y, ldy, C, os) ||
        !aligned_elem(W, wsz) || !aligned_elem(scale, 4))
        return set_error(HLA2_ERR_INVALID, "%s: a row stride below C=%d or a pointer not aligned to its element", what, C);
    const bool vec = C % 8 == 0 && row_vec(X, ldx, es, 16) && row_vec(R, ldr, es, 16) && row_vec(S, lds, es, 16) &&
                     row_vec(Y, ldy, os, out == kOutE4M3 ? 8 : 16) && reinterpret_cast<uintptr_t>(W) % 16 == 0;
    NormParams p{X, R, W, S, Y, scale, rows, ldx, ldr, lds, ldy, C, wdtype, eps, 1.f / (float)C};
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (dtype == HLA2_DTYPE_BF16)
        e = out == kOutF32 ? pick_norm<bf16, kOutF32>(p, vec, s)
            : out == kOutBF16 ? pick_norm<bf16, kOutBF16>(p, vec, s) : pick_norm<bf16, kOutE4M3>(p, vec, s);
    else
        e = out == kOutF32 ? pick_norm<float, kOutF32>(p, vec, s)
            : out == kOutBF16 ? pick_norm<float, kOutBF16>(p, vec, s) : pick_norm<float, kOutE4M3>(p, vec, s);
    if (e != cudaSuccess) return set_error(HLA2_ERR_LAUNCH, "%s: %s", what, cudaGetErrorString(e));
    return HLA2_OK;
}

}  // namespace
}  // namespace hla2

extern "C" int hla2_rmsnorm(const void* X, const void* R, const void* W, void* S, void* Y, long long rows, int C,
                            long long ldx, long long ldr, long long lds, long long ldy, float eps, int dtype,
                            int wdtype, int out_dtype, hla2_stream_t stream) {
    using namespace hla2;
    if (!known_dtype(out_dtype)) return set_error(HLA2_ERR_UNSUPPORTED, "rmsnorm: unknown output dtype %d", out_dtype);
    return norm_common("rmsnorm", X, R, W, S, Y, nullptr, rows, C, ldx, ldr, lds, ldy, eps, dtype, wdtype,
                       out_dtype == HLA2_DTYPE_F32 ? kOutF32 : kOutBF16, stream);
}

extern "C" int hla2_rmsnorm_q8(const void* X, const void* R, const void* W, void* S, void* Q, float* scale,
                               long long rows, int C, long long ldx, long long ldr, long long lds, long long ldq,
                               float eps, int dtype, int wdtype, hla2_stream_t stream) {
    using namespace hla2;
    return norm_common("rmsnorm_q8", X, R, W, S, Q, scale, rows, C, ldx, ldr, lds, ldq, eps, dtype, wdtype, kOutE4M3,
                       stream);
}

extern "C" size_t hla2_rmsnorm_backward_workspace(long long rows, int C) {
    using namespace hla2;
    if (rows <= 0 || rows > 0x7fffffffLL || C <= 0 || C > kMaxC) return 0;
    const BwdPlan b = bwd_plan(rows, C);
    return ((size_t)b.blocks * C * 4 + 255) & ~size_t(255);
}

extern "C" int hla2_rmsnorm_backward(const void* S, const void* dY, const void* W, const void* dS, void* dX, float* dW,
                                     long long rows, int C, const long long* ld, float eps, int dtype, int wdtype,
                                     int out_dtype, void* workspace, size_t ws_bytes, hla2_stream_t stream) {
    using namespace hla2;
    const char* what = "rmsnorm_backward";
    if (int rc = check_rows(what, rows, C, dtype, wdtype, W)) return rc;
    if (!known_dtype(out_dtype)) return set_error(HLA2_ERR_UNSUPPORTED, "%s: unknown dtype %d of dY", what, out_dtype);
    if (!S || !dY || !dX) return set_error(HLA2_ERR_INVALID, "%s: null pointer", what);
    if (!(eps >= 0.f)) return set_error(HLA2_ERR_INVALID, "%s: eps must not be negative", what);
    const long long dense[4] = {C, C, C, C};
    if (!ld) ld = dense;
    const int es = dtype_size(dtype), os = dtype_size(out_dtype), wsz = W ? dtype_size(wdtype) : 4;
    if (!row_ok(S, ld[0], C, es) || !row_ok(dY, ld[1], C, os) || !row_ok(dS, ld[2], C, es) ||
        !row_ok(dX, ld[3], C, es) || !aligned_elem(W, wsz) || !aligned_elem(dW, 4))
        return set_error(HLA2_ERR_INVALID, "%s: a row stride below C=%d or a pointer not aligned to its element", what, C);
    const BwdPlan b = bwd_plan(rows, C);
    if (dW && (!workspace || ws_bytes < (size_t)b.blocks * C * 4))
        return set_error(HLA2_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", what, ws_bytes, (size_t)b.blocks * C * 4);
    if (dW && reinterpret_cast<uintptr_t>(workspace) % 16) return set_error(HLA2_ERR_INVALID, "%s: workspace not 16-byte aligned", what);
    const bool vec = C % 8 == 0 && row_vec(S, ld[0], es, 16) && row_vec(dY, ld[1], os, 16) &&
                     row_vec(dS, ld[2], es, 16) && row_vec(dX, ld[3], es, 16) &&
                     reinterpret_cast<uintptr_t>(W) % 16 == 0;
    NormBwdParams p{S, dY, W, dS, dX, dW, static_cast<float*>(workspace), rows, ld[0], ld[1], ld[2], ld[3], C, wdtype, eps, 1.f / (float)C};
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (dtype == HLA2_DTYPE_BF16)
        e = out_dtype == HLA2_DTYPE_BF16 ? pick_bwd<bf16, bf16>(p, b, vec, s) : pick_bwd<bf16, float>(p, b, vec, s);
    else
        e = out_dtype == HLA2_DTYPE_BF16 ? pick_bwd<float, bf16>(p, b, vec, s) : pick_bwd<float, float>(p, b, vec, s);
    if (e == cudaSuccess && dW) {
        fold_columns_kernel<<<(C + kFoldColumns - 1) / kFoldColumns, kFoldThreads, 0, s>>>(p.part, dW, b.blocks, C);
        note_launches(1);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) return set_error(HLA2_ERR_LAUNCH, "%s: %s", what, cudaGetErrorString(e));
    return HLA2_OK;
}
