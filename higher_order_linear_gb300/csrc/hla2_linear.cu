// hla2_linear.cu -- first-order linear attention with a decay for each head:
// entries, segment plan, scan of the segments' states, CUDA-core walk and the
// single-token step.
//
//   S_t = g_h S_{t-1} + k_t v_t^T,  o_t = S_t^T q_t.
//
// The CUDA-core walk computes in fp32 and carries what the tensor cores do not
// (fp32 inputs, widths or strides without 16-byte steps): chunks of 64 tokens,
//   P = tril(A B^T) o g^(i-j),  O = P C + g^(i+1) A S,  S = g^n S + (B g^(n-1-j))^T C,
// with tiles and state in shared memory and register blocks of up to 8 x 8.  Its
// products bound it: 2 x 3 heads of 1023 tokens, 80 and 48 wide, 12 us for the
// states and 25 for the outputs (a chunk to a CTA), 152 us for forward and gradients.
#include "hla2_linear.cuh"

namespace hla2 {
namespace {

constexpr int kTokens = 64;  // a chunk of the CUDA-core walk
constexpr int kWalkThreads = 256;

template <int D>
struct SimpleLayout {  // floats
    static constexpr int LD = D + 4;  // rows four banks apart: 16-byte reads down a column of rows do not collide
    static constexpr int A = 0, B = kTokens * LD, C = 2 * kTokens * LD, P = 3 * kTokens * LD;
    static constexpr int LP = kTokens + 4;
    static constexpr int S = P + kTokens * LP, G = S + D * D;
    static constexpr int kBytes = (G + kTokens + 1) * 4;
};

template <typename T, int D, bool OUT>
__global__ void __launch_bounds__(kWalkThreads, 1) lin_walk_kernel(const LinWalk p) {
    using LY = SimpleLayout<D>;
    constexpr int LD = LY::LD, LP = LY::LP;
    extern __shared__ __align__(16) float sm[];
    float *const sA = sm + LY::A, *const sB = sm + LY::B, *const sC = sm + LY::C, *const sP = sm + LY::P,
                 *const sS = sm + LY::S, *const pw = sm + LY::G;
    const int tid = threadIdx.x;
    const int bh = blockIdx.y, w = blockIdx.x, seg = p.rev ? p.nseg - 1 - w : w;
    const int b = bh / p.H, h = bh % p.H;
    const int len = length_of(p, b);
    if (tid <= kTokens) pw[tid] = power(__ldg(p.gamma + h), tid);
    follow();
    const size_t R = (size_t)p.da * p.dc;
    // the state that enters
    {
        const float* src = nullptr;
        long long sr = 0, sc = 0;
        if (OUT && p.nseg > 1) {
            src = p.rec + ((size_t)bh * (p.nseg + 1) + w) * R; sr = p.rec_r; sc = p.rec_c;
        } else if (OUT && p.s_in) {
            src = p.s_in + (size_t)bh * R; sr = p.in_r; sc = p.in_c;
        }
        const bool turned = sr == 1 && sc != 1;  // neighbours in memory to neighbouring threads
#pragma unroll 16
        for (int i = 0; i < D * D / kWalkThreads; ++i) {
            const int e = tid + i * kWalkThreads, r = turned ? e % D : e / D, c = turned ? e / D : e % D;
            sS[r * D + c] = src && r < p.da && c < p.dc ? src[r * sr + c * sc] : 0.f;
        }
    }
    const T* const ga = static_cast<const T*>(p.a) + b * p.sa[0] + h * p.sa[1];
    const T* const gb = static_cast<const T*>(p.b) + b * p.sb[0] + h * p.sb[1];
    const T* const gc = static_cast<const T*>(p.c) + b * p.sc[0] + h * p.sc[1];
    T* const go = static_cast<T*>(p.o) + (OUT ? b * p.so[0] + h * p.so[1] : 0);
    const int c0 = seg * p.seglen, c1 = min(c0 + p.seglen, p.nchunk);
    for (int i = 0; i < c1 - c0; ++i) {
        const int t0 = (p.rev ? c1 - 1 - i : c0 + i) * kTokens;
        const int n = min(kTokens, len - t0);
        if (n <= 0) continue;  // behind the sequence's end: all threads agree
        __syncthreads();
        // rows of four values at a time where they allow it, eight loads on their way to a thread
        auto load = [&](float* dst, const T* src, long long st, int width, bool four) {
            if (four) {
                constexpr int RUN = D / 4, N = kTokens * RUN / kWalkThreads;
                Lane<T, 4, true> v[N];
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const int e = tid + k * kWalkThreads, r = e / RUN, c = e % RUN * 4;
                    if (r < n && c < width) v[k].load(src + (t0 + r) * st + c, 4);
                }
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const int e = tid + k * kWalkThreads, r = e / RUN, c = e % RUN * 4;
                    const bool in = r < n && c < width;
                    *reinterpret_cast<float4*>(dst + r * LD + c) =
                        in ? make_float4(v[k].get(0), v[k].get(1), v[k].get(2), v[k].get(3)) : make_float4(0.f, 0.f, 0.f, 0.f);
                }
            } else {
#pragma unroll 8
                for (int k = 0; k < kTokens * D / kWalkThreads; ++k) {
                    const int e = tid + k * kWalkThreads, r = e / D, c = e % D;
                    dst[r * LD + c] = r < n && c < width ? to_f32(src[(t0 + r) * st + c]) : 0.f;
                }
            }
        };
        if (OUT) load(sA, ga, p.sa[2], p.da, p.fours & 1);
        load(sB, gb, p.sb[2], p.da, p.fours & 2);
        load(sC, gc, p.sc[2], p.dc, p.fours & 4);
        __syncthreads();
        if (OUT) {
            // P: rows 4 (tid / 16) .. + 3, columns tid % 16 + 16 q
            const int r0 = tid / 16 * 4, q0 = tid % 16;
            float acc[4][4] = {};
            for (int x = 0; x < p.da; x += 4) {  // (zeros up to a whole step)
                float4 a[4], bb[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    a[q] = *reinterpret_cast<const float4*>(sA + (r0 + q) * LD + x);
                    bb[q] = *reinterpret_cast<const float4*>(sB + (q0 + 16 * q) * LD + x);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        acc[r][q] = fmaf(a[r].x, bb[q].x, acc[r][q]);
                        acc[r][q] = fmaf(a[r].y, bb[q].y, acc[r][q]);
                        acc[r][q] = fmaf(a[r].z, bb[q].z, acc[r][q]);
                        acc[r][q] = fmaf(a[r].w, bb[q].w, acc[r][q]);
                    }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int ii = r0 + r, jj = q0 + 16 * q, far = p.rev ? jj - ii : ii - jj;
                    sP[ii * LP + jj] = far >= 0 ? acc[r][q] * pw[far] : 0.f;
                }
            __syncthreads();
            // O: 4 columns, R rows to a thread
            constexpr int TC = D / 4, RO = kTokens * TC / kWalkThreads;
            const int col = tid % TC * 4, row = tid / TC * RO;
            float o[RO][4] = {};
            for (int x = 0; x < p.da; x += 4) {
                float4 s[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) s[q] = *reinterpret_cast<const float4*>(sS + (x + q) * D + col);
#pragma unroll
                for (int r = 0; r < RO; ++r) {
                    const float4 a = *reinterpret_cast<const float4*>(sA + (row + r) * LD + x);
                    const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        o[r][0] = fmaf(av[q], s[q].x, o[r][0]);
                        o[r][1] = fmaf(av[q], s[q].y, o[r][1]);
                        o[r][2] = fmaf(av[q], s[q].z, o[r][2]);
                        o[r][3] = fmaf(av[q], s[q].w, o[r][3]);
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < RO; ++r) {
                const float f = row + r < n ? pw[p.rev ? n - 1 - (row + r) : row + r + 1] : 0.f;
#pragma unroll
                for (int q = 0; q < 4; ++q) o[r][q] *= f;
            }
            for (int j = 0; j < kTokens; j += 4) {
                float4 s[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) s[q] = *reinterpret_cast<const float4*>(sC + (j + q) * LD + col);
#pragma unroll
                for (int r = 0; r < RO; ++r) {
                    const float4 a = *reinterpret_cast<const float4*>(sP + (row + r) * LP + j);
                    const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        o[r][0] = fmaf(av[q], s[q].x, o[r][0]);
                        o[r][1] = fmaf(av[q], s[q].y, o[r][1]);
                        o[r][2] = fmaf(av[q], s[q].z, o[r][2]);
                        o[r][3] = fmaf(av[q], s[q].w, o[r][3]);
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < RO; ++r)
                if (row + r < n) {
                    T* dst = go + (t0 + row + r) * p.so[2] + col;
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (col + q < p.dc) dst[q] = from_f32<T>(o[r][q]);
                }
            __syncthreads();  // every read of S precedes its update
        }
        // S = g^n S + (B g^(..))^T C: NS x NS values to a thread, columns in steps of four
        constexpr int NS = D == 128 ? 8 : 4, TS = D / NS;
        const int x0 = tid / TS * NS, cc = tid % TS * 4;
        const bool wide = NS == 4 || p.dc > 4 * TS;  // the second half of the columns
        if (x0 >= p.da) continue;
        float acc[NS][NS];
        const float gn = pw[n];
#pragma unroll
        for (int r = 0; r < NS; ++r)
#pragma unroll
            for (int q = 0; q < NS; q += 4) {
                const float4 s = *reinterpret_cast<const float4*>(sS + (x0 + r) * D + cc + q * TS);
                acc[r][q] = gn * s.x; acc[r][q + 1] = gn * s.y; acc[r][q + 2] = gn * s.z; acc[r][q + 3] = gn * s.w;
            }
        for (int j = 0; j < n; ++j) {
            const float f = pw[p.rev ? j + 1 : n - 1 - j];
            float bv[NS], cv[NS];
#pragma unroll
            for (int q = 0; q < NS; q += 4) {
                const float4 x = *reinterpret_cast<const float4*>(sB + j * LD + x0 + q);
                bv[q] = f * x.x; bv[q + 1] = f * x.y; bv[q + 2] = f * x.z; bv[q + 3] = f * x.w;
                if (q == 0 || wide) {
                    const float4 y = *reinterpret_cast<const float4*>(sC + j * LD + cc + q * TS);
                    cv[q] = y.x; cv[q + 1] = y.y; cv[q + 2] = y.z; cv[q + 3] = y.w;
                }
            }
#pragma unroll
            for (int q = 0; q < NS; q += 4)
                if (q == 0 || wide) {
#pragma unroll
                    for (int r = 0; r < NS; ++r)
#pragma unroll
                        for (int k = q; k < q + 4; ++k) acc[r][k] = fmaf(bv[r], cv[k], acc[r][k]);
                }
        }
#pragma unroll
        for (int r = 0; r < NS; ++r)
#pragma unroll
            for (int q = 0; q < NS; q += 4)
                *reinterpret_cast<float4*>(sS + (x0 + r) * D + cc + q * TS) =
                    make_float4(acc[r][q], acc[r][q + 1], acc[r][q + 2], acc[r][q + 3]);
    }
    __syncthreads();
    if (!OUT) {
        float* dst = p.rec + ((size_t)bh * (p.nseg + 1) + w + 1) * R;
        for (int e = tid; e < (int)R; e += kWalkThreads) dst[e] = sS[e / p.dc * D + e % p.dc];
    } else if (p.s_out && p.nseg == 1) {
        for (int e = tid; e < (int)R; e += kWalkThreads) {
            const int r = e / p.dc, c = e % p.dc;
            p.s_out[(size_t)bh * R + r * p.out_r + c * p.out_c] = sS[r * D + c];
        }
    }
}

// The states that enter the segments, in place: slot 0 is the state before the
// first, slot w + 1 becomes g^(tokens of w) slot w + (its own sum); `segments`
// have one.  A thread
// for each element (or four: N); the loads do not wait for the sums.
template <int N>
__global__ void __launch_bounds__(256) lin_scan_kernel(const LinWalk p, int chunk, int segments) {
    const int R = p.da * p.dc, e = (blockIdx.x * 256 + threadIdx.x) * N, bh = blockIdx.y;
    __shared__ float f[256];
    const int len = length_of(p, bh / p.H);
    const float g = __ldg(p.gamma + bh % p.H);
    float* const rec = p.rec + (size_t)bh * (p.nseg + 1) * R + e;
    Lane<float, 4, N == 4> acc;
    auto first = [&](int j) { return p.s_in ? p.s_in[(size_t)bh * R + ((e + j) / p.dc) * p.in_r + ((e + j) % p.dc) * p.in_c] : 0.f; };
    auto powers = [&](int base) {
        const int w = base + threadIdx.x;
        if (w < segments) {
            const int seg = p.rev ? p.nseg - 1 - w : w;
            const long long t0 = (long long)seg * p.seglen * chunk, t1 = t0 + (long long)p.seglen * chunk;
            f[threadIdx.x] = power(g, (int)max(0LL, min(t1, (long long)len) - t0));
        }
    };
    powers(0);
    follow();
    if (e < R) {
#pragma unroll
        for (int j = 0; j < N; ++j) acc.v[j] = first(j);
        acc.store(rec, N);
    }
    for (int base = 0; base < segments; base += 256) {
        if (base) powers(base);
        __syncthreads();
        const int m = min(256, segments - base);
        if (e < R) {
            for (int i0 = 0; i0 < m; i0 += 8) {  // eight loads on their way at a time
                float* const slot = rec + (size_t)(base + i0 + 1) * R;
                Lane<float, 4, N == 4> own[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i0 + i < m) own[i].load(slot + (size_t)i * R, N);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i0 + i < m) {
#pragma unroll
                        for (int j = 0; j < N; ++j) acc.v[j] = fmaf(f[i0 + i], acc.v[j], own[i].v[j]);
                        acc.store(slot + (size_t)i * R, N);
                    }
            }
        }
        __syncthreads();
    }
    if (e < R && p.s_out) {
#pragma unroll
        for (int j = 0; j < N; ++j)
            p.s_out[(size_t)bh * R + ((e + j) / p.dc) * p.out_r + ((e + j) % p.dc) * p.out_c] = acc.v[j];
    }
}

// Zeros in the rows behind each sequence's end (the gradients there).
template <typename T>
__global__ void __launch_bounds__(256) lin_tail_kernel(const LinWalk p) {
    const int b = blockIdx.z, h = blockIdx.y, len = length_of(p, b);
    T* const o = static_cast<T*>(p.o) + b * p.so[0] + h * p.so[1];
    const long long n = (long long)(p.T - len) * p.dc;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256)
        o[(len + i / p.dc) * p.so[2] + i % p.dc] = from_f32<T>(0.f);
}

// One token.  The state crosses HBM once each way and is all the work: a block
// takes `cols` columns (four to a thread) of one head's state, its rows over the
// rest of the block, and sums q over the rows in shared memory.  Few heads are cut
// into up to eight blocks each.  4096 heads of 128 x 128 (545 MB): 84 us, 0.96 of
// the copy bandwidth; 16 heads: a launch.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) lin_step_kernel(const float* state, const T* q, const T* k, const T* v,
                                                       const float* gamma, T* o, float* state_out, int H, int d,
                                                       int dv, int cols, int slices, long long ldq, long long ldk, long long ldv,
                                                       long long ldo) {
    constexpr int N = VEC ? 4 : 1;
    __shared__ float sq[128], sk[128];
    __shared__ float part[256 * N];
    const int head = blockIdx.x / slices, tid = threadIdx.x;
    const int per = (cols + N - 1) / N;  // threads to a row
    const int lines = 256 / per, line = tid / per, c = blockIdx.x % slices * cols + tid % per * N;
    if (tid < d) {
        sq[tid] = to_f32(q[head * ldq + tid]);
        sk[tid] = to_f32(k[head * ldk + tid]);
    }
    const bool live = line < lines && c < dv;
    float vv[N], acc[N] = {};
#pragma unroll
    for (int j = 0; j < N; ++j) vv[j] = live ? to_f32(v[head * ldv + c + j]) : 0.f;
    const float g = __ldg(gamma + head % H);
    __syncthreads();
    if (live) {
        const float* s = state + (size_t)head * d * dv + c;
        float* so = state_out + (size_t)head * d * dv + c;
        constexpr int U = 8;
        for (int r0 = line; r0 < d; r0 += lines * U) {
            Lane<float, 4, true> x4[U];
            float x1[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = r0 + u * lines;
                if (r < d) {
                    if constexpr (VEC) x4[u].load(s + (size_t)r * dv, 4);
                    else x1[u] = s[(size_t)r * dv];
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = r0 + u * lines;
                if (r < d) {
                    float y[N];
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        y[j] = fmaf(g, VEC ? x4[u].get(j) : x1[u], sk[r] * vv[j]);
                        acc[j] = fmaf(sq[r], y[j], acc[j]);
                    }
                    if constexpr (VEC) *reinterpret_cast<float4*>(so + (size_t)r * dv) = make_float4(y[0], y[1], y[2], y[3]);
                    else so[(size_t)r * dv] = y[0];
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < N; ++j) part[tid * N + j] = acc[j];
    __syncthreads();
    if (line == 0 && live) {
        for (int l = 1; l < lines; ++l)
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] += part[(l * per + tid) * N + j];
#pragma unroll
        for (int j = 0; j < N; ++j) o[head * ldo + c + j] = from_f32<T>(acc[j]);
    }
}

// ------------------------------------------------------------------ host ----
// Segments per head, each a CTA.  The count with the least time, in units of a
// chunk of the output walk: rounds of CTAs, each its chunks and about one to
// start; the states' walk, the scan and two more launches where there are several
// segments.  Measured: a chunk takes 2.8 us on the tensor cores (1.25 times that where
// CTAs are more than SMs: two share one up to width 64; above it the factor is a price
// on further rounds that was not measured by itself), the states' walk 0.6 of the output walk, the scan and the
// launches 17 us (alone; the overlap of a call's kernels gives some back); the CUDA
// cores take some 20 us for a chunk and 0.45 for its states.
struct SegmentCost {
    int ctas;  // to an SM
    double shared, states, extra;
};
SegmentCost segment_cost(bool tc, int d, int dv) {
    return tc ? SegmentCost{lin_tc_ctas(d, dv), 1.25, 0.6, 6.0} : SegmentCost{1, 1.0, 0.45, 0.5};
}
void plan_segments(int BH, int T, int chunk, const SegmentCost& c, int* nseg, int* seglen, int* nchunk) {
    const int n = T / chunk + (T % chunk != 0), sms = sm_count();
    double best = 0;
    *nchunk = n; *nseg = 1; *seglen = n;
    for (int want = 1; want <= n && want <= 1024; ++want) {
        const int len = (n + want - 1) / want, segs = (n + len - 1) / len;
        if (segs != want) continue;
        const long long blocks = (long long)BH * segs, slots = (long long)sms * c.ctas;
        double cost = (double)((blocks + slots - 1) / slots) * (len + 1) * (blocks > sms ? c.shared : 1.0);
        if (segs > 1) cost = cost * (1.0 + c.states) + c.extra + 0.05 * segs;
        if (want == 1 || cost < best) {
            best = cost;
            *nseg = segs;
            *seglen = len;
        }
        if (blocks > 4 * slots) break;
    }
}

template <typename T, int D>
cudaError_t launch_simple(const LinWalk& w, bool states, cudaStream_t s) {
    auto kernel = states ? lin_walk_kernel<T, D, false> : lin_walk_kernel<T, D, true>;
    const int bytes = SimpleLayout<D>::kBytes;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    return launch_following(kernel, dim3(states ? lin_state_segments(w) : w.nseg, w.B * w.H), kWalkThreads, bytes, s,
                            w.after, w);
}

// The path and the segments of a walk.
bool plan_walk(LinWalk& w, int dtype) {
    const bool tc = lin_tc_supported(w, dtype);
    plan_segments(w.B * w.H, w.T, tc ? kLinTcChunk : kTokens, segment_cost(tc, w.da, w.dc), &w.nseg, &w.seglen, &w.nchunk);
    w.rec_r = w.dc;
    w.rec_c = 1;
    const int es = dtype_size(dtype);
    auto four = [&](const void* ptr, const long long (&st)[3], int n) { return n % 4 == 0 && aligned_to(ptr, es, st, 3, 4 * es); };
    w.fours = (four(w.a, w.sa, w.da) ? 1 : 0) | (four(w.b, w.sb, w.da) ? 2 : 0) | (four(w.c, w.sc, w.dc) ? 4 : 0);
    return tc;
}
cudaError_t launch_walk(const LinWalk& w, int dtype, bool tc, bool states, cudaStream_t s) {
    if (tc) return launch_lin_tc(w, states, s);
    const bool small = w.da <= 64 && w.dc <= 64;
    if (dtype == HLA2_DTYPE_BF16) return small ? launch_simple<bf16, 64>(w, states, s) : launch_simple<bf16, 128>(w, states, s);
    return small ? launch_simple<float, 64>(w, states, s) : launch_simple<float, 128>(w, states, s);
}
// The states that enter the segments, where there are several (and the last state).
cudaError_t enter_states(const LinWalk& w, int dtype, bool tc, cudaStream_t s) {
    if (w.nseg == 1) return cudaSuccess;
    if (cudaError_t e = launch_walk(w, dtype, tc, true, s)) return e;
    const int R = w.da * w.dc, per = R % 4 ? 256 : 1024;
    auto scan = R % 4 ? lin_scan_kernel<1> : lin_scan_kernel<4>;
    return launch_following(scan, dim3((R + per - 1) / per, w.B * w.H), 256, 0, s, true, w, tc ? kLinTcChunk : kTokens,
                            lin_state_segments(w));
}
cudaError_t run_walk(LinWalk w, int dtype, cudaStream_t s) {
    const bool tc = plan_walk(w, dtype);
    if (cudaError_t e = enter_states(w, dtype, tc, s)) return e;
    w.after |= w.nseg > 1;
    return launch_walk(w, dtype, tc, false, s);
}

int check_linear(const char* what, int B, int H, int T, int d, int dv, int dtype) {
    if (B <= 0 || H <= 0 || T <= 0 || d <= 0 || dv <= 0)
        return set_error(HLA2_ERR_INVALID, "%s: sizes must be positive (B=%d H=%d T=%d d=%d dv=%d)", what, B, H, T, d, dv);
    if (d > 128 || dv > 128) return set_error(HLA2_ERR_UNSUPPORTED, "%s: d=%d or dv=%d exceeds 128", what, d, dv);
    if ((long long)B * H > 65535) return set_error(HLA2_ERR_UNSUPPORTED, "%s: B*H=%lld exceeds 65535", what, (long long)B * H);
    if (!known_dtype(dtype)) return set_error(HLA2_ERR_UNSUPPORTED, "%s: unknown dtype %d", what, dtype);
    return HLA2_OK;
}

// Two state tensors are one or apart.
int check_apart(const char* what, const float* in, const float* out, size_t n) {
    if (!in || !out || in == out) return HLA2_OK;
    const uintptr_t a = reinterpret_cast<uintptr_t>(in), b = reinterpret_cast<uintptr_t>(out), bytes = n * 4;
    if (a < b + bytes && b < a + bytes) return set_error(HLA2_ERR_INVALID, "%s: states overlap without being one tensor", what);
    return HLA2_OK;
}

void take(long long (&s)[3], const long long* strides, int i, int H, int T, int d) {
    if (strides) {
        for (int k = 0; k < 3; ++k) s[k] = strides[3 * i + k];
    } else {
        s[0] = (long long)H * T * d; s[1] = (long long)T * d; s[2] = d;
    }
}

size_t walk_bytes(int B, int H, int T, int d, int dv) {
    size_t most = 0;
    for (int chunk : {kLinTcChunk, kTokens}) {
        int nseg, seglen, nchunk;
        plan_segments(B * H, T, chunk, segment_cost(chunk == kLinTcChunk, d, dv), &nseg, &seglen, &nchunk);
        if (nseg > 1) most = max(most, (size_t)B * H * (nseg + 1) * d * dv * 4);
    }
    return (most + 255) & ~size_t(255);
}

int check_workspace(const char* what, size_t need, const void* workspace, size_t ws_bytes) {
    if (need && (!workspace || ws_bytes < need))
        return set_error(HLA2_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", what, ws_bytes, need);
    if (need && reinterpret_cast<uintptr_t>(workspace) % 16)
        return set_error(HLA2_ERR_INVALID, "%s: workspace not 16-byte aligned", what);
    return HLA2_OK;
}

}  // namespace
}  // namespace hla2

extern "C" size_t hla2_linear_workspace(int B, int H, int T, int d, int dv) {
    using namespace hla2;
    if (B <= 0 || H <= 0 || T <= 0 || d <= 0 || dv <= 0 || d > 128 || dv > 128 || (long long)B * H > 65535) return 0;
    return walk_bytes(B, H, T, d, dv);
}

extern "C" int hla2_linear_forward(const void* Q, const void* K, const void* V, const float* gamma, const int* lengths,
                                   const float* state_in, void* O, float* state_out, int B, int H, int T, int d,
                                   int dv, const long long* strides, int dtype, void* workspace, size_t ws_bytes,
                                   hla2_stream_t stream) {
    using namespace hla2;
    const char* what = "linear_forward";
    if (int rc = check_linear(what, B, H, T, d, dv, dtype)) return rc;
    if (!Q || !K || !V || !gamma || !O) return set_error(HLA2_ERR_INVALID, "%s: null pointer", what);
    const int es = dtype_size(dtype);
    for (const void* p : {Q, K, V, static_cast<const void*>(O)})
        if (!aligned_elem(p, es)) return set_error(HLA2_ERR_INVALID, "%s: pointer not aligned to its element", what);
    for (const void* p : {static_cast<const void*>(gamma), static_cast<const void*>(lengths),
                          static_cast<const void*>(state_in), static_cast<const void*>(state_out)})
        if (!aligned_elem(p, 4)) return set_error(HLA2_ERR_INVALID, "%s: pointer not aligned to its element", what);
    if (O == Q || O == K || O == V) return set_error(HLA2_ERR_INVALID, "%s: the output must not be an input", what);
    if (int rc = check_apart(what, state_in, state_out, (size_t)B * H * d * dv)) return rc;
    if (int rc = check_workspace(what, hla2_linear_workspace(B, H, T, d, dv), workspace, ws_bytes)) return rc;
    LinWalk w{};
    w.a = Q; w.b = K; w.c = V; w.o = O;
    take(w.sa, strides, 0, H, T, d);
    take(w.sb, strides, 1, H, T, d);
    take(w.sc, strides, 2, H, T, dv);
    take(w.so, strides, 3, H, T, dv);
    w.B = B; w.H = H; w.T = T; w.da = d; w.dc = dv;
    w.gamma = gamma; w.lengths = lengths;
    w.s_in = state_in; w.s_out = state_out;
    w.in_r = w.out_r = dv; w.in_c = w.out_c = 1;
    w.rec = static_cast<float*>(workspace);
    w.status = device_status_word();
    if (!w.status) return set_error(HLA2_ERR_LAUNCH, "%s: cannot resolve the device status word", what);
    const cudaError_t e = run_walk(w, dtype, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return set_error(HLA2_ERR_LAUNCH, "%s: %s", what, cudaGetErrorString(e));
    return HLA2_OK;
}

extern "C" int hla2_linear_backward(const void* Q, const void* K, const void* V, const float* gamma,
                                    const int* lengths, const float* state_in, const void* dO,
                                    const float* dstate_out, void* dQ, void* dK, void* dV, float* dstate_in, int B,
                                    int H, int T, int d, int dv, const long long* strides, int dtype, void* workspace,
                                    size_t ws_bytes, hla2_stream_t stream) {
    using namespace hla2;
    const char* what = "linear_backward";
    if (int rc = check_linear(what, B, H, T, d, dv, dtype)) return rc;
    if (!Q || !K || !V || !gamma || !dO || !dQ || !dK || !dV) return set_error(HLA2_ERR_INVALID, "%s: null pointer", what);
    const int es = dtype_size(dtype);
    for (const void* p : {Q, K, V, dO, static_cast<const void*>(dQ), static_cast<const void*>(dK), static_cast<const void*>(dV)})
        if (!aligned_elem(p, es)) return set_error(HLA2_ERR_INVALID, "%s: pointer not aligned to its element", what);
    for (const void* p : {static_cast<const void*>(gamma), static_cast<const void*>(lengths), static_cast<const void*>(state_in),
                          static_cast<const void*>(dstate_out), static_cast<const void*>(dstate_in)})
        if (!aligned_elem(p, 4)) return set_error(HLA2_ERR_INVALID, "%s: pointer not aligned to its element", what);
    for (const void* out : {static_cast<const void*>(dQ), static_cast<const void*>(dK), static_cast<const void*>(dV)})
        for (const void* in : {Q, K, V, dO})
            if (out == in) return set_error(HLA2_ERR_INVALID, "%s: an output must not be an input", what);
    if (dQ == dK || dQ == dV || dK == dV) return set_error(HLA2_ERR_INVALID, "%s: two outputs are one tensor", what);
    if (int rc = check_apart(what, dstate_out, dstate_in, (size_t)B * H * d * dv)) return rc;
    if (int rc = check_apart(what, state_in, dstate_in, (size_t)B * H * d * dv)) return rc;
    if (int rc = check_workspace(what, hla2_linear_workspace(B, H, T, d, dv), workspace, ws_bytes)) return rc;
    LinWalk base{};
    base.B = B; base.H = H; base.T = T;
    base.gamma = gamma; base.lengths = lengths;
    base.rec = static_cast<float*>(workspace);
    base.status = device_status_word();
    if (!base.status) return set_error(HLA2_ERR_LAUNCH, "%s: cannot resolve the device status word", what);
    struct Role { const void* p; int i, n; };
    const Role q{Q, 0, d}, k{K, 1, d}, v{V, 2, dv}, g{dO, 3, dv};
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    auto walk = [&](const Role& a, const Role& b, const Role& c, void* o, int oi, bool rev, const float* s_in,
                    bool transposed, float* s_out) {
        LinWalk w = base;
        w.a = a.p; w.b = b.p; w.c = c.p; w.o = o;
        take(w.sa, strides, a.i, H, T, a.n);
        take(w.sb, strides, b.i, H, T, b.n);
        take(w.sc, strides, c.i, H, T, c.n);
        take(w.so, strides, oi, H, T, c.n);
        w.da = a.n; w.dc = c.n; w.rev = rev;
        w.s_in = s_in; w.s_out = s_out;
        w.in_r = transposed ? 1 : dv; w.in_c = transposed ? dv : 1;
        w.out_r = dv; w.out_c = 1;
        return w;
    };
    LinWalk wq = walk(g, v, k, dQ, 4, false, state_in, true, nullptr);
    LinWalk wk = walk(v, g, q, dK, 5, true, dstate_out, true, nullptr);
    LinWalk wv = walk(k, q, g, dV, 6, true, dstate_out, false, dstate_in);
    // dQ first, and dV, which writes dstate_in, after whatever reads dstate_out: dstate_in may be either state
    cudaError_t e = run_walk(wq, dtype, s);
    wk.after = wv.after = 1;
    const bool tk = plan_walk(wk, dtype), tv = plan_walk(wv, dtype);
    if (e == cudaSuccess && tk == tv && wv.nseg > 1) {
        // the states of dK are those of dV, transposed
        e = enter_states(wv, dtype, tv, s);
        wk.rec_r = 1;
        wk.rec_c = dv;
        if (e == cudaSuccess) e = launch_walk(wk, dtype, tk, false, s);
        if (e == cudaSuccess) e = launch_walk(wv, dtype, tv, false, s);
    } else {
        if (e == cudaSuccess) e = run_walk(wk, dtype, s);
        if (e == cudaSuccess) e = run_walk(wv, dtype, s);
    }
    if (e == cudaSuccess && lengths)
        for (const LinWalk& w : {wq, wk, wv}) {
            if (dtype == HLA2_DTYPE_BF16) lin_tail_kernel<bf16><<<dim3(8, H, B), 256, 0, s>>>(w);
            else lin_tail_kernel<float><<<dim3(8, H, B), 256, 0, s>>>(w);
            note_launches(1);
            if ((e = cudaGetLastError()) != cudaSuccess) break;
        }
    if (e != cudaSuccess) return set_error(HLA2_ERR_LAUNCH, "%s: %s", what, cudaGetErrorString(e));
    return HLA2_OK;
}

extern "C" int hla2_linear_step(float* state, const void* q, const void* k, const void* v, const float* gamma, void* o,
                                float* state_out, int n, int H, int d, int dv, const long long* ld, int dtype,
                                hla2_stream_t stream) {
    using namespace hla2;
    const char* what = "linear_step";
    if (n <= 0 || H <= 0 || d <= 0 || dv <= 0 || n % H)
        return set_error(HLA2_ERR_INVALID, "%s: sizes must be positive and n a multiple of H (n=%d H=%d d=%d dv=%d)", what, n, H, d, dv);
    if (d > 128 || dv > 128) return set_error(HLA2_ERR_UNSUPPORTED, "%s: d=%d or dv=%d exceeds 128", what, d, dv);
    if (!known_dtype(dtype)) return set_error(HLA2_ERR_UNSUPPORTED, "%s: unknown dtype %d", what, dtype);
    if (!state || !q || !k || !v || !gamma || !o) return set_error(HLA2_ERR_INVALID, "%s: null pointer", what);
    const int es = dtype_size(dtype);
    if (!aligned_elem(state, 4) || !aligned_elem(state_out, 4) || !aligned_elem(gamma, 4) || !aligned_elem(q, es) ||
        !aligned_elem(k, es) || !aligned_elem(v, es) || !aligned_elem(o, es))
        return set_error(HLA2_ERR_INVALID, "%s: pointer not aligned to its element", what);
    if (int rc = check_apart(what, state, state_out, (size_t)n * d * dv)) return rc;
    if (!state_out) state_out = state;
    const long long ldq = ld ? ld[0] : d, ldk = ld ? ld[1] : d, ldv = ld ? ld[2] : dv, ldo = ld ? ld[3] : dv;
    // Few heads are cut into blocks that each read all of q and k and write their own columns: an output among the
    // inputs would be read by one block before and by another after its writing.  v's columns are read by the
    // block that writes them in o.
    const Rows rq{q, n, ldq * es, (long long)d * es}, rk{k, n, ldk * es, (long long)d * es},
        rv{v, n, ldv * es, (long long)dv * es}, ro{o, n, ldo * es, (long long)dv * es};
    const long long all = (long long)n * d * dv * 4;
    const Rows before{state, 1, all, all}, behind{state_out, 1, all, all};
    if (rows_meet(ro, rq) || rows_meet(ro, rk) || (!(o == v && ldo == ldv) && rows_meet(ro, rv)))
        return set_error(HLA2_ERR_INVALID, "%s: the output overlaps an input", what);
    if (rows_meet(ro, before) || rows_meet(ro, behind) || rows_meet(rq, behind) || rows_meet(rk, behind) ||
        rows_meet(rv, behind))
        return set_error(HLA2_ERR_INVALID, "%s: a state overlaps the output or an input", what);
    const bool vec = dv % 4 == 0 && aligned_to(state, 4, nullptr, 0, 16) && aligned_to(state_out, 4, nullptr, 0, 16);
    int cols = dv;
    while (cols > 16 && (long long)n * ((dv + cols - 1) / cols) < 2LL * sm_count()) cols = (cols + 1) / 2;
    if (vec) cols = (cols + 3) / 4 * 4;
    const int slices = (dv + cols - 1) / cols;  // (several only of few heads)
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    auto go = [&](auto t) {
        using T = decltype(t);
        auto kernel = vec ? lin_step_kernel<T, true> : lin_step_kernel<T, false>;
        kernel<<<(unsigned)n * slices, 256, 0, s>>>(state, static_cast<const T*>(q), static_cast<const T*>(k),
                                    static_cast<const T*>(v), gamma, static_cast<T*>(o), state_out, H, d, dv, cols,
                                    slices, ldq, ldk, ldv, ldo);
    };
    if (dtype == HLA2_DTYPE_BF16) go(bf16{});
    else go(float{});
    note_launches(1);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return set_error(HLA2_ERR_LAUNCH, "%s: %s", what, cudaGetErrorString(e));
    return HLA2_OK;
}
