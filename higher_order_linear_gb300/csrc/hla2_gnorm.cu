// hla2_gnorm.cu -- group norm, channels last, with an activation or a gate, and
// its gradient.
//
//   x [N][L][C], G groups of cg = C / G channels; mean and variance over a
//   sample's L positions and a group's channels:
//   n = (x - mean) / sqrt(var + eps),  z = n w + b,
//   y = act(z), or z act(gate);  act: identity or silu.
// Gradient, with dz = dy act'(z) (or dy act(gate)) and t = dz w:
//   dx = rstd (t - mean(t) - n mean(t n)),  dw = sum dz n,  db = sum dz,
//   dgate = dy z act'(gate).
//
// Two forms.  A unit (a sample's group, L cg values) of up to 2048 values stays
// in the registers of up to 256 threads, eight values each: x crosses HBM once, the
// variance is taken about the mean.  Larger units are summed by channel over
// runs of positions (moments of a few positions at a time about one of them, joined, so that
// neither a large mean nor an untypical value costs the others' digits), folded in a second launch
// and read again by a third.
//
// Measured, 16 bits: gated silu, 16384 rows of 2048 in 16 groups (203 MB), 41 us, 0.74
// of the copy bandwidth, instructions (an element takes a power of two, a
// reciprocal and some 25 more; the SMs issue in 76 % of their clocks) and HBM together; its gradient
// on 1024 channels (170 MB) 41 us with the lines of dw and db.  8 maps of 4096 x 512 with silu (67
// MB: 10 us at the copy bandwidth): 33 us for moments, fold and the second pass, 61 us for the gradient.
#include <type_traits>

#include "hla2_layer.cuh"

namespace hla2 {
namespace {

constexpr int kThreads = 256;
constexpr int kUnit = kThreads * 8;  // the most values of a unit in registers
constexpr int kMaxChannels = 16384;
constexpr int kFwdBlocks = 4, kBwdBlocks = 2;  // blocks of units in registers that an SM holds
constexpr int kRunBlocks = 3;                  // and of runs of large units

struct View {
    const void* p;
    long long sn, sl;  // strides of samples and positions
};

struct GNormParams {
    View x, z, dy;  // input, gate (p null: none), gradient of the output
    void *y, *dz;   // output (dx in the gradient), gradient of the gate
    long long yn, yl, dzn, dzl;
    const void *w, *b;  // [C], wdtype, or null
    float* stats;       // [N][G][2]: mean and reciprocal deviation
    float* part;        // gradient and large units: partial sums
    float* dw;          // [2][C] in the gradient: dw, then db
    long long N;
    int L, C, G, cg, wdtype;
    bool silu;
    float eps;
    // units in registers: threads to a unit, units of one sample to a block, samples to a block
    int tpr, gpb, spb;
    // large units: runs of `run` positions, `runs` of them
    int run, runs;
};

// 1 / (1 + 2^(-x log2 e)): one power of two and one reciprocal, good to (1.5 |x| + 10) 2^-24 of itself, and zero below
// -87.3, where it is less than the smallest normal number (x times it less than 1.1e-36)
__device__ __forceinline__ float sigmoid(float x) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}
// the activation and its slope
template <bool SILU>
__device__ __forceinline__ float act(float x) { return SILU ? x * sigmoid(x) : x; }
template <bool SILU>
__device__ __forceinline__ void act_slope(float x, float& v, float& s) {
    if (SILU) {
        const float g = sigmoid(x);
        v = x * g;
        s = fmaf(v, 1.f - g, g);
    } else {
        v = x;
        s = 1.f;
    }
}
__device__ __forceinline__ float weight_at(const void* w, int wdtype, int c, float none) {
    if (!w) return none;
    return wdtype == HLA2_DTYPE_F32 ? __ldg(static_cast<const float*>(w) + c)
                                    : __bfloat162float(static_cast<const bf16*>(w)[c]);
}
// eight channels in a row, from a 16-byte step on
__device__ __forceinline__ void weights8(const void* w, int wdtype, int c, float none, float (&v)[8]) {
    if (!w) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = none;
    } else if (wdtype == HLA2_DTYPE_F32) {
        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(w) + c);
        const float4 a = __ldg(q), b = __ldg(q + 1);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(static_cast<const bf16*>(w) + c));
        const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(u[j] << 16);
            v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
        }
    }
}

// Where the eight values of a thread are: VEC, eight channels in a row of one
// position; else every tpr-th value of the unit.
template <bool VEC>
struct Spots {
    int pos[VEC ? 1 : 8], ch[VEC ? 1 : 8], n;
    __device__ __forceinline__ Spots(int lane, int tpr, int values, int cg) {
        n = 0;
        if (VEC) {
            const int e = lane * 8;
            pos[0] = e / cg;
            ch[0] = e - pos[0] * cg;
            n = e < values ? 8 : 0;
        } else {
#pragma unroll
            for (int j = 0; j < (VEC ? 1 : 8); ++j) {
                const int e = lane + j * tpr;
                pos[j] = e / cg;
                ch[j] = e - pos[j] * cg;
                n += e < values;
            }
        }
    }
    __device__ __forceinline__ int channel(int j) const { return VEC ? ch[0] + j : ch[VEC ? 0 : j]; }
    __device__ __forceinline__ void weights(const void* w, int wdtype, int c0, float none, float (&v)[8]) const {
        if constexpr (VEC) {
            if (n) weights8(w, wdtype, c0 + ch[0], none, v);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = j < n ? weight_at(w, wdtype, c0 + ch[j], none) : 0.f;
        }
    }
    // eight values as they lie in memory
    template <typename T>
    struct Raw {
        Lane<T, 8, VEC> l;
        __device__ __forceinline__ float get(int j) const { return l.get(j); }
    };
    template <typename T>
    __device__ __forceinline__ void load(const T* p, long long sl, Raw<T>& r) const {
        if constexpr (VEC) {
            if (n) r.l.load(p + pos[0] * sl + ch[0], 8);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n) r.l.v[j] = p[pos[j] * sl + ch[j]];
        }
    }
    template <typename T>
    __device__ __forceinline__ void store(T* p, long long sl, const float (&v)[8]) const {
        if constexpr (VEC) {
            Lane<T, 8, true> l;
            l.set(v);
            if (n) l.store(p + pos[0] * sl + ch[0], 8);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n) p[pos[j] * sl + ch[j]] = from_f32<T>(v[j]);
        }
    }
};

// Sums over a unit's threads (B: two of them); sh: two rows of kThreads / 32, used alternately.
template <bool B>
__device__ __forceinline__ void unit_sum(float& a, float& b, int tpr, float2* sh) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o < tpr) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            if (B) b += __shfl_xor_sync(0xffffffffu, b, o);
        }
    if (tpr > 32) {
        const int warp = threadIdx.x >> 5, nw = tpr >> 5, w0 = warp / nw * nw;
        if ((threadIdx.x & 31) == 0) sh[warp] = make_float2(a, b);
        __syncthreads();
        a = b = 0.f;
        for (int i = 0; i < nw; ++i) {
            a += sh[w0 + i].x;
            if (B) b += sh[w0 + i].y;
        }
    }
}

// A running sum with its rounding errors kept (64-bit sums would take 60 times as long here)
struct LongSum {
    float hi = 0.f, lo = 0.f;
    __device__ __forceinline__ void add(float x) {
        const float s = hi + x, t = s - hi;
        lo += (hi - (s - t)) + (x - t);
        hi = s;
    }
    __device__ __forceinline__ float value() const { return hi + lo; }
};
// Long sums are taken in pieces of this many terms, and the pieces so: a thousand equal terms added one after another
// are off by 160 roundings, all to one side.
constexpr int kPiece = 16;

// --------------------------------------------- units in registers ----
// A block keeps its groups and takes every gridDim.x-th run of samples: its
// weights stay in registers, and the next samples' values are on their way.
template <typename T, bool VEC, bool GATE, bool SILU>
__global__ void __launch_bounds__(kThreads, VEC ? kFwdBlocks : 2) gnorm_unit_kernel(const GNormParams p) {
    __shared__ float2 sh[2][kThreads / 32];
    const int unit = threadIdx.x / p.tpr, lane = threadIdx.x % p.tpr;
    const int s = unit / p.gpb, g = blockIdx.y * p.gpb + unit % p.gpb;
    const int values = p.L * p.cg, c0 = g * p.cg;
    const Spots<VEC> at(lane, p.tpr, s < p.spb && g < p.G ? values : 0, p.cg);
    const bool mine = at.n > 0;
    const float inv = 1.f / (float)values;
    const bool even = (values & (values - 1)) == 0;  // the reciprocal is exact
    typename Spots<VEC>::template Raw<T> xr{}, zr{};  // (two samples ahead, with three blocks to an SM: 43 us instead of 41)
    auto fetch = [&](long long n) {
        if (n >= p.N) return;
        at.load(static_cast<const T*>(p.x.p) + n * p.x.sn + c0, p.x.sl, xr);
        if (GATE) at.load(static_cast<const T*>(p.z.p) + n * p.z.sn + c0, p.z.sl, zr);
    };
    long long n = (long long)blockIdx.x * p.spb + s;
    const long long step = (long long)gridDim.x * p.spb;
    fetch(n);
    float w[8], b[8];
    at.weights(p.w, p.wdtype, c0, 1.f, w);
    at.weights(p.b, p.wdtype, c0, 0.f, b);
    for (long long n0 = (long long)blockIdx.x * p.spb; n0 < p.N; n0 += step, n += step) {
        float x[8], z[8], sum = 0.f, sq = 0.f, rest = 0.f, none = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[j] = VEC || j < at.n ? xr.get(j) : 0.f;
            if (GATE) z[j] = VEC || j < at.n ? zr.get(j) : 0.f;
            sum += x[j];
        }
        fetch(n + step);
        if (!mine) sum = 0.f;
        unit_sum<false>(sum, none, p.tpr, sh[0]);
        // Equal values are their mean.  In 16 bits by themselves: 2048 of them add up exactly.  In 32 bits the
        // sum has been rounded, and the mean of what is left is taken off as well.
        constexpr bool TWICE = sizeof(T) == 4;
        float mean = even ? sum * inv : sum / (float)values;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[j] -= mean;
            if (VEC || j < at.n) {
                sq = fmaf(x[j], x[j], sq);
                if (TWICE) rest += x[j];
            }
        }
        if (!mine) sq = rest = 0.f;
        unit_sum<TWICE>(sq, rest, p.tpr, sh[1]);
        if (!mine || n >= p.N) continue;
        float var = sq * inv;
        if (TWICE) {
            rest *= inv;
            mean += rest;
            var = fmaf(-rest, rest, var);
            if (var < 0.f) var = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] -= rest;
        }
        const float rstd = rsqrtf(var + p.eps);
        if (p.stats && lane == 0) *reinterpret_cast<float2*>(p.stats + (n * p.G + g) * 2) = make_float2(mean, rstd);
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float v = fmaf(x[j] * rstd, w[j], b[j]);
            y[j] = GATE ? v * act<SILU>(z[j]) : act<SILU>(v);
        }
        at.store(static_cast<T*>(p.y) + n * p.yn + c0, p.yl, y);
    }
}

// The gradient.  A block keeps its groups and takes every gridDim.x-th run of
// samples, so that a thread's channels stay its own and dw and db add up in
// registers, a piece at a time; then the block's threads add theirs, one line of sums to a block.
template <typename T, bool VEC, bool GATE, bool SILU>
__global__ void __launch_bounds__(kThreads, VEC ? kBwdBlocks : 1) gnorm_unit_bwd_kernel(const GNormParams p) {
    __shared__ float2 sh[2][kThreads / 32];
    __shared__ float4 sofar[8][kThreads];  // dw and db of a thread's values, each as a LongSum
    follow();
    const int unit = threadIdx.x / p.tpr, lane = threadIdx.x % p.tpr;
    const int s = unit / p.gpb, g = blockIdx.y * p.gpb + unit % p.gpb;
    const int values = p.L * p.cg, c0 = g * p.cg;
    const Spots<VEC> at(lane, p.tpr, s < p.spb && g < p.G ? values : 0, p.cg);
    const bool mine = at.n > 0;
    const float inv = 1.f / (float)values;
    typename Spots<VEC>::template Raw<T> xr{}, yr{}, zr{};
    float2 sr = make_float2(0.f, 0.f);
    auto fetch = [&](long long n) {
        if (!mine || n >= p.N) return;
        at.load(static_cast<const T*>(p.x.p) + n * p.x.sn + c0, p.x.sl, xr);
        at.load(static_cast<const T*>(p.dy.p) + n * p.dy.sn + c0, p.dy.sl, yr);
        if (GATE) at.load(static_cast<const T*>(p.z.p) + n * p.z.sn + c0, p.z.sl, zr);
        sr = __ldg(reinterpret_cast<const float2*>(p.stats + (n * p.G + g) * 2));
    };
    const long long step = (long long)gridDim.x * p.spb;
    fetch((long long)blockIdx.x * p.spb + s);
    float w[8], b[8], dw[8] = {}, db[8] = {};
    at.weights(p.w, p.wdtype, c0, 1.f, w);
    at.weights(p.b, p.wdtype, c0, 0.f, b);
#pragma unroll
    for (int j = 0; j < 8; ++j) sofar[j][threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
    auto keep = [&]() {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float4 f = sofar[j][threadIdx.x];
            LongSum first{f.x, f.y}, second{f.z, f.w};
            first.add(dw[j]);
            second.add(db[j]);
            sofar[j][threadIdx.x] = make_float4(first.hi, first.lo, second.hi, second.lo);
            dw[j] = db[j] = 0.f;
        }
    };
    int turn = 0;
    for (long long n0 = (long long)blockIdx.x * p.spb; n0 < p.N; n0 += step, ++turn) {
        if (turn && turn % kPiece == 0) keep();
        const long long n = n0 + s;
        const bool live = mine && n < p.N;
        float x[8], dy[8], z[8], dgate[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const bool in = VEC || j < at.n;
            x[j] = in ? xr.get(j) : 0.f;
            dy[j] = in ? yr.get(j) : 0.f;
            if (GATE) z[j] = in ? zr.get(j) : 0.f;
        }
        const float2 st = sr;
        fetch(n + step);
        float m1 = 0.f, m2 = 0.f;
        if (live)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (!VEC && j >= at.n) break;
                x[j] = (x[j] - st.x) * st.y;
                const float v = fmaf(x[j], w[j], b[j]);
                float value, slope;
                act_slope<SILU>(GATE ? z[j] : v, value, slope);
                if (GATE) dgate[j] = dy[j] * v * slope;
                const float d = dy[j] * (GATE ? value : slope);
                db[j] += d;
                dw[j] = fmaf(d, x[j], dw[j]);
                dy[j] = d * w[j];
                m1 += dy[j];
                m2 = fmaf(dy[j], x[j], m2);
            }
        unit_sum<true>(m1, m2, p.tpr, sh[turn & 1]);
        if (!live) continue;
        m1 *= inv;
        m2 *= inv;
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = st.y * (dy[j] - m1 - x[j] * m2);
        at.store(static_cast<T*>(p.y) + n * p.yn + c0, p.yl, x);
        if (GATE) at.store(static_cast<T*>(p.dz) + n * p.dzn + c0, p.dzl, dgate);
    }
    keep();
    __syncthreads();
    float* const line = p.part + (long long)blockIdx.x * 2 * p.C;
    const int width = min(p.gpb, p.G - (int)blockIdx.y * p.gpb) * p.cg;
    for (int c = threadIdx.x; c < width; c += kThreads) {
        const int u = c / p.cg, ch = c - u * p.cg;
        LongSum first, second;
        for (int i = 0; i < p.spb; ++i)
            for (int l = 0; l < p.L; ++l) {
                const int e = l * p.cg + ch, t = (i * p.gpb + u) * p.tpr;
                const float4 f = VEC ? sofar[e % 8][t + e / 8] : sofar[e / p.tpr][t + e % p.tpr];
                first.add(f.x + f.y);
                second.add(f.z + f.w);
            }
        line[blockIdx.y * p.gpb * p.cg + c] = first.value();
        line[p.C + blockIdx.y * p.gpb * p.cg + c] = second.value();
    }
}

// ------------------------------------------------------ large units ----
// A block takes one run of positions of one sample and up to 2048 channels, a
// thread eight of them and every rows-th position.
struct RunSpot {
    long long n;
    int l0, l1, c, cols, rows, row, live;
};
__device__ __forceinline__ RunSpot run_spot(const GNormParams& p) {
    RunSpot r;
    r.cols = min((p.C + 7) / 8, kThreads);  // threads along the channels
    r.n = blockIdx.x / p.runs;
    r.l0 = (int)(blockIdx.x % p.runs) * p.run;
    r.l1 = r.l0 + min(p.run, p.L - r.l0);  // (sums of positions may pass 2^31 - 1 next to the largest L)
    r.rows = kThreads / r.cols;
    r.row = threadIdx.x / r.cols;
    r.c = (blockIdx.y * kThreads + threadIdx.x % r.cols) * 8;
    r.live = r.row < r.rows ? min(8, p.C - r.c) : 0;
    return r;
}
// Mean and sum of squares about it of each channel of a run.  A thread takes its positions in pieces of kPiece, each
// about its own first value, and joins them: with count n, mean and squares of what it has and m, mean + d, squares'
// of a piece,  mean + d m / (n + m),  squares + squares' + d^2 n m / (n + m).  So a value far from the others
// costs the digits of one piece, not of the run (a zero in front of 4096 values of 1000 +- 1 moved a variance by 2e-3
// where the run was summed about it, by 4e-6 now), and long runs are sums of few levels.  What a thread has so
// far waits in shared memory.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads, VEC ? kRunBlocks : 2) gnorm_moments_kernel(const GNormParams p) {
    __shared__ float4 sofar[8][kThreads];  // mean and squares, each as a LongSum
    follow();
    const RunSpot r = run_spot(p);
    constexpr int M = sizeof(T) == 4 ? 2 : 4;  // positions on their way to a thread
    const int len = r.l1 - r.l0;
#pragma unroll
    for (int j = 0; j < 8; ++j) sofar[j][threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r.live > 0) {
        const T* const x = static_cast<const T*>(p.x.p) + r.n * p.x.sn + r.l0 * p.x.sl + r.c;
        float done = 0.f;
#pragma unroll 1
        for (int l0 = r.row; l0 < len; l0 += kPiece * r.rows) {
            Lane<T, 8, VEC> pivot;
            float a[8] = {}, q[8] = {};
            const int m = min(kPiece, (len - l0 + r.rows - 1) / r.rows);
#pragma unroll 1
            for (int i0 = 0; i0 < m; i0 += M) {
                Lane<T, 8, VEC> v[M];
#pragma unroll
                for (int i = 0; i < M; ++i)
                    if (i0 + i < m) v[i].load(x + (l0 + (i0 + i) * r.rows) * p.x.sl, r.live);
                if (i0 == 0) pivot = v[0];
#pragma unroll
                for (int i = 0; i < M; ++i) {
                    if (i0 + i >= m) break;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float d = v[i].get(j) - pivot.get(j);
                        a[j] += d;
                        q[j] = fmaf(d, d, q[j]);
                    }
                }
            }
            const float inv = 1.f / (float)m, part = (float)m / (done + (float)m);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float4 f = sofar[j][threadIdx.x];
                LongSum mean{f.x, f.y}, squares{f.z, f.w};
                const float shift = a[j] * inv, d = (pivot.get(j) - mean.hi) + (shift - mean.lo);
                // (d is the value itself in the first piece: its square, which counts nothing there, is not formed)
                squares.add(fmaf(d * part, d * done, fmaxf(fmaf(-a[j], shift, q[j]), 0.f)));
                mean.add(d * part);
                sofar[j][threadIdx.x] = make_float4(mean.hi, mean.lo, squares.hi, squares.lo);
            }
            done += (float)m;
            asm volatile("" ::: "memory");  // (it is to wait there, not in registers)
        }
    }
    __syncthreads();
    // the block's rows, joined in order about the first one's mean: a channel to a thread
    float* const line = p.part + (long long)blockIdx.x * 2 * p.C;
    for (int e = threadIdx.x; e < r.cols * 8; e += kThreads) {
        const int col = e % r.cols, j = e / r.cols, c = blockIdx.y * kUnit + col * 8 + j;
        if (c >= p.C) continue;
        const float4* const own = sofar[j] + col;  // row i at i cols
        const int whole = len / r.rows, more = len % r.rows;
        const float first = own->x + own->y;
        LongSum moved, all;
#pragma unroll 4
        for (int i = 1; i < r.rows; ++i) {
            const float4 f = own[i * r.cols];
            moved.add((float)(whole + (i < more)) * ((f.x - first) + f.y));
        }
        const float middle = first + moved.value() / (float)len;
#pragma unroll 4
        for (int i = 0; i < r.rows; ++i) {
            const float4 f = own[i * r.cols];
            const float d = (f.x - middle) + f.y;
            all.add(fmaf((float)(whole + (i < more)) * d, d, f.z + f.w));
        }
        line[c] = middle;
        line[p.C + c] = all.value();
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, int n, float (&v)[8]) {
    Lane<T, 8, VEC> l;
    l.load(p, n);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = l.get(j);
}
// The gradient's sums of each channel of a run: dz n and dz, in pieces.  Three blocks to an SM where 80 registers hold it without
// spills, two elsewhere (gradient of 512 maps of 1024 x 256, silu without a gate: 336 us by two, 468 by three; of
// 8 x 4096 x 512 with a gate: 66 by three, 68 by two).
template <typename T, bool VEC, bool GATE, bool SILU>
__global__ void __launch_bounds__(kThreads, VEC && sizeof(T) == 2 && (GATE || !SILU) ? kRunBlocks : 2) gnorm_sums_kernel(const GNormParams p) {
    __shared__ float4 sofar[8][kThreads];  // two LongSums
    follow();
    const RunSpot r = run_spot(p);
    const int len = r.l1 - r.l0;
#pragma unroll
    for (int j = 0; j < 8; ++j) sofar[j][threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r.live > 0) {
        const T* const x = static_cast<const T*>(p.x.p) + r.n * p.x.sn + r.l0 * p.x.sl + r.c;
        const T* const g = static_cast<const T*>(p.dy.p) + r.n * p.dy.sn + r.l0 * p.dy.sl + r.c;
        const T* const gate = static_cast<const T*>(p.z.p) + r.n * p.z.sn + r.l0 * p.z.sl + r.c;
        float w[8], b[8], mean[8], rstd[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = min(r.c + j, p.C - 1);
            const float2 st = __ldg(reinterpret_cast<const float2*>(p.stats) + r.n * p.G + c / p.cg);
            mean[j] = st.x;
            rstd[j] = st.y;
            w[j] = weight_at(p.w, p.wdtype, c, 1.f);
            b[j] = weight_at(p.b, p.wdtype, c, 0.f);
        }
#pragma unroll 1
        for (int l0 = r.row; l0 < len; l0 += kPiece * r.rows) {
            float a[8] = {}, q[8] = {};
            const int end = min(len, l0 + kPiece * r.rows);
#pragma unroll 2
            for (int l = l0; l < end; l += r.rows) {
                float v[8], dy[8], z[8];
                load8<T, VEC>(x + l * p.x.sl, r.live, v);
                load8<T, VEC>(g + l * p.dy.sl, r.live, dy);
                if (GATE) load8<T, VEC>(gate + l * p.z.sl, r.live, z);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float n = (v[j] - mean[j]) * rstd[j];
                    float value, slope;
                    act_slope<SILU>(GATE ? z[j] : fmaf(n, w[j], b[j]), value, slope);
                    const float d = dy[j] * (GATE ? value : slope);
                    a[j] = fmaf(d, n, a[j]);
                    q[j] += d;
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float4 f = sofar[j][threadIdx.x];
                LongSum first{f.x, f.y}, second{f.z, f.w};
                first.add(a[j]);
                second.add(q[j]);
                sofar[j][threadIdx.x] = make_float4(first.hi, first.lo, second.hi, second.lo);
            }
            asm volatile("" ::: "memory");  // (they are to wait there, not in registers)
        }
    }
    __syncthreads();
    float* const line = p.part + (long long)blockIdx.x * 2 * p.C;
    for (int e = threadIdx.x; e < r.cols * 8; e += kThreads) {
        const int col = e % r.cols, j = e / r.cols, c = blockIdx.y * kUnit + col * 8 + j;
        if (c >= p.C) continue;
        LongSum first, second;
#pragma unroll 4
        for (int i = 0; i < r.rows; ++i) {
            const float4 f = sofar[j][col + i * r.cols];
            first.add(f.x + f.y);
            second.add(f.z + f.w);
        }
        line[c] = first.value();
        line[p.C + c] = second.value();
    }
}

__device__ __forceinline__ float block_sum(const LongSum& sum, float* sh) {
    float v = sum.value();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) v += sh[i];
    return v;
}

// dw and db: the lines of partial sums added in a fixed order, 16 columns to a
// block, each THREADS / 16 threads' sums of every (THREADS / 16)th line.
constexpr int kFoldColumns = 16, kFoldThreads = 1024;
template <int THREADS>
__device__ __forceinline__ void fold_lines(const float* part, float* out, long long lines,
                                           int width, int block, bool add, float (*sh)[kFoldColumns]) {
    const int col = threadIdx.x % kFoldColumns, line = threadIdx.x / kFoldColumns;
    const int c = block * kFoldColumns + col;
    LongSum sum;
    if (c < width) {
#pragma unroll 8
        for (long long g = line; g < lines; g += THREADS / kFoldColumns) sum.add(part[g * width + c]);
    }
    float a = sum.value();
    a += __shfl_down_sync(0xffffffffu, a, 16);
    if ((threadIdx.x & 31) < kFoldColumns) sh[threadIdx.x >> 5][col] = a;
    __syncthreads();
    if (threadIdx.x < kFoldColumns && c < width) {
        a = 0.f;
#pragma unroll
        for (int i = 0; i < THREADS / 32; ++i) a += sh[i][col];
        out[c] = add ? out[c] + a : a;
    }
}
__global__ void __launch_bounds__(kFoldThreads) gnorm_lines_kernel(const float* part, float* out,
                                                                   long long lines, int width) {
    __shared__ float sh[kFoldThreads / 32][kFoldColumns];
    follow();
    fold_lines<kFoldThreads>(part, out, lines, width, blockIdx.x, false, sh);
}

// A group's runs and channels folded: mean and reciprocal deviation, or (GRAD)
// the means of t and t n, which go behind the partial sums.  The blocks behind the
// groups' fold the gradient's lines (add: to those of the samples before).
template <bool GRAD>
__global__ void __launch_bounds__(kThreads) gnorm_fold_kernel(const GNormParams p, float* out, bool add) {
    __shared__ float sh[kThreads / 32];
    follow();
    if (GRAD && blockIdx.x >= p.N * p.G) {
        __shared__ float columns[kThreads / 32][kFoldColumns];
        fold_lines<kThreads>(p.part, p.dw, p.N * p.runs, 2 * p.C, (int)(blockIdx.x - p.N * p.G), add, columns);
        return;
    }
    const long long n = blockIdx.x / p.G;
    const int g = (int)(blockIdx.x % p.G), items = p.runs * p.cg;
    const float* const part = p.part + n * p.runs * 2 * p.C + g * p.cg;
    const float count = (float)p.L * (float)p.cg;
    const float about = GRAD ? 0.f : part[0];  // means are added about one of them: equal values are their mean
    LongSum first, second;
    for (int i = threadIdx.x; i < items; i += kThreads) {
        const int k = i / p.cg, c = i - k * p.cg;
        const float* v = part + (long long)k * 2 * p.C + c;
        if (GRAD) {
            const float w = weight_at(p.w, p.wdtype, g * p.cg + c, 1.f);
            first.add(w * v[p.C]);
            second.add(w * v[0]);
        } else {
            first.add((float)min(p.run, p.L - k * p.run) * (v[0] - about));
        }
    }
    const float a = about + block_sum(first, sh) / count;
    if (!GRAD)
        for (int i = threadIdx.x; i < items; i += kThreads) {
            const int k = i / p.cg, c = i - k * p.cg;
            const float* v = part + (long long)k * 2 * p.C + c;
            const float d = v[0] - a;
            second.add(fmaf((float)min(p.run, p.L - k * p.run) * d, d, v[p.C]));
        }
    const float q = block_sum(second, sh) / count;
    if (threadIdx.x == 0)
        *reinterpret_cast<float2*>(out + 2 * (long long)blockIdx.x) = make_float2(a, GRAD ? q : 1.f / sqrtf(q + p.eps));
}

// y, or (GRAD) dx and dgate; means: the gradient's, [N][G][2].  A few positions on
// their way to a thread at a time.
template <typename T, bool VEC, bool GRAD, bool GATE, bool SILU>
__global__ void __launch_bounds__(kThreads, VEC ? (GRAD ? 2 : kRunBlocks) : 1) gnorm_apply_kernel(const GNormParams p, const float* means) {
    const RunSpot r = run_spot(p);
    if (r.live <= 0) {
        follow();
        return;
    }
    constexpr int M = sizeof(T) == 4 || GRAD || GATE ? 2 : 4;
    float w[8], b[8], mean[8], rstd[8], m1[8], m2[8];
    if (VEC) {
        weights8(p.w, p.wdtype, r.c, 1.f, w);
        weights8(p.b, p.wdtype, r.c, 0.f, b);
    }
    follow();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int c = min(r.c + j, p.C - 1);
        const float2 st = *(reinterpret_cast<const float2*>(p.stats) + r.n * p.G + c / p.cg);
        mean[j] = st.x;
        rstd[j] = st.y;
        if (!VEC) {
            w[j] = weight_at(p.w, p.wdtype, c, 1.f);
            b[j] = weight_at(p.b, p.wdtype, c, 0.f);
        }
        if (!GRAD) w[j] *= st.y;
        if (GRAD) {
            const float2 m = *(reinterpret_cast<const float2*>(means) + r.n * p.G + c / p.cg);
            m1[j] = m.x;
            m2[j] = m.y;
        }
    }
    const T* const xp = static_cast<const T*>(p.x.p) + r.n * p.x.sn + r.l0 * p.x.sl + r.c;
    const T* const zp = static_cast<const T*>(p.z.p) + r.n * p.z.sn + r.l0 * p.z.sl + r.c;
    const T* const gp = static_cast<const T*>(p.dy.p) + r.n * p.dy.sn + r.l0 * p.dy.sl + r.c;
    T* const yp = static_cast<T*>(p.y) + r.n * p.yn + r.l0 * p.yl + r.c;
    T* const dp = static_cast<T*>(p.dz) + r.n * p.dzn + r.l0 * p.dzl + r.c;
    const int len = r.l1 - r.l0;
    for (int l0 = r.row; l0 < len; l0 += M * r.rows) {
        Lane<T, 8, VEC> xv[M], zv[M], gv[M];
#pragma unroll
        for (int i = 0; i < M; ++i) {
            const int l = l0 + i * r.rows;
            if (l < len) {
                xv[i].load(xp + l * p.x.sl, r.live);
                if (GATE) zv[i].load(zp + l * p.z.sl, r.live);
                if (GRAD) gv[i].load(gp + l * p.dy.sl, r.live);
            }
        }
#pragma unroll
        for (int i = 0; i < M; ++i) {
            const int l = l0 + i * r.rows;
            if (l >= len) break;
            float x[8], z[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (!GRAD) {
                    const float v = fmaf(xv[i].get(j) - mean[j], w[j], b[j]);
                    x[j] = GATE ? v * act<SILU>(zv[i].get(j)) : act<SILU>(v);
                } else {
                    const float n = (xv[i].get(j) - mean[j]) * rstd[j], v = fmaf(n, w[j], b[j]);
                    float value, slope;
                    act_slope<SILU>(GATE ? zv[i].get(j) : v, value, slope);
                    const float dy = gv[i].get(j), t = dy * (GATE ? value : slope) * w[j];
                    z[j] = dy * v * slope;
                    x[j] = rstd[j] * (t - m1[j] - n * m2[j]);
                }
            }
            Lane<T, 8, VEC> o;
            o.set(x);
            o.store(yp + l * p.yl, r.live);
            if (GRAD && GATE) {
                o.set(z);
                o.store(dp + l * p.dzl, r.live);
            }
        }
    }
}

// ------------------------------------------------------------------ host ----
struct GPlan {
    bool unit;
    int tpr, gpb, spb, blocks;  // units in registers; blocks along the samples in the gradient
    int run, runs;
    long long slab;      // large units: samples whose sums are held at a time
    long long lines;     // of partial sums
    size_t part, means;  // floats of partial sums; of the gradient's means behind them
};

// Large units take their samples in slabs whose partial sums have this many bytes at most (16384 blocks or more then).
// A run of a wide row is one position, whose sums are twice the size of an fp32 row: 65536 x 16384 held 8.6 GB of
// them.  (16384 x 8192 in 16 bits, of 1.07 GB: 1.91 ms at once, 2.00 by 256 MB, 2.23 by 64 MB.)
constexpr size_t kPartBytes = size_t(256) << 20;

GPlan gnorm_plan(long long N, int L, int C, int G, bool grad) {
    GPlan g{};
    const int cg = C / G;
    g.unit = (long long)L * cg <= kUnit;
    if (g.unit) {
        g.tpr = 1;
        while (g.tpr * 8 < L * cg) g.tpr *= 2;
        const int units = kThreads / g.tpr;
        g.gpb = G < units ? G : units;
        g.spb = units / g.gpb;
        const int across = (G + g.gpb - 1) / g.gpb;
        const long long need = (N + g.spb - 1) / g.spb, most = ((long long)(grad ? kBwdBlocks : kFwdBlocks) * sm_count() + across - 1) / across;
        g.blocks = (int)(need < most ? need : most);
        g.lines = g.blocks;
        g.part = grad ? (size_t)g.lines * 2 * C : 0;
        return g;
    }
    const int across = (C + kUnit - 1) / kUnit;
    // enough blocks to fill the SMs, runs of 16 positions or more
    long long runs = ((long long)kRunBlocks * sm_count() + N * across - 1) / (N * across);
    const long long most = (L + 15LL) / 16;
    if (runs > most) runs = most;
    g.run = (int)((L + runs - 1) / runs);
    g.runs = (int)((L + (long long)g.run - 1) / g.run);
    const long long fit = (long long)(kPartBytes / ((size_t)g.runs * 2 * C * 4));  // (one sample's runs are far below)
    g.slab = N < fit ? N : fit;
    g.lines = g.slab * g.runs;
    g.part = (size_t)g.lines * 2 * C;
    g.means = (size_t)g.slab * G * 2;
    return g;
}

int check_gnorm(const char* what, long long N, int L, int C, int G, float eps, int dtype, int wdtype, int act) {
    if (N <= 0 || L <= 0 || C <= 0 || G <= 0 || C % G)
        return set_error(HLA2_ERR_INVALID, "%s: sizes must be positive and C a multiple of G (N=%lld L=%d C=%d G=%d)", what, N, L, C, G);
    if (C > kMaxChannels) return set_error(HLA2_ERR_UNSUPPORTED, "%s: C=%d exceeds %d", what, C, kMaxChannels);
    if (N > 0x7fffffffLL || N * L > 0x7fffffffLL || N * G > 0x7fff0000LL)
        return set_error(HLA2_ERR_UNSUPPORTED, "%s: N*L or N*G exceeds 2^31 - 1 (N=%lld L=%d G=%d)", what, N, L, G);
    if (!known_dtype(dtype) || !known_dtype(wdtype)) return set_error(HLA2_ERR_UNSUPPORTED, "%s: unknown dtype", what);
    if (act != HLA2_ACT_NONE && act != HLA2_ACT_SILU) return set_error(HLA2_ERR_UNSUPPORTED, "%s: unknown activation %d", what, act);
    if (!(eps >= 0.f)) return set_error(HLA2_ERR_INVALID, "%s: eps must not be negative", what);
    return HLA2_OK;
}

int check_gws(const char* what, size_t need, const void* ws, size_t bytes) {
    if (need && (!ws || bytes < need)) return set_error(HLA2_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", what, bytes, need);
    if (need && reinterpret_cast<uintptr_t>(ws) % 16) return set_error(HLA2_ERR_INVALID, "%s: workspace not 16-byte aligned", what);
    return HLA2_OK;
}
size_t gnorm_bytes(const GPlan& g) { return ((g.part + g.means) * 4 + 255) & ~size_t(255); }

// what the kernels take 16 bytes of at a time
bool wide(const void* p, long long sn, long long sl, long long N, int L, int es) {
    if (!p) return true;
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (N == 1 || sn * es % 16 == 0) && (L == 1 || sl * es % 16 == 0);
}

template <bool GRAD>
cudaError_t run_gnorm(GNormParams p, const GPlan& g, int dtype, bool vec, cudaStream_t s) {
    auto typed = [&](auto t, auto v, auto gate, auto silu) {
        using T = decltype(t);
        constexpr bool VEC = decltype(v)::value, GATE = decltype(gate)::value, SILU = decltype(silu)::value;
        if (g.unit) {
            const dim3 grid(g.blocks, (p.G + g.gpb - 1) / g.gpb);
            if (GRAD)
                return launch_following(gnorm_unit_bwd_kernel<T, VEC, GATE, SILU>, grid, kThreads, 0, s, false, p);
            gnorm_unit_kernel<T, VEC, GATE, SILU><<<grid, kThreads, 0, s>>>(p);
            note_launches(1);
            return cudaGetLastError();
        }
        float* const means = p.part + g.part;
        const unsigned lines = GRAD && p.dw ? (2 * p.C + kFoldColumns - 1) / kFoldColumns : 0;
        for (long long n0 = 0; n0 < p.N; n0 += g.slab) {
            GNormParams q = p;
            q.N = p.N - n0 < g.slab ? p.N - n0 : g.slab;
            auto ahead = [&](auto* at, long long stride) {
                using P = std::conditional_t<std::is_const_v<std::remove_pointer_t<decltype(at)>>, const T, T>;
                return at ? static_cast<P*>(at) + n0 * stride : nullptr;
            };
            q.x.p = ahead(p.x.p, p.x.sn);
            q.z.p = ahead(p.z.p, p.z.sn);
            q.dy.p = ahead(p.dy.p, p.dy.sn);
            q.y = ahead(p.y, p.yn);
            q.dz = ahead(p.dz, p.dzn);
            if (p.stats) q.stats = p.stats + n0 * p.G * 2;
            float* const folded = GRAD || !p.stats ? means : q.stats;
            const dim3 grid((unsigned)(q.N * g.runs), (p.C + kUnit - 1) / kUnit);
            cudaError_t e;
            if constexpr (GRAD) e = launch_following(gnorm_sums_kernel<T, VEC, GATE, SILU>, grid, kThreads, 0, s, n0 > 0, q);
            else e = launch_following(gnorm_moments_kernel<T, VEC>, grid, kThreads, 0, s, n0 > 0, q);
            if (e == cudaSuccess)
                e = launch_following(gnorm_fold_kernel<GRAD>, dim3((unsigned)(q.N * p.G) + lines), kThreads, 0, s, true, q, folded,
                                     n0 > 0);
            if (!GRAD) q.stats = folded;
            if (e == cudaSuccess)
                e = launch_following(gnorm_apply_kernel<T, VEC, GRAD, GATE, SILU>, grid, kThreads, 0, s, true, q, means);
            if (e != cudaSuccess) return e;
        }
        return cudaSuccess;
    };
    using yes = std::true_type;
    using no = std::false_type;
    auto acted = [&](auto t, auto v) {
        if (p.z.p) return p.silu ? typed(t, v, yes{}, yes{}) : typed(t, v, yes{}, no{});
        return p.silu ? typed(t, v, no{}, yes{}) : typed(t, v, no{}, no{});
    };
    cudaError_t e;
    if (dtype == HLA2_DTYPE_BF16) e = vec ? acted(bf16{}, yes{}) : acted(bf16{}, no{});
    else e = vec ? acted(float{}, yes{}) : acted(float{}, no{});
    if (GRAD && e == cudaSuccess && p.dw && g.unit) {
        e = launch_following(gnorm_lines_kernel, dim3((2 * p.C + kFoldColumns - 1) / kFoldColumns), kFoldThreads, 0, s, true,
                             p.part, p.dw, g.lines, 2 * p.C);
    }
    return e;
}

}  // namespace
}  // namespace hla2

extern "C" size_t hla2_groupnorm_workspace(long long N, int L, int C, int G, int backward) {
    using namespace hla2;
    if (check_gnorm("groupnorm_workspace", N, L, C, G, 0.f, HLA2_DTYPE_F32, HLA2_DTYPE_F32, HLA2_ACT_NONE)) return 0;
    return gnorm_bytes(gnorm_plan(N, L, C, G, backward != 0));
}

extern "C" int hla2_groupnorm(const void* X, const void* W, const void* Bias, const void* gate, void* Y, float* stats,
                              long long N, int L, int C, int G, const long long* strides, float eps, int act, int dtype,
                              int wdtype, void* workspace, size_t ws_bytes, hla2_stream_t stream) {
    using namespace hla2;
    const char* what = "groupnorm";
    if (int rc = check_gnorm(what, N, L, C, G, eps, dtype, wdtype, act)) return rc;
    if (!X || !Y) return set_error(HLA2_ERR_INVALID, "%s: null pointer", what);
    const int es = dtype_size(dtype), wsz = dtype_size(wdtype);
    if (!aligned_elem(X, es) || !aligned_elem(gate, es) || !aligned_elem(Y, es) || !aligned_elem(W, wsz) ||
        !aligned_elem(Bias, wsz) || !aligned_elem(stats, 8))
        return set_error(HLA2_ERR_INVALID, "%s: pointer not aligned to its element", what);
    const GPlan g = gnorm_plan(N, L, C, G, false);
    if (int rc = check_gws(what, gnorm_bytes(g), workspace, ws_bytes)) return rc;
    const long long dense[2] = {(long long)L * C, C};
    auto st = [&](int i, int k) { return strides ? strides[2 * i + k] : dense[k]; };
    GNormParams p{};
    p.x = {X, st(0, 0), st(0, 1)};
    p.z = {gate, st(1, 0), st(1, 1)};
    p.y = Y; p.yn = st(2, 0); p.yl = st(2, 1);
    p.w = W; p.b = Bias; p.wdtype = wdtype; p.stats = stats; p.part = static_cast<float*>(workspace);
    p.N = N; p.L = L; p.C = C; p.G = G; p.cg = C / G; p.silu = act == HLA2_ACT_SILU; p.eps = eps;
    p.tpr = g.tpr; p.gpb = g.gpb; p.spb = g.spb; p.run = g.run; p.runs = g.runs;
    const bool vec = (g.unit ? p.cg : C) % 8 == 0 && wide(X, p.x.sn, p.x.sl, N, L, es) &&
                     wide(gate, p.z.sn, p.z.sl, N, L, es) && wide(Y, p.yn, p.yl, N, L, es) &&
                     wide(W, 0, 0, 1, 1, wsz) && wide(Bias, 0, 0, 1, 1, wsz);
    const cudaError_t e = run_gnorm<false>(p, g, dtype, vec, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return set_error(HLA2_ERR_LAUNCH, "%s: %s", what, cudaGetErrorString(e));
    return HLA2_OK;
}

extern "C" int hla2_groupnorm_backward(const void* X, const void* dY, const float* stats, const void* W,
                                       const void* Bias, const void* gate, void* dX, void* dgate, float* dWB,
                                       long long N, int L, int C, int G, const long long* strides, int act, int dtype,
                                       int wdtype, void* workspace, size_t ws_bytes, hla2_stream_t stream) {
    using namespace hla2;
    const char* what = "groupnorm_backward";
    if (int rc = check_gnorm(what, N, L, C, G, 0.f, dtype, wdtype, act)) return rc;
    if (!X || !dY || !stats || !dX || (gate != nullptr) != (dgate != nullptr))
        return set_error(HLA2_ERR_INVALID, "%s: null pointer, or one of gate and dgate without the other", what);
    const int es = dtype_size(dtype), wsz = dtype_size(wdtype);
    if (!aligned_elem(X, es) || !aligned_elem(dY, es) || !aligned_elem(gate, es) || !aligned_elem(dX, es) ||
        !aligned_elem(dgate, es) || !aligned_elem(W, wsz) || !aligned_elem(Bias, wsz) || !aligned_elem(stats, 8) ||
        !aligned_elem(dWB, 4))
        return set_error(HLA2_ERR_INVALID, "%s: pointer not aligned to its element", what);
    if (dX == dgate) return set_error(HLA2_ERR_INVALID, "%s: two outputs are one tensor", what);
    const GPlan g = gnorm_plan(N, L, C, G, true);
    if (int rc = check_gws(what, gnorm_bytes(g), workspace, ws_bytes)) return rc;
    const long long dense[2] = {(long long)L * C, C};
    auto st = [&](int i, int k) { return strides ? strides[2 * i + k] : dense[k]; };
    GNormParams p{};
    p.x = {X, st(0, 0), st(0, 1)};
    p.dy = {dY, st(1, 0), st(1, 1)};
    p.z = {gate, st(2, 0), st(2, 1)};
    p.y = dX; p.yn = st(3, 0); p.yl = st(3, 1);
    p.dz = dgate; p.dzn = st(4, 0); p.dzl = st(4, 1);
    p.w = W; p.b = Bias; p.wdtype = wdtype; p.stats = const_cast<float*>(stats);
    p.part = static_cast<float*>(workspace); p.dw = dWB;
    p.N = N; p.L = L; p.C = C; p.G = G; p.cg = C / G; p.silu = act == HLA2_ACT_SILU;
    p.tpr = g.tpr; p.gpb = g.gpb; p.spb = g.spb; p.run = g.run; p.runs = g.runs;
    const bool vec = (g.unit ? p.cg : C) % 8 == 0 && wide(X, p.x.sn, p.x.sl, N, L, es) &&
                     wide(dY, p.dy.sn, p.dy.sl, N, L, es) && wide(gate, p.z.sn, p.z.sl, N, L, es) &&
                     wide(dX, p.yn, p.yl, N, L, es) && wide(dgate, p.dzn, p.dzl, N, L, es) && wide(W, 0, 0, 1, 1, wsz) &&
                     wide(Bias, 0, 0, 1, 1, wsz);
    const cudaError_t e = run_gnorm<true>(p, g, dtype, vec, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return set_error(HLA2_ERR_LAUNCH, "%s: %s", what, cudaGetErrorString(e));
    return HLA2_OK;
}
