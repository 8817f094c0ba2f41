// hla2_gated.cu -- gated linear recurrence along the tokens of each head and
// channel: forward, gradient and the single-token step.
//
//   h_t = a_t h_{t-1} + u_t
//   decay:   a = g, u = x
//   sigmoid: a = 1 / (1 + e^-g), u = (1 - a) x, taken as h += z (x - h) with
//            z = 1 - a = e^-g / (1 + e^-g): z keeps its relative precision where
//            a is next to 1, which is where the memory is long.
// A reset at t makes h_{t-1} zero there (chosen, not multiplied: nothing of an
// earlier document passes, not even inf or NaN).
//
// Gradient, lam_t = dh_t + a_{t+1} lam_{t+1}:
//   decay:   dx = lam,    dg = lam h_{t-1}
//   sigmoid: dx = z lam,  dg = z (1 - z) lam (h_{t-1} - x)
//
// One pass over the data.  A run of tokens maps the state before it to the
// state after it by h -> A h + X, and such maps compose, so a tile of tokens
// can be read once, long before the state that enters it is known:
//   - a block holds a tile in registers: a thread 4 channels of kTok tokens, a
//     "run"; the runs' maps are composed in shared memory;
//   - the tile's map goes to the workspace; the state that enters the tile is
//     the state that entered its super-group of 128 tiles, passed through the
//     maps of the groups of 8 tiles, then of the tiles, before it; warps of their
//     own do this, so that no thread holds its tokens and these maps at once;
//   - every thread then walks its tokens again, from registers, from the state
//     that enters its run.
// Tiles are taken by ticket, all heads' first tiles first, so whoever waits
// waits for a tile that a running block holds.  Which maps are composed, and in
// which order, depends on the tile's place alone: the same call gives the same
// bits, whatever the timing.  The last tile of a group publishes the group's
// map and the last of a super-group the state after it, so a tile reads at most
// 22 maps and one state, and the only chain along the sequence has one link for
// each 128 tiles.
#include <map>
#include <mutex>

#include "hla2_layer.cuh"

namespace hla2 {
namespace {

constexpr int kTok = 8;         // tokens of a thread's run
constexpr int kCh = 4;          // channels of a thread
constexpr int kData = 256;      // threads that hold a tile
constexpr int kGroup = 8;       // tiles to a group
constexpr int kSuper = 16;      // groups to a super-group
constexpr unsigned long long kGateWaitNs = 2000000000ull;  // bounded waits: 2 s

// Lanes that share a token: they cover 4 channels each, d <= 4 lanes.
__host__ __device__ constexpr int lanes_of(int d) { return d <= 64 ? 16 : 32; }
// Tokens of a tile: a state is kept for the gradient at the start of each.
__host__ __device__ constexpr int tile_of(int lanes) { return kData / lanes * kTok; }
// Threads of a block: those that hold the tile, and a warp for each 32 channels that joins tiles.
__host__ __device__ constexpr int block_threads(int lanes) { return kData + lanes * kCh; }

struct GateParams {
    const void *x, *g, *dout;
    const unsigned char* reset;
    const float *state_in, *dstate_out;
    void *o, *dx, *dg;
    float *state_out, *dstate_in, *carry;
    int B, H, T, d;
    long long sx[3], sg[3], so[3], sdo[3], sdx[3], sdg[3];
    // workspace (null for one tile): see Lookback
    unsigned long long* words;
    int tiles, out_bf16;
    unsigned total;  // rows * tiles
    int* status;
};

// z = 1 - a of the sigmoid gate
__device__ __forceinline__ float keep_out(float g) {
    const float e = __expf(-g);
    return isinf(e) ? 1.f : __fdividef(e, 1.f + e);
}

// ---- maps h -> A h + X -------------------------------------------------------
// A run that holds a reset forgets what entered it: its A is -0, which nothing
// else is (products that are zero are made +0), and then only X counts.
__device__ __forceinline__ float cut() { return __uint_as_float(0x80000000u); }
__device__ __forceinline__ bool is_cut(float A) { return __float_as_uint(A) == 0x80000000u; }
__device__ __forceinline__ float pass(float2 m, float h) { return is_cut(m.x) ? m.y : fmaf(m.x, h, m.y); }
// first `a`, then `b`
__device__ __forceinline__ float2 then(float2 a, float2 b) {
    return make_float2(is_cut(b.x) || is_cut(a.x) ? cut() : a.x * b.x + 0.f, pass(b, a.y));
}

// ---- the workspace -----------------------------------------------------------
// A ticket word and a word that says that a wait ran out; then the maps of the
// tiles and of the groups (A, X for each of a row's channels), then the states
// that enter the super-groups (h, 0).  Each pair is one 64-bit word, written and
// read whole, so it is its own flag: the words are set to all ones before the
// launch, which no pair is (arithmetic gives one NaN, 0x7fffffff), and whoever
// needs one reads it until it is something else.
struct Lookback {
    int rows, tiles, groups, supers, cb;  // cb: channels of a map
    __host__ __device__ Lookback(int rows, int tiles, int cb)
        : rows(rows), tiles(tiles), groups((tiles + kGroup - 1) / kGroup),
          supers((groups + kSuper - 1) / kSuper), cb(cb) {}
    __host__ __device__ size_t tile_map(int r, int t) const { return 1 + ((size_t)r * tiles + t) * cb; }
    __host__ __device__ size_t group_map(int r, int g) const { return tile_map(rows, 0) + ((size_t)r * groups + g) * cb; }
    __host__ __device__ size_t super_state(int r, int s) const {
        return group_map(rows, 0) + ((size_t)r * supers + s) * cb;
    }
    __host__ __device__ size_t words() const { return super_state(rows, 0); }
};

using u64 = unsigned long long;
constexpr u64 kNothing = ~0ull;

__device__ __forceinline__ u64 ld_word(const u64* p) {
    u64 v;
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void st_pair(u64* p, float2 m) {
    u64 v = ((u64)__float_as_uint(m.y) << 32) | __float_as_uint(m.x);
    if (v == kNothing) v = 0x7fffffff7fffffffull;
    asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(v) : "memory");
}
__device__ __forceinline__ float2 as_pair(u64 v) {
    return make_float2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
}
__device__ __forceinline__ u64 gate_timer() {
    u64 t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    return t;
}

// Reads w[i] = p[i * step] for i < n until every one is there.  Gives up after
// 2 s: then this call's results are void, the status word says so, and every
// later wait of the call ends at once.
template <int N>
__device__ __forceinline__ void read_words(const GateParams& p, const u64* src, size_t step, int n, u64 (&w)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = i < n ? ld_word(src + i * step) : 0;
    u64 t0 = 0;
    while (true) {
        bool all = true;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (w[i] == kNothing) {
                w[i] = ld_word(src + i * step);
                all = all && w[i] != kNothing;
            }
        if (all) return;
        const u64 now = gate_timer();
        if (t0 == 0) t0 = now;
        unsigned* const run_out = reinterpret_cast<unsigned*>(p.words) + 1;
        if (now - t0 > kGateWaitNs || *(volatile unsigned*)run_out != ~0u) {
            atomicExch(run_out, 0u);
            atomicExch(p.status, (int)kDevWaitTimeout);
            return;
        }
    }
}

// One thread's part, for its channel: publishes the tile's map `m`, returns the
// state that enters the tile.  `start`: the state that enters the sequence.
// `n` counts tiles in the order of the walk.
__device__ __forceinline__ float enter_tile(const GateParams& p, const Lookback& lb, int row, int n, int ch, float2 m,
                                            float start) {
    const int g = n / kGroup, s = g / kSuper;
    const int nt = n % kGroup, ng = g % kSuper;  // tiles before this one in its group, groups before it in the super-group
    const bool last = n + 1 == lb.tiles, ends_group = nt == kGroup - 1, ends_super = ends_group && ng == kSuper - 1;
    if (!last) st_pair(p.words + lb.tile_map(row, n) + ch, m);
    // the tiles of the group first: the group's map waits for nothing else
    u64 w[kGroup - 1];
    read_words(p, p.words + lb.tile_map(row, n - nt) + ch, lb.cb, nt, w);
    if (ends_group && !last) {
        float2 all = as_pair(w[0]);
#pragma unroll
        for (int i = 1; i < kGroup - 1; ++i) all = then(all, as_pair(w[i]));
        st_pair(p.words + lb.group_map(row, g) + ch, then(all, m));
    }
    float h = start;
    if (s > 0) {
        u64 v[1];
        read_words(p, p.words + lb.super_state(row, s) + ch, 0, 1, v);
        h = as_pair(v[0]).x;
    }
#pragma unroll
    for (int half = 0; half < kSuper; half += kSuper / 2) {
        u64 v[kSuper / 2];
        const int here = min(ng - half, kSuper / 2);
        if (here > 0) {
            read_words(p, p.words + lb.group_map(row, g - ng + half) + ch, lb.cb, here, v);
#pragma unroll
            for (int i = 0; i < kSuper / 2; ++i)
                if (i < here) h = pass(as_pair(v[i]), h);
        }
    }
#pragma unroll
    for (int i = 0; i < kGroup - 1; ++i)
        if (i < nt) h = pass(as_pair(w[i]), h);
    if (ends_super && !last) st_pair(p.words + lb.super_state(row, s + 1) + ch, make_float2(pass(m, h), 0.f));
    return h;
}

// The tiles of a block, by ticket where tiles wait for one another.  The
// joining warps take the next ticket between the two barriers of a tile.
struct Tickets {
    unsigned* word;  // starts at ~0
    unsigned* slot;  // shared
    __device__ unsigned first() {
        if (!word) return blockIdx.x;
        if (threadIdx.x == 0) *slot = atomicAdd(word, 1u) + 1u;
        __syncthreads();
        return *slot;
    }
    __device__ unsigned take(unsigned k) { return word ? atomicAdd(word, 1u) + 1u : k + gridDim.x; }
};

// Loads a run: x and gates of tokens [0, nt), the bits of its resets.
template <typename T, bool SHARED, bool VEC>
struct Run {
    Lane<T, kCh, VEC> x[kTok];
    Lane<T, SHARED ? 1 : kCh, VEC && !SHARED> g[kTok];
    unsigned resets;
    __device__ __forceinline__ void load(const GateParams& p, int b, int hd, int t0, int c, int nc, int nt) {
        const T* xp = static_cast<const T*>(p.x) + b * p.sx[0] + hd * p.sx[1] + t0 * p.sx[2] + c;
        const T* gp = static_cast<const T*>(p.g) + b * p.sg[0] + hd * p.sg[1] + t0 * p.sg[2] + (SHARED ? 0 : c);
#pragma unroll
        for (int i = 0; i < kTok; ++i)
            if (i < nt) {
                x[i].load(xp + i * p.sx[2], nc);
                g[i].load(gp + i * p.sg[2], SHARED ? 1 : nc);
            }
        resets = 0;
        if (p.reset) {
            const unsigned char* rp = p.reset + (long long)b * p.T + t0;
#pragma unroll
            for (int i = 0; i < kTok; ++i)
                if (i < nt && rp[i]) resets |= 1u << i;
        }
    }
    __device__ __forceinline__ bool reset(int i) const { return (resets >> i) & 1u; }
};

// ---- forward -----------------------------------------------------------------
// LANES x 4 channels to a token, kData / LANES runs of kTok tokens to a tile.
template <typename T, bool SIG, bool SHARED, int LANES, bool VEC>
__global__ void __launch_bounds__(block_threads(LANES), sizeof(T) == 2 ? 2 : 1)
gated_scan_kernel(const GateParams p) {
    constexpr int CB = LANES * kCh, RUNS = kData / LANES, TILE = RUNS * kTok, NG = SHARED ? 1 : kCh;
    __shared__ float2 runs[RUNS][CB];  // maps of the runs, then of what is before each in the tile
    __shared__ float entering[CB];
    __shared__ unsigned slot;
    const int rows = p.B * p.H;
    const Lookback lb(rows, p.tiles, CB);
    Tickets tickets{reinterpret_cast<unsigned*>(p.words), &slot};
    unsigned k = tickets.first();
    if (threadIdx.x >= kData) {  // joins the tiles: one thread to a channel
        const int ch = threadIdx.x - kData;
        while (k < p.total) {
            const int n = (int)(k / (unsigned)rows), row = (int)(k - (unsigned)n * (unsigned)rows);
            float h = p.state_in && ch < p.d ? p.state_in[(long long)row * p.d + ch] : 0.f;
            __syncthreads();  // the runs' maps are there
            if (ch == 0) slot = tickets.take(k);
            float2 m = make_float2(1.f, 0.f);
#pragma unroll 8
            for (int r = 0; r < RUNS; ++r) {
                const float2 f = runs[r][ch];
                runs[r][ch] = m;
                m = then(m, f);
            }
            if (p.words) h = enter_tile(p, lb, row, n, ch, m, h);
            entering[ch] = h;
            if (p.carry && ch < p.d) p.carry[((long long)row * p.tiles + n) * p.d + ch] = h;
            __syncthreads();  // what enters each run is there
            k = slot;
        }
        return;
    }
    const int lane = threadIdx.x % LANES, run = threadIdx.x / LANES;
    const int c = lane * kCh, nc = p.d - c;
    while (k < p.total) {
        const int n = (int)(k / (unsigned)rows), row = (int)(k - (unsigned)n * (unsigned)rows);
        const int b = row / p.H, hd = row - b * p.H;
        const int t0 = n * TILE + run * kTok;
        const int nt = nc > 0 ? min(kTok, p.T - t0) : 0;  // tokens of this thread, none where <= 0
        Run<T, SHARED, VEC> in;
        in.load(p, b, hd, t0, c, nc, nt);
        float gate[kTok][NG];  // z of the sigmoid, a of the decay
        float A[kCh], X[kCh];
#pragma unroll
        for (int j = 0; j < kCh; ++j) { A[j] = 1.f; X[j] = 0.f; }
#pragma unroll
        for (int i = 0; i < kTok; ++i)
            if (i < nt) {
#pragma unroll
                for (int j = 0; j < NG; ++j) gate[i][j] = SIG ? keep_out(in.g[i].get(j)) : in.g[i].get(j);
#pragma unroll
                for (int j = 0; j < kCh; ++j) {
                    const float ga = gate[i][SHARED ? 0 : j], xv = in.x[i].get(j);
                    if (in.reset(i)) X[j] = 0.f;
                    X[j] = SIG ? fmaf(ga, xv - X[j], X[j]) : fmaf(ga, X[j], xv);
                    A[j] = SIG ? fmaf(-ga, A[j], A[j]) : ga * A[j];
                }
            }
#pragma unroll
        for (int j = 0; j < kCh; ++j) runs[run][c + j] = make_float2(in.resets ? cut() : A[j] + 0.f, X[j]);
        __syncthreads();
        __syncthreads();
        k = slot;
        if (nt > 0) {
            float h[kCh];
#pragma unroll
            for (int j = 0; j < kCh; ++j) h[j] = pass(runs[run][c + j], entering[c + j]);
            const long long off = b * p.so[0] + hd * p.so[1] + t0 * p.so[2] + c;
#pragma unroll
            for (int i = 0; i < kTok; ++i)
                if (i < nt) {
#pragma unroll
                    for (int j = 0; j < kCh; ++j) {
                        const float ga = gate[i][SHARED ? 0 : j], xv = in.x[i].get(j);
                        if (in.reset(i)) h[j] = 0.f;
                        h[j] = SIG ? fmaf(ga, xv - h[j], h[j]) : fmaf(ga, h[j], xv);
                    }
                    if (p.out_bf16) {
                        Lane<bf16, kCh, VEC> ov;
                        ov.set(h);
                        ov.store(static_cast<bf16*>(p.o) + off + i * p.so[2], nc);
                    } else {
                        Lane<float, kCh, VEC> ov;
                        ov.set(h);
                        ov.store(static_cast<float*>(p.o) + off + i * p.so[2], nc);
                    }
                }
            if (p.state_out && t0 + nt == p.T) {
#pragma unroll
                for (int j = 0; j < kCh; ++j)
                    if (j < nc) p.state_out[(long long)row * p.d + c + j] = h[j];
            }
        }
    }
}

// ---- gradient ----------------------------------------------------------------
// The same walk from the last tile to the first for mu_t = a_t lam_t, the part of
// the gradient that reaches h_{t-1}: mu_t = a_t (dh_t + mu_{t+1}), so a run maps
// the mu behind it to the mu before it by the same A and a Y of its own.  The
// states inside the tile are formed anew, from the kept state that enters it; a
// thread's h_{t-1} wait in shared memory until its way back.
template <typename T, typename TO, bool SIG, bool SHARED, int LANES, bool VEC>
__global__ void __launch_bounds__(block_threads(LANES), sizeof(T) == 2 ? 2 : 1)
gated_scan_bwd_kernel(const GateParams p) {
    constexpr int CB = LANES * kCh, RUNS = kData / LANES, TILE = RUNS * kTok, NG = SHARED ? 1 : kCh;
    __shared__ float2 fwd[RUNS][CB];   // maps of h; .x becomes the state that enters the run
    __shared__ float2 back[RUNS][CB];  // maps of mu, then of what is behind each run in the tile
    __shared__ float entering[CB];
    __shared__ unsigned slot;
    extern __shared__ float4 before[];  // [kTok][kData]: h_{t-1}
    const int rows = p.B * p.H;
    const Lookback lb(rows, p.tiles, CB);
    Tickets tickets{reinterpret_cast<unsigned*>(p.words), &slot};
    unsigned k = tickets.first();
    if (threadIdx.x >= kData) {
        const int ch = threadIdx.x - kData;
        while (k < p.total) {
            const int n = (int)(k / (unsigned)rows), row = (int)(k - (unsigned)n * (unsigned)rows);
            float mu = 0.f, h = 0.f;
            if (ch < p.d) {
                if (p.dstate_out) mu = p.dstate_out[(long long)row * p.d + ch];
                h = p.carry[((long long)row * p.tiles + (p.tiles - 1 - n)) * p.d + ch];
            }
            __syncthreads();
            if (ch == 0) slot = tickets.take(k);
            float2 m = make_float2(1.f, 0.f);
#pragma unroll 8
            for (int r = RUNS - 1; r >= 0; --r) {
                const float2 f = back[r][ch];
                back[r][ch] = m;
                m = then(m, f);
            }
#pragma unroll 8
            for (int r = 0; r < RUNS; ++r) {
                const float2 f = fwd[r][ch];
                fwd[r][ch].x = h;
                h = pass(f, h);
            }
            if (p.words) mu = enter_tile(p, lb, row, n, ch, m, mu);
            entering[ch] = mu;
            __syncthreads();
            k = slot;
        }
        return;
    }
    const int tid = threadIdx.x, lane = tid % LANES, run = tid / LANES;
    const int c = lane * kCh, nc = p.d - c;
    while (k < p.total) {
        const int n = (int)(k / (unsigned)rows), row = (int)(k - (unsigned)n * (unsigned)rows);
        const int b = row / p.H, hd = row - b * p.H;
        const int t0 = (p.tiles - 1 - n) * TILE + run * kTok;
        const int nt = nc > 0 ? min(kTok, p.T - t0) : 0;
        Run<T, SHARED, VEC> in;
        in.load(p, b, hd, t0, c, nc, nt);
        Lane<TO, kCh, VEC> dh[kTok];
        const TO* up = static_cast<const TO*>(p.dout) + b * p.sdo[0] + hd * p.sdo[1] + t0 * p.sdo[2] + c;
#pragma unroll
        for (int i = 0; i < kTok; ++i)
            if (i < nt) dh[i].load(up + i * p.sdo[2], nc);
        float gate[kTok][NG];
        float A[kCh], X[kCh], Y[kCh];
#pragma unroll
        for (int j = 0; j < kCh; ++j) { A[j] = 1.f; X[j] = 0.f; Y[j] = 0.f; }
#pragma unroll
        for (int i = 0; i < kTok; ++i)
            if (i < nt) {
#pragma unroll
                for (int j = 0; j < NG; ++j) gate[i][j] = SIG ? keep_out(in.g[i].get(j)) : in.g[i].get(j);
#pragma unroll
                for (int j = 0; j < kCh; ++j) {
                    const float ga = gate[i][SHARED ? 0 : j], xv = in.x[i].get(j);
                    if (in.reset(i)) X[j] = 0.f;
                    X[j] = SIG ? fmaf(ga, xv - X[j], X[j]) : fmaf(ga, X[j], xv);
                    A[j] = SIG ? fmaf(-ga, A[j], A[j]) : ga * A[j];
                }
            }
#pragma unroll
        for (int i = kTok - 1; i >= 0; --i)
            if (i < nt) {
#pragma unroll
                for (int j = 0; j < kCh; ++j) {
                    const float ga = gate[i][SHARED ? 0 : j], lam = dh[i].get(j) + Y[j];
                    Y[j] = in.reset(i) ? 0.f : SIG ? fmaf(-ga, lam, lam) : ga * lam;
                }
            }
#pragma unroll
        for (int j = 0; j < kCh; ++j) {
            const float a = in.resets ? cut() : A[j] + 0.f;
            fwd[run][c + j] = make_float2(a, X[j]);
            back[run][c + j] = make_float2(a, Y[j]);
        }
        __syncthreads();
        __syncthreads();
        k = slot;
        float mu[kCh];
        if (nt > 0) {
            float h[kCh];
#pragma unroll
            for (int j = 0; j < kCh; ++j) {
                h[j] = fwd[run][c + j].x;
                mu[j] = pass(back[run][c + j], entering[c + j]);
            }
#pragma unroll
            for (int i = 0; i < kTok; ++i)
                if (i < nt) {
#pragma unroll
                    for (int j = 0; j < kCh; ++j)
                        if (in.reset(i)) h[j] = 0.f;
                    before[i * kData + tid] = make_float4(h[0], h[1], h[2], h[3]);
#pragma unroll
                    for (int j = 0; j < kCh; ++j) {
                        const float ga = gate[i][SHARED ? 0 : j], xv = in.x[i].get(j);
                        h[j] = SIG ? fmaf(ga, xv - h[j], h[j]) : fmaf(ga, h[j], xv);
                    }
                }
        }
        T* dxp = static_cast<T*>(p.dx) + b * p.sdx[0] + hd * p.sdx[1] + t0 * p.sdx[2] + c;
        T* dgp = static_cast<T*>(p.dg) + b * p.sdg[0] + hd * p.sdg[1] + t0 * p.sdg[2] + (SHARED ? 0 : c);
#pragma unroll
        for (int i = kTok - 1; i >= 0; --i) {
            float gx[kCh], gg[kCh];
            const bool live = i < nt;
            if (live) {
                const float4 hb4 = before[i * kData + tid];
                const float hb[kCh] = {hb4.x, hb4.y, hb4.z, hb4.w};
#pragma unroll
                for (int j = 0; j < kCh; ++j) {
                    const float ga = gate[i][SHARED ? 0 : j], lam = dh[i].get(j) + mu[j];
                    if (SIG) {
                        gx[j] = ga * lam;
                        gg[j] = fmaf(-ga, gx[j], gx[j]) * (hb[j] - in.x[i].get(j));
                        mu[j] = in.reset(i) ? 0.f : fmaf(-ga, lam, lam);
                    } else {
                        gx[j] = lam;
                        gg[j] = lam * hb[j];
                        mu[j] = in.reset(i) ? 0.f : ga * lam;
                    }
                }
                Lane<T, kCh, VEC> ov;
                ov.set(gx);
                ov.store(dxp + i * p.sdx[2], nc);
            }
            if (SHARED) {  // the sum over the token's channels
                float s = 0.f;
#pragma unroll
                for (int j = 0; j < kCh; ++j) s += live && j < nc ? gg[j] : 0.f;
#pragma unroll
                for (int w = LANES / 2; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
                if (live && lane == 0) dgp[i * p.sdg[2]] = from_f32<T>(s);
            } else if (live) {
                Lane<T, kCh, VEC> ov;
                ov.set(gg);
                ov.store(dgp + i * p.sdg[2], nc);
            }
        }
        if (p.dstate_in && t0 == 0 && nt > 0) {
#pragma unroll
            for (int j = 0; j < kCh; ++j)
                if (j < nc) p.dstate_in[(long long)row * p.d + c + j] = mu[j];
        }
    }
}

// One token: a read and a write of the state and of the token's n d values are
// the whole work; four channels to a thread where d and the strides allow.
template <typename T, typename TO, bool SIG, bool SHARED, bool VEC>
__global__ void __launch_bounds__(256) gated_step_kernel(const float* state, const T* x, const T* g, TO* o,
                                                         float* state_out, int n, int d, long long ldx, long long ldg,
                                                         long long ldo) {
    constexpr int N = VEC ? 4 : 1;
    const unsigned per = (unsigned)d / N;  // threads to a row
    const unsigned long long i = (unsigned long long)blockIdx.x * 256 + threadIdx.x;
    const long long row = (long long)(i / per);
    if (row >= n) return;
    const int c = (int)(i - (unsigned long long)row * per) * N;
    Lane<float, N, VEC> h;
    Lane<T, N, VEC> xv, gv;
    h.load(state + row * d + c, N);
    xv.load(x + row * ldx + c, N);
    if (!SHARED) gv.load(g + row * ldg + c, N);
    const float gate0 = SHARED ? to_f32(__ldg(g + row * ldg)) : 0.f;
    float out[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const float gate = SHARED ? gate0 : gv.get(j);
        out[j] = SIG ? fmaf(keep_out(gate), xv.get(j) - h.get(j), h.get(j)) : fmaf(gate, h.get(j), xv.get(j));
    }
    h.set(out);
    h.store(state_out + row * d + c, N);
    Lane<TO, N, VEC> ov;
    ov.set(out);
    ov.store(o + row * ldo + c, N);
}

template <typename F>
cudaError_t by_types(int dtype, int out_dtype, F&& f) {
    if (dtype == HLA2_DTYPE_BF16) return out_dtype == HLA2_DTYPE_BF16 ? f(bf16{}, bf16{}) : f(bf16{}, float{});
    return out_dtype == HLA2_DTYPE_BF16 ? f(float{}, bf16{}) : f(float{}, float{});
}
template <typename F>
cudaError_t by_form(int form, int shared, F&& f) {
    using std::false_type;
    using std::true_type;
    if (form == HLA2_GATE_SIGMOID) return shared ? f(true_type{}, true_type{}) : f(true_type{}, false_type{});
    return shared ? f(false_type{}, true_type{}) : f(false_type{}, false_type{});
}

int check_gated(const char* what, int B, int H, int T, int d, int form, int dtype, int out_dtype) {
    if (B <= 0 || H <= 0 || T <= 0 || d <= 0)
        return set_error(HLA2_ERR_INVALID, "%s: sizes must be positive (B=%d H=%d T=%d d=%d)", what, B, H, T, d);
    if (d > 128) return set_error(HLA2_ERR_UNSUPPORTED, "%s: d=%d: this build supports d <= 128", what, d);
    if ((long long)B * H > 65535) return set_error(HLA2_ERR_UNSUPPORTED, "%s: B*H=%lld exceeds 65535", what, (long long)B * H);
    if (form != HLA2_GATE_SIGMOID && form != HLA2_GATE_DECAY) return set_error(HLA2_ERR_UNSUPPORTED, "%s: unknown form %d", what, form);
    if (!known_dtype(dtype) || !known_dtype(out_dtype))
        return set_error(HLA2_ERR_UNSUPPORTED, "%s: unknown dtype %d or output dtype %d", what, dtype, out_dtype);
    if (T > (1 << 30) || (long long)B * H * T > (1LL << 33)) return set_error(HLA2_ERR_UNSUPPORTED, "%s: problem too large", what);
    return HLA2_OK;
}

// strides of operand i of `strides`, or those of a dense [B][H][T][d] (or [B][H][T]) tensor
void take_strides(long long (&s)[3], const long long* strides, int i, int H, int T, int d) {
    if (strides) {
        for (int k = 0; k < 3; ++k) s[k] = strides[3 * i + k];
    } else {
        s[0] = (long long)H * T * d; s[1] = (long long)T * d; s[2] = d;
    }
}


size_t lookback_bytes(int rows, int tiles, int cb) {
    if (tiles <= 1) return 0;
    return Lookback(rows, tiles, cb).words() * 8;
}

// Blocks of a kernel that fit the device at once, at most one to a tile.  What
// an SM holds is asked once for each kernel and device.
cudaError_t persistent_blocks(const void* kernel, int threads, size_t smem, unsigned total, unsigned* blocks) {
    static std::mutex mu;
    static std::map<std::pair<const void*, int>, unsigned> known;
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    unsigned fit = 0;
    {
        std::lock_guard<std::mutex> lk(mu);
        auto it = known.find({kernel, dev});
        if (it != known.end()) fit = it->second;
    }
    if (!fit) {
        if (smem)
            if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem))
                return e;
        int per_sm = 0;
        if (cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem)) return e;
        fit = (unsigned)(per_sm > 0 ? per_sm : 1) * (unsigned)sm_count();
        std::lock_guard<std::mutex> lk(mu);
        known[{kernel, dev}] = fit;
    }
    *blocks = total < fit ? total : fit;
    return cudaSuccess;
}

// Sets the workspace's words to "nothing yet".
cudaError_t begin_lookback(GateParams& p, int cb, void* workspace, cudaStream_t s) {
    p.total = (unsigned)((long long)p.B * p.H * p.tiles);
    if (p.tiles <= 1) return cudaSuccess;
    p.words = static_cast<unsigned long long*>(workspace);
    p.status = device_status_word();
    return cudaMemsetAsync(p.words, 0xff, Lookback(p.B * p.H, p.tiles, cb).words() * 8, s);
}

template <int N>
using Int = std::integral_constant<int, N>;

template <typename F>
cudaError_t by_lanes(int d, bool vec, F&& f) {
    using std::false_type;
    using std::true_type;
    if (d <= 64) return vec ? f(Int<16>{}, true_type{}) : f(Int<16>{}, false_type{});
    return vec ? f(Int<32>{}, true_type{}) : f(Int<32>{}, false_type{});
}

}  // namespace
}  // namespace hla2

extern "C" size_t hla2_gated_scan_workspace(int B, int H, int T, int d) {
    using namespace hla2;
    if (B <= 0 || H <= 0 || T <= 0 || d <= 0 || d > 128 || (long long)B * H > 65535) return 0;
    const int lanes = lanes_of(d), rows = B * H;
    return (lookback_bytes(rows, (T + tile_of(lanes) - 1) / tile_of(lanes), lanes * kCh) + 255) & ~size_t(255);
}

extern "C" size_t hla2_gated_scan_carry_len(int T, int d) {
    using namespace hla2;
    if (T <= 0 || d <= 0 || d > 128) return 0;
    const int kept = tile_of(lanes_of(d));
    return (size_t)((T + kept - 1) / kept) * d;
}

extern "C" int hla2_gated_scan(const void* X, const void* G, const unsigned char* reset, const float* state_in, void* O,
                               float* state_out, float* carry, int B, int H, int T, int d, const long long* strides,
                               int form, int gate_shared, int dtype, int out_dtype, void* workspace, size_t ws_bytes,
                               hla2_stream_t stream) {
    using namespace hla2;
    const char* what = "gated_scan";
    if (int rc = check_gated(what, B, H, T, d, form, dtype, out_dtype)) return rc;
    if (!X || !G || !O) return set_error(HLA2_ERR_INVALID, "%s: null pointer", what);
    const int es = dtype_size(dtype), os = dtype_size(out_dtype);
    if (!aligned_elem(X, es) || !aligned_elem(G, es) || !aligned_elem(O, os) || !aligned_elem(state_in, 4) ||
        !aligned_elem(state_out, 4) || !aligned_elem(carry, 4))
        return set_error(HLA2_ERR_INVALID, "%s: pointer not aligned to its element", what);
    const size_t need = hla2_gated_scan_workspace(B, H, T, d);
    if (need && (!workspace || ws_bytes < need))
        return set_error(HLA2_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", what, ws_bytes, need);
    if (need && reinterpret_cast<uintptr_t>(workspace) % 16)
        return set_error(HLA2_ERR_INVALID, "%s: workspace not 16-byte aligned", what);
    GateParams p{};
    p.x = X; p.g = G; p.reset = reset; p.state_in = state_in; p.o = O; p.state_out = state_out; p.carry = carry;
    p.B = B; p.H = H; p.T = T; p.d = d;
    take_strides(p.sx, strides, 0, H, T, d);
    take_strides(p.sg, strides, 1, H, T, gate_shared ? 1 : d);
    take_strides(p.so, strides, 2, H, T, d);
    const int lanes = lanes_of(d), tile = tile_of(lanes);
    p.tiles = (T + tile - 1) / tile;
    const bool vec = d % kCh == 0 && aligned_to(X, es, p.sx, 3, kCh * es) && aligned_to(O, os, p.so, 3, kCh * os) &&
                     (gate_shared || aligned_to(G, es, p.sg, 3, kCh * es));
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = begin_lookback(p, lanes * kCh, workspace, s);
    p.out_bf16 = out_dtype == HLA2_DTYPE_BF16;
    if (e == cudaSuccess) e = by_types(dtype, HLA2_DTYPE_F32, [&](auto tin, auto) {
        return by_form(form, gate_shared, [&](auto sig, auto shared) {
            return by_lanes(d, vec, [&](auto ln, auto v) {
                constexpr int threads = block_threads(decltype(ln)::value);
                auto kernel = gated_scan_kernel<decltype(tin), decltype(sig)::value, decltype(shared)::value,
                                                decltype(ln)::value, decltype(v)::value>;
                unsigned blocks = 0;
                if (cudaError_t e2 = persistent_blocks(reinterpret_cast<const void*>(kernel), threads, 0, p.total, &blocks)) return e2;
                kernel<<<blocks, threads, 0, s>>>(p);
                return cudaGetLastError();
            });
        });
    });
    note_launches(1);
    if (e != cudaSuccess) return set_error(HLA2_ERR_LAUNCH, "%s: %s", what, cudaGetErrorString(e));
    return HLA2_OK;
}

extern "C" int hla2_gated_scan_backward(const void* X, const void* G, const unsigned char* reset, const float* carry,
                                        const void* dO, const float* dstate_out, void* dX, void* dG, float* dstate_in,
                                        int B, int H, int T, int d, const long long* strides, int form, int gate_shared,
                                        int dtype, int out_dtype, void* workspace, size_t ws_bytes,
                                        hla2_stream_t stream) {
    using namespace hla2;
    const char* what = "gated_scan_backward";
    if (int rc = check_gated(what, B, H, T, d, form, dtype, out_dtype)) return rc;
    if (!X || !G || !carry || !dO || !dX || !dG) return set_error(HLA2_ERR_INVALID, "%s: null pointer", what);
    const int es = dtype_size(dtype), os = dtype_size(out_dtype);
    if (!aligned_elem(X, es) || !aligned_elem(G, es) || !aligned_elem(dX, es) || !aligned_elem(dG, es) ||
        !aligned_elem(dO, os) || !aligned_elem(carry, 4) || !aligned_elem(dstate_out, 4) || !aligned_elem(dstate_in, 4))
        return set_error(HLA2_ERR_INVALID, "%s: pointer not aligned to its element", what);
    const size_t need = hla2_gated_scan_workspace(B, H, T, d);
    if (need && (!workspace || ws_bytes < need))
        return set_error(HLA2_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", what, ws_bytes, need);
    if (need && reinterpret_cast<uintptr_t>(workspace) % 16)
        return set_error(HLA2_ERR_INVALID, "%s: workspace not 16-byte aligned", what);
    GateParams p{};
    p.x = X; p.g = G; p.reset = reset; p.carry = const_cast<float*>(carry); p.dout = dO; p.dstate_out = dstate_out;
    p.dx = dX; p.dg = dG; p.dstate_in = dstate_in;
    p.B = B; p.H = H; p.T = T; p.d = d;
    take_strides(p.sx, strides, 0, H, T, d);
    take_strides(p.sg, strides, 1, H, T, gate_shared ? 1 : d);
    take_strides(p.sdo, strides, 2, H, T, d);
    take_strides(p.sdx, strides, 3, H, T, d);
    take_strides(p.sdg, strides, 4, H, T, gate_shared ? 1 : d);
    const int lanes = lanes_of(d), tile = tile_of(lanes);
    p.tiles = (T + tile - 1) / tile;
    const bool vec = d % kCh == 0 && aligned_to(X, es, p.sx, 3, kCh * es) && aligned_to(dX, es, p.sdx, 3, kCh * es) &&
                     aligned_to(dO, os, p.sdo, 3, kCh * os) &&
                     (gate_shared || (aligned_to(G, es, p.sg, 3, kCh * es) && aligned_to(dG, es, p.sdg, 3, kCh * es)));
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = begin_lookback(p, lanes * kCh, workspace, s);
    if (e == cudaSuccess) e = by_types(dtype, out_dtype, [&](auto tin, auto tout) {
        return by_form(form, gate_shared, [&](auto sig, auto shared) {
            return by_lanes(d, vec, [&](auto ln, auto v) {
                auto kernel = gated_scan_bwd_kernel<decltype(tin), decltype(tout), decltype(sig)::value,
                                                    decltype(shared)::value, decltype(ln)::value, decltype(v)::value>;
                constexpr int threads = block_threads(decltype(ln)::value);
                constexpr size_t smem = (size_t)kTok * kData * sizeof(float4);
                unsigned blocks = 0;
                if (cudaError_t e2 = persistent_blocks(reinterpret_cast<const void*>(kernel), threads, smem, p.total, &blocks)) return e2;
                kernel<<<blocks, threads, smem, s>>>(p);
                return cudaGetLastError();
            });
        });
    });
    note_launches(1);
    if (e != cudaSuccess) return set_error(HLA2_ERR_LAUNCH, "%s: %s", what, cudaGetErrorString(e));
    return HLA2_OK;
}

extern "C" int hla2_gated_step(float* state, const void* x, const void* g, void* o, float* state_out, int n, int d,
                               const long long* ld, int form, int gate_shared, int dtype, int out_dtype,
                               hla2_stream_t stream) {
    using namespace hla2;
    const char* what = "gated_step";
    if (int rc = check_gated(what, 1, 1, n, d, form, dtype, out_dtype)) return rc;
    if (!state || !x || !g || !o) return set_error(HLA2_ERR_INVALID, "%s: null pointer", what);
    const int es = dtype_size(dtype), os = dtype_size(out_dtype);
    if (!aligned_elem(state, 4) || !aligned_elem(state_out, 4) || !aligned_elem(x, es) || !aligned_elem(g, es) ||
        !aligned_elem(o, os))
        return set_error(HLA2_ERR_INVALID, "%s: pointer not aligned to its element", what);
    if (!state_out) state_out = state;
    const long long ldx = ld ? ld[0] : d, ldg = ld ? ld[1] : gate_shared ? 1 : d, ldo = ld ? ld[2] : d;
    const bool vec = d % 4 == 0 && aligned_to(state, 4, nullptr, 0, 16) && aligned_to(state_out, 4, nullptr, 0, 16) &&
                     aligned_to(x, es, &ldx, 1, 4 * es) && aligned_to(o, os, &ldo, 1, 4 * os) &&
                     (gate_shared || aligned_to(g, es, &ldg, 1, 4 * es));
    const long long threads = (long long)n * (vec ? d / 4 : d);
    const unsigned grid = (unsigned)((threads + 255) / 256);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = by_types(dtype, out_dtype, [&](auto tin, auto tout) {
        return by_form(form, gate_shared, [&](auto sig, auto shared) {
            using T = decltype(tin);
            using TO = decltype(tout);
            if (vec)
                gated_step_kernel<T, TO, decltype(sig)::value, decltype(shared)::value, true><<<grid, 256, 0, s>>>(
                    state, static_cast<const T*>(x), static_cast<const T*>(g), static_cast<TO*>(o), state_out, n, d,
                    ldx, ldg, ldo);
            else
                gated_step_kernel<T, TO, decltype(sig)::value, decltype(shared)::value, false><<<grid, 256, 0, s>>>(
                    state, static_cast<const T*>(x), static_cast<const T*>(g), static_cast<TO*>(o), state_out, n, d,
                    ldx, ldg, ldo);
            return cudaGetLastError();
        });
    });
    note_launches(1);
    if (e != cudaSuccess) return set_error(HLA2_ERR_LAUNCH, "%s: %s", what, cudaGetErrorString(e));
    return HLA2_OK;
}
