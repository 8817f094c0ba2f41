// hla2_gated.cuh -- what the forward (hla2_gated.cu) and the gradient
// (hla2_gated_bwd.cu) of the gated linear recurrence share: the maps of runs of
// tokens, how tiles are joined through the workspace, and the host side.
#pragma once

#include <map>
#include <mutex>
#include <new>

#include "hla2_layer.cuh"
#include "hla2_tc_common.cuh"

namespace hla2 {
namespace {

constexpr int kTok = 8;         // tokens of a run
constexpr int kCh = 4;          // channels of a thread
constexpr int kData = 256;      // threads that share a tile: one to a run and four channels
constexpr int kGroup = 8;       // tiles to a group: a state is published at the end of each
constexpr unsigned long long kGateWaitNs = 2000000000ull;  // bounded waits: 2 s

// Lanes that share a token: they cover 4 channels each, d <= 4 lanes.
__host__ __device__ constexpr int lanes_of(int d) { return d <= 64 ? 16 : 32; }
// Tokens of a tile: a state is kept for the gradient at the start of each.
__host__ __device__ constexpr int tile_of(int lanes) { return kData / lanes * kTok; }
// Tiles of T > 0 tokens; T may be any int.
__host__ __device__ constexpr int tiles_of(int T, int tile) { return (T - 1) / tile + 1; }
// Threads of a block of the register kernels: those that hold the tile, and a warp for each 32 channels that joins tiles.
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
    unsigned long long per_rows, per_h;  // 2^64 / rows and 2^64 / H, for quotients
    int* status;
};

// The sigmoid gate is kept as the smaller of a = 1 / (1 + e^-g) and z = 1 - a, which
// is c = e / (1 + e) with e = e^-|g|, and its sign says which: c where it is a (g < 0),
// -c where it is z.  Either end keeps its relative precision: the long memory where a
// is next to 1, and what is left of the state and of the gate's gradient where a is
// next to 0.  Held as z alone, a = 1 - z was off by 1e-2 of itself at g = -12 and
// zero from -17 on.
//
// The power of two and the reciprocal are the approximate instructions (2 ulp and
// 1 ulp) without their handling of subnormal numbers: a c below 2^-126 is 0.  The
// rounding of g log2(e) adds |g| 2^-24 of c: what half a unit in the last place of an
// fp32 g makes of c, and 2^-15 of that for a 16-bit g.
__device__ __forceinline__ float sigmoid_gate(float g) {
    constexpr float kLog2e = 1.4426950408889634f;
    const float t = fabsf(g) * -kLog2e;
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return __uint_as_float(__float_as_uint(e * r) | (~__float_as_uint(g) & 0x80000000u));
}
__device__ __forceinline__ bool holds_z(float gate) { return (int)__float_as_uint(gate) < 0; }

// What a gate (a itself in the decay form) does to a state and to a decay.  The sigmoid
// form is a step from the nearer of x and h towards the other: x + a (h - x) or
// h + z (x - h).
template <bool SIG>
__device__ __forceinline__ float next_state(float gate, float h, float x) {
    return SIG ? fmaf(gate, h - x, holds_z(gate) ? h : x) : fmaf(gate, h, x);
}
template <bool SIG>
__device__ __forceinline__ float decayed(float gate, float v) {  // a v
    return SIG ? fmaf(gate, v, holds_z(gate) ? v : 0.f) : gate * v;
}
// One token of the gradient: lam = dh + mu -> dx, dg and the mu that reaches h_{t-1}.
template <bool SIG>
__device__ __forceinline__ void back_token(float gate, float lam, float before, float x, float& dx, float& dg, float& mu) {
    if (SIG) {
        const bool z = holds_z(gate);
        mu = fmaf(gate, lam, z ? lam : 0.f);    // a lam
        dx = fmaf(-gate, lam, z ? 0.f : lam);   // z lam
        dg = fabsf(gate) * (z ? mu : dx) * (before - x);
    } else {
        dx = lam;
        dg = lam * before;
        mu = gate * lam;
    }
}

// The pipelined kernels take the sigmoid gate as E = e^g, a = E / (1 + E), z = 1 / (1 + E):
// positive factors alone, so both keep their relative precision, and a run's map needs
// one quotient in all.  Over the tokens of a run D = prod (1 + E), P = prod E, and
//   X = N / D,  N -> E N + x D;      A = P / D = 1 - Q / D,  Q -> E Q + D;
// A is taken from the smaller of P and Q, so that a long memory's 1 - A is good to its
// own size and not to A's.  For the gradient Y = M / D, M -> (1 + E) M + P dh.
// Every token's E and 1 are scaled by 2^-6: D then holds for gates of 14 at every token
// of a run, and an A below 2^-78 loses bits.  A run of larger gates, with inf or NaN, or
// of inputs all below 2^-74 is walked with sigmoid_gate() instead.  Scan of
// 65536 x 16 x 128 with gates of 2 +- 1.5: 184 us, 9: 186, 12: 208, 14: 348 (unscaled,
// 9: 510).  Per element and token this takes 7.5 operations in the map and 7 in the walk
// that writes; sigmoid_gate() and its selections took 12 and 10, which made that scan
// 240 us.
// Two elements to an instruction (f32x2) halve that again.
template <int N, typename F>
__device__ __forceinline__ void by_pairs(float (&o)[N], const float (&a)[N], const float (&b)[N], const float (&c)[N], F&& f) {
    static_assert(N % 2 == 0, "pairs");
#pragma unroll
    for (int j = 0; j < N; j += 2) {
        unsigned long long x, y, z;
        asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a[j]), "f"(a[j + 1]));
        asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b[j]), "f"(b[j + 1]));
        asm("mov.b64 %0, {%1, %2};" : "=l"(z) : "f"(c[j]), "f"(c[j + 1]));
        asm("mov.b64 {%0, %1}, %2;" : "=f"(o[j]), "=f"(o[j + 1]) : "l"(f(x, y, z)));
    }
}
template <int N>
__device__ __forceinline__ void fmas(float (&o)[N], const float (&a)[N], const float (&b)[N], const float (&c)[N]) {
    using u = unsigned long long;
    by_pairs(o, a, b, c, [](u x, u y, u z) { u r; asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z)); return r; });
}
template <int N>
__device__ __forceinline__ void products(float (&o)[N], const float (&a)[N], const float (&b)[N]) {
    using u = unsigned long long;
    by_pairs(o, a, b, b, [](u x, u y, u) { u r; asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y)); return r; });
}
template <int N>
__device__ __forceinline__ void sums(float (&o)[N], const float (&a)[N], const float (&b)[N]) {
    using u = unsigned long long;
    by_pairs(o, a, b, b, [](u x, u y, u) { u r; asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y)); return r; });
}
template <int N>
__device__ __forceinline__ void fill(float (&o)[N], float v) {
#pragma unroll
    for (int j = 0; j < N; ++j) o[j] = v;
}
// Gates of a token: one for each channel, or a shared one twice, which is the pair that
// every pair of channels takes (formed for each use, the moves made the scan of
// 65536 x 16 x 128 with a shared gate 190 us for 174).
template <int N, int NG>
__device__ __forceinline__ void each(float (&o)[N], const float (&g)[NG]) {
    static_assert(NG == N || NG == 2, "gates of the channels, or a pair");
#pragma unroll
    for (int j = 0; j < N; ++j) o[j] = g[j % NG];
}

// e^g, or e^g 2^-6 where `scaled`
constexpr float kGateScale = 0x1p-6f;
template <int N>
__device__ __forceinline__ void gate_powers(float (&g)[N], bool scaled) {
    float l[N], shift[N];
    fill(l, 1.4426950408889634f);
    fill(shift, -6.f);
    if (scaled) fmas(g, g, l, shift);
    else products(g, g, l);
#pragma unroll
    for (int j = 0; j < N; ++j) {
        if (N == 2 && j) g[j] = g[0];
        else asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(g[j]) : "f"(g[j]));
    }
}
__device__ __forceinline__ float reciprocal(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
template <int N>
__device__ __forceinline__ void keeps(float (&z)[N], const float (&E)[N]) {  // 1 / (1 + E)
    float one[N];
    fill(one, 1.f);
    sums(z, E, one);
#pragma unroll
    for (int j = 0; j < N; ++j) z[j] = N == 2 && j ? z[0] : reciprocal(z[j]);
}
template <int NG>
struct Powers {
    float D[NG], P[NG], Q[NG];
    __device__ __forceinline__ Powers() {
        fill(D, 1.f);
        fill(P, 1.f);
        fill(Q, 0.f);
    }
    // a token, E scaled: X is N
    __device__ __forceinline__ void token(const float (&E)[NG], float (&X)[kCh], const float (&x)[kCh]) {
        float e[kCh], d[kCh], one[NG];
        fill(one, kGateScale);
        products(one, one, D);
        each(e, E);
        each(d, one);
        products(d, d, x);
        fmas(X, e, X, d);
        fmas(Q, E, Q, one);
        fmas(D, D, E, one);
        products(P, P, E);
    }
    // Y is M; u counts where `open`
    __device__ __forceinline__ void back_token(const float (&E)[NG], float (&Y)[kCh], const float (&u)[kCh], bool open) const {
        float e[kCh], q[kCh], one[kCh];
        each(e, E);
        each(q, P);
        fill(one, kGateScale);
        products(one, one, Y);
        fmas(Y, Y, e, one);
        if (open) fmas(Y, q, u, Y);
    }
    // N becomes X, and A is formed
    __device__ __forceinline__ void close(float (&X)[kCh], float (&A)[kCh]) const {
        float per[NG], a[NG], all[kCh];
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            per[j] = NG == 2 && j ? per[0] : reciprocal(D[j]);
            a[j] = P[j] < Q[j] ? P[j] * per[j] : fmaf(-Q[j], per[j], 1.f);
        }
        each(A, a);
        each(all, per);
        products(X, X, all);
    }
    __device__ __forceinline__ void close_back(float (&Y)[kCh]) const {  // M becomes Y
        float per[NG], all[kCh];
#pragma unroll
        for (int j = 0; j < NG; ++j) per[j] = NG == 2 && j ? per[0] : reciprocal(D[j]);
        each(all, per);
        products(Y, Y, all);
    }
};
// The largest and the smallest of |v| and what top and low are; NaN stays.
template <int N>
__device__ __forceinline__ void span(const float (&v)[N], float& top, float& low) {
#pragma unroll
    for (int j = 0; j < N; j += 2) {
        asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(top) : "f"(v[j]), "f"(v[j + 1]));
        asm("min.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(low) : "f"(v[j]), "f"(v[j + 1]));
    }
}
// Ranges of the D of a run of kTok tokens: below the first no E is above 2^126, below
// the second the products hold, but each E must be looked at.
constexpr float kSurely = 0x1p78f, kPerhaps = 0x1p120f, kLargestGate = 83.f;  // e^83 < 2^120
// At the other end N, M >= 2^-48 of X, Y.  Below the first of these they may lose 2^-149
// a token, 2^-98 of X and Y: a run's inputs above the second are 2^24 times that.
constexpr float kSmall = 0x1p-78f, kSmallInput = 0x1p-74f;

// A token with E: h -> a h + z x
template <int NG>
__device__ __forceinline__ void next_by_power(const float (&E)[NG], float (&h)[kCh], const float (&x)[kCh]) {
    float z[NG], a[NG], zs[kCh], as[kCh];
    keeps(z, E);
    products(a, E, z);
    each(zs, z);
    each(as, a);
    products(zs, zs, x);
    fmas(h, as, h, zs);
}
// One token of the gradient: lam = u + mu -> dx = z lam, mu = a lam, dg = a z lam (before - x)
template <int NG>
__device__ __forceinline__ void back_by_power(const float (&E)[NG], const float (&u)[kCh], const float (&before)[kCh],
                                              const float (&x)[kCh], float (&dx)[kCh], float (&dg)[kCh], float (&mu)[kCh]) {
    float z[NG], zs[kCh], es[kCh], minus[kCh];
    keeps(z, E);
    each(zs, z);
    each(es, E);
    sums(mu, u, mu);
    products(dx, zs, mu);
    products(mu, es, dx);
    products(dg, zs, mu);
    fill(minus, -1.f);
    fmas(minus, x, minus, before);
    products(dg, dg, minus);
}

// ---- maps h -> A h + X -------------------------------------------------------
// A run that holds a reset forgets what entered it: its A is -0, which nothing
// else is (a product that is zero is made +0, by an addition that may not be
// contracted with it: an fma of a negative product that underflows is -0), and then
// only X counts.
__device__ __forceinline__ float cut() { return __uint_as_float(0x80000000u); }
__device__ __forceinline__ bool is_cut(float A) { return __float_as_uint(A) == 0x80000000u; }
__device__ __forceinline__ float no_cut(float A) { return __fadd_rn(A, 0.f); }
__device__ __forceinline__ float pass(float2 m, float h) { return is_cut(m.x) ? m.y : fmaf(m.x, h, m.y); }
// first `a`, then `b`
__device__ __forceinline__ float2 then(float2 a, float2 b) {
    return make_float2(is_cut(b.x) || is_cut(a.x) ? cut() : no_cut(__fmul_rn(a.x, b.x)), pass(b, a.y));
}

// x / y for the y whose 2^64 / y (rounded up; 0 stands for y = 1) is `per`
__device__ __forceinline__ unsigned quotient(unsigned x, unsigned long long per) {
    return per ? (unsigned)__umul64hi((unsigned long long)x, per) : x;
}

// ---- the workspace -----------------------------------------------------------
// A ticket word and a word that says that a wait ran out; then the maps of the
// tiles (A, X for each of a row's channels), then the states that enter the groups
// (h, 0).  Each pair is one 64-bit word, written and read whole, so it is its own
// flag: the words are set to all ones before the launch, which no pair is
// (arithmetic gives one NaN, 0x7fffffff), and whoever needs one reads it until it
// is something else.
struct Lookback {
    int rows, tiles, groups, cb;  // cb: channels of a map
    __host__ __device__ Lookback(int rows, int tiles, int cb)
        : rows(rows), tiles(tiles), groups((tiles + kGroup - 1) / kGroup), cb(cb) {}
    __host__ __device__ size_t tile_map(int r, int t) const { return 1 + ((size_t)r * tiles + t) * cb; }
    __host__ __device__ size_t state(int r, int g) const { return tile_map(rows, 0) + ((size_t)r * groups + g) * cb; }
    __host__ __device__ size_t words() const { return state(rows, 0); }
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

// Reads w[i] = src[i * step] for i < n.
template <int N>
__device__ __forceinline__ void ask_words(const u64* src, size_t step, int n, u64 (&w)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = i < n ? ld_word(src + i * step) : 0;
}
// Reads those that were not there again until every one is.  Gives up after 2 s:
// then this call's results are void, the status word says so, and every later
// wait of the call ends at once.
template <int N>
__device__ __forceinline__ void wait_words(const GateParams& p, const u64* src, size_t step, u64 (&w)[N]) {
    u64 t0 = 0;
    for (unsigned tries = 1;; ++tries) {
        bool all = true;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (w[i] == kNothing) {
                w[i] = ld_word(src + i * step);
                all = all && w[i] != kNothing;
            }
        if (all) return;
        if (tries % 64 == 0) {
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
}

// Publishes one channel of a tile's map.  `n` counts tiles in the order of the walk.
__device__ __forceinline__ void publish_tile(const GateParams& p, const Lookback& lb, int row, int n, int ch, float2 m) {
    if (n + 1 < lb.tiles) st_pair(p.words + lb.tile_map(row, n) + ch, m);
}

// What enters tile n, for one channel.  First the maps w of the tiles of its group
// before it: `mapped()` is called between the first look at their words and the
// waiting for those that are missing; it waits for the tile's own map (false: give
// up), by which time the tiles before it have theirs too.  Polling from the start
// took more of the L2's bandwidth than the data.
template <typename F>
__device__ __forceinline__ bool maps_before(const GateParams& p, const Lookback& lb, int row, int n, int ch,
                                            u64 (&w)[kGroup - 1], F&& mapped) {
    const int nt = n % kGroup;
    const u64* const tiles = p.words + lb.tile_map(row, n - nt) + ch;
    ask_words(tiles, lb.cb, nt, w);
    if (!mapped()) return false;
    wait_words(p, tiles, lb.cb, w);
    return true;
}
__device__ __forceinline__ float2 compose(const u64 (&w)[kGroup - 1], int nt) {
    float2 m = make_float2(1.f, 0.f);
#pragma unroll
    for (int i = 0; i < kGroup - 1; ++i)
        if (i < nt) m = then(m, as_pair(w[i]));
    return m;
}
__device__ __forceinline__ float pass_all(const u64 (&w)[kGroup - 1], int nt, float h) {
#pragma unroll
    for (int i = 0; i < kGroup - 1; ++i)
        if (i < nt) h = pass(as_pair(w[i]), h);
    return h;
}
// Then the state that enters the group (`start` enters the sequence), waited for
// last: from group to group only this passes, so the tile that ends a group has
// composed all that it can before it comes.
__device__ __forceinline__ float group_state(const GateParams& p, const Lookback& lb, int row, int n, int ch,
                                             float start) {
    const int g = n / kGroup;
    if (g == 0) return start;
    u64 u[1];
    const u64* const state = p.words + lb.state(row, g) + ch;
    ask_words(state, 0, 1, u);
    wait_words(p, state, 0, u);
    return as_pair(u[0]).x;
}

__device__ __forceinline__ bool ends_group(const Lookback& lb, int n) {
    return n % kGroup == kGroup - 1 && n + 1 < lb.tiles;
}
// Publishes the state `h` after tile n where the tile ends a group.
__device__ __forceinline__ void publish_state(const GateParams& p, const Lookback& lb, int row, int n, int ch, float h) {
    if (ends_group(lb, n)) st_pair(p.words + lb.state(row, n / kGroup + 1) + ch, make_float2(h, 0.f));
}

// One channel's part in the register kernels: publishes the tile's map, returns the state that enters it.
__device__ __forceinline__ float join_tile(const GateParams& p, const Lookback& lb, int row, int n, int ch, float2 m,
                                           float start) {
    publish_tile(p, lb, row, n, ch, m);
    u64 w[kGroup - 1];
    maps_before(p, lb, row, n, ch, w, [] { return true; });
    const float h = pass_all(w, n % kGroup, group_state(p, lb, row, n, ch, start));
    publish_state(p, lb, row, n, ch, pass(m, h));
    return h;
}

// The tiles of a block, by ticket where tiles wait for one another.
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

// ---- the pipelined kernels ---------------------------------------------------
constexpr int kComposers = 64;  // threads that compose a tile's map
constexpr int kMostJoin = 3;    // sets of joiners, every so-many-th tile each
constexpr int kFar = 2;         // tiles are asked into L2 this many rounds of the grid ahead: 217 -> 203 us
constexpr unsigned kNapNs = 40;  // between two tries of a wait

// A tile in a stage, worked out once by the loader: n counts tiles in the order of
// the walk (-1: there is no further tile); t0 is its first token; the offsets are
// those of the tile's first element in each strided operand that is not loaded by
// tensor copies.
struct TileInfo {
    int n, row, b, t0;
    long long reset, g, o, o2;
};
// A role's place in the ring of stages.
template <int S, int STEP>
struct Ring {
    int s;
    uint32_t phase;
    __device__ explicit Ring(int first) : s(first), phase(0) {}
    __device__ void next() {
        s += STEP;
        if (s >= S) {
            s -= S;
            phase ^= 1u;
        }
    }
};

// Waits on a barrier of the block, at most 2 x kGateWaitNs (longer than a joiner
// waits for other blocks); false when that ran out, or when another wait of the
// block did.  Between two tries the warp sleeps, which leaves the issue slots to the
// warps that work.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
    if (mbar_try(bar, parity)) return *abort_flag == 0;
    unsigned long long t0 = 0;
    for (unsigned tries = 1;; ++tries) {
        __nanosleep(kNapNs);
        if (mbar_try(bar, parity)) return *abort_flag == 0;
        if (tries % 64 == 0) {
            if (*abort_flag) return false;
            const unsigned long long now = globaltimer();
            if (t0 == 0) t0 = now;
            if (now - t0 > 2 * kGateWaitNs) {
                *abort_flag = 1;
                atomicExch(status, (int)kDevWaitTimeout);
                return false;
            }
        }
    }
}
__device__ __forceinline__ void mbar_arrive(uint32_t a) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(a) : "memory");
}
__device__ __forceinline__ void tma_prefetch_l2_4d(const CUtensorMap* map, int x, int y, int z, int w) {
    asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global [%0, {%1, %2, %3, %4}];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w)
                 : "memory");
}

// The resets of a run of kTok tokens from t0 on, as bits, for the LANES lanes of a
// warp that share the run: each of the first kTok loads one byte.
template <int LANES>
__device__ __forceinline__ unsigned run_resets(const unsigned char* rp, int t0, int T) {
    const int lane = threadIdx.x & 31, i = lane % LANES;
    const bool r = i < kTok && t0 + i < T && rp[t0 + i];
    return (__ballot_sync(0xffffffffu, r) >> (lane - i)) & ((1u << kTok) - 1u);
}

// four channels of one token in shared memory, as fp32
__device__ __forceinline__ void four(const float* p, float (&v)[4]) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}
__device__ __forceinline__ void four(const bf16* p, float (&v)[4]) {
    const uint2 a = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(a.x << 16); v[1] = __uint_as_float(a.x & 0xffff0000u);
    v[2] = __uint_as_float(a.y << 16); v[3] = __uint_as_float(a.y & 0xffff0000u);
}

// ------------------------------------------------------------ host side ----
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


// The words, then room for the states that enter the sequences (begin_states).
size_t lookback_bytes(int rows, int tiles, int cb, int d) {
    if (tiles <= 1) return 0;
    return Lookback(rows, tiles, cb).words() * 8 + (size_t)rows * d * 4;
}

// The state that a call leaves may take the place of the one that enters, but not a part of it.
int check_states(const char* what, const float* in, const float* out, size_t n) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(in), b = reinterpret_cast<uintptr_t>(out), bytes = n * 4;
    if (in && out && a != b && a < b + bytes && b < a + bytes)
        return set_error(HLA2_ERR_INVALID, "%s: the state after overlaps the state before without being it", what);
    return HLA2_OK;
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
        try {
            std::lock_guard<std::mutex> lk(mu);
            known[{kernel, dev}] = fit;
        } catch (const std::bad_alloc&) {  // not remembered: nothing leaves a C entry as an exception
        }
    }
    *blocks = total < fit ? total : fit;
    return cudaSuccess;
}

// Sets the workspace's words to "nothing yet".
cudaError_t begin_lookback(GateParams& p, int cb, void* workspace, cudaStream_t s) {
    p.total = (unsigned)((long long)p.B * p.H * p.tiles);
    const auto per = [](unsigned long long y) { return y == 1 ? 0ull : ~0ull / y + 1; };
    p.per_rows = per((unsigned long long)p.B * p.H);
    p.per_h = per((unsigned long long)p.H);
    if (p.tiles <= 1) return cudaSuccess;
    p.words = static_cast<unsigned long long*>(workspace);
    return cudaMemsetAsync(p.words, 0xff, Lookback(p.B * p.H, p.tiles, cb).words() * 8, s);
}

// Where a call leaves its last state in the place of the one that enters, the tiles
// read a copy: a row's last tile waits for the other tiles' maps only, so it may be
// written before a tile of the first group has read what enters.  A row of one tile
// reads its state before it writes.
cudaError_t begin_states(const GateParams& p, int cb, void* workspace, const float** in, const float* out, cudaStream_t s) {
    if (!*in || *in != out || p.tiles <= 1) return cudaSuccess;
    const int rows = p.B * p.H;
    float* const copy = reinterpret_cast<float*>(static_cast<u64*>(workspace) + Lookback(rows, p.tiles, cb).words());
    const float* const from = *in;
    *in = copy;
    return cudaMemcpyAsync(copy, from, (size_t)rows * p.d * 4, cudaMemcpyDeviceToDevice, s);
}

template <int N>
using Int = std::integral_constant<int, N>;

template <typename F>
cudaError_t by_lanes(int d, F&& f) {
    return lanes_of(d) == 16 ? f(Int<16>{}) : f(Int<32>{});
}
template <typename F>
cudaError_t by_bool(bool v, F&& f) {
    return v ? f(std::true_type{}) : f(std::false_type{});
}

// A map of a strided [B][H][T][d] tensor, box of TILE tokens; false where its
// strides or address do not allow bulk tensor copies.
bool gate_map(CUtensorMap* m, const void* base, int es, const long long (&s)[3], int B, int H, int T, int d, int tile) {
    EncodeTiledFn fn = encode_fn();
    if (!fn || (reinterpret_cast<uintptr_t>(base) & 15u) || (d * es) % 16) return false;
    const int sizes[3] = {T, H, B};
    const long long st[3] = {s[2], s[1], s[0]};
    cuuint64_t strides[3];
    for (int i = 0; i < 3; ++i) {
        strides[i] = (cuuint64_t)(sizes[i] == 1 ? (long long)d * es : st[i] * es);  // a single index needs none
        if (sizes[i] > 1 && (st[i] <= 0 || (st[i] * es) % 16 || st[i] * es >= (1LL << 40))) return false;
    }
    const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)T, (cuuint64_t)H, (cuuint64_t)B};
    const cuuint32_t box[4] = {(cuuint32_t)d, (cuuint32_t)tile, 1, 1}, step[4] = {1, 1, 1, 1};
    return fn(m, es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4,
              const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

}  // namespace
}  // namespace hla2
