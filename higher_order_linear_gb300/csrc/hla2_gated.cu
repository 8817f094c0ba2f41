// hla2_gated.cu -- gated linear recurrence along the tokens of each head and
// channel: forward, gradient and the single-token step.
//
//   h_t = a_t h_{t-1} + u_t
//   decay:   a = g, u = x
//   sigmoid: a = 1 / (1 + e^-g), u = z x, z = 1 - a = 1 / (1 + e^g): each of a and
//            z keeps its relative precision, z where a is next to 1 (a long memory)
//            and a where it is next to 0 (what a closing gate leaves).
// A reset at t makes h_{t-1} zero there (chosen, not multiplied: nothing of an
// earlier document passes, not even inf or NaN).
//
// Gradient, lam_t = dh_t + a_{t+1} lam_{t+1}:
//   decay:   dx = lam,    dg = lam h_{t-1}
//   sigmoid: dx = z lam,  dg = a z lam (h_{t-1} - x)
//
// One pass over the data.  A run of tokens maps the state before it to the state
// after it by h -> A h + X, and such maps compose, so a tile of tokens can be read
// once, long before the state that enters it is known: the maps of its runs are
// composed to the tile's, which goes to the workspace; the state that enters the
// tile is the state that entered its group of 8 tiles, passed through the maps of
// the tiles before it in the group; and the tokens are walked again, on chip, from
// the state that enters each run.
//
// Tiles are taken by ticket, all heads' first tiles first, so whoever waits waits
// for a tile that a running block holds.  Which maps are passed, and in which
// order, depends on the tile's place alone: the same call gives the same bits,
// whatever the timing.  Along the sequence one state for each group is handed on.
//
// What bounds it.  Forward of 1 x 16 x 65536 x 128, 16-bit in, 32-bit out (1.07 GB,
// 158 us at the copy bandwidth of 6.8 TB/s): 185 us, 0.85 of it; 16-bit out
// (0.81 GB, 118 us): 174 us.  An earlier stand of the pipeline took 170 us with the
// waits between blocks left out: they cost the rest, by the way of a state from
// group to group, about 1.3 us a hop through L2, and by the maps to be read for
// each tile (groups of 6 tiles took 215 us where 8 took 200, 12 211 and 16 237, all
// before the last two steps below).  Steps, same sizes: a
// thread to a channel, token by token, 34.7 ms; tiles in registers, flags beside
// the maps, 0.78 ms; a map that is its own flag 0.48 ms; tiles by bulk copies into
// a ring and a warp to a role 0.33 ms; the gate as a power of two and a reciprocal
// 0.24 ms; joiners apart from composers, three sets of them, 0.20 ms; the state
// waited for last and handed on first 0.185 ms.
#include "hla2_gated.cuh"

namespace hla2 {
namespace {

// ---- forward in registers: operands that bulk tensor copies do not take ---------
// (strides or addresses that are no multiple of 16 bytes).  A block holds a tile in
// registers, 4 channels of 8 tokens to a thread; warps of their own join tiles, so
// that no thread holds its tokens and the maps of other tiles at once.
// LANES x 4 channels to a token, kData / LANES runs of kTok tokens to a tile.
template <typename T, bool SIG, bool SHARED, int LANES>
__global__ void __launch_bounds__(block_threads(LANES), 1)
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
            if (p.words) h = join_tile(p, lb, row, n, ch, m, h);
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
        Run<T, SHARED, false> in;
        in.load(p, b, hd, t0, c, nc, nt);
        float gate[kTok][NG];
        float A[kCh], X[kCh];
#pragma unroll
        for (int j = 0; j < kCh; ++j) { A[j] = 1.f; X[j] = 0.f; }
#pragma unroll
        for (int i = 0; i < kTok; ++i)
            if (i < nt) {
#pragma unroll
                for (int j = 0; j < NG; ++j) gate[i][j] = SIG ? sigmoid_gate(in.g[i].get(j)) : in.g[i].get(j);
#pragma unroll
                for (int j = 0; j < kCh; ++j) {
                    const float ga = gate[i][SHARED ? 0 : j], xv = in.x[i].get(j);
                    if (in.reset(i)) X[j] = 0.f;
                    X[j] = next_state<SIG>(ga, X[j], xv);
                    A[j] = decayed<SIG>(ga, A[j]);
                }
            }
#pragma unroll
        for (int j = 0; j < kCh; ++j) runs[run][c + j] = make_float2(in.resets ? cut() : no_cut(A[j]), X[j]);
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
                        h[j] = next_state<SIG>(ga, h[j], xv);
                    }
                    if (p.out_bf16) {
                        Lane<bf16, kCh, false> ov;
                        ov.set(h);
                        ov.store(static_cast<bf16*>(p.o) + off + i * p.so[2], nc);
                    } else {
                        Lane<float, kCh, false> ov;
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


// ---- the pipelined forward -----------------------------------------------------
// One block to an SM and a ring of tiles in shared memory, so that several tiles
// of a block wait for the states that enter them while others are loaded,
// mapped and written.  Warps have one role each and meet on mbarriers:
//   loader   takes tickets and loads tiles of x (and gates) by bulk tensor copies;
//   mappers  form the maps of the tile's runs;
//   composers compose them to the tile's map and publish it;
//   joiners  (three sets, every third tile each: one waits about 3 us for other
//            blocks, a tile has 1.5 us) find the state that enters the tile, hand on
//            the one that leaves a group, and leave in each run's entry the state
//            that enters it;
//   writers  walk the runs again and write the outputs.
// Every wait is bounded in time, as in the other kernels of this library.

template <typename T, bool SHARED, int LANES>
struct PipeLayout {
    static constexpr int CB = LANES * kCh, RUNS = kData / LANES, TILE = RUNS * kTok;
    static constexpr uint32_t kTileBytes = TILE * CB * sizeof(T);  // of x, and of the gates
    static constexpr uint32_t kMaps = RUNS * CB * 8;
    static constexpr uint32_t kStage = kTileBytes * (SHARED ? 1 : 2);
    // The maps of a tile live from its mapping to its writing, a part of the time
    // that its data does: they have a ring of their own, of fewer slots.
    static constexpr int kSlots = sizeof(T) == 2 ? 4 : 2;
    static constexpr int kFit = (int)((225 * 1024 - kMaps * kSlots) / kStage);
    static constexpr int kStages = kFit > 8 ? 8 : kFit;
    static constexpr uint32_t kBytes = kStage * kStages + kMaps * kSlots + 128;  // and alignment to 128 bytes
    static constexpr int kJoin = kSlots < kMostJoin ? kSlots : kMostJoin;
    static constexpr int kThreads = 32 + kData + kJoin * CB + kComposers + kData;
};

template <typename T, bool SIG, bool SHARED, int LANES>
__global__ void __launch_bounds__(PipeLayout<T, SHARED, LANES>::kThreads, 1)
gated_pipe_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mg, const GateParams p) {
    using LY = PipeLayout<T, SHARED, LANES>;
    constexpr int CB = LY::CB, RUNS = LY::RUNS, TILE = LY::TILE, S = LY::kStages, M = LY::kSlots, kJoin = LY::kJoin;
    extern __shared__ __align__(128) unsigned char raw[];
    __shared__ __align__(8) unsigned long long bars[5 * S + 2 * M];
    static_assert(S >= kJoin, "the ends of the tickets take a stage for each group of joiners");
    __shared__ TileInfo info[S];
    __shared__ unsigned reset_bits[S][RUNS];
    __shared__ unsigned wide[S][kData / 32];  // lanes whose runs leave the range of Powers, for each warp
    __shared__ volatile int abort_flag;
    unsigned char* const base = raw + ((128u - (smem_u32(raw) & 127u)) & 127u);
    const int tid = threadIdx.x, warp = tid >> 5;
    auto full = [&](int s) { return smem_u32(&bars[s]); };            // the tile is loaded
    auto mapped = [&](int s) { return smem_u32(&bars[S + s]); };      // its runs' maps and its own are there
    auto joined = [&](int s) { return smem_u32(&bars[2 * S + s]); };  // the states that enter its runs are there
    auto empty = [&](int s) { return smem_u32(&bars[3 * S + s]); };   // its outputs are written
    auto known = [&](int s) { return smem_u32(&bars[4 * S + s]); };   // the stage's next tile is known
    auto sx = [&](int s) { return reinterpret_cast<T*>(base + (size_t)s * LY::kStage); };
    auto sg = [&](int s) { return reinterpret_cast<T*>(base + (size_t)s * LY::kStage + LY::kTileBytes); };
    auto maps = [&](int m) { return reinterpret_cast<float2*>(base + (size_t)S * LY::kStage + m * LY::kMaps); };
    auto runs = [&](int m) { return smem_u32(&bars[5 * S + m]); };      // every mapper's runs are mapped
    auto taken = [&](int m) { return smem_u32(&bars[5 * S + M + m]); };  // the slot's maps have been read
    if (tid == 0) {
        abort_flag = 0;
        for (int s = 0; s < S; ++s) {
            mbar_init(full(s), 1);
            mbar_init(mapped(s), kComposers / 32);
            mbar_init(joined(s), CB / 32);
            mbar_init(empty(s), kData / 32);
            mbar_init(known(s), 1);
        }
        for (int m = 0; m < M; ++m) {
            mbar_init(runs(m), kData / 32);
            mbar_init(taken(m), kData / 32);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    auto wait = [&](uint32_t bar, uint32_t parity) { return bar_wait(bar, parity, &abort_flag, p.status); };
    const int rows = p.B * p.H;
    const Lookback lb(rows, p.tiles, CB);
    auto place = [&](unsigned k, int& n, int& row, int& b, int& hd) {
        n = (int)quotient(k, p.per_rows);
        row = (int)(k - (unsigned)n * (unsigned)rows);
        b = (int)quotient((unsigned)row, p.per_h);
        hd = row - b * p.H;
    };
    if (warp == 0) {  // loader
        if (tid != 0) return;
        int n, row, b, hd;
        Tickets tickets{reinterpret_cast<unsigned*>(p.words), nullptr};
        LoadLedger<S> loads(full(0));
        // Tickets come in order, so the tiles of the rounds ahead are known: each block
        // asks L2 for as many tiles as it loads, whichever block will load them.
        auto ask = [&](unsigned long long k) {
            if (k >= p.total) return;
            place((unsigned)k, n, row, b, hd);
            tma_prefetch_l2_4d(&mx, 0, n * TILE, hd, b);
            if (!SHARED) tma_prefetch_l2_4d(&mg, 0, n * TILE, hd, b);
        };
        for (int r = 1; r < kFar; ++r) ask((unsigned long long)r * gridDim.x + blockIdx.x);
        unsigned next = p.words ? tickets.take(0) : blockIdx.x;
        int ends = 0;
        for (Ring<S, 1> at(0); ends < kJoin; at.next()) {
            const int s = at.s;
            const unsigned k = next;
            if (!wait(empty(s), at.phase ^ 1u)) break;
            if (k >= p.total) {  // one end to each group of joiners
                info[s].n = -1;
                mbar_arrive(known(s));
                mbar_arrive(full(s));
                ++ends;
                continue;
            }
            place(k, n, row, b, hd);
            const long long t = (long long)n * TILE;
            info[s] = TileInfo{n, row, b, n * TILE, (long long)b * p.T, b * p.sg[0] + hd * p.sg[1] + t * p.sg[2],
                               b * p.so[0] + hd * p.so[1] + t * p.so[2], 0};
            mbar_arrive(known(s));
            loads.note(s);
            mbar_expect_tx(full(s), (uint32_t)(TILE * p.d * sizeof(T)) * (SHARED ? 1u : 2u));
            tma_load_4d(smem_u32(sx(s)), &mx, 0, n * TILE, hd, b, full(s));
            if (!SHARED) tma_load_4d(smem_u32(sg(s)), &mg, 0, n * TILE, hd, b, full(s));
            ask((unsigned long long)kFar * gridDim.x + k);
            // a ticket held longer than it must be holds up the tiles after it in its row
            next = tickets.take(k);
        }
        if (abort_flag && !loads.settle()) atomicExch(p.status, (int)kDevWaitTimeout);
        return;
    }
    constexpr int kFirstJoiner = 32 + kData, kFirstComposer = kFirstJoiner + kJoin * CB;
    if (tid >= kFirstJoiner && tid < kFirstComposer) {  // joiners
        const int j = (tid - kFirstJoiner) / CB, ch = tid - kFirstJoiner - j * CB;
        Ring<M, kJoin> slot(j);
        for (Ring<S, kJoin> at(j);; at.next(), slot.next()) {
            const int s = at.s;
            if (!wait(known(s), at.phase)) return;
            const int n = info[s].n, row = info[s].row;
            if (n >= 0) {
                const float start = p.state_in && ch < p.d ? p.state_in[(long long)row * p.d + ch] : 0.f;
                const auto own = [&] { return wait(mapped(s), at.phase); };
                float2 f[RUNS];
                u64 w[kGroup - 1];
                if (!(p.words ? maps_before(p, lb, row, n, ch, w, own) : own())) return;
                float2* m = maps(slot.s) + ch;
#pragma unroll
                for (int r = 0; r < RUNS; ++r) f[r] = m[r * CB];
                float h = start;
                if (p.words && ends_group(lb, n)) {
                    float2 all = compose(w, kGroup - 1);
#pragma unroll
                    for (int r = 0; r < RUNS; ++r) all = then(all, f[r]);
                    h = group_state(p, lb, row, n, ch, start);
                    publish_state(p, lb, row, n, ch, pass(all, h));  // first: tiles of other blocks wait for it
                } else if (p.words) {
                    h = group_state(p, lb, row, n, ch, start);
                }
                if (p.words) h = pass_all(w, n % kGroup, h);
                if (p.carry && ch < p.d) p.carry[((long long)row * p.tiles + n) * p.d + ch] = h;
#pragma unroll
                for (int r = 0; r < RUNS; ++r) {
                    m[r * CB].x = h;
                    h = pass(f[r], h);
                }
            }
            __syncwarp();
            if ((tid & 31) == 0) mbar_arrive(joined(s));
            if (n < 0) return;
        }
    }
    if (tid >= kFirstComposer && tid < kFirstComposer + kComposers) {  // composers: N channels to a thread
        constexpr int N = CB / kComposers;
        const int ch = (tid - kFirstComposer) * N;
        Ring<M, 1> slot(0);
        for (Ring<S, 1> at(0);; at.next(), slot.next()) {
            const int s = at.s;
            if (!wait(known(s), at.phase)) return;
            const int n = info[s].n, row = info[s].row;
            if (n < 0) return;
            if (!wait(runs(slot.s), slot.phase)) return;
            if (p.words && n + 1 < p.tiles) {
                float2 m[N];
#pragma unroll
                for (int r = 0; r < RUNS; ++r)
#pragma unroll
                    for (int q = 0; q < N; ++q) {
                        const float2 f = maps(slot.s)[r * CB + ch + q];
                        m[q] = r ? then(m[q], f) : f;
                    }
#pragma unroll
                for (int q = 0; q < N; ++q) publish_tile(p, lb, row, n, ch + q, m[q]);
            }
            __syncwarp();
            if ((tid & 31) == 0) mbar_arrive(mapped(s));
        }
    }
    const bool mapper = warp < 1 + kData / 32;
    const int at = mapper ? tid - 32 : tid - (LY::kThreads - kData);
    const int lane = at % LANES, run = at / LANES;
    const int c = lane * kCh, nc = p.d - c;
    constexpr int NG = SHARED ? 2 : kCh;
    Ring<M, 1> slot(0);
    for (Ring<S, 1> ring(0);; ring.next(), slot.next()) {
        const int s = ring.s;
        const uint32_t phase = ring.phase;
        if (!wait(mapper ? known(s) : joined(s), phase)) return;
        const int n = info[s].n;
        if (n < 0) return;
        const int t0 = info[s].t0 + run * kTok;
        const int nt = nc > 0 ? min(kTok, p.T - t0) : 0;
        unsigned resets = 0;  // asked for while the tile is loaded
        if (p.reset) {
            if (mapper) {
                resets = run_resets<LANES>(p.reset + info[s].reset, t0, p.T);
                if (lane == 0) reset_bits[s][run] = resets;
            } else {
                resets = reset_bits[s][run];
            }
        }
        if (!wait(full(s), phase)) return;
        const T* xs = sx(s) + run * kTok * p.d + c;
        const T* gs = sg(s) + run * kTok * p.d + c;
        const T* gp = static_cast<const T*>(p.g) + info[s].g + run * kTok * p.sg[2];
        float gl[SHARED ? kTok : 1];
        if (SHARED) {
#pragma unroll
            for (int i2 = 0; i2 < kTok; ++i2)
                if (i2 < nt) gl[i2] = to_f32(gp[i2 * p.sg[2]]);
        }
        auto gates_of = [&](int i2, float (&ga)[NG]) {
            if constexpr (SHARED) ga[0] = ga[1] = gl[i2];
            else four(gs + i2 * p.d, ga);
        };
        auto gates = [&](int i2, float (&ga)[NG], bool by_power) {  // e^g, or gates as next_state() takes them
            gates_of(i2, ga);
            if (!SIG) return;
            if (by_power) {
                gate_powers(ga, mapper);
                return;
            }
#pragma unroll
            for (int j = 0; j < NG; ++j) ga[j] = sigmoid_gate(ga[j]);
        };
        if (mapper) {
            float A[kCh], X[kCh];
            // whole: a run of kTok tokens; clean: one without resets
            auto walk = [&](auto whole, auto clean) {
#pragma unroll
                for (int j = 0; j < kCh; ++j) { A[j] = 1.f; X[j] = 0.f; }
#pragma unroll(SIG && !SHARED ? 1 : kTok)
                for (int i2 = 0; i2 < kTok; ++i2)
                    if (whole || i2 < nt) {
                        float xv[kCh], ga[NG];
                        four(xs + i2 * p.d, xv);
                        gates(i2, ga, false);
#pragma unroll
                        for (int j = 0; j < kCh; ++j) {
                            const float gate = ga[SHARED ? 0 : j];
                            if (!clean && ((resets >> i2) & 1u)) X[j] = 0.f;
                            X[j] = next_state<SIG>(gate, X[j], xv[j]);
                            A[j] = decayed<SIG>(gate, A[j]);
                        }
                    }
            };
            auto powers = [&](auto whole, auto clean) {  // false: out of range
                Powers<NG> w;
#pragma unroll
                for (int j = 0; j < kCh; ++j) X[j] = 0.f;
#pragma unroll
                for (int i2 = 0; i2 < kTok; ++i2)
                    if (whole || i2 < nt) {
                        float xv[kCh], E[NG];
                        four(xs + i2 * p.d, xv);
                        gates(i2, E, true);
                        if (!clean && ((resets >> i2) & 1u)) fill(X, 0.f);
                        w.token(E, X, xv);
                    }
                float d = 0.f, top = 0.f, low = INFINITY, any = 0.f;
                span(w.D, d, any);
                span(X, top, low);
                bool in = d < kPerhaps && top < INFINITY;
                if (in && !(d < kSurely && low >= kSmall)) {  // looked at closer
                    float gate = 0.f, x = 0.f;
#pragma unroll 1
                    for (int i2 = 0; i2 < nt; ++i2) {
                        float xv[kCh], ga[NG];
                        four(xs + i2 * p.d, xv);
                        span(xv, x, any);
                        if constexpr (SHARED) ga[0] = ga[1] = to_f32(gp[i2 * p.sg[2]]);
                        else four(gs + i2 * p.d, ga);
#pragma unroll
                        for (int j = 0; j < NG; ++j) gate = fmaxf(gate, ga[j]);
                    }
                    in = gate < kLargestGate && (x == 0.f || x >= kSmallInput);
                }
                w.close(X, A);
                return in;
            };
            using yes = std::true_type;
            using no = std::false_type;
            if constexpr (SIG) {
                const bool in = nt == kTok && resets == 0 ? powers(yes{}, yes{})
                                : nt == kTok              ? powers(yes{}, no{})
                                                          : powers(no{}, no{});
                if (!in) walk(no{}, no{});
                const unsigned out = __ballot_sync(0xffffffffu, !in);
                if ((tid & 31) == 0) wide[s][at >> 5] = out;
            } else {
                if (nt == kTok && resets == 0) walk(yes{}, yes{});
                else if (nt == kTok) walk(yes{}, no{});
                else walk(no{}, no{});
            }
            if (!wait(taken(slot.s), slot.phase ^ 1u)) return;
            float4* m4 = reinterpret_cast<float4*>(maps(slot.s) + run * CB + c);
#pragma unroll
            for (int j = 0; j < kCh; ++j) A[j] = resets ? cut() : no_cut(A[j]);
            m4[0] = make_float4(A[0], X[0], A[1], X[1]);
            m4[1] = make_float4(A[2], X[2], A[3], X[3]);
            __syncwarp();
            if ((tid & 31) == 0) mbar_arrive(runs(slot.s));
        } else {
            float h[kCh];
            const float4* m4 = reinterpret_cast<const float4*>(maps(slot.s) + run * CB + c);
            const float4 lo = m4[0], hi = m4[1];
            h[0] = lo.x; h[1] = lo.z; h[2] = hi.x; h[3] = hi.z;
            __syncwarp();
            if ((tid & 31) == 0) mbar_arrive(taken(slot.s));
            const long long off = info[s].o + run * kTok * p.so[2] + c;
            auto walk = [&](auto whole, auto clean, auto by_power, auto* o) {
#pragma unroll(!SIG || SHARED || by_power ? kTok : 1)
                for (int i2 = 0; i2 < kTok; ++i2)
                    if (whole || i2 < nt) {
                        float xv[kCh], ga[NG];
                        four(xs + i2 * p.d, xv);
                        gates(i2, ga, by_power);
                        if (!clean && ((resets >> i2) & 1u)) fill(h, 0.f);
                        if (by_power) {
                            next_by_power(ga, h, xv);
                        } else {
#pragma unroll
                            for (int j = 0; j < kCh; ++j) h[j] = next_state<SIG>(ga[SHARED ? 0 : j], h[j], xv[j]);
                        }
                        Lane<std::remove_pointer_t<decltype(o)>, kCh, true> ov;
                        ov.set(h);
                        ov.store(o + off + i2 * p.so[2], nc);
                    }
            };
            auto go = [&](auto* o) {
                using power = std::integral_constant<bool, SIG>;
                using yes = std::true_type;
                using no = std::false_type;
                if (SIG && wide[s][at >> 5]) walk(no{}, no{}, no{}, o);
                else if (nt == kTok && resets == 0) walk(yes{}, yes{}, power{}, o);
                else if (nt == kTok) walk(yes{}, no{}, power{}, o);
                else walk(no{}, no{}, power{}, o);
            };
            if (p.out_bf16) go(static_cast<bf16*>(p.o));
            else go(static_cast<float*>(p.o));
            const int row = info[s].row;
            __syncwarp();
            if ((tid & 31) == 0) mbar_arrive(empty(s));
            if (p.state_out && nt > 0 && t0 + nt == p.T)
                *reinterpret_cast<float4*>(p.state_out + (long long)row * p.d + c) = make_float4(h[0], h[1], h[2], h[3]);
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
        out[j] = next_state<SIG>(SIG ? sigmoid_gate(gate) : gate, h.get(j), xv.get(j));
    }
    h.set(out);
    h.store(state_out + row * d + c, N);
    Lane<TO, N, VEC> ov;
    ov.set(out);
    ov.store(o + row * ldo + c, N);
}


}  // namespace
}  // namespace hla2

extern "C" size_t hla2_gated_scan_workspace(int B, int H, int T, int d) {
    using namespace hla2;
    if (B <= 0 || H <= 0 || T <= 0 || d <= 0 || d > 128 || (long long)B * H > 65535) return 0;
    const int lanes = lanes_of(d), rows = B * H;
    return (lookback_bytes(rows, tiles_of(T, tile_of(lanes)), lanes * kCh, d) + 255) & ~size_t(255);
}

extern "C" size_t hla2_gated_scan_carry_len(int T, int d) {
    using namespace hla2;
    if (T <= 0 || d <= 0 || d > 128) return 0;
    return (size_t)tiles_of(T, tile_of(lanes_of(d))) * d;
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
    if (int rc = check_states(what, state_in, state_out, (size_t)B * H * d)) return rc;
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
    p.tiles = tiles_of(T, tile);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    p.status = device_status_word();  // where a wait that runs out is reported
    if (!p.status) return set_error(HLA2_ERR_LAUNCH, "%s: cannot resolve the device status word", what);
    cudaError_t e = begin_lookback(p, lanes * kCh, workspace, s);
    if (e == cudaSuccess) e = begin_states(p, lanes * kCh, workspace, &p.state_in, state_out, s);
    p.out_bf16 = out_dtype == HLA2_DTYPE_BF16;
    CUtensorMap mx{}, mg{};
    const bool pipe = gate_map(&mx, X, es, p.sx, B, H, T, d, tile) &&
                      (gate_shared || gate_map(&mg, G, es, p.sg, B, H, T, d, tile)) && d % kCh == 0 &&
                      aligned_to(O, os, p.so, 3, kCh * os) && aligned_to(state_out, 4, nullptr, 0, 16);
    if (e == cudaSuccess) e = by_types(dtype, HLA2_DTYPE_F32, [&](auto tin, auto) {
        return by_form(form, gate_shared, [&](auto sig, auto shared) {
            return by_lanes(d, [&](auto ln) {
                using T_ = decltype(tin);
                constexpr bool SIG = decltype(sig)::value, SHARED = decltype(shared)::value;
                constexpr int LANES = decltype(ln)::value;
                unsigned blocks = 0;
                if (pipe) {
                    using LY = PipeLayout<T_, SHARED, LANES>;
                    auto kernel = gated_pipe_kernel<T_, SIG, SHARED, LANES>;
                    if (cudaError_t e2 = persistent_blocks(reinterpret_cast<const void*>(kernel), LY::kThreads, LY::kBytes, p.total, &blocks)) return e2;
                    kernel<<<blocks, LY::kThreads, LY::kBytes, s>>>(mx, mg, p);
                } else {
                    constexpr int threads = block_threads(LANES);
                    auto kernel = gated_scan_kernel<T_, SIG, SHARED, LANES>;
                    if (cudaError_t e2 = persistent_blocks(reinterpret_cast<const void*>(kernel), threads, 0, p.total, &blocks)) return e2;
                    kernel<<<blocks, threads, 0, s>>>(p);
                }
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
    if (int rc = check_states(what, state, state_out, (size_t)n * d)) return rc;
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
