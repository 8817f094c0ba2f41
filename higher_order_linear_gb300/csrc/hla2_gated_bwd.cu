// hla2_gated_bwd.cu -- gradient of the gated linear recurrence (hla2_gated.cu).
//
//   lam_t = dh_t + a_{t+1} lam_{t+1}
//   decay:   dx = lam,    dg = lam h_{t-1}
//   sigmoid: dx = z lam,  dg = a z lam (h_{t-1} - x),  z = 1 - a
//
// The forward's walk from the last tile to the first, for mu_t = a_t lam_t, the part
// of the gradient that reaches h_{t-1}: mu_t = a_t (dh_t + mu_{t+1}), so a run maps
// the mu behind it to the mu before it by the same A and a Y of its own, and tiles
// are joined by the same workspace.  The states inside a tile are formed anew from
// x, the gates and the state that the forward kept at its beginning (fp32): they
// need no rounding to 16 bits, and reading x costs what reading h would.
//
// What bounds it.  4 x 16 x 4096 x 64, 16 bits (168 MB, 25 us at the copy
// bandwidth): 60 us; with the forward (100 MB, 15 us) of 36 us a training pass
// takes 94 us (129 with sigmoid_gate() throughout).  A tile is on chip for about 7 us
// (loads 0.8, mapping 1.0, waiting for tiles of other blocks 2.6, writing 1.7) and
// shared memory holds three, so one leaves every 2.5 to 2.9 us against 1.8 us for its
// bytes; a launch of 13 tiles to an SM also pays for the filling and emptying of that
// pipeline.  In registers, without the ring and with wide accesses: about 85 us.  Tried
// and left out, when the writers still kept a run's gates: a fourth stage, with h_{t-1}
// in the place of the 16-bit x and gate (62 us for 56: they then kept x as loaded too,
// and spilled more than the stage gave).
#include "hla2_gated.cuh"

namespace hla2 {
namespace {

// ---- gradient in registers: fp32 operands, and those that bulk tensor copies do
// not take.  A tile of fp32 x, gates and dh leaves no room for a second one in
// shared memory.  A thread's h_{t-1} wait in shared memory until its way back.
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
            if (p.words) mu = join_tile(p, lb, row, n, ch, m, mu);
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
        for (int i = kTok - 1; i >= 0; --i)
            if (i < nt) {
#pragma unroll
                for (int j = 0; j < kCh; ++j) {
                    const float ga = gate[i][SHARED ? 0 : j], lam = dh[i].get(j) + Y[j];
                    Y[j] = in.reset(i) ? 0.f : decayed<SIG>(ga, lam);
                }
            }
#pragma unroll
        for (int j = 0; j < kCh; ++j) {
            const float a = in.resets ? cut() : no_cut(A[j]);
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
                        h[j] = next_state<SIG>(ga, h[j], xv);
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
                    back_token<SIG>(ga, lam, hb[j], in.x[i].get(j), gx[j], gg[j], mu[j]);
                    if (in.reset(i)) mu[j] = 0.f;
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


// ---- the pipelined gradient (16-bit x and gates) --------------------------------
// The forward's pipeline (hla2_gated.cu) over tiles of x, gates and dh.  A run's
// entry is (A, X, Y); the joiners wait for the mu behind the tile and read the
// kept state that enters it, and leave in X and Y what enters each run from
// either side.  A writer's thread walks its run forwards, leaving h_{t-1} in
// shared memory and the gates in registers, and then backwards.
template <typename TO, bool SHARED, int LANES>
struct BackLayout {
    static constexpr int CB = LANES * kCh, RUNS = kData / LANES, TILE = RUNS * kTok;
    static constexpr uint32_t kTileBytes = TILE * CB * 2, kUpBytes = TILE * CB * sizeof(TO);
    static constexpr uint32_t kPlane = RUNS * CB * 4;  // of A, of X, of Y
    static constexpr uint32_t kStage = kTileBytes * (SHARED ? 1 : 2) + kUpBytes + 3 * kPlane;
    static constexpr uint32_t kBefore = kTok * kData * 16;
    static constexpr int kFit = (int)((222 * 1024 - kBefore) / kStage);
    static constexpr int kStages = kFit > 6 ? 6 : kFit;
    static constexpr uint32_t kBytes = kStage * kStages + kBefore + 128;
    static constexpr int kJoin = 2;  // as many as the smallest ring has stages
    static constexpr int kThreads = 32 + kData + kJoin * CB + kComposers + kData;
};

template <typename TO, bool SIG, bool SHARED, int LANES>
__global__ void __launch_bounds__(BackLayout<TO, SHARED, LANES>::kThreads, 1)
gated_pipe_bwd_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mg,
                      const __grid_constant__ CUtensorMap mu_, const GateParams p) {
    using T = bf16;
    using LY = BackLayout<TO, SHARED, LANES>;
    constexpr int CB = LY::CB, RUNS = LY::RUNS, TILE = LY::TILE, S = LY::kStages, kJoin = LY::kJoin, NG = SHARED ? 2 : kCh;
    extern __shared__ __align__(128) unsigned char raw[];
    __shared__ __align__(8) unsigned long long bars[6 * S];
    static_assert(S >= kJoin, "the ends of the tickets take a stage for each group of joiners");
    __shared__ TileInfo info[S];
    __shared__ unsigned reset_bits[S][RUNS];
    __shared__ unsigned wide[S][kData / 32];  // lanes whose runs leave the range of Powers, for each warp
    __shared__ volatile int abort_flag;
    unsigned char* const base = raw + ((128u - (smem_u32(raw) & 127u)) & 127u);
    float4* const before = reinterpret_cast<float4*>(base + (size_t)LY::kStage * S);  // [kTok][kData]: h_{t-1}
    const int tid = threadIdx.x, warp = tid >> 5;
    auto full = [&](int s) { return smem_u32(&bars[s]); };
    auto mapped = [&](int s) { return smem_u32(&bars[S + s]); };
    auto joined = [&](int s) { return smem_u32(&bars[2 * S + s]); };
    auto empty = [&](int s) { return smem_u32(&bars[3 * S + s]); };
    auto runs = [&](int s) { return smem_u32(&bars[4 * S + s]); };
    auto known = [&](int s) { return smem_u32(&bars[5 * S + s]); };
    auto stage = [&](int s) { return base + (size_t)s * LY::kStage; };
    constexpr uint32_t kG = LY::kTileBytes, kUp = kG * (SHARED ? 1 : 2), kMapA = kUp + LY::kUpBytes;
    auto plane = [&](int s, int which) { return reinterpret_cast<float*>(stage(s) + kMapA + which * LY::kPlane); };
    if (tid == 0) {
        abort_flag = 0;
        for (int s = 0; s < S; ++s) {
            mbar_init(full(s), 1);
            mbar_init(mapped(s), kComposers / 32);
            mbar_init(joined(s), CB / 32);
            mbar_init(empty(s), kData / 32);
            mbar_init(runs(s), kData / 32);
            mbar_init(known(s), 1);
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
            tma_prefetch_l2_4d(&mx, 0, (p.tiles - 1 - n) * TILE, hd, b);
            if (!SHARED) tma_prefetch_l2_4d(&mg, 0, (p.tiles - 1 - n) * TILE, hd, b);
            tma_prefetch_l2_4d(&mu_, 0, (p.tiles - 1 - n) * TILE, hd, b);
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
            const int t = (p.tiles - 1 - n) * TILE;
            info[s] = TileInfo{n, row, b, t, (long long)b * p.T, b * p.sg[0] + hd * p.sg[1] + t * p.sg[2],
                               b * p.sdx[0] + hd * p.sdx[1] + t * p.sdx[2], b * p.sdg[0] + hd * p.sdg[1] + t * p.sdg[2]};
            mbar_arrive(known(s));
            loads.note(s);
            mbar_expect_tx(full(s), (uint32_t)(TILE * p.d) * (2u * (SHARED ? 1u : 2u) + (uint32_t)sizeof(TO)));
            tma_load_4d(smem_u32(stage(s)), &mx, 0, t, hd, b, full(s));
            if (!SHARED) tma_load_4d(smem_u32(stage(s) + kG), &mg, 0, t, hd, b, full(s));
            tma_load_4d(smem_u32(stage(s) + kUp), &mu_, 0, t, hd, b, full(s));
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
        for (Ring<S, kJoin> at(j);; at.next()) {
            const int s = at.s;
            if (!wait(known(s), at.phase)) return;
            const int n = info[s].n, row = info[s].row;
            if (n >= 0) {
                float start = 0.f, h = 0.f;
                if (ch < p.d) {
                    if (p.dstate_out) start = p.dstate_out[(long long)row * p.d + ch];
                    h = p.carry[((long long)row * p.tiles + (p.tiles - 1 - n)) * p.d + ch];
                }
                const auto own = [&] { return wait(mapped(s), at.phase); };
                float2 f[RUNS];
                u64 w[kGroup - 1];
                if (!(p.words ? maps_before(p, lb, row, n, ch, w, own) : own())) return;
                float *X = plane(s, 1) + ch, *Y = plane(s, 2) + ch;
#pragma unroll
                for (int r = 0; r < RUNS; ++r) f[r] = make_float2(plane(s, 0)[r * CB + ch], X[r * CB]);
#pragma unroll
                for (int r = 0; r < RUNS; ++r) {
                    X[r * CB] = h;
                    h = pass(f[r], h);
                }
#pragma unroll
                for (int r = 0; r < RUNS; ++r) f[r].y = Y[r * CB];
                float mu = start;
                if (p.words && ends_group(lb, n)) {
                    float2 all = compose(w, kGroup - 1);
#pragma unroll
                    for (int r = RUNS - 1; r >= 0; --r) all = then(all, f[r]);
                    mu = group_state(p, lb, row, n, ch, start);
                    publish_state(p, lb, row, n, ch, pass(all, mu));  // first: tiles of other blocks wait for it
                } else if (p.words) {
                    mu = group_state(p, lb, row, n, ch, start);
                }
                if (p.words) mu = pass_all(w, n % kGroup, mu);
#pragma unroll
                for (int r = RUNS - 1; r >= 0; --r) {
                    Y[r * CB] = mu;
                    mu = pass(f[r], mu);
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
        for (Ring<S, 1> at(0);; at.next()) {
            const int s = at.s;
            if (!wait(known(s), at.phase)) return;
            const int n = info[s].n, row = info[s].row;
            if (n < 0) return;
            if (!wait(runs(s), at.phase)) return;
            if (p.words && n + 1 < p.tiles) {
                const float *A = plane(s, 0) + ch, *Y = plane(s, 2) + ch;
                float2 m[N];
#pragma unroll
                for (int r = RUNS - 1; r >= 0; --r)  // from the tile's last run to its first
#pragma unroll
                    for (int q = 0; q < N; ++q) {
                        const float2 f = make_float2(A[r * CB + q], Y[r * CB + q]);
                        m[q] = r < RUNS - 1 ? then(m[q], f) : f;
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
    for (Ring<S, 1> ring(0);; ring.next()) {
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
        const T* xs = reinterpret_cast<const T*>(stage(s)) + run * kTok * p.d + c;
        const T* gs = reinterpret_cast<const T*>(stage(s) + kG) + run * kTok * p.d + c;
        const TO* us = reinterpret_cast<const TO*>(stage(s) + kUp) + run * kTok * p.d + c;
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
            // (A, X) forwards; Y = sum over the run of dh_t times the decays a_t .. of its beginning
            float A[kCh], X[kCh], Y[kCh];
            // whole: a run of kTok tokens; clean: one without resets
            auto walk = [&](auto whole, auto clean) {
                bool open = true;  // no reset so far
#pragma unroll
                for (int j = 0; j < kCh; ++j) { A[j] = 1.f; X[j] = 0.f; Y[j] = 0.f; }
#pragma unroll(SIG && !SHARED ? 1 : kTok)
                for (int i2 = 0; i2 < kTok; ++i2)
                    if (whole || i2 < nt) {
                        float xv[kCh], uv[kCh], ga[NG];
                        four(xs + i2 * p.d, xv);
                        four(us + i2 * p.d, uv);
                        gates(i2, ga, false);
                        if (!clean && ((resets >> i2) & 1u)) open = false;
#pragma unroll
                        for (int j = 0; j < kCh; ++j) {
                            const float gate = ga[SHARED ? 0 : j];
                            if (!clean && ((resets >> i2) & 1u)) X[j] = 0.f;
                            X[j] = next_state<SIG>(gate, X[j], xv[j]);
                            A[j] = decayed<SIG>(gate, A[j]);
                            if (clean || open) Y[j] = fmaf(A[j], uv[j], Y[j]);
                        }
                    }
            };
            auto powers = [&](auto whole, auto clean) {  // false: out of range
                Powers<NG> w;
                bool open = true;
#pragma unroll
                for (int j = 0; j < kCh; ++j) X[j] = Y[j] = 0.f;
#pragma unroll
                for (int i2 = 0; i2 < kTok; ++i2)
                    if (whole || i2 < nt) {
                        float xv[kCh], uv[kCh], E[NG];
                        four(xs + i2 * p.d, xv);
                        four(us + i2 * p.d, uv);
                        gates(i2, E, true);
                        if (!clean && ((resets >> i2) & 1u)) open = false;
                        if (!clean && ((resets >> i2) & 1u)) fill(X, 0.f);
                        w.token(E, X, xv);
                        w.back_token(E, Y, uv, clean || open);
                    }
                float d = 0.f, top = 0.f, low = INFINITY, any = 0.f;
                span(w.D, d, any);
                span(X, top, low);
                span(Y, top, low);
                bool in = d < kPerhaps && top < INFINITY;
                if (in && !(d < kSurely && low >= kSmall)) {  // looked at closer
                    float gate = 0.f, x = 0.f, u = 0.f;
#pragma unroll 1
                    for (int i2 = 0; i2 < nt; ++i2) {
                        float xv[kCh], ga[NG];
                        four(xs + i2 * p.d, xv);
                        span(xv, x, any);
                        four(us + i2 * p.d, xv);
                        span(xv, u, any);
                        if constexpr (SHARED) ga[0] = ga[1] = to_f32(gp[i2 * p.sg[2]]);
                        else four(gs + i2 * p.d, ga);
#pragma unroll
                        for (int j = 0; j < NG; ++j) gate = fmaxf(gate, ga[j]);
                    }
                    in = gate < kLargestGate && (x == 0.f || x >= kSmallInput) && (u == 0.f || u >= kSmallInput);
                }
                w.close(X, A);
                w.close_back(Y);
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
            const int o = run * CB + c;
            if (resets) {
#pragma unroll
                for (int j = 0; j < kCh; ++j) A[j] = cut();
            } else {
#pragma unroll
                for (int j = 0; j < kCh; ++j) A[j] = no_cut(A[j]);
            }
            *reinterpret_cast<float4*>(plane(s, 0) + o) = make_float4(A[0], A[1], A[2], A[3]);
            *reinterpret_cast<float4*>(plane(s, 1) + o) = make_float4(X[0], X[1], X[2], X[3]);
            *reinterpret_cast<float4*>(plane(s, 2) + o) = make_float4(Y[0], Y[1], Y[2], Y[3]);
            __syncwarp();
            if ((tid & 31) == 0) mbar_arrive(runs(s));
        } else {
            float h[kCh], mu[kCh];
            four(plane(s, 1) + run * CB + c, h);
            four(plane(s, 2) + run * CB + c, mu);
            T* const dxp = static_cast<T*>(p.dx) + info[s].o + run * kTok * p.sdx[2] + c;
            T* const dgp = static_cast<T*>(p.dg) + info[s].o2 + run * kTok * p.sdg[2] + (SHARED ? 0 : c);
            // A gate for each channel is formed on either way from the tile: kept, the run's 32
            // went to local memory (63 us for 58).  Shared ones are formed once.
            auto walk = [&](auto whole, auto clean, auto by_power) {
                if (SHARED && SIG) {
#pragma unroll
                    for (int i2 = 0; i2 < kTok; ++i2)
                        if (whole || i2 < nt) {
                            float ga[NG];
                            gates(i2, ga, by_power);
                            gl[SHARED ? i2 : 0] = ga[0];
                        }
                }
                auto formed = [&](int i2, float (&ga)[NG]) {
                    if (SHARED) gates_of(i2, ga);
                    else gates(i2, ga, by_power);
                };
#pragma unroll
                for (int i2 = 0; i2 < kTok; ++i2)
                    if (whole || i2 < nt) {
                        float xv[kCh], ga[NG];
                        four(xs + i2 * p.d, xv);
                        formed(i2, ga);
                        if (!clean && ((resets >> i2) & 1u)) {
#pragma unroll
                            for (int j = 0; j < kCh; ++j) h[j] = 0.f;
                        }
                        before[i2 * kData + at] = make_float4(h[0], h[1], h[2], h[3]);
                        if (by_power) {
                            next_by_power(ga, h, xv);
                        } else {
#pragma unroll
                            for (int j = 0; j < kCh; ++j) h[j] = next_state<SIG>(ga[SHARED ? 0 : j], h[j], xv[j]);
                        }
                    }
#pragma unroll
                for (int i2 = kTok - 1; i2 >= 0; --i2) {
                    const bool live = whole || i2 < nt;
                    float gx[kCh], gg[kCh];
                    if (live) {
                        float xv[kCh], uv[kCh], ga[NG];
                        four(xs + i2 * p.d, xv);
                        four(us + i2 * p.d, uv);
                        formed(i2, ga);
                        const float4 hb4 = before[i2 * kData + at];
                        const float hb[kCh] = {hb4.x, hb4.y, hb4.z, hb4.w};
                        if (by_power) {
                            back_by_power(ga, uv, hb, xv, gx, gg, mu);
                        } else {
#pragma unroll
                            for (int j = 0; j < kCh; ++j)
                                back_token<SIG>(ga[SHARED ? 0 : j], uv[j] + mu[j], hb[j], xv[j], gx[j], gg[j], mu[j]);
                        }
                        if (!clean && ((resets >> i2) & 1u)) fill(mu, 0.f);
                        Lane<T, kCh, true> ov;
                        ov.set(gx);
                        ov.store(dxp + i2 * p.sdx[2], nc);
                    }
                    if constexpr (SHARED) {  // the sum over the token's channels
                        float sum = 0.f;
#pragma unroll
                        for (int j = 0; j < kCh; ++j) sum += live ? gg[j] : 0.f;
#pragma unroll
                        for (int w = LANES / 2; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
                        if (live && lane == 0) dgp[i2 * p.sdg[2]] = from_f32<T>(sum);
                    } else if (live) {
                        Lane<T, kCh, true> ov;
                        ov.set(gg);
                        ov.store(dgp + i2 * p.sdg[2], nc);
                    }
                }
            };
            // the same path for a warp's lanes: a shared gate's gradient is summed over them
            const bool whole = __all_sync(0xffffffffu, nt == kTok), clean = __all_sync(0xffffffffu, resets == 0);
            using power = std::integral_constant<bool, SIG>;
            using yes = std::true_type;
            using no = std::false_type;
            if (SIG && wide[s][at >> 5]) walk(no{}, no{}, no{});
            else if (whole && clean) walk(yes{}, yes{}, power{});
            else if (whole) walk(yes{}, no{}, power{});
            else walk(no{}, no{}, power{});
            const int row = info[s].row;
            __syncwarp();
            if ((tid & 31) == 0) mbar_arrive(empty(s));
            if (p.dstate_in && nt > 0 && t0 == 0) {
#pragma unroll
                for (int j = 0; j < kCh; ++j) p.dstate_in[(long long)row * p.d + c + j] = mu[j];
            }
        }
    }
}

}  // namespace
}  // namespace hla2

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
    if (int rc = check_states(what, dstate_out, dstate_in, (size_t)B * H * d)) return rc;
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
    p.tiles = tiles_of(T, tile);
    const bool vec = d % kCh == 0 && aligned_to(X, es, p.sx, 3, kCh * es) && aligned_to(dX, es, p.sdx, 3, kCh * es) &&
                     aligned_to(dO, os, p.sdo, 3, kCh * os) &&
                     (gate_shared || (aligned_to(G, es, p.sg, 3, kCh * es) && aligned_to(dG, es, p.sdg, 3, kCh * es)));
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    p.status = device_status_word();  // where a wait that runs out is reported
    if (!p.status) return set_error(HLA2_ERR_LAUNCH, "%s: cannot resolve the device status word", what);
    cudaError_t e = begin_lookback(p, lanes * kCh, workspace, s);
    if (e == cudaSuccess) e = begin_states(p, lanes * kCh, workspace, &p.dstate_out, dstate_in, s);
    CUtensorMap mx{}, mg{}, mu{};
    const bool pipe = dtype == HLA2_DTYPE_BF16 && vec && gate_map(&mx, X, es, p.sx, B, H, T, d, tile) &&
                      (gate_shared || gate_map(&mg, G, es, p.sg, B, H, T, d, tile)) &&
                      gate_map(&mu, dO, os, p.sdo, B, H, T, d, tile);
    if (e == cudaSuccess) e = by_types(dtype, out_dtype, [&](auto tin, auto tout) {
        return by_form(form, gate_shared, [&](auto sig, auto shared) {
            return by_lanes(d, [&](auto ln) {
                using T_ = decltype(tin);
                using TO = decltype(tout);
                constexpr bool SIG = decltype(sig)::value, SHARED = decltype(shared)::value;
                constexpr int LANES = decltype(ln)::value;
                unsigned blocks = 0;
                if constexpr (std::is_same<T_, bf16>::value) {
                    if (pipe) {
                        using LY = BackLayout<TO, SHARED, LANES>;
                        auto kernel = gated_pipe_bwd_kernel<TO, SIG, SHARED, LANES>;
                        if (cudaError_t e2 = persistent_blocks(reinterpret_cast<const void*>(kernel), LY::kThreads,
                                                               LY::kBytes, p.total, &blocks)) return e2;
                        kernel<<<blocks, LY::kThreads, LY::kBytes, s>>>(mx, mg, mu, p);
                        return cudaGetLastError();
                    }
                }
                // wide accesses only for fp32: 16-bit operands that allow them took the pipeline
                return by_bool(vec && std::is_same<T_, float>::value, [&](auto v) {
                    constexpr bool VEC = decltype(v)::value && std::is_same<T_, float>::value;
                    constexpr int threads = block_threads(LANES);
                    constexpr size_t smem = (size_t)kTok * kData * sizeof(float4);
                    auto kernel = gated_scan_bwd_kernel<T_, TO, SIG, SHARED, LANES, VEC>;
                    if (cudaError_t e2 = persistent_blocks(reinterpret_cast<const void*>(kernel), threads, smem,
                                                           p.total, &blocks)) return e2;
                    kernel<<<blocks, threads, smem, s>>>(p);
                    return cudaGetLastError();
                });
            });
        });
    });
    note_launches(1);
    if (e != cudaSuccess) return set_error(HLA2_ERR_LAUNCH, "%s: %s", what, cudaGetErrorString(e));
    return HLA2_OK;
}

