// hla2_gated_bwd.cu -- gradient of the gated linear recurrence (hla2_gated.cu).
#include "hla2_gated.cuh"

namespace hla2 {
namespace {

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
            if (p.words) {
                publish_tile(p, lb, row, n, ch, m);
                publish_group(p, lb, row, n, ch, m);
            }
#pragma unroll 8
            for (int r = 0; r < RUNS; ++r) {
                const float2 f = fwd[r][ch];
                fwd[r][ch].x = h;
                h = pass(f, h);
            }
            if (p.words) {
                mu = enter_tile(p, lb, row, n, ch, mu);
                publish_state(p, lb, row, n, ch, pass(m, mu));
            }
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
            return by_lanes(d, [&](auto ln) { return by_bool(vec, [&](auto v) {
                auto kernel = gated_scan_bwd_kernel<decltype(tin), decltype(tout), decltype(sig)::value,
                                                    decltype(shared)::value, decltype(ln)::value, decltype(v)::value>;
                constexpr int threads = block_threads(decltype(ln)::value);
                constexpr size_t smem = (size_t)kTok * kData * sizeof(float4);
                unsigned blocks = 0;
                if (cudaError_t e2 = persistent_blocks(reinterpret_cast<const void*>(kernel), threads, smem, p.total, &blocks)) return e2;
                kernel<<<blocks, threads, smem, s>>>(p);
                return cudaGetLastError();
            }); });
        });
    });
    note_launches(1);
    if (e != cudaSuccess) return set_error(HLA2_ERR_LAUNCH, "%s: %s", what, cudaGetErrorString(e));
    return HLA2_OK;
}

