// hla2_linear_tc.cu -- the walk of the first-order linear attention on GB300
// tensor cores (hla2_linear.cuh says which walks there are).
//
// One CTA walks one segment of one head in chunks of 128 tokens.  With the
// chunk's tiles A, B, C (queries, keys, values of a forward walk), n its
// tokens, g the head's decay and S the state that enters it:
//   P  = A B^T                    P~ = P o g^(i-j) where j <= i (bf16, in tensor memory)
//   O1 = P~ C     O2 = A S        o_i = O1_i + g^(i+1) O2_i
//   U  = B~^T C,  B~_j = g^(n-1-j) B_j           S <- g^n S + U
// (backward in time: j >= i, g^(j-i), g^(n-1-i) and g^(j+1)).  All factors are
// powers with exponents >= 0, so no decay overflows, zero included.
//
// Precision.  P~ and the copy of S that A is multiplied with are rounded to
// bf16 (half a unit each, like the bf16 result itself).  S is fp32, in the
// registers of the warps that update it: the tensor cores only form U, one
// chunk's sum, from B~ as three bf16 terms (24 bits), so neither a rounded
// decay nor a sum of many chunks in the accumulator costs it bits.
//
// Roles.  X warps (8): P from tensor memory, decayed, masked and packed back;
// o_i from O1 and O2 to global memory.  Y warps (8): B~ in quarters of 32
// tokens (first terms in place of B, the others in a ring of two slots), then S
// and its bf16 copy.  One warp issues the products, one the loads.
#include "hla2_linear.cuh"
#include "hla2_tc_common.cuh"

namespace hla2 {
namespace {

static_assert(kL == kLinTcChunk, "a chunk is the M of the products");

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int t, int h, int b,
                                            uint32_t mbar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(t), "r"(h), "r"(b), "r"(mbar)
        : "memory");
}

// 16 packed words of this thread's lane
__device__ __forceinline__ void tmem_store16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

constexpr int kQuarter = 32;  // tokens of B~ at a time

// Shared memory.  Tiles of A: NA, of B and C: NB; the ring's slots hold the
// second and third terms of a quarter of B~.  At D = 64 the products' A operand
// still has 128 rows: those past the tile's 64 columns read what follows it in
// this allocation, and nobody reads their results.
template <int D, bool OUT>
struct TcLayout {
    static constexpr int NA = OUT ? (D == 64 ? 2 : 1) : 0, NB = OUT ? (D == 64 ? 3 : 2) : 3;
    static constexpr uint32_t kTile = kL * D * 2, kPart = kQuarter * D * 2;
    static constexpr uint32_t A = 0, B = NA * kTile, C = B + NB * kTile, ring = C + NB * kTile;
    static constexpr uint32_t S = ring + 4 * kPart, kBytes = S + (D == 64 || OUT ? D * D * 2 : 0);
};

template <int D, bool OUT>
struct TcRoles {
    static constexpr int kX = OUT ? 8 : 0, kY = 8;
    static constexpr int kThreads = (kX + kY + 2) * 32;
    static constexpr int kState = D / 32 * 2;  // Y warps that hold rows of the state
};

template <int D, bool REV, bool OUT>
__global__ void __launch_bounds__(TcRoles<D, OUT>::kThreads, 1)
lin_tc_kernel(const __grid_constant__ CUtensorMap mA, const __grid_constant__ CUtensorMap mB,
              const __grid_constant__ CUtensorMap mC, const LinWalk p) {
    using LY = TcLayout<D, OUT>;
    using RO = TcRoles<D, OUT>;
    constexpr int NA = LY::NA, NB = LY::NB;
    extern __shared__ __align__(1024) unsigned char dsm_raw[];
    // loads | buffers free | P ready, packed | ring filled, free | U ready, drained | S copy ready, read |
    // O ready, drained | last wait
    enum { LA, LB = LA + NA, LC = LB + NB, FA = LC + NB, FB = FA + NA, FC = FB + NB, CP = FC + NB, DP, KQ, RF = KQ + 2,
           CU = RF + 2, DU, DS, CS, CO, DO, FIN, NBAR };
    __shared__ __align__(8) unsigned long long bars[NBAR];
    __shared__ __align__(16) float pw[kL + 4];  // g^0 .. g^128
    __shared__ __align__(16) float down[32];    // g^31 .. g^0
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool xwarp = warp < RO::kX, ywarp = !xwarp && warp < RO::kX + RO::kY;
    const bool issuer = warp == RO::kX + RO::kY, loader = warp == RO::kX + RO::kY + 1;
    const int quarter = warp & 3, row = quarter * 32 + lane;  // lanes of tensor memory
    const int part = (warp >> 2) & 1;                         // which half of the columns
    const int bh = blockIdx.y, w = blockIdx.x, seg = REV ? p.nseg - 1 - w : w;
    const int b = bh / p.H, h = bh % p.H;
    const int len = length_of(p, b);
    const int c0 = seg * p.seglen, c1 = min(min(c0 + p.seglen, p.nchunk), (len + kL - 1) / kL);
    const int nchunks = max(0, c1 - c0);
    auto chunk_of = [&](int it) { return REV ? c1 - 1 - it : c0 + it; };
    auto tokens_of = [&](int it) { return min(kL, len - chunk_of(it) * kL); };

    const uint32_t dsm = (smem_u32(dsm_raw) + 1023u) & ~1023u;
    auto tA = [&](int it) { return Tile{dsm + LY::A + (uint32_t)(it % (NA ? NA : 1)) * LY::kTile, kL}; };
    auto tB = [&](int it) { return Tile{dsm + LY::B + (uint32_t)(it % NB) * LY::kTile, kL}; };
    auto tC = [&](int it) { return Tile{dsm + LY::C + (uint32_t)(it % NB) * LY::kTile, kL}; };
    auto tR = [&](int slot, int term) { return Tile{dsm + LY::ring + (uint32_t)(slot * 2 + term) * LY::kPart, kQuarter}; };
    const Tile tS{dsm + LY::S, D};
    auto bar = [&](int i) -> uint32_t { return smem_u32(&bars[i]); };

    if (tid == 0) {
        abort_flag = 0;
        for (int i = 0; i < NBAR; ++i) {
            uint32_t count = 1;
            if (i == DP || i == DO) count = OUT ? RO::kX : 1;
            if (i == KQ || i == KQ + 1) count = RO::kY;
            if (i == DU || i == DS) count = RO::kState;
            mbar_init(bar(i), count);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (tid <= kL) {
        const float f = (float)power((double)__ldg(p.gamma + h), tid);
        pw[tid] = f;
        if (tid < 32) down[31 - tid] = f;
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const uint32_t tP = tmem, tO1 = tmem + 128, tO2 = tmem + 128 + D, tU = tmem + 128 + 2 * D;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;

    auto wait_bar = [&](int i, uint32_t parity) -> bool {
        const uint32_t a = bar(i);
        if (abort_flag) return false;
        if (mbar_try(a, parity)) return true;
        const unsigned long long t0 = globaltimer();
        while (!mbar_try(a, parity)) {
            if (abort_flag) return false;
            if (globaltimer() - t0 > kWaitNs) {
                abort_flag = 1;
                atomicExch(p.status, (int)kDevWaitTimeout);
                return false;
            }
        }
        return true;
    };
    auto arrive = [&](int i) {
        __syncwarp();
        if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar(i)) : "memory");
    };

    constexpr uint32_t iPP = idesc_bf16(128, 128, false, false);  // A B^T: both along the channels
    constexpr uint32_t iAS = idesc_bf16(128, D, false, true);     // A S, P~ C: the second along its rows
    constexpr uint32_t iBC = idesc_bf16(128, D, true, true);      // B~^T C: both along the tokens

    if (issuer) {
        if (lane == 0) {
            // packed pairs of tokens 16 ks.. of P~ (each group of 32 columns packed into its first 16)
            auto packed = [](int ks) -> uint32_t { return (uint32_t)(32 * (ks / 2) + 8 * (ks % 2)); };
            for (int it = 0; it < nchunks; ++it) {
                const uint32_t ph = it & 1, before = ph ^ 1;
                const int sb = it % NB;
                const uint32_t kb = (uint32_t)(it / NB) & 1;
                const Tile B = tB(it), C = tC(it);
                if (OUT) {
                    // P, once the previous chunk's P~ C has read its columns
                    if (it > 0 && !wait_bar(CO, before)) break;
                    if (!wait_bar(LA + it % (NA ? NA : 1), (uint32_t)(it / (NA ? NA : 1)) & 1) || !wait_bar(LB + sb, kb)) break;
                    tc_fence_after();
                    const Tile A = tA(it);
                    for (int ks = 0; ks < D / 16; ++ks) mma_bf16(tP, A.kmaj(ks), B.kmaj(ks), iPP, ks > 0);
                    mma_commit(bar(CP));
                }
                // U, a quarter of the tokens at a time as Y fills the ring
                if (!wait_bar(LC + sb, kb)) break;
                if (it > 0 && !wait_bar(DU, before)) break;
                bool ok = true;
                for (int q = 0; q < 4 && ok; ++q) {
                    if (OUT && q == 2) {
                        // O2 = A S beside Y's third quarter
                        if (!wait_bar(DS, ph) || (it > 0 && !wait_bar(DO, before))) { ok = false; break; }
                        tc_fence_after();
                        const Tile A = tA(it);
                        for (int ks = 0; ks < D / 16; ++ks) mma_bf16(tO2, A.kmaj(ks), tS.mnmaj(ks), iAS, ks > 0);
                        mma_commit(bar(CS));
                        mma_commit(bar(FA + it % (NA ? NA : 1)));
                    }
                    const int slot = q & 1;
                    if (!wait_bar(KQ + slot, (uint32_t)((2 * it + (q >> 1)) & 1))) { ok = false; break; }
                    tc_fence_after();
                    const Tile mid = tR(slot, 0), lo = tR(slot, 1);
                    for (int ks = 0; ks < 2; ++ks) {
                        const uint64_t c = C.mnmaj(2 * q + ks);
                        mma_bf16(tU, B.mnmaj(2 * q + ks), c, iBC, q + ks > 0);
                        mma_bf16(tU, mid.mnmaj(ks), c, iBC, 1);
                        mma_bf16(tU, lo.mnmaj(ks), c, iBC, 1);
                    }
                    mma_commit(bar(RF + slot));
                }
                if (!ok) break;
                mma_commit(bar(CU));
                mma_commit(bar(FB + sb));
                if (OUT) {
                    if (!wait_bar(DP, ph)) break;
                    tc_fence_after();
                    for (int ks = 0; ks < kL / 16; ++ks) mma_bf16_tmem_a(tO1, tP + packed(ks), C.mnmaj(ks), iAS, ks > 0);
                    mma_commit(bar(CO));
                }
                mma_commit(bar(FC + sb));
            }
            if (!mma_wait_all(bar(FIN))) atomicExch(p.status, (int)kDevWaitTimeout);
        }
    } else if (loader) {
        if (lane == 0) {
            LoadLedger<NA + 2 * NB> loads(bar(0));
            auto load = [&](int l, const CUtensorMap* map, const Tile& t, int it) {
                loads.note(l);
                mbar_expect_tx(bar(l), LY::kTile);
#pragma unroll
                for (int k = 0; k < D / 64; ++k)
                    tma_load_4d(t.base + k * t.block_bytes(), map, k * 64, chunk_of(it) * kL, h, b, bar(l));
            };
            for (int it = 0; it < nchunks; ++it) {
                const int sb = it % NB, ub = it / NB;
                if (ub > 0 && !wait_bar(FB + sb, (uint32_t)(ub - 1) & 1)) break;
                load(LB + sb, &mB, tB(it), it);
                if (ub > 0 && !wait_bar(FC + sb, (uint32_t)(ub - 1) & 1)) break;
                load(LC + sb, &mC, tC(it), it);
                if (OUT) {
                    const int sa = it % (NA ? NA : 1), ua = it / (NA ? NA : 1);
                    if (ua > 0 && !wait_bar(FA + sa, (uint32_t)(ua - 1) & 1)) break;
                    load(LA + sa, &mA, tA(it), it);
                }
            }
            if (!loads.settle()) atomicExch(p.status, (int)kDevWaitTimeout);
        }
    } else if (OUT && xwarp) {
        bf16* const out = static_cast<bf16*>(p.o) + b * p.so[0] + h * p.so[1];
        for (int it = 0; it < nchunks; ++it) {
            const uint32_t ph = it & 1;
            const int n = tokens_of(it);
            if (!wait_bar(CP, ph)) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int col = (k == 0 ? part : 3 - part) * 32;  // both halves get a full and a short one
                uint32_t hi[16];
                const bool none = REV ? col < quarter * 32 : col > quarter * 32;
                if (none) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) hi[j] = 0u;
                } else {
                    uint32_t r[32];
                    tmem_ld32(tP + lane_off + col, r);
                    tmem_ld_wait();
                    float v[32];
                    if (col == quarter * 32) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const int far = REV ? j - lane : lane - j;
                            const bool in = far >= 0 && (!REV || col + j < n);
                            v[j] = in ? __uint_as_float(r[j]) * pw[in ? far : 0] : 0.f;
                        }
                    } else {
                        // the row's distance to the group's near edge, then the group's own powers
                        const float f = pw[REV ? col - row : row - col - 31];
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            const float4 u = REV ? *reinterpret_cast<const float4*>(pw + j)
                                                 : *reinterpret_cast<const float4*>(down + j);
                            const float uu[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                v[j + i] = !REV || col + j + i < n ? __uint_as_float(r[j + i]) * (f * uu[i]) : 0.f;
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j) hi[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
                }
                tmem_store16(tP + lane_off + col, hi);
            }
            tmem_st_wait();
            tc_fence_before();
            arrive(DP);
            if (!wait_bar(CO, ph)) break;
            tc_fence_after();
            const float f = row < n ? pw[REV ? n - 1 - row : row + 1] : 0.f;
            bf16* const dst = out + (long long)(chunk_of(it) * kL + row) * p.so[2];
            constexpr int G = D / 64;  // groups of 32 columns to a warp
#pragma unroll
            for (int k = 0; k < G; ++k) {
                const int col = (part * G + k) * 32;
                uint32_t r1[32], r2[32];
                tmem_ld32(tO1 + lane_off + col, r1);
                tmem_ld32(tO2 + lane_off + col, r2);
                tmem_ld_wait();
                if (k == G - 1) {
                    tc_fence_before();
                    arrive(DO);
                }
                if (row < n) {
#pragma unroll
                    for (int j = 0; j < 32; j += 8) {
                        if (col + j >= p.dc) break;
                        uint32_t o[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            o[i] = pack_bf16(fmaf(f, __uint_as_float(r2[j + 2 * i]), __uint_as_float(r1[j + 2 * i])),
                                             fmaf(f, __uint_as_float(r2[j + 2 * i + 1]), __uint_as_float(r1[j + 2 * i + 1])));
                        *reinterpret_cast<uint4*>(dst + col + j) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                }
            }
        }
    } else if (ywarp) {
        constexpr int W = D / 2;  // columns of S to a thread
        const int yw = warp - RO::kX;
        const bool holds = quarter < D / 32;
        const int scol = part * W;
        const size_t R = (size_t)p.da * p.dc;
        float S[W];
#pragma unroll
        for (int j = 0; j < W; ++j) S[j] = 0.f;
        if (OUT && holds && row < p.da) {
            const float* src = nullptr;
            long long step = 1;
            if (p.nseg > 1) {
                src = p.rec + ((size_t)bh * p.nseg + w) * R + (size_t)row * p.dc;
            } else if (p.s_in) {
                src = p.s_in + (size_t)bh * R + row * p.in_r;
                step = p.in_c;
            }
            if (src) {
#pragma unroll
                for (int j = 0; j < W; ++j)
                    if (scol + j < p.dc) S[j] = src[(scol + j) * step];
            }
        }
        auto copy_state = [&]() {  // bf16 S for A S
#pragma unroll
            for (int j = 0; j < W; j += 8) {
                const int col = scol + j;
                st_shared_v4(tS.chunk(row, col >> 6, (col & 63) >> 3), pack_bf16(S[j], S[j + 1]),
                             pack_bf16(S[j + 2], S[j + 3]), pack_bf16(S[j + 4], S[j + 5]), pack_bf16(S[j + 6], S[j + 7]));
            }
            fence_proxy_async();
            arrive(DS);
        };
        if (OUT && holds && nchunks > 0) copy_state();
        for (int it = 0; it < nchunks; ++it) {
            const uint32_t ph = it & 1;
            const int n = tokens_of(it), sb = it % NB;
            const uint32_t kb = (uint32_t)(it / NB) & 1;
            const Tile B = tB(it), C = tC(it);
            if (!wait_bar(LB + sb, kb)) break;
            if (n < kL) {
                // rows behind the end: zeros in C, whatever they hold (B~'s are zeros below)
                if (!wait_bar(LC + sb, kb)) break;
                for (int i = (n << 3) + yw * 32 + lane; i < kL * 8; i += RO::kY * 32)
#pragma unroll
                    for (int k = 0; k < D / 64; ++k) st_shared_v4(C.chunk(i >> 3, k, i & 7), 0u, 0u, 0u, 0u);
            }
            if (OUT && !wait_bar(CP, ph)) break;  // A B^T has read B
            bool ok = true;
            for (int q = 0; q < 4; ++q) {
                const int slot = q & 1, use = 2 * it + (q >> 1);
                if (use > 0 && !wait_bar(RF + slot, (uint32_t)(use - 1) & 1)) { ok = false; break; }
                const Tile mid = tR(slot, 0), lo = tR(slot, 1);
                const int r = 4 * yw + (lane >> 3), t = kQuarter * q + r;
                const bool live = t < n;
                const float f = live ? pw[REV ? t + 1 : n - 1 - t] : 0.f;
#pragma unroll
                for (int k = 0; k < D / 64; ++k) {
                    const uint32_t a = B.chunk(t, k, lane & 7);
                    uint32_t x[4], y[4], z[4];
                    ld_shared_v4(a, x[0], x[1], x[2], x[3]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float u = live ? __uint_as_float(x[i] << 16) * f : 0.f;
                        const float v = live ? __uint_as_float(x[i] & 0xffff0000u) * f : 0.f;
                        const __nv_bfloat162 h0 = __floats2bfloat162_rn(u, v);
                        const float u1 = u - __low2float(h0), v1 = v - __high2float(h0);
                        const __nv_bfloat162 h1 = __floats2bfloat162_rn(u1, v1);
                        x[i] = *reinterpret_cast<const uint32_t*>(&h0);
                        y[i] = *reinterpret_cast<const uint32_t*>(&h1);
                        z[i] = pack_bf16(u1 - __low2float(h1), v1 - __high2float(h1));
                    }
                    st_shared_v4(a, x[0], x[1], x[2], x[3]);
                    st_shared_v4(mid.chunk(r, k, lane & 7), y[0], y[1], y[2], y[3]);
                    st_shared_v4(lo.chunk(r, k, lane & 7), z[0], z[1], z[2], z[3]);
                }
                fence_proxy_async();
                arrive(KQ + slot);
            }
            if (!ok) break;
            if (holds) {
                if (!wait_bar(CU, ph)) break;
                tc_fence_after();
                const float gn = pw[n];
#pragma unroll
                for (int k = 0; k < W / 32; ++k) {
                    uint32_t r[32];
                    tmem_ld32(tU + lane_off + scol + 32 * k, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j) S[32 * k + j] = fmaf(gn, S[32 * k + j], __uint_as_float(r[j]));
                }
                tc_fence_before();
                arrive(DU);
                if (OUT && it + 1 < nchunks) {
                    if (!wait_bar(CS, ph)) break;  // A S has read the copy
                    copy_state();
                }
            }
        }
        // (a wait that ran out leaves here too: the status word says so)
        float* dst = nullptr;
        long long step = 1;
        if (!OUT) {
            dst = p.rec + ((size_t)bh * p.nseg + w + 1) * R + (size_t)row * p.dc;
        } else if (p.s_out && w == p.nseg - 1) {
            dst = p.s_out + (size_t)bh * R + row * p.out_r;
            step = p.out_c;
        }
        if (dst && holds && row < p.da) {
#pragma unroll
            for (int j = 0; j < W; ++j)
                if (scol + j < p.dc) dst[(scol + j) * step] = S[j];
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

// ------------------------------------------------------------------ host ----
bool steps_of_16(const void* p, const long long (&s)[3], int B, int H, int T, int d) {
    if (reinterpret_cast<uintptr_t>(p) % 16 || d % 8) return false;
    const int sizes[3] = {B, H, T};
    for (int i = 0; i < 3; ++i)
        if (sizes[i] > 1 && (s[i] <= 0 || s[i] % 8 || s[i] * 2 >= (1LL << 40))) return false;
    return true;
}

// [B][H][T][d] in boxes of 128 tokens by 64 channels, 128-byte swizzle
bool tile_map(CUtensorMap* m, const void* base, const long long (&s)[3], int B, int H, int T, int d) {
    const int sizes[3] = {T, H, B};
    const long long st[3] = {s[2], s[1], s[0]};
    cuuint64_t strides[3];
    for (int i = 0; i < 3; ++i) strides[i] = (cuuint64_t)(sizes[i] == 1 ? (long long)d * 2 : st[i] * 2);
    const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)T, (cuuint64_t)H, (cuuint64_t)B};
    const cuuint32_t box[4] = {64, kL, 1, 1}, step[4] = {1, 1, 1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, step,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool REV, bool OUT>
cudaError_t launch(const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mc, const LinWalk& w,
                   cudaStream_t s) {
    auto kernel = lin_tc_kernel<D, REV, OUT>;
    const int bytes = (int)TcLayout<D, OUT>::kBytes + 1024;
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) return e;
    kernel<<<dim3(OUT ? w.nseg : w.nseg - 1, w.B * w.H), TcRoles<D, OUT>::kThreads, bytes, s>>>(ma, mb, mc, w);
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace

bool lin_tc_supported(const LinWalk& w, int dtype) {
    return dtype == HLA2_DTYPE_BF16 && encode_fn() && steps_of_16(w.a, w.sa, w.B, w.H, w.T, w.da) &&
           steps_of_16(w.b, w.sb, w.B, w.H, w.T, w.da) && steps_of_16(w.c, w.sc, w.B, w.H, w.T, w.dc) &&
           steps_of_16(w.o, w.so, w.B, w.H, w.T, w.dc);
}

cudaError_t launch_lin_tc(const LinWalk& w, bool states, cudaStream_t s) {
    CUtensorMap ma{}, mb{}, mc{};
    if (!tile_map(&mb, w.b, w.sb, w.B, w.H, w.T, w.da) || !tile_map(&mc, w.c, w.sc, w.B, w.H, w.T, w.dc) ||
        (!states && !tile_map(&ma, w.a, w.sa, w.B, w.H, w.T, w.da)))
        return cudaErrorInvalidValue;
    const bool small = w.da <= 64 && w.dc <= 64;
    if (states) {
        if (small) return w.rev ? launch<64, true, false>(ma, mb, mc, w, s) : launch<64, false, false>(ma, mb, mc, w, s);
        return w.rev ? launch<128, true, false>(ma, mb, mc, w, s) : launch<128, false, false>(ma, mb, mc, w, s);
    }
    if (small) return w.rev ? launch<64, true, true>(ma, mb, mc, w, s) : launch<64, false, true>(ma, mb, mc, w, s);
    return w.rev ? launch<128, true, true>(ma, mb, mc, w, s) : launch<128, false, true>(ma, mb, mc, w, s);
}

}  // namespace hla2
