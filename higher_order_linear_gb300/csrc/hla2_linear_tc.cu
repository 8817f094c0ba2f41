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
// chunk's sum, so neither a rounded decay nor a sum of many chunks in the
// accumulator costs it bits.  B~ is a sum of bf16 terms: three (24 bits), split off
// the fp32 product, where S leaves the walk in fp32; two (16 bits) where only
// the copy of S is used, by packed bf16 operations alone: with g^.. = f1 + f2 in
// bf16 pieces, h = rn(b f1) and m = rn(b f2 + (b f1 - h)), the error of a bf16
// product being a bf16 number.  (Four such terms for 24 bits cost the tensor cores more
// than they save: states of 65536 x 16 x 128 in 133 us instead of 119.)
//
// Roles.  X warps (4): P from tensor memory, decayed, masked and packed back.
// O warps (4): o_i from O1 and O2, through shared memory, to global memory.  Y
// warps (16): B~ in steps of 16 to 64 tokens (first terms in place of B, the
// others in a ring of two slots), then S and its bf16 copy.  Two warps issue
// products, U and the other three, so that a wait in one chain does not hold up
// the other; one warp loads.  Code is kept short and nothing may spill: seven
// roles share the instruction caches, and local memory goes to L2 (shared memory
// takes all of L1).
//
// Measured (device time of a launch alone, 16 heads, 16 bits).  65536 x 128: states 97
// us, 537 MB at 0.82 of the copy bandwidth; outputs 174 us, 1.07 GB at 0.91.  Shorter
// walks also pay for their start and end: 16384 x 128, 31 us (0.64) and 54 us (0.73).
// 4 x 4096 x 64 (four segments of eight chunks a head, three of them with states):
// 21 us and 35 us, 0.36 and 0.57 of the copy bandwidth were the tiles not in L2; the
// chain P, its packing, P~ C and the drain takes 3.3 us a chunk, two CTAs to an SM.
// Tried and slower: packing P in groups of 32 columns or with the next group on its way
// (outputs of 65536 x 128 at a stand of 196 us: 210, 207), a factor for P's columns, the
// state and the rows so that both terms share one accumulator (201 at a stand of 176),
// four-term keys (above).
#include "hla2_linear.cuh"
#include "hla2_tc_common.cuh"

namespace hla2 {
namespace {

static_assert(kL == kLinTcChunk, "a chunk is the M of the products");

// 8 packed words of this thread's lane
__device__ __forceinline__ void tmem_store8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

__device__ __forceinline__ void tmem_load8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
// 16 columns of this thread's lane
__device__ __forceinline__ void tmem_load16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// (a, b) op (c, d), two fp32 operations to an instruction
struct Pair {
    float x, y;
};
__device__ __forceinline__ unsigned long long bits(Pair a) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
    return r;
}
__device__ __forceinline__ Pair pair_of(unsigned long long v) {
    Pair r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
    return pair_of(r);
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
    return pair_of(r);
}
__device__ __forceinline__ Pair unpack_bf16(uint32_t w) { return {__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)}; }
__device__ __forceinline__ __nv_bfloat162 as_pair(uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); }
__device__ __forceinline__ uint32_t as_word(__nv_bfloat162 v) { return *reinterpret_cast<const uint32_t*>(&v); }
__device__ __forceinline__ Pair at(const uint32_t* r) { return {__uint_as_float(r[0]), __uint_as_float(r[1])}; }

__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r != 0;
}
// One try that may suspend the warp for up to a millisecond: a waiting warp takes no issue slots from the others.
__device__ __forceinline__ bool mbar_long_try(uint32_t a, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(a), "r"(parity), "r"(1000000u)
        : "memory");
    return ok != 0;
}

// Warps and shared memory.  One tile of A (outputs), NB of B and C; the ring's slots hold
// the terms of STEP tokens of B~ but the first; the stage a group of SC
// output columns of each O warp.  At D = 64 two CTAs share an SM: sixteen warps of
// 64 registers each (X and O are the same four), half of tensor memory, and
// half of shared memory; a walk of one chunk after another leaves gaps that the other
// CTA fills.  At D = 64 the products' A operand still has 128 rows: those past
// the tile's 64 columns read what follows it in this allocation, and nobody
// reads their results.
template <int D, bool OUT, int TERMS>
struct TcLayout {
    static constexpr int kCtas = D == 64 ? 2 : 1;
    static constexpr int kX = OUT ? 4 : 0, kO = OUT && D == 128 ? 4 : 0, kY = D == 64 ? 8 : 16;
    static constexpr int kY0 = kX + kO, kStates = kY0 + kY, kLoader = kStates + 1, kOuts = kLoader + 1;
    static constexpr int kThreads = (OUT ? kOuts + 1 : kOuts) * 32;
    static constexpr int kParts = kY / 4;           // Y warps to 32 rows of the state
    static constexpr int kState = D / 32 * kParts;  // Y warps that hold rows of the state
    static constexpr int kCols = D == 128 ? 512 : OUT ? 256 : 128;  // of tensor memory

    static constexpr int STEP = !OUT ? 64 : TERMS == 3 ? 16 : 32;
    static constexpr int kItems = STEP / 4 * (D / 64);  // of 4 tokens by 64 channels in a step
    static constexpr int PER = kItems < kY ? kItems : kY;  // warps that share a step, kItems / PER items each
    static constexpr int SC = D == 128 && TERMS == 2 ? 64 : 32;
    static constexpr int NB = 2;
    static constexpr uint32_t kTile = kL * D * 2, kPart = STEP * D * 2, kStage = 32 * SC * 2;
    static constexpr uint32_t A = 0, B = OUT ? kTile : 0, C = B + NB * kTile, ring = C + NB * kTile;
    static constexpr uint32_t S = ring + 2 * (TERMS - 1) * kPart;
    static constexpr uint32_t stage = S + (D == 64 || OUT ? D * D * 2 : 0), kBytes = stage + (OUT ? 4 * kStage : 0);
};

template <int D, bool REV, bool OUT, int TERMS>
__global__ void __launch_bounds__(TcLayout<D, OUT, TERMS>::kThreads, TcLayout<D, OUT, TERMS>::kCtas)
lin_tc_kernel(const __grid_constant__ CUtensorMap mA, const __grid_constant__ CUtensorMap mB,
              const __grid_constant__ CUtensorMap mC, const LinWalk p) {
    using LY = TcLayout<D, OUT, TERMS>;
    constexpr int NB = LY::NB, STEP = LY::STEP, STEPS = kL / STEP, PER = LY::PER, ITEMS = LY::kItems / PER;
    extern __shared__ __align__(1024) unsigned char dsm_raw[];
    // A barrier's next phase never completes before everybody has seen this one: it takes an arrival that each waiter
    // gives after its wait.  (P of the next chunk needs no arrival of Y, so its barriers go by turns.)
    // loads | A read (O2 = A S done) | B and C read (by both issuers) | P ready, packed | ring filled, free |
    // U ready, drained | S copy ready | O ready (P's columns free), drained | last waits
    enum { LA, LB, LC = LB + NB, FA = LC + NB, FB, CP = FB + NB, DP = CP + 2, KQ, RF = KQ + 2, CU = RF + 2,
           DU = CU + 2, DS = DU + 2, CO, DO, FIN, NBAR = FIN + 2 };
    __shared__ __align__(8) unsigned long long bars[NBAR];
    __shared__ __align__(16) float pw[kL + 4];  // g^0 .. g^128
    __shared__ __align__(16) float down[16];    // g^15 .. g^0
    __shared__ uint32_t pieces[TERMS == 2 ? kL + 1 : 1];  // f1 (low half) and f2 of each power
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool xwarp = warp < LY::kX, owarp = LY::kO ? !xwarp && warp < LY::kY0 : xwarp;
    const bool ywarp = warp >= LY::kY0 && warp < LY::kStates;
    const int quarter = warp & 3, row = quarter * 32 + lane;  // lanes of tensor memory
    const int bh = blockIdx.y, w = blockIdx.x, seg = REV ? p.nseg - 1 - w : w;
    const int b = bh / p.H, h = bh % p.H;
    const int len = length_of(p, b);
    const int c0 = seg * p.seglen, c1 = min(min(c0 + p.seglen, p.nchunk), len / kL + (len % kL != 0));
    const int nchunks = max(0, c1 - c0);
    auto chunk_of = [&](int it) { return REV ? c1 - 1 - it : c0 + it; };
    auto tokens_of = [&](int it) { return min(kL, len - chunk_of(it) * kL); };

    const uint32_t dsm = (smem_u32(dsm_raw) + 1023u) & ~1023u;
    const Tile tA{dsm + LY::A, kL};
    auto tB = [&](int it) { return Tile{dsm + LY::B + (uint32_t)(it % NB) * LY::kTile, kL}; };
    auto tC = [&](int it) { return Tile{dsm + LY::C + (uint32_t)(it % NB) * LY::kTile, kL}; };
    auto tR = [&](int slot, int term) {
        return Tile{dsm + LY::ring + (uint32_t)(slot * (TERMS - 1) + term) * LY::kPart, STEP};
    };
    const Tile tS{dsm + LY::S, D};
    auto bar = [&](int i) -> uint32_t { return smem_u32(&bars[i]); };

    // the loader's first lane sets up the barriers and sends for the first tiles at once; they are on their way while
    // the others form the powers and take tensor memory
    LoadLedger<1 + 2 * NB> loads(bar(0));
    auto load = [&](int l, const CUtensorMap* map, const Tile& t, int it) {
        loads.note(l);
        mbar_expect_tx(bar(l), LY::kTile);
#pragma unroll
        for (int k = 0; k < D / 64; ++k)
            tma_load_4d(t.base + k * t.block_bytes(), map, k * 64, chunk_of(it) * kL, h, b, bar(l));
    };
    if (warp == LY::kLoader && lane == 0) {
        abort_flag = 0;
        for (int i = 0; i < NBAR; ++i) {
            uint32_t count = 1;
            if (i == DP || i == DO) count = OUT ? LY::kX : 1;
            if (i >= FB && i < FB + NB) count = OUT ? 2 : 1;
            if (i == KQ || i == KQ + 1) count = PER;
            if (i == DU || i == DU + 1 || i == DS) count = LY::kState;
            mbar_init(bar(i), count);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async();
        for (int it = 0; it < NB && it < nchunks; ++it) {
            load(LB + it, &mB, tB(it), it);
            if (OUT && it == 0) load(LA, &mA, tA, it);
            load(LC + it, &mC, tC(it), it);
        }
    }
    if (tid <= kL) {
        const float f = power(__ldg(p.gamma + h), tid);
        pw[tid] = f;
        if (tid < 16) down[15 - tid] = f;
        if (TERMS == 2) {
            const bf16 f1 = __float2bfloat16_rn(f), f2 = __float2bfloat16_rn(f - __bfloat162float(f1));
            pieces[tid] = (uint32_t)__bfloat16_as_ushort(f1) | (uint32_t)__bfloat16_as_ushort(f2) << 16;
        }
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                     "r"(LY::kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    follow();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    // outputs: P | O2 | U | O1, which at D = 64 takes the half of P's columns that P~ leaves free; states: U
    // twice, by turns
    const uint32_t tP = tmem, tO2 = tmem + 128, tO1 = D == 64 ? tmem + 64 : tmem + 128 + 2 * D;
    auto tU = [&](int it) -> uint32_t { return OUT ? tmem + 128 + D : tmem + D * (it & 1); };
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;

    auto wait_bar = [&](int i, uint32_t parity) -> bool {
        const uint32_t a = bar(i);
        if (mbar_long_try(a, parity)) return true;
        const unsigned long long t0 = globaltimer();
        while (!mbar_long_try(a, parity)) {
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

    // Zeros in the rows of C behind the end, whatever they hold, by warp `i` of `count`.  Y writes them before U, X
    // before P~ C: neither set of products waits for the other's.
    auto zero_behind = [&](const Tile& C, int n, int i, int count) {
        for (int e = (n << 3) + i * 32 + lane; e < kL * 8; e += count * 32)
#pragma unroll
            for (int k = 0; k < D / 64; ++k) st_shared_v4(C.chunk(e >> 3, k, e & 7), 0u, 0u, 0u, 0u);
    };

    constexpr uint32_t iPP = idesc_bf16(128, 128, false, false);  // A B^T: both along the channels
    constexpr uint32_t iAS = idesc_bf16(128, D, false, true);     // A S, P~ C: the second along its rows
    constexpr uint32_t iBC = idesc_bf16(128, D, true, true);      // B~^T C: both along the tokens

    // a tile's descriptors: its first one, then steps along the channels (16 of them) or the rows (16)
    constexpr uint32_t kBlock = kL * 128u;
    auto along = [](uint64_t first, int ks) { return first + (uint64_t)((((ks >> 2) * kBlock) + (ks & 3) * 32u) >> 4); };
    auto down_rows = [](uint64_t first, int ks) { return first + (uint64_t)(ks * 128); };

    // The issuing warps stay together: their values are uniform, so that descriptors are formed once for the warp
    // (a single lane's way through its own registers took 180 clocks a product), and one lane issues each batch.
    auto wait_warp = [&](int i, uint32_t parity) -> bool {
        const uint32_t a = bar(i);
        bool ok = mbar_long_try(a, parity);
        if (!__all_sync(0xffffffffu, ok)) {
            const unsigned long long t0 = globaltimer();
            while (!ok && !abort_flag) {
                ok = mbar_long_try(a, parity);
                if (!ok && globaltimer() - t0 > kWaitNs) {
                    abort_flag = 1;
                    atomicExch(p.status, (int)kDevWaitTimeout);
                }
            }
            __syncwarp();
        }
        return __all_sync(0xffffffffu, ok) != 0;
    };
    // no product may still run when the CTA gives its memory back, whatever ended the walk
    auto finish = [&](int i) {
        if (elect_one()) mma_commit(bar(i));
        __syncwarp();
        const unsigned long long t0 = globaltimer();
        while (!mbar_long_try(bar(i), 0))
            if (globaltimer() - t0 > kWaitNs) {
                atomicExch(p.status, (int)kDevWaitTimeout);
                break;
            }
        __syncwarp();
    };

    if (warp == LY::kStates) {
        // U, a step of the tokens at a time as Y fills the ring, once its columns have been drained
        int sb = 0;
        uint32_t pb = 0;
        for (int it = 0; it < nchunks; ++it) {
            const uint64_t dB = sdesc(dsm + LY::B + (uint32_t)sb * LY::kTile, kBlock, 1024u);
            const uint64_t dC = sdesc(dsm + LY::C + (uint32_t)sb * LY::kTile, kBlock, 1024u);
            if (!wait_warp(LC + sb, pb)) break;
            if (OUT ? it > 0 && !wait_warp(DU, (uint32_t)(it - 1) & 1)
                    : it > 1 && !wait_warp(DU + (it & 1), (uint32_t)((it >> 1) - 1) & 1)) break;
            const uint32_t u = tU(it);
            bool ok = true;
#pragma unroll
            for (int q = 0; q < STEPS; ++q) {
                const int slot = q & 1;
                ok = ok && wait_warp(KQ + slot, (uint32_t)((STEPS / 2 * it + q / 2) & 1));
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < STEP / 16; ++ks) {
                        const int kk = q * (STEP / 16) + ks;
                        mma_bf16(u, down_rows(dB, kk), down_rows(dC, kk), iBC, kk > 0);
#pragma unroll
                        for (int t = 0; t < TERMS - 1; ++t)
                            mma_bf16(u, down_rows(sdesc(dsm + LY::ring + (uint32_t)(slot * (TERMS - 1) + t) * LY::kPart, STEP * 128u, 1024u), ks),
                                     down_rows(dC, kk), iBC, 1);
                    }
                    mma_commit(bar(RF + slot));
                    if (q == STEPS - 1) {
                        mma_commit(bar(CU + (OUT ? 0 : it & 1)));
                        mma_commit(bar(FB + sb));
                    }
                }
                __syncwarp();
            }
            if (!ok) break;
            if (++sb == NB) { sb = 0; pb ^= 1; }
        }
        finish(FIN);
    } else if (OUT && warp == LY::kOuts) {
        // P, O2, O1, with an issuer of their own: a wait of one chain of products does not hold up the other
        const uint64_t dS = sdesc(dsm + LY::S, D * 128u, 1024u);
        int sb = 0;
        uint32_t pb = 0;
        for (int it = 0; it < nchunks; ++it) {
            const uint32_t ph = it & 1, before = ph ^ 1;
            const uint64_t dA = sdesc(dsm + LY::A, 16u, 1024u);
            const uint64_t dB = sdesc(dsm + LY::B + (uint32_t)sb * LY::kTile, 16u, 1024u);
            const uint64_t dC = sdesc(dsm + LY::C + (uint32_t)sb * LY::kTile, kBlock, 1024u);
            // P, once the last chunk's P~ C has read its columns (and what it left there has been drained)
            if (it > 0 && !wait_warp(D == 64 ? DO : CO, before)) break;
            if (!wait_warp(LA, ph) || !wait_warp(LB + sb, pb)) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) mma_bf16(tP, along(dA, ks), along(dB, ks), iPP, ks > 0);
                mma_commit(bar(CP + ph));
            }
            __syncwarp();
            // O2 = A S, once the last chunk's outputs have been drained
            if (!wait_warp(DS, ph) || (D == 128 && it > 0 && !wait_warp(DO, before))) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) mma_bf16(tO2, along(dA, ks), down_rows(dS, ks), iAS, ks > 0);
                mma_commit(bar(FA));
            }
            __syncwarp();
            // O1 = P~ C
            if (!wait_warp(LC + sb, pb) || !wait_warp(DP, ph)) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < kL / 16; ++ks) mma_bf16_tmem_a(tO1, tP + 8 * ks, down_rows(dC, ks), iAS, ks > 0);
                mma_commit(bar(CO));
                mma_commit(bar(FB + sb));
            }
            __syncwarp();
            if (++sb == NB) { sb = 0; pb ^= 1; }
        }
        finish(FIN + 1);
    } else if (warp == LY::kLoader) {
        if (lane == 0) {
            for (int it = 1; it < nchunks; ++it) {
                const int sb = it % NB, ub = it / NB;
                if (it >= NB) {
                    if (!wait_bar(FB + sb, (uint32_t)(ub - 1) & 1)) break;
                    load(LB + sb, &mB, tB(it), it);
                    load(LC + sb, &mC, tC(it), it);
                }
                if (OUT) {
                    if (!wait_bar(FA, (uint32_t)(it - 1) & 1)) break;
                    load(LA, &mA, tA, it);
                }
            }
            if (!loads.settle()) atomicExch(p.status, (int)kDevWaitTimeout);
        }
    } else if (OUT && (xwarp || owarp)) {
        bf16* const out = static_cast<bf16*>(p.o) + b * p.so[0] + h * p.so[1];
        const uint32_t stage = dsm + LY::stage + (uint32_t)quarter * LY::kStage;
        for (int it = 0; it < nchunks; ++it) {
            const uint32_t ph = it & 1;
            const int n = tokens_of(it);
            if (xwarp) {
                if (!wait_bar(CP + ph, (uint32_t)(it >> 1) & 1)) break;
                tc_fence_after();
#pragma unroll 1
                for (int col = 0; col < kL; col += 16) {  // packed two to a column, from the first on
                    const int gap = REV ? col - row : row - col - 15;  // the row's distance to the group's near edge
                    const int nearest = REV ? col - quarter * 32 - 16 : quarter * 32 - col;  // -16 or 0 on the diagonal
                    uint32_t hi[8];
                    if (nearest < -16) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) hi[j] = 0u;
                    } else {
                        uint32_t r[16];
                        tmem_load16(tP + lane_off + col, r);
                        tmem_ld_wait();
                        if (nearest <= 0) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                const int far = REV ? gap + j : gap + 15 - j;
                                r[j] = far >= 0 ? __float_as_uint(__uint_as_float(r[j]) * pw[max(far, 0)]) : 0u;
                            }
#pragma unroll
                            for (int j = 0; j < 8; ++j) hi[j] = pack_bf16(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
                        } else {
                            const float f = pw[gap];
#pragma unroll
                            for (int j = 0; j < 16; j += 4) {
                                const float4 u = *reinterpret_cast<const float4*>((REV ? pw : down) + j);
                                const Pair x = mul2(mul2(at(r + j), {f, f}), {u.x, u.y});
                                const Pair y = mul2(mul2(at(r + j + 2), {f, f}), {u.z, u.w});
                                hi[j / 2] = pack_bf16(x.x, x.y);
                                hi[j / 2 + 1] = pack_bf16(y.x, y.y);
                            }
                        }
                    }
                    tmem_store8(tP + lane_off + col / 2, hi);
                }
                if (REV && n < kL) {
                    // scores of tokens behind the end: zeros, whatever they held
                    tmem_st_wait();
#pragma unroll 1
                    for (int col = n & ~15; col < kL; col += 16) {
                        uint32_t hi[8];
                        tmem_load8(tP + lane_off + col / 2, hi);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 8; ++j) hi[j] = col + 2 * j >= n ? 0u : col + 2 * j + 1 >= n ? hi[j] & 0xffffu : hi[j];
                        tmem_store8(tP + lane_off + col / 2, hi);
                    }
                }
                if (n < kL) {
                    if (!wait_bar(LC + it % NB, (uint32_t)(it / NB) & 1)) break;
                    zero_behind(tC(it), n, quarter, LY::kX);
                    fence_proxy_async();
                }
                tmem_st_wait();
                tc_fence_before();
                arrive(DP);
            }
            if (!owarp) continue;
            if (!wait_bar(CO, ph)) break;
            tc_fence_after();
            const float f = row < n ? pw[REV ? n - 1 - row : row + 1] : 0.f;
            // the lane's place in a line of SC columns, and its rows: row0, row0 + RI, ..
            constexpr int CH = LY::SC / 8, RI = 32 / CH;
            const int row0 = lane / CH, c8 = lane % CH, left = n - quarter * 32 - row0;
            bf16* const dst = out + (long long)(chunk_of(it) * kL + quarter * 32 + row0) * p.so[2] + c8 * 8;
            auto spot = [&](int r, int c) {  // 16 bytes c of row r, so that neither side's accesses collide
                return stage + (uint32_t)r * (LY::SC * 2) + (uint32_t)((c ^ (CH == 8 ? r & 7 : (r >> 1) & 3)) << 4);
            };
#pragma unroll 1
            for (int g = 0; g < D / LY::SC; ++g) {
#pragma unroll
                for (int k = 0; k < LY::SC / 16; ++k) {
                    const int col = LY::SC * g + 16 * k;
                    uint32_t r1[16], r2[16];
                    tmem_load16(tO1 + lane_off + col, r1);
                    tmem_load16(tO2 + lane_off + col, r2);
                    tmem_ld_wait();
                    if (col == D - 16) {
                        tc_fence_before();
                        arrive(DO);
                    }
#pragma unroll
                    for (int j = 0; j < 16; j += 8) {
                        uint32_t o[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const Pair v = fma2({f, f}, at(r2 + j + 2 * i), at(r1 + j + 2 * i));
                            o[i] = pack_bf16(v.x, v.y);
                        }
                        st_shared_v4(spot(lane, 2 * k + j / 8), o[0], o[1], o[2], o[3]);
                    }
                }
                // whole lines to global memory
                __syncwarp();
                bf16* to = dst + LY::SC * g;
                const bool wide = LY::SC * g + c8 * 8 < p.dc;
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    uint4 v;
                    ld_shared_v4(spot(RI * i + row0, c8), v.x, v.y, v.z, v.w);
                    if (wide && RI * i < left) *reinterpret_cast<uint4*>(to) = v;
                    to += RI * p.so[2];
                }
                __syncwarp();
            }
        }
    } else if (ywarp) {
        constexpr int W = D / LY::kParts;  // columns of S to a thread
        const int yw = warp - LY::kY0, part = yw >> 2;
        const bool holds = quarter < D / 32;
        const int scol = part * W;
        const size_t R = (size_t)p.da * p.dc;
        float S[W];
#pragma unroll
        for (int j = 0; j < W; ++j) S[j] = 0.f;
        // a row of a state that can be taken 16 bytes at a time (dc is a multiple of eight here)
        auto whole_steps = [](const float* at, long long step) {
            return step == 1 && reinterpret_cast<uintptr_t>(at) % 16 == 0;
        };
        if (OUT && holds && row < p.da) {
            const float* src = nullptr;
            long long step = 1;
            if (p.nseg > 1) {
                src = p.rec + ((size_t)bh * (p.nseg + 1) + w) * R + (size_t)row * p.rec_r;
                step = p.rec_c;
            } else if (p.s_in) {
                src = p.s_in + (size_t)bh * R + row * p.in_r;
                step = p.in_c;
            }
            if (src && whole_steps(src, step)) {
#pragma unroll
                for (int j = 0; j < W; j += 4)
                    if (scol + j < p.dc) {
                        const float4 v = *reinterpret_cast<const float4*>(src + scol + j);
                        S[j] = v.x; S[j + 1] = v.y; S[j + 2] = v.z; S[j + 3] = v.w;
                    }
            } else if (src) {
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
        auto update = [&](int it) -> bool {  // S of chunk it's end
            if (!wait_bar(CU + (OUT ? 0 : it & 1), OUT ? (uint32_t)it & 1 : (uint32_t)(it >> 1) & 1)) return false;
            tc_fence_after();
            const float gn = pw[tokens_of(it)];
#pragma unroll
            for (int k = 0; k < W / 16; ++k) {
                uint32_t r[16];
                tmem_load16(tU(it) + lane_off + scol + 16 * k, r);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    const Pair v = fma2({gn, gn}, {S[16 * k + j], S[16 * k + j + 1]}, at(r + j));
                    S[16 * k + j] = v.x;
                    S[16 * k + j + 1] = v.y;
                }
            }
            tc_fence_before();
            arrive(DU + (OUT ? 0 : it & 1));
            return true;
        };
        if (OUT && holds && nchunks > 0) copy_state();
        // items of 4 tokens by 64 channels of a step; where a step has fewer than there are warps, half the warps
        // take every other step
        constexpr int GROUPS = LY::kY / PER;
        const int group = yw / PER, item = yw % PER;
        int it = 0;
        for (; it < nchunks; ++it) {
            const uint32_t ph = it & 1;
            const int n = tokens_of(it), sb = it % NB;
            const uint32_t kb = (uint32_t)(it / NB) & 1;
            const Tile B = tB(it), C = tC(it);
            if (!wait_bar(LB + sb, kb) || (OUT && !wait_bar(CP + ph, (uint32_t)(it >> 1) & 1))) break;  // A B^T has read B
            if (n < kL) {
                if (!wait_bar(LC + sb, kb)) break;
                zero_behind(C, n, item, PER);  // by each group of warps, so that the arrivals of either say so
            }
            bool ok = true;
#pragma unroll 1
            for (int q = group; q < STEPS; q += GROUPS) {
                const int slot = q & 1, use = STEPS / 2 * it + (q >> 1);
                uint32_t more[ITEMS][TERMS - 1][4], place[ITEMS];
#pragma unroll
                for (int i = 0; i < ITEMS; ++i) {
                    const int m = item + PER * i, r = 4 * (m % (STEP / 4)) + (lane >> 3), t = STEP * q + r;
                    const uint32_t a = B.chunk(t, m / (STEP / 4), lane & 7);
                    place[i] = tR(slot, 0).chunk(r, m / (STEP / 4), lane & 7);
                    uint32_t x[4];
                    ld_shared_v4(a, x[0], x[1], x[2], x[3]);
                    const bool in = t < n;
                    const int far = in ? (REV ? t + 1 : n - 1 - t) : 0;
                    if constexpr (TERMS == 2) {
                        const uint32_t f12 = pieces[far];
                        const __nv_bfloat162 f1 = as_pair(__byte_perm(f12, 0u, 0x1010)), f2 = as_pair(__byte_perm(f12, 0u, 0x3232));
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const __nv_bfloat162 v = as_pair(in ? x[j] : 0u), h1 = __hmul2_rn(v, f1);
                            x[j] = as_word(h1);
                            more[i][0][j] = as_word(__hfma2(v, f2, __hfma2(v, f1, __hneg2(h1))));
                        }
                    } else {
                        const float f = pw[far];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            Pair u = mul2(unpack_bf16(in ? x[j] : 0u), {f, f});
                            x[j] = pack_bf16(u.x, u.y);
                            u = fma2(unpack_bf16(x[j]), {-1.f, -1.f}, u);
                            more[i][0][j] = pack_bf16(u.x, u.y);
                            u = fma2(unpack_bf16(more[i][0][j]), {-1.f, -1.f}, u);
                            more[i][TERMS - 2][j] = pack_bf16(u.x, u.y);
                        }
                    }
                    st_shared_v4(a, x[0], x[1], x[2], x[3]);
                }
                if (use > 0 && !wait_bar(RF + slot, (uint32_t)(use - 1) & 1)) { ok = false; break; }
#pragma unroll
                for (int i = 0; i < ITEMS; ++i)
#pragma unroll
                    for (int t = 0; t < TERMS - 1; ++t)
                        st_shared_v4(place[i] + t * LY::kPart, more[i][t][0], more[i][t][1], more[i][t][2], more[i][t][3]);
                fence_proxy_async();
                arrive(KQ + slot);
            }
            if (!ok) break;
            if (holds) {
                if (OUT) {
                    if (!update(it)) break;
                    if (it + 1 < nchunks) {
                        if (!wait_bar(FA, ph)) break;  // A S has read the copy
                        copy_state();
                    }
                } else if (it > 0 && !update(it - 1)) {  // the previous chunk's, beside this one's products
                    break;
                }
            }
        }
        if (!OUT && holds && it == nchunks && nchunks > 0) update(nchunks - 1);
        // (a wait that ran out leaves here too: the status word says so)
        float* dst = nullptr;
        long long step = 1;
        if (!OUT) {
            dst = p.rec + ((size_t)bh * (p.nseg + 1) + w + 1) * R + (size_t)row * p.dc;
        } else if (p.s_out && p.nseg == 1) {
            dst = p.s_out + (size_t)bh * R + row * p.out_r;
            step = p.out_c;
        }
        if (dst && holds && row < p.da) {
            if (whole_steps(dst, step)) {
#pragma unroll
                for (int j = 0; j < W; j += 4)
                    if (scol + j < p.dc)
                        *reinterpret_cast<float4*>(dst + scol + j) = make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
            } else {
#pragma unroll
                for (int j = 0; j < W; ++j)
                    if (scol + j < p.dc) dst[(scol + j) * step] = S[j];
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_slot), "r"(LY::kCols) : "memory");
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

template <int D, bool REV, bool OUT, int TERMS>
cudaError_t launch(const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mc, const LinWalk& w,
                   cudaStream_t s) {
    auto kernel = lin_tc_kernel<D, REV, OUT, TERMS>;
    using LY = TcLayout<D, OUT, TERMS>;
    const int bytes = (int)LY::kBytes + 1024;
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) return e;
    return launch_following(kernel, dim3(OUT ? w.nseg : lin_state_segments(w), w.B * w.H), LY::kThreads, bytes, s, w.after,
                            ma, mb, mc, w);
}

// states: three terms.  outputs: three where the walk itself leaves the last state.
template <int D, bool REV>
cudaError_t pick(const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mc, const LinWalk& w, bool states,
                 cudaStream_t s) {
    if (states) return launch<D, REV, false, 3>(ma, mb, mc, w, s);
    return w.s_out && w.nseg == 1 ? launch<D, REV, true, 3>(ma, mb, mc, w, s) : launch<D, REV, true, 2>(ma, mb, mc, w, s);
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
    if (w.da <= 64 && w.dc <= 64) return w.rev ? pick<64, true>(ma, mb, mc, w, states, s) : pick<64, false>(ma, mb, mc, w, states, s);
    return w.rev ? pick<128, true>(ma, mb, mc, w, states, s) : pick<128, false>(ma, mb, mc, w, states, s);
}

}  // namespace hla2
