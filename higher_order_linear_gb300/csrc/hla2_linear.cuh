// hla2_linear.cuh -- what the walks of the first-order linear attention share
// (hla2_linear.cu: CUDA cores and the entries, hla2_linear_tc.cu: tensor cores).
//
// Every pass of the operator is one kind of walk over the tokens of a head:
//   forward in time   o_i = sum_{j<=i} g^(i-j) (a_i . b_j) c_j + g^(i+1) S_in^T a_i
//   backward in time  o_j = sum_{i>=j} g^(i-j) (a_j . b_i) c_i + g^(T-1-j) S_in^T a_j
// with a state S = sum of the decayed b c^T, [da][dc].  The output is the walk
// (q, k, v); the gradients are dQ = (dO, v, k) forwards, with S transposed, and
// dK = (v, dO, q) and dV = (k, q, dO) backwards, from the last state's gradient.
//
// A head's chunks are cut into nseg segments, a CTA each.  Walk index w counts
// segments in walk order.  With more than one: every segment (the last one
// only where the last state is wanted) leaves its own sum (from zero) in slot
// w + 1 of the head's records, a scan turns the slots into the states that
// enter the segments and writes the last state, and the second walk starts from
// slot w.  A single segment's walk writes the last state itself.
#pragma once

#include "hla2_layer.cuh"

namespace hla2 {

struct LinWalk {
    const void *a, *b, *c;
    void* o;
    long long sa[3], sb[3], sc[3], so[3];  // element strides of b, h, t
    int B, H, T, da, dc;
    const float* gamma;  // [H]
    const int* lengths;  // [B] or null: all T
    const float* s_in;   // [BH][da * dc], element (r, c) at r in_r + c in_c; null: zero
    float* s_out;        // the same with out_r, out_c; null: not wanted
    long long in_r, in_c, out_r, out_c;
    float* rec;  // [BH][nseg + 1][da * dc] (nseg > 1), a state that enters has (r, c) at r rec_r + c rec_c
    long long rec_r, rec_c;  // (dK's walk reads dV's states, transposed)
    int nseg, seglen, nchunk;
    int rev;
    int fours;  // CUDA cores: bits 0..2, a, b, c are read four values at a time
    int* status;
    int after;  // host: what the stream was given last is a kernel of the same call
};

// segments whose own sums are formed
inline int lin_state_segments(const LinWalk& w) { return w.s_out ? w.nseg : w.nseg - 1; }

// Tensor cores (hla2_linear_tc.cu): bf16, da and dc up to 128, rows and bases
// of whole 16-byte steps.  chunks of 128 tokens.
constexpr int kLinTcChunk = 128;
inline int lin_tc_ctas(int da, int dc) { return da <= 64 && dc <= 64 ? 2 : 1; }  // to an SM
bool lin_tc_supported(const LinWalk& w, int dtype);
cudaError_t launch_lin_tc(const LinWalk& w, bool states, cudaStream_t s);

namespace {

// g^n, n >= 0 (g^0 = 1 for any g), by squaring with sums of two fp32 numbers, so
// that far powers of decays next to one keep all 24 bits (64-bit products are
// 60 times as slow here, which a CTA's start would notice)
struct Twofold {
    float hi, lo;
};
__device__ __forceinline__ Twofold operator*(Twofold a, Twofold b) {
    const float p = a.hi * b.hi, e = fmaf(a.hi, b.hi, -p) + fmaf(a.hi, b.lo, a.lo * b.hi), s = p + e;
    return {s, e - (s - p)};
}
__device__ __forceinline__ float power(float g, int n) {
    Twofold r{1.f, 0.f}, q{g, 0.f};
    for (; n; n >>= 1) {
        if (n & 1) r = r * q;
        q = q * q;
    }
    return r.hi;
}
__device__ __forceinline__ int length_of(const LinWalk& p, int b) {
    return p.lengths ? min(max(__ldg(p.lengths + b), 0), p.T) : p.T;
}

}  // namespace
}  // namespace hla2
