// hla2_rotary.cu -- rotary positions with several axes on queries and keys.
//
// Pair p of a head turns by the angle pos[axis(p)][b][t] * freq[p]:
//   (x, y) -> (x cos - y sin, x sin + y cos);
// the inverse turn (the gradient) flips the sine.
//
// The work is one read and one write of every element; the angle, its
// reduction and the sine and cosine depend on the token and the pair alone.
// So a thread owns V pairs of one token, takes their sines once into
// registers and then walks over the heads of Q and of K, four heads' loads in
// flight: 65536 tokens x 32 heads need 4M sines instead of 134M.
//
// The angle is reduced in revolutions: freq / (2 pi) is carried as a sum of two
// fp32 numbers, its product with the position as a sum of two more (the
// rounding error of a product comes from one fma), and the nearest whole
// number is subtracted exactly; positions of 2^24 and more go through fp64.
// So the angle is good to fp32 at every position.
#include "hla2_layer.cuh"

namespace hla2 {
namespace {

constexpr int kRotThreads = 256;
constexpr int kRotHeads = 4;  // heads whose loads are in flight together

struct RotParams {
    const void *q, *k;
    void *oq, *ok;
    const int* pos;
    const float* freq;
    int B, H, HK, T, d, rot;
    int ends[4];  // axis of pair p: the first a with p < ends[a]
    int slots;    // threads for each token: pairs / V, then 2 V copied channels each
    int heads_per_group;
    int inverse;
    long long total;  // B * T * slots
    long long sq[3], soq[3], sk[3], sok[3], sp[2];
};

// 1 / (2 pi) as a sum of two fp32 numbers
constexpr double kInvTwoPi = 0.15915494309189533577;
constexpr float kInvTwoPiHi = (float)kInvTwoPi;
constexpr float kInvTwoPiLo = (float)(kInvTwoPi - (double)kInvTwoPiHi);

// pos * (hi + lo) less the nearest whole number, for a whole |pos| < 2^24: the
// pair holds about 48 bits, so the result is off by less than 2^-26 of a turn
__device__ __forceinline__ float turn_fraction(float pos, float hi, float lo) {
    const float p = pos * hi;
    const float e = fmaf(pos, hi, -p) + pos * lo;
    return (p - rintf(p)) + e;
}

template <typename T, int V, bool IL>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const RotParams p) {
    constexpr bool VEC = V > 1;
    const long long idx = (long long)blockIdx.x * kRotThreads + threadIdx.x;
    if (idx >= p.total) return;
    int b, t, slot;
    if (p.total <= 0x7fffffffLL) {
        const unsigned i = (unsigned)idx, bt = i / (unsigned)p.slots;
        slot = (int)(i - bt * (unsigned)p.slots);
        b = (int)(bt / (unsigned)p.T);
        t = (int)(bt - (unsigned)b * (unsigned)p.T);
    } else {
        const long long bt = idx / p.slots;
        slot = (int)(idx - bt * p.slots);
        b = (int)(bt / p.T);
        t = (int)(bt - (long long)b * p.T);
    }
    const int pairs = p.rot >> 1;
    const int p0 = slot * V;
    const bool turns = p0 < pairs;
    // channels of this thread: two runs of V, the partners of V pairs or copied ones
    const int c0 = turns ? (IL ? 2 * p0 : p0) : p.rot + (p0 - pairs) * 2;
    const int c1 = turns ? (IL ? 2 * p0 + V : p0 + pairs) : c0 + V;
    const int n0 = min(V, p.d - c0), n1 = min(V, p.d - c1);  // copied runs may end the head

    const int heads = p.H + p.HK;
    const int h_begin = blockIdx.y * p.heads_per_group, h_end = min(heads, h_begin + p.heads_per_group);
    auto src = [&](int h) -> const T* {
        return h < p.H ? static_cast<const T*>(p.q) + b * p.sq[0] + h * p.sq[1] + t * p.sq[2]
                       : static_cast<const T*>(p.k) + b * p.sk[0] + (h - p.H) * p.sk[1] + t * p.sk[2];
    };
    auto dst = [&](int h) -> T* {
        return h < p.H ? static_cast<T*>(p.oq) + b * p.soq[0] + h * p.soq[1] + t * p.soq[2]
                       : static_cast<T*>(p.ok) + b * p.sok[0] + (h - p.H) * p.sok[1] + t * p.sok[2];
    };
    Lane<T, V, VEC> x[kRotHeads], y[kRotHeads];
    auto load = [&](int h0) {
#pragma unroll
        for (int i = 0; i < kRotHeads; ++i)
            if (h0 + i < h_end) {
                if (n0 > 0) x[i].load(src(h0 + i) + c0, n0);
                if (n1 > 0) y[i].load(src(h0 + i) + c1, n1);
            }
    };
    load(h_begin);  // the first heads' loads pass the sines

    float co[V], si[V];
    if (turns) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int pr = p0 + j;
            const int a = (pr >= p.ends[0]) + (pr >= p.ends[1]) + (pr >= p.ends[2]);
            const int ps = __ldg(p.pos + a * p.sp[0] + b * p.sp[1] + t);
            const float f = __ldg(p.freq + pr);
            const float hi = f * kInvTwoPiHi;
            const float lo = fmaf(f, kInvTwoPiHi, -hi) + f * kInvTwoPiLo;
            float r;
            if (ps > -(1 << 24) && ps < (1 << 24)) {
                r = turn_fraction((float)ps, hi, lo);
            } else {  // beyond what 48 bits of revolutions resolve
                const double turns = (double)ps * ((double)f * kInvTwoPi);
                r = (float)(turns - rint(turns));
            }
            sincospif(2.f * r, &si[j], &co[j]);
            if (p.inverse) si[j] = -si[j];
        }
    }
    for (int h0 = h_begin; h0 < h_end; h0 += kRotHeads) {
        if (h0 != h_begin) load(h0);
#pragma unroll
        for (int i = 0; i < kRotHeads; ++i) {
            if (h0 + i >= h_end) break;
            if (turns) {
                float u[V], v[V];
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    if (IL && VEC) {  // pair j: elements 2j, 2j + 1 of the 2 V channels
                        const float a = 2 * j < V ? x[i].get((2 * j) % V) : y[i].get((2 * j) % V);
                        const float c = 2 * j < V ? x[i].get((2 * j + 1) % V) : y[i].get((2 * j + 1) % V);
                        const float r0 = a * co[j] - c * si[j], r1 = a * si[j] + c * co[j];
                        if (2 * j < V) { u[(2 * j) % V] = r0; u[(2 * j + 1) % V] = r1; }
                        else { v[(2 * j) % V] = r0; v[(2 * j + 1) % V] = r1; }
                    } else {
                        const float a = x[i].get(j), c = y[i].get(j);
                        u[j] = a * co[j] - c * si[j];
                        v[j] = a * si[j] + c * co[j];
                    }
                }
                x[i].set(u);
                y[i].set(v);
            }
            T* o = dst(h0 + i);
            if (n0 > 0) x[i].store(o + c0, n0);
            if (n1 > 0) y[i].store(o + c1, n1);
        }
    }
}

template <typename T, int V>
cudaError_t launch_rotary(RotParams& p, bool interleaved, int sms, cudaStream_t s) {
    const int pairs = p.rot / 2, rest = p.d - p.rot;
    p.slots = pairs / V + (rest + 2 * V - 1) / (2 * V);
    p.total = (long long)p.B * p.T * p.slots;
    // Heads are split over thread groups only as far as the tokens leave SMs
    // idle: each group takes its sines anew.
    const int heads = p.H + p.HK;
    const long long want = (long long)sms * 1024;
    long long groups = (want + p.total - 1) / p.total;
    if (groups > heads) groups = heads;
    if (groups < 1) groups = 1;
    p.heads_per_group = (int)((heads + groups - 1) / groups);
    groups = (heads + p.heads_per_group - 1) / p.heads_per_group;
    const dim3 grid((unsigned)((p.total + kRotThreads - 1) / kRotThreads), (unsigned)groups);
    if (interleaved) rotary_kernel<T, V, true><<<grid, kRotThreads, 0, s>>>(p);
    else rotary_kernel<T, V, false><<<grid, kRotThreads, 0, s>>>(p);
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace
}  // namespace hla2

extern "C" int hla2_rotary(const void* Q, void* OQ, const void* K, void* OK, const int* pos, const float* freq, int B,
                           int H, int HK, int T, int d, int rot, int naxes, const int* sections, int interleaved,
                           int inverse, const long long* strides, int dtype, hla2_stream_t stream) {
    using namespace hla2;
    if (B <= 0 || H <= 0 || HK < 0 || T <= 0 || d <= 0)
        return set_error(HLA2_ERR_INVALID, "sizes must be positive (B=%d H=%d HK=%d T=%d d=%d)", B, H, HK, T, d);
    if (!Q || !OQ || !pos || !freq || !sections) return set_error(HLA2_ERR_INVALID, "null pointer");
    if ((HK > 0) != (K != nullptr) || (HK > 0) != (OK != nullptr))
        return set_error(HLA2_ERR_INVALID, "K and OK are given exactly when HK > 0");
    if (!known_dtype(dtype)) return set_error(HLA2_ERR_UNSUPPORTED, "unknown dtype %d", dtype);
    if (d > 128) return set_error(HLA2_ERR_UNSUPPORTED, "d=%d: this build supports d <= 128", d);
    if (rot <= 0 || rot > d || (rot & 1)) return set_error(HLA2_ERR_INVALID, "rot=%d must be even and in 2..d", rot);
    if (naxes < 1 || naxes > 4) return set_error(HLA2_ERR_INVALID, "naxes=%d must be in 1..4", naxes);
    if ((long long)B * ((long long)H + HK) > 65535)
        return set_error(HLA2_ERR_UNSUPPORTED, "B*(H+HK)=%lld exceeds 65535", (long long)B * ((long long)H + HK));
    if ((long long)B * T > (1LL << 31)) return set_error(HLA2_ERR_UNSUPPORTED, "B*T exceeds 2^31");
    int end = 0;
    RotParams p{};
    for (int a = 0; a < 4; ++a) {
        if (a < naxes) {
            if (sections[a] <= 0 || sections[a] > rot / 2) return set_error(HLA2_ERR_INVALID, "sections[%d]=%d", a, sections[a]);
            end += sections[a];
        }
        p.ends[a] = end;
    }
    if (end != rot / 2) return set_error(HLA2_ERR_INVALID, "sections add up to %d, not rot/2=%d", end, rot / 2);
    const int es = dtype_size(dtype);
    if (!aligned_elem(Q, es) || !aligned_elem(OQ, es) || !aligned_elem(K, es) || !aligned_elem(OK, es) ||
        !aligned_elem(pos, 4) || !aligned_elem(freq, 4))
        return set_error(HLA2_ERR_INVALID, "pointer not aligned to its element");
    p.q = Q; p.k = K; p.oq = OQ; p.ok = OK; p.pos = pos; p.freq = freq;
    p.B = B; p.H = H; p.HK = HK; p.T = T; p.d = d; p.rot = rot; p.inverse = inverse != 0;
    if (strides) {
        for (int i = 0; i < 3; ++i) {
            p.sq[i] = strides[i]; p.soq[i] = strides[3 + i]; p.sk[i] = strides[6 + i]; p.sok[i] = strides[9 + i];
        }
        p.sp[0] = strides[12]; p.sp[1] = strides[13];
    } else {
        p.sq[0] = p.soq[0] = (long long)H * T * d; p.sk[0] = p.sok[0] = (long long)HK * T * d;
        p.sq[1] = p.soq[1] = p.sk[1] = p.sok[1] = (long long)T * d;
        p.sq[2] = p.soq[2] = p.sk[2] = p.sok[2] = d;
        p.sp[0] = (long long)B * T; p.sp[1] = T;
    }
    auto fits = [&](int bytes) {
        return aligned_to(Q, es, p.sq, 3, bytes) && aligned_to(OQ, es, p.soq, 3, bytes) &&
               aligned_to(K, es, p.sk, 3, bytes) && aligned_to(OK, es, p.sok, 3, bytes);
    };
    // V pairs to a thread need both runs of channels, and the copied ones, whole and aligned
    const int pairs = rot / 2, rest = d - rot;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int sms = sm_count();
    cudaError_t e;
    if (dtype == HLA2_DTYPE_BF16) {
        if (pairs % 8 == 0 && rest % 8 == 0 && fits(16)) e = launch_rotary<bf16, 8>(p, interleaved != 0, sms, s);
        else if (pairs % 4 == 0 && rest % 4 == 0 && fits(8)) e = launch_rotary<bf16, 4>(p, interleaved != 0, sms, s);
        else e = launch_rotary<bf16, 1>(p, interleaved != 0, sms, s);
    } else {
        if (pairs % 4 == 0 && rest % 4 == 0 && fits(16)) e = launch_rotary<float, 4>(p, interleaved != 0, sms, s);
        else e = launch_rotary<float, 1>(p, interleaved != 0, sms, s);
    }
    if (e != cudaSuccess) return set_error(HLA2_ERR_LAUNCH, "rotary: %s", cudaGetErrorString(e));
    return HLA2_OK;
}
