// hla2_rotary.cu -- rotary positions with several axes on queries and keys.
//
// Pair p of a head turns by the angle pos[axis(p)][b][t] * freq[p]:
//   (x, y) -> (x cos - y sin, x sin + y cos);
// the inverse turn (the gradient) flips the sine.
//
// The work is one read and one write of every element; the angle, its
// reduction and the sine and cosine depend on the token and the pair alone.
// So a block takes the sines of a few tokens once, into shared memory, and then
// streams the tokens' heads, of Q and of K, through its threads, a run of
// channels and its partners at a time: 65536 tokens x 32 heads need 4M sines
// instead of 134M.  It walks the heads (or the tokens) in the order in which
// they lie in memory: a walk that has all blocks at the same head of different
// tokens, 4 KB apart, reached 0.54 of the copy bandwidth.  For the same reason a
// block takes about 64 KB of Q and K, one row in flight to a thread and eight
// blocks to an SM: few addresses, close together.  65536 tokens x 32 heads x 128
// in 16 bits (1.07 GB): 168 us, 0.94 of the copy bandwidth; with 16 and 32 tokens
// to a block (128 and 256 KB) 172 and 184 us, with two and four rows in flight
// (and 32 tokens) 197 and 228 us.
//
// The angle is reduced in revolutions: freq / (2 pi) is carried as a sum of two
// fp32 numbers, its product with the position as a sum of two more (the
// rounding error of a product comes from one fma), and the nearest whole
// number is subtracted exactly; positions of 2^24 and more, and angles of 2^23 and
// more, go through sums of two fp64 numbers.  So the angle is good to fp32 at every
// position and frequency.
#include <cstdlib>

#include "hla2_layer.cuh"

namespace hla2 {
namespace {

constexpr int kRotThreads = 256;
constexpr int kRotTokens = 32;         // tokens to a block, at most
constexpr int kRotBytes = 64 * 1024;   // of Q and K to a block, about

struct RotParams {
    const void *q, *k;
    void *oq, *ok;
    const int* pos;
    const float* freq;
    int B, H, HK, T, d, rot;
    int ends[4];   // axis of pair p: the first a with p < ends[a]
    int slots;     // threads to a row: pairs / V, then 2 V copied channels each
    int tokens;    // of a block
    int head_inner;  // heads of a token, not tokens of a head, are neighbours in memory
    int inverse;
    long long total;  // B * T
    long long sq[3], soq[3], sk[3], sok[3], sp[2];
};

// 1 / (2 pi) as a sum of two fp32 numbers
constexpr double kInvTwoPi = 0.15915494309189533577;
constexpr float kInvTwoPiHi = (float)kInvTwoPi;
constexpr float kInvTwoPiLo = (float)(kInvTwoPi - (double)kInvTwoPiHi);
constexpr double kInvTwoPiRest = -9.839338337591243477019410e-18;  // 1 / (2 pi) less kInvTwoPi

// pos * (hi + lo) less the nearest whole number, of fewer than 2^21 turns of a whole
// |pos| < 2^24: the pair holds about 48 bits, so the result is off by less than 2^-26
// of a turn
__device__ __forceinline__ float turn_fraction(float pos, float hi, float lo) {
    const float p = pos * hi;
    const float e = fmaf(pos, hi, -p) + pos * lo;
    return (p - rintf(p)) + e;
}

// sine and cosine of pos * f
__device__ __forceinline__ void turn_of(int ps, float f, float& si, float& co) {
    const float hi = f * kInvTwoPiHi;
    const float lo = fmaf(f, kInvTwoPiHi, -hi) + f * kInvTwoPiLo;
    float r;
    if (ps > -(1 << 24) && ps < (1 << 24) && fabsf((float)ps * f) < 0x1p23f) {
        r = turn_fraction((float)ps, hi, lo);
    } else {  // beyond what 48 bits of revolutions resolve: the same in fp64, 106 bits
        const double dh = (double)f * kInvTwoPi, dl = fma((double)f, kInvTwoPi, -dh) + (double)f * kInvTwoPiRest;
        const double p = ps * dh, e = fma((double)ps, dh, -p) + ps * dl;
        const double t = (p - rint(p)) + e;
        r = (float)(t - rint(t));
    }
    sincospif(2.f * r, &si, &co);
}

template <typename T, int V, bool IL>
__global__ void __launch_bounds__(kRotThreads, V == 8 ? 8 : 1) rotary_kernel(const __grid_constant__ RotParams p) {
    constexpr bool VEC = V > 1;
    extern __shared__ __align__(16) unsigned char raw[];
    // where each token's heads are: element offsets of Q, OQ, K, OK
    __shared__ long long at[4][kRotTokens];
    __shared__ int pos_at[kRotTokens][2];  // b, t
    const int tid = threadIdx.x, pairs = p.rot >> 1, turning = pairs / V;
    const long long first = (long long)blockIdx.x * p.tokens;
    const int nt = (int)min((long long)p.tokens, p.total - first);
    if (tid < nt) {
        const long long bt = first + tid;
        const long long b = bt / p.T, t = bt - b * p.T;
        at[0][tid] = b * p.sq[0] + t * p.sq[2];
        at[1][tid] = b * p.soq[0] + t * p.soq[2];
        at[2][tid] = b * p.sk[0] + t * p.sk[2];
        at[3][tid] = b * p.sok[0] + t * p.sok[2];
        pos_at[tid][0] = (int)b;
        pos_at[tid][1] = (int)t;
    }
    __syncthreads();
    const int slot = tid % p.slots, group = tid / p.slots, groups = kRotThreads / p.slots;
    const int heads = p.H + p.HK;
    const unsigned rows = (unsigned)nt * (unsigned)heads;
    const bool turns = slot < turning;
    // this thread's channels: two runs of V, the partners of V pairs or copied ones
    const int p0 = slot * V;
    const int c0 = turns ? (IL ? 2 * p0 : p0) : p.rot + (p0 - pairs) * 2;
    const int c1 = turns ? (IL ? 2 * p0 + V : p0 + pairs) : c0 + V;
    const int n0 = min(V, p.d - c0), n1 = min(V, p.d - c1);  // copied runs may end the head
    auto locate = [&](unsigned r, int& tok, int& h) {
        if (p.head_inner) { tok = (int)(r / (unsigned)heads); h = (int)(r - (unsigned)tok * (unsigned)heads); }
        else { h = (int)(r / (unsigned)nt); tok = (int)(r - (unsigned)h * (unsigned)nt); }
    };
    Lane<T, V, VEC> x, y;
    auto load = [&](unsigned r) {
        int tok, h;
        locate(r, tok, h);
        const T* s = h < p.H ? static_cast<const T*>(p.q) + at[0][tok] + h * p.sq[1]
                             : static_cast<const T*>(p.k) + at[2][tok] + (h - p.H) * p.sk[1];
        if (n0 > 0) x.load(s + c0, n0);
        if (n1 > 0) y.load(s + c1, n1);
    };
    const bool works = group < groups && (unsigned)group < rows;
    if (works) load(group);  // on its way while the sines are taken

    // sines: 4 pairs' cosines (or sines) are one 16-byte word; a token's words lie
    // so that the threads of a row read neighbouring ones
    float* const table = reinterpret_cast<float*>(raw);
    auto entry = [&](int tok, int pr, int which) -> int {
        if (VEC) {
            const int s = pr / V, j = pr % V;  // thread of the row, pair of the thread
            return ((tok * (V / 4) * 2 + (j / 4) * 2 + which) * turning + s) * 4 + j % 4;
        }
        return (tok * 2 + which) * pairs + pr;
    };
    for (int i = tid; i < nt * pairs; i += kRotThreads) {
        const int tok = i / pairs, pr = i - tok * pairs;
        const int a = (pr >= p.ends[0]) + (pr >= p.ends[1]) + (pr >= p.ends[2]);
        const int ps = __ldg(p.pos + a * p.sp[0] + pos_at[tok][0] * p.sp[1] + pos_at[tok][1]);
        float si, co;
        turn_of(ps, __ldg(p.freq + pr), si, co);
        table[entry(tok, pr, 0)] = co;
        table[entry(tok, pr, 1)] = p.inverse ? -si : si;
    }
    __syncthreads();
    if (!works) return;
    for (unsigned r = group; r < rows; r += groups) {
        if (r != (unsigned)group) load(r);
        int tok, h;
        locate(r, tok, h);
        if (turns) {
            float co[V], si[V];
            if constexpr (VEC) {
#pragma unroll
                for (int q = 0; q < V / 4; ++q) {
                    const float4 c4 = *reinterpret_cast<const float4*>(table + entry(tok, p0 + 4 * q, 0));
                    const float4 s4 = *reinterpret_cast<const float4*>(table + entry(tok, p0 + 4 * q, 1));
                    co[4 * q] = c4.x; co[4 * q + 1] = c4.y; co[4 * q + 2] = c4.z; co[4 * q + 3] = c4.w;
                    si[4 * q] = s4.x; si[4 * q + 1] = s4.y; si[4 * q + 2] = s4.z; si[4 * q + 3] = s4.w;
                }
            } else {
                co[0] = table[entry(tok, p0, 0)];
                si[0] = table[entry(tok, p0, 1)];
            }
            float u[V], v[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (IL && VEC) {  // pair j: elements 2j, 2j + 1 of the 2 V channels
                    const float a = 2 * j < V ? x.get((2 * j) % V) : y.get((2 * j) % V);
                    const float c = 2 * j < V ? x.get((2 * j + 1) % V) : y.get((2 * j + 1) % V);
                    const float r0 = a * co[j] - c * si[j], r1 = a * si[j] + c * co[j];
                    if (2 * j < V) { u[(2 * j) % V] = r0; u[(2 * j + 1) % V] = r1; }
                    else { v[(2 * j) % V] = r0; v[(2 * j + 1) % V] = r1; }
                } else {
                    const float a = x.get(j), c = y.get(j);
                    u[j] = a * co[j] - c * si[j];
                    v[j] = a * si[j] + c * co[j];
                }
            }
            x.set(u);
            y.set(v);
        }
        T* o = h < p.H ? static_cast<T*>(p.oq) + at[1][tok] + h * p.soq[1]
                       : static_cast<T*>(p.ok) + at[3][tok] + (h - p.H) * p.sok[1];
        if (n0 > 0) x.store(o + c0, n0);
        if (n1 > 0) y.store(o + c1, n1);
    }
}

template <typename T, int V>
cudaError_t launch_rotary(RotParams& p, bool interleaved, int sms, cudaStream_t s) {
    const int pairs = p.rot / 2, rest = p.d - p.rot;
    p.slots = pairs / V + (rest + 2 * V - 1) / (2 * V);
    p.total = (long long)p.B * p.T;
    p.tokens = kRotTokens;
    while (p.tokens > 1 && (long long)p.tokens * (p.H + p.HK) * p.d * sizeof(T) > kRotBytes) p.tokens /= 2;
    // and as few as leave four blocks to an SM
    while (p.tokens > 1 && (p.total + p.tokens - 1) / p.tokens < 4LL * sms) p.tokens /= 2;
    const unsigned blocks = (unsigned)((p.total + p.tokens - 1) / p.tokens);
    const size_t smem = (size_t)p.tokens * pairs * 8;
    if (interleaved) rotary_kernel<T, V, true><<<blocks, kRotThreads, smem, s>>>(p);
    else rotary_kernel<T, V, false><<<blocks, kRotThreads, smem, s>>>(p);
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
    p.head_inner = T == 1 || std::llabs(p.sq[1]) <= std::llabs(p.sq[2]);
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
