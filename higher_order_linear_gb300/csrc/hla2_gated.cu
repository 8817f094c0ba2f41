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
#include "hla2_layer.cuh"

namespace hla2 {
namespace {

constexpr int kTile = 64;  // tokens between two kept states

struct GateParams {
    const void *x, *g, *dout;
    const unsigned char* reset;
    const float *state_in, *dstate_out;
    void *o, *dx, *dg;
    float *state_out, *dstate_in, *carry;
    int B, H, T, d;
    long long sx[3], sg[3], so[3], sdo[3], sdx[3], sdg[3];
};

// z = 1 - a of the sigmoid gate
__device__ __forceinline__ float keep_out(float g) {
    const float e = __expf(-g);
    return isinf(e) ? 1.f : __fdividef(e, 1.f + e);
}

template <typename T, typename TO, bool SIG, bool SHARED>
__global__ void __launch_bounds__(128) gated_simple_kernel(const GateParams p) {
    const int c = threadIdx.x, b = blockIdx.x / p.H, hd = blockIdx.x % p.H;
    if (c >= p.d) return;
    const long long row = (long long)blockIdx.x * p.d + c;
    const int tiles = (p.T + kTile - 1) / kTile;
    const T* x = static_cast<const T*>(p.x) + b * p.sx[0] + hd * p.sx[1] + c;
    const T* g = static_cast<const T*>(p.g) + b * p.sg[0] + hd * p.sg[1] + (SHARED ? 0 : c);
    TO* o = static_cast<TO*>(p.o) + b * p.so[0] + hd * p.so[1] + c;
    float h = p.state_in ? p.state_in[row] : 0.f;
    for (int t = 0; t < p.T; ++t) {
        if (p.carry && t % kTile == 0) p.carry[((long long)blockIdx.x * tiles + t / kTile) * p.d + c] = h;
        if (p.reset && p.reset[(long long)b * p.T + t]) h = 0.f;
        const float xv = to_f32(x[t * p.sx[2]]), gv = to_f32(g[t * p.sg[2]]);
        h = SIG ? fmaf(keep_out(gv), xv - h, h) : fmaf(gv, h, xv);
        o[t * p.so[2]] = from_f32<TO>(h);
    }
    if (p.state_out) p.state_out[row] = h;
}

template <typename T, typename TO, bool SIG, bool SHARED>
__global__ void __launch_bounds__(128) gated_simple_bwd_kernel(const GateParams p) {
    __shared__ float before[kTile][128];  // h_{t-1} of this tile's tokens
    __shared__ float part[128];
    const int c = threadIdx.x, b = blockIdx.x / p.H, hd = blockIdx.x % p.H;
    const bool in = c < p.d;
    const long long row = (long long)blockIdx.x * p.d + c;
    const int tiles = (p.T + kTile - 1) / kTile;
    const int cc = in ? c : 0;
    const T* x = static_cast<const T*>(p.x) + b * p.sx[0] + hd * p.sx[1] + cc;
    const T* g = static_cast<const T*>(p.g) + b * p.sg[0] + hd * p.sg[1] + (SHARED ? 0 : cc);
    const TO* dout = static_cast<const TO*>(p.dout) + b * p.sdo[0] + hd * p.sdo[1] + cc;
    T* dx = static_cast<T*>(p.dx) + b * p.sdx[0] + hd * p.sdx[1] + cc;
    T* dg = static_cast<T*>(p.dg) + b * p.sdg[0] + hd * p.sdg[1] + (SHARED ? 0 : cc);
    float mu = in && p.dstate_out ? p.dstate_out[row] : 0.f;  // a_{t+1} lam_{t+1}
    for (int tile = tiles - 1; tile >= 0; --tile) {
        const int t0 = tile * kTile, t1 = min(p.T, t0 + kTile);
        float h = in ? p.carry[((long long)blockIdx.x * tiles + tile) * p.d + c] : 0.f;
        for (int t = t0; t < t1; ++t) {
            if (p.reset && p.reset[(long long)b * p.T + t]) h = 0.f;
            before[t - t0][c] = h;
            const float xv = to_f32(x[t * p.sx[2]]), gv = to_f32(g[t * p.sg[2]]);
            h = SIG ? fmaf(keep_out(gv), xv - h, h) : fmaf(gv, h, xv);
        }
        for (int t = t1 - 1; t >= t0; --t) {
            const float xv = to_f32(x[t * p.sx[2]]), gv = to_f32(g[t * p.sg[2]]), hb = before[t - t0][c];
            const float lam = to_f32(dout[t * p.sdo[2]]) + mu;
            float gx, gg, a;
            if (SIG) {
                const float z = keep_out(gv);
                a = 1.f - z;
                gx = z * lam;
                gg = gx * a * (hb - xv);
            } else {
                a = gv;
                gx = lam;
                gg = lam * hb;
            }
            mu = (p.reset && p.reset[(long long)b * p.T + t]) ? 0.f : a * lam;
            if (in) dx[t * p.sdx[2]] = from_f32<T>(gx);
            if (SHARED) {
                __syncthreads();
                part[c] = in ? gg : 0.f;
                __syncthreads();
                if (c == 0) {
                    float s = 0.f;
                    for (int i = 0; i < p.d; ++i) s += part[i];
                    dg[t * p.sdg[2]] = from_f32<T>(s);
                }
            } else if (in) {
                dg[t * p.sdg[2]] = from_f32<T>(gg);
            }
        }
    }
    if (in && p.dstate_in) p.dstate_in[row] = mu;
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

}  // namespace
}  // namespace hla2

extern "C" size_t hla2_gated_scan_workspace(int B, int H, int T, int d) {
    (void)B; (void)H; (void)T; (void)d;
    return 0;
}

extern "C" size_t hla2_gated_scan_carry_len(int T, int d) {
    if (T <= 0 || d <= 0) return 0;
    return (size_t)((T + hla2::kTile - 1) / hla2::kTile) * d;
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
    GateParams p{};
    p.x = X; p.g = G; p.reset = reset; p.state_in = state_in; p.o = O; p.state_out = state_out; p.carry = carry;
    p.B = B; p.H = H; p.T = T; p.d = d;
    take_strides(p.sx, strides, 0, H, T, d);
    take_strides(p.sg, strides, 1, H, T, gate_shared ? 1 : d);
    take_strides(p.so, strides, 2, H, T, d);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = by_types(dtype, out_dtype, [&](auto tin, auto tout) {
        return by_form(form, gate_shared, [&](auto sig, auto shared) {
            gated_simple_kernel<decltype(tin), decltype(tout), decltype(sig)::value, decltype(shared)::value>
                <<<B * H, 128, 0, s>>>(p);
            return cudaGetLastError();
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
    GateParams p{};
    p.x = X; p.g = G; p.reset = reset; p.carry = const_cast<float*>(carry); p.dout = dO; p.dstate_out = dstate_out;
    p.dx = dX; p.dg = dG; p.dstate_in = dstate_in;
    p.B = B; p.H = H; p.T = T; p.d = d;
    take_strides(p.sx, strides, 0, H, T, d);
    take_strides(p.sg, strides, 1, H, T, gate_shared ? 1 : d);
    take_strides(p.sdo, strides, 2, H, T, d);
    take_strides(p.sdx, strides, 3, H, T, d);
    take_strides(p.sdg, strides, 4, H, T, gate_shared ? 1 : d);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = by_types(dtype, out_dtype, [&](auto tin, auto tout) {
        return by_form(form, gate_shared, [&](auto sig, auto shared) {
            gated_simple_bwd_kernel<decltype(tin), decltype(tout), decltype(sig)::value, decltype(shared)::value>
                <<<B * H, 128, 0, s>>>(p);
            return cudaGetLastError();
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
