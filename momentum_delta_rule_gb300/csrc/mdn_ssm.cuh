// Declarations shared by the state-space layer's translation units: problem
// structs, launchers, packets of elements and the elementwise functions.
#pragma once

#include "mdn_internal.cuh"

namespace mdn {

struct ConvProblem {
    const void *x, *dy;
    const float *w, *bias;
    const void *state0, *dstate_T;
    void *y, *state_T;              // forward, step (state0 -> state_T)
    void *dx, *dstate0;             // gradient
    float *dw, *dbias, *partial;
    const int32_t *cu;              // device, or nullptr for equal lengths
    int n_seq, T, T_total, D, width, act;
    long ld_x, ld_dy;
    mdn_dtype dtype;
    int *status;
};

struct ScanProblem {
    const void *u, *dt, *z, *Bm, *Cm, *dy;
    const float *A, *D_skip, *dt_bias;
    const float *h0;                // initial states (fwd), state before the token (step)
    void *y;
    float *h_T, *h_chunks;
    // gradient
    const float *dh_T;
    void *du, *ddt, *dz, *dB, *dC;
    float *dA, *dD, *ddt_bias, *dh0;
    long ld_u, ld_dt, ld_z, ld_B, ld_C, ld_dy;
    const int32_t *cu;
    int n_seq, T, T_total, D, G, N, softplus;
    mdn_dtype dtype;
    int *status;
    unsigned char *ws;
};

struct NormProblem {
    const void *y, *x, *gate, *dx_out, *dh;
    const float *w_post, *w_pre, *scale;
    void *x_out, *h, *dy, *dx, *dgate;
    float *stats, *dw_post, *dw_pre, *dscale, *partial;
    int rows, D, gate_act;
    float eps;
    long ld_y, ld_x, ld_gate, ld_dx_out, ld_dh;
    mdn_dtype dtype;
};

cudaError_t launch_conv_fwd(const ConvProblem &p, cudaStream_t st);
cudaError_t launch_conv_bwd(const ConvProblem &p, cudaStream_t st);
cudaError_t launch_conv_step(const ConvProblem &p, cudaStream_t st);
size_t conv_bwd_workspace(int T_total, int D, int width, mdn_dtype dtype);
cudaError_t launch_scan_fwd(const ScanProblem &p, cudaStream_t st);
cudaError_t launch_scan_bwd(const ScanProblem &p, cudaStream_t st);
cudaError_t launch_scan_step(const ScanProblem &p, cudaStream_t st);
size_t scan_fwd_workspace(int n_seq, int T_total, int D, int G, int N, mdn_dtype dtype);
size_t scan_bwd_workspace(int n_seq, int T_total, int D, int G, int N, mdn_dtype dtype);
cudaError_t launch_norm_fwd(const NormProblem &p, cudaStream_t st);
cudaError_t launch_norm_bwd(const NormProblem &p, cudaStream_t st);
size_t norm_bwd_workspace(int rows, int D, mdn_dtype dtype);

// Supported device check and the device status word's address (mdn_api.cu).
mdn_status current_device_status(int **status);

inline size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

// Whether `bytes`-wide packets reach every row of a [rows, width] array of
// `el`-byte elements whose rows lie ld elements apart.
inline bool rows_aligned(const void *ptr, long ld, int el, int bytes) {
    return ptr == nullptr || (((uintptr_t)ptr % bytes) == 0 && (ld * el) % bytes == 0);
}

// ---------------------------------------------------------------- device

// V consecutive elements as one packet (V * sizeof(T) = 2 .. 32 bytes) <-> fp32.
template <typename T, int V>
struct alignas(V * sizeof(T) < 16 ? V * sizeof(T) : 16) Packet {
    T e[V];
};

template <typename T, int V>
__device__ __forceinline__ void unpack(const Packet<T, V> &p, float *f) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = to_f32(p.e[i]);
}
template <typename T, int V>
__device__ __forceinline__ Packet<T, V> pack(const float *f) {
    Packet<T, V> p;
#pragma unroll
    for (int i = 0; i < V; ++i) p.e[i] = from_f32<T>(f[i]);
    return p;
}
template <typename T, int V>
__device__ __forceinline__ Packet<T, V> load_packet(const T *src) {
    return *reinterpret_cast<const Packet<T, V> *>(src);
}
template <typename T, int V>
__device__ __forceinline__ void store_packet(T *dst, const Packet<T, V> &p) {
    *reinterpret_cast<Packet<T, V> *>(dst) = p;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// 1 / (1 + e^{-x}); a large e^{-x} gives 0.
__device__ __forceinline__ float sigmoid_f(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// log(1 + e^x) = max(x, 0) + log(1 + e), e = e^{-|x|} in (0, 1], with
// log(1 + e) = 2 atanh(r), r = e / (2 + e) <= 1/3, from the series
// 2 r (1 + r^2/3 + r^4/5 + ...): its terms up to r^14 leave out less than
// 1e-8 of the sum, and a small e keeps its relative accuracy, which
// log(1.f + e) would lose in rounding the sum.
__device__ __forceinline__ float softplus_rel(float x) {
    const float e = expf(-fabsf(x));
    const float r = __fdividef(e, 2.f + e);
    const float q = r * r;
    float s = fmaf(q, 1.f / 15.f, 1.f / 13.f);
    s = fmaf(q, s, 1.f / 11.f);
    s = fmaf(q, s, 1.f / 9.f);
    s = fmaf(q, s, 1.f / 7.f);
    s = fmaf(q, s, 1.f / 5.f);
    s = fmaf(q, s, 1.f / 3.f);
    s = fmaf(q, s, 1.f);
    return fmaf(2.f * r, s, fmaxf(x, 0.f));
}

// The sequence that token t of a packed batch belongs to: the largest s with
// cu[s] <= t.  In bounds for any array contents.
__device__ __forceinline__ int seq_of_token(const int32_t *cu, int n_seq, long t) {
    int lo = 0, hi = n_seq;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid; else hi = mid;
    }
    return lo;
}

// Whether cu_seqlens is well formed (whole CTA; uniform result).
__device__ __forceinline__ bool cu_well_formed(const int32_t *cu, int n_seq, int T_total) {
    int bad = 0;
    for (int s = threadIdx.x; s < n_seq; s += blockDim.x) bad |= cu[s] > cu[s + 1];
    if (threadIdx.x == 0) bad |= cu[0] != 0 || cu[n_seq] != T_total;
    return !__syncthreads_or(bad);
}

}  // namespace mdn
