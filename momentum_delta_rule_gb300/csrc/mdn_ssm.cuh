// Declarations shared by the state-space layer's translation units: problem
// structs, launchers, packets of elements and the elementwise functions.
#pragma once

#include <type_traits>

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
    bool bc_wide;                   // four neighbouring states of B and C make one packet
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

// Lets a kernel have `bytes` of dynamic shared memory, the most that any of its
// launches takes: once on each device, since the limit is the device's and not
// the call's, and another host thread may be between its limit and its launch.
template <auto Kernel>
inline cudaError_t allow_shared(int bytes) {
    static std::atomic<uint64_t> done{0};
    // 48 KiB need no asking; the kernels' own static arrays count towards them
    if (bytes <= 47 * 1024) return cudaSuccess;
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    err = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return err;
}

// The widest packet (elements: `most`, 2 or 1) for which `fits(bytes)` holds;
// 2 only for two-byte elements, which it lets be copied asynchronously.  What
// the width is worth, in us, for bf16 rows of 2048, 2044 and 2047 channels
// (the convolution's widest is 4): gated norm of 16384 rows 51, 115, 258;
// its gradient 122, 189, 335; scan of 8192 tokens 108, 128, 271.
template <typename F>
inline int packet_width(int most, int el, F fits) {
    if (fits(most, most * el)) return most;
    return el == 2 && fits(2, 4) ? 2 : 1;
}

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

template <int BYTES>
__device__ __forceinline__ void cp_async(void *dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src), "n"(BYTES)
                 : "memory");
}
// Copies one packet from global to shared memory: asynchronously (visible to
// this thread after wait_copies) where it is 4, 8 or 16 bytes, at once
// otherwise.
template <typename T, int V>
__device__ __forceinline__ void copy_packet(Packet<T, V> *dst, const T *src) {
    if constexpr (V * sizeof(T) >= 4) cp_async<V * (int)sizeof(T)>(dst, src);
    else *dst = load_packet<T, V>(src);
}
// The same for N packets at a time, without a wait whatever their size: packets
// too small for an asynchronous copy are loaded into registers, and stored when
// the next N are asked for (or by `put`), by when they have arrived.
template <typename T, int V, int N>
struct Copies {
    static constexpr bool kAsync = V * sizeof(T) >= 4;
    static constexpr uint32_t kNone = 0xffffffffu;
    Packet<T, V> held[kAsync ? 1 : N];
    uint32_t at[kAsync ? 1 : N];      // shared-memory addresses, kNone for none

    __device__ __forceinline__ void clear() {
        if constexpr (!kAsync) {
#pragma unroll
            for (int i = 0; i < N; ++i) at[i] = kNone;
        }
    }
    __device__ __forceinline__ void put() {
        if constexpr (!kAsync) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (at[i] != kNone)
                    asm volatile("st.shared.b16 [%0], %1;" ::"r"(at[i]),
                                 "h"(*reinterpret_cast<const unsigned short *>(&held[i]))
                                 : "memory");
            clear();
        }
    }
    __device__ __forceinline__ void get(int i, Packet<T, V> *dst, const T *src) {
        if constexpr (kAsync) {
            copy_packet<T, V>(dst, src);
        } else {
            held[i] = load_packet<T, V>(src);
            at[i] = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
        }
    }
};
// The same without registers, for the scan's helper warps: a place for one
// packet that a thread copies for itself.  Packets of 4, 8 or 16 bytes are
// copied as they are.  A single two-byte element comes as the aligned word
// around it; which half it is follows from its address.  The array's first and
// last elements, whose words may reach past the array, are loaded and stored
// instead.  (Rows of 2047 bf16 channels, 8192 tokens: the convolution, the
// norm and the scan's gradient, which have registers to spare for Copies, take
// 164, 639 and 511 us with those and 234, 716 and 882 us with these.)
template <typename T, int V>
struct Slot {
    static constexpr bool kWord = V * sizeof(T) < 4;
    Packet<typename std::conditional<kWord, uint32_t, T>::type, V> p;
};
// The elements of an array whose words may reach past it.
template <typename T>
struct Span {
    const T *first, *last;
};
// `rows` rows of `width` elements, ld apart.
template <typename T>
__device__ __forceinline__ Span<T> span_of(const void *base, long rows, long ld, int width) {
    const T *b = static_cast<const T *>(base);
    return Span<T>{b, b + (rows - 1) * ld + width - 1};
}

template <typename T, int V>
__device__ __forceinline__ void copy_slot(Slot<T, V> *dst, const T *src, const Span<T> &span) {
    if constexpr (!Slot<T, V>::kWord) {
        cp_async<V * (int)sizeof(T)>(dst, src);
    } else {
        const uintptr_t a = (uintptr_t)src;
        if (src == span.first || src == span.last)
            dst->p.e[0] = (uint32_t) * reinterpret_cast<const unsigned short *>(src) << (a & 2 ? 16 : 0);
        else
            cp_async<4>(dst, reinterpret_cast<const void *>(a & ~(uintptr_t)3));
    }
}
// `src`: where the slot was copied from.
template <typename T, int V>
__device__ __forceinline__ void unpack_slot(const Slot<T, V> &s, const T *src, float *f) {
    if constexpr (!Slot<T, V>::kWord) {
        unpack<T, V>(s.p, f);
    } else {
        static_assert(std::is_same<T, __nv_bfloat16>::value, "bf16 is the upper half of an fp32");
        f[0] = __uint_as_float((uintptr_t)src & 2 ? s.p.e[0] & 0xffff0000u : s.p.e[0] << 16);
    }
}
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most N of this thread's committed groups are in flight.
template <int N>
__device__ __forceinline__ void wait_copies() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Pairs of fp32 values in one 64-bit register: one instruction, the same
// rounding of each half.
struct Pair {
    unsigned long long v;
};
__device__ __forceinline__ Pair make_pair(float x, float y) {
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p.v) : "f"(x), "f"(y));
    return p;
}
__device__ __forceinline__ void split_pair(Pair p, float &x, float &y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p.v));
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
    Pair d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return d;
}

constexpr float kLog2e = 1.4426950408889634f;
// Added to the arguments of the decays 2^(delta A log2 e), in the same fma.
// ex2.approx falls short of 2^x by 1.5e-8 on average for x in [-0.5, 0]
// (measured over 4 M arguments), and a decay a that enters 1 / (1 - a) times
// turns that into up to 1e-5 of a state; raising the argument by 1.5e-8 / ln 2
// takes the mean out.  Errors of dA at 8 x 2048 tokens against 64 bits: 1.8e-6
// without it, 7.7e-7 with.  2^kDecayBias rounds to 1: delta = 0 changes nothing.
constexpr float kDecayBias = 2.2e-8f;

// 1 / (1 + e^{-x}); a large e^{-x} gives 0.
__device__ __forceinline__ float sigmoid_f(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// log(1 + e^x) = max(x, 0) + log(1 + e), e = e^{-|x|} in (0, 1], with
// log(1 + e) = 2 atanh(r), r = e / (2 + e) <= 1/3, so that a small e keeps its
// relative accuracy, which log(1.f + e) would lose in rounding the sum.
// atanh(r) / r is a polynomial in r^2 through the five Chebyshev points of
// [0, 1/9]: within 4.1e-9 of it there.  e is 2^(-|x| log2 e) with the argument
// rounded once: |x| 2^-24 of relative error, and e itself vanishes as |x| grows.
__device__ __forceinline__ float softplus_rel(float x) {
    const float e = ex2(-fabsf(x) * kLog2e);
    const float r = __fdividef(e, 2.f + e);
    const float q = r * r;
    float s = fmaf(q, 0.14078889f, 0.13982579f);
    s = fmaf(q, s, 0.20012298f);
    s = fmaf(q, s, 0.33333161f);
    s = fmaf(q, s, 1.0000000038f);
    return fmaf(r + r, s, fmaxf(x, 0.f));
}

__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The same functions for V values, two to an instruction where V is even.
// x <- softplus(x + bias), or x + bias.
template <int V>
__device__ __forceinline__ void step_sizes(float *x, const float *bias, bool softplus) {
    if constexpr (V % 2 == 0) {
        auto two = [](float c) { return make_pair(c, c); };
#pragma unroll
        for (int v = 0; v < V; v += 2) {
            const Pair s = add2(make_pair(x[v], x[v + 1]), make_pair(bias[v], bias[v + 1]));
            split_pair(s, x[v], x[v + 1]);
            if (!softplus) continue;
            float e0, e1, d0, d1;
            split_pair(mul2(make_pair(fabsf(x[v]), fabsf(x[v + 1])), two(-kLog2e)), e0, e1);
            const Pair e = make_pair(ex2(e0), ex2(e1));
            split_pair(add2(e, two(2.f)), d0, d1);
            const Pair r = mul2(e, make_pair(rcp(d0), rcp(d1))), q = mul2(r, r);
            Pair p = fma2(q, two(0.14078889f), two(0.13982579f));
            p = fma2(q, p, two(0.20012298f));
            p = fma2(q, p, two(0.33333161f));
            p = fma2(q, p, two(1.0000000038f));
            split_pair(fma2(add2(r, r), p, make_pair(fmaxf(x[v], 0.f), fmaxf(x[v + 1], 0.f))), x[v], x[v + 1]);
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            x[v] += bias[v];
            if (softplus) x[v] = softplus_rel(x[v]);
        }
    }
}
// s <- sigmoid(x)
template <int V>
__device__ __forceinline__ void sigmoids(const float *x, float *s) {
    if constexpr (V % 2 == 0) {
#pragma unroll
        for (int v = 0; v < V; v += 2) {
            float e0, e1;
            split_pair(mul2(make_pair(x[v], x[v + 1]), make_pair(-kLog2e, -kLog2e)), e0, e1);
            split_pair(add2(make_pair(ex2(e0), ex2(e1)), make_pair(1.f, 1.f)), e0, e1);
            s[v] = rcp(e0);
            s[v + 1] = rcp(e1);
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = sigmoid_f(x[v]);
    }
}
// y <- y z sigmoid(z)
template <int V>
__device__ __forceinline__ void apply_gate(float *y, const float *z) {
    float s[V];
    sigmoids<V>(z, s);
#pragma unroll
    for (int v = 0; v < V; ++v) y[v] *= z[v] * s[v];
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
