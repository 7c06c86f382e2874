// Group norm with an activation, channels last, and its gradient.
//
//   n = (x - mean) rstd over a group,  u = n weight + bias,
//   y = act(u), or with a gate u act(gate)
//   du = dy act'(u) or dy act(gate),  dgate = dy u act'(gate),  dn = du weight
//   dx = rstd (dn - mean(dn) - n mean(dn n)),  dweight = sum du n,  dbias = sum du
//
// A group is D / G neighbouring columns, of one token or of all tokens of a
// sequence.  Without centering the mean is zero and so is its gradient's term.
//
// Memory bound.  A token's group is read once: its elements stay in the
// registers of a few threads, which take the same group of every so-manieth
// token, so that weights and the parameters' sums stay in registers too.  With 16
// groups of 128 bf16 columns and a gate, 32768 tokens take 81 us (403 MB: 0.73 of
// the copy rate), forward and gradient of 16384 tokens 114 (0.52): the activation
// and its derivative on the CUDA cores, at 24 and 16 warps a multiprocessor.
// (Times here and below: calls one behind another, through the binding.)
// Groups too wide for that are read again from the caches, in loops.
// The groups of a sequence are read once where a cluster's shared memory holds
// them, twice otherwise: the second time after the sums of tiles of its tokens
// have been joined (from the L2 cache, if the batch fits it).
#include <cooperative_groups.h>

#include <algorithm>

#include "mdn_attn.cuh"

namespace mdn {
namespace {

constexpr int kThreads = 256;

// A call's kernels follow one another by programmatic dependent launch: each lets
// the next one be set up once its own blocks run, and waits for the one before
// it, every thread of it, before it reads.
__device__ __forceinline__ void grid_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... P, typename... A>
cudaError_t follow(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// Sums over the threads of a group: tpg threads (a power of two).  The halves of
// `red` alternate, as one barrier a call then is enough.
template <int N>
struct Sums {
    float v[N];
};
template <int N>
__device__ __forceinline__ Sums<N> group_sum(Sums<N> s, int tpg, Sums<N> *red, int &turn) {
    for (int o = min(tpg, 32) >> 1; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) s.v[i] += __shfl_xor_sync(0xffffffffu, s.v[i], o);
    if (tpg <= 32) return s;
    Sums<N> *r = red + turn;
    turn ^= 32;
    if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = s;
    __syncthreads();
    const int wpg = tpg >> 5;
    s = r[((threadIdx.x >> 5) & ~(wpg - 1)) + (threadIdx.x & (wpg - 1))];
    for (int o = wpg >> 1; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) s.v[i] += __shfl_xor_sync(0xffffffffu, s.v[i], o);
    return s;
}

// V values as pairs of fp32, two to an instruction (a single one beside a zero
// that no sum takes).
template <int V>
struct Vals {
    static constexpr int N = (V + 1) / 2;
    Pair p[N];
};
__device__ __forceinline__ Pair both(float x) { return make_pair(x, x); }
template <typename T, int V>
__device__ __forceinline__ Vals<V> values(const Packet<T, V> &p) {
    Vals<V> r;
    if constexpr (V == 1) {
        r.p[0] = make_pair(to_f32(p.e[0]), 0.f);
    } else if constexpr (sizeof(T) == 2) {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(&p);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) r.p[i] = make_pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) r.p[i] = make_pair(p.e[2 * i], p.e[2 * i + 1]);
    }
    return r;
}
template <typename T, int V>
__device__ __forceinline__ Packet<T, V> packet(const Vals<V> &r) {
    float f[2 * Vals<V>::N];
#pragma unroll
    for (int i = 0; i < Vals<V>::N; ++i) split_pair(r.p[i], f[2 * i], f[2 * i + 1]);
    return pack<T, V>(f);
}
template <int V>
__device__ __forceinline__ float sum_of(const Vals<V> &r) {
    Pair s = r.p[0];
#pragma unroll
    for (int i = 1; i < Vals<V>::N; ++i) s = add2(s, r.p[i]);
    float x, y;
    split_pair(s, x, y);
    return V == 1 ? x : x + y;
}
template <int V>
__device__ __forceinline__ Vals<V> zeros() {
    Vals<V> r;
#pragma unroll
    for (int i = 0; i < Vals<V>::N; ++i) r.p[i] = both(0.f);
    return r;
}
template <int V>
__device__ __forceinline__ Vals<V> load_weights(const float *w, long c, float none) {
    Vals<V> r;
#pragma unroll
    for (int i = 0; i < Vals<V>::N; ++i)
        r.p[i] = w ? make_pair(__ldg(w + c + 2 * i), V == 1 ? none : __ldg(w + c + 2 * i + 1)) : both(none);
    return r;
}

__device__ __forceinline__ Pair sigmoid2(Pair x) {
    float a, b;
    split_pair(mul2(x, both(-kLog2e)), a, b);
    split_pair(add2(make_pair(ex2(a), ex2(b)), both(1.f)), a, b);
    return make_pair(rcp(a), rcp(b));
}
__device__ __forceinline__ Pair act2(Pair x, int act) {
    if (act == MDN_ACT_NONE) return x;
    const Pair s = sigmoid2(x);
    return act == MDN_ACT_SILU ? mul2(x, s) : s;
}
// a <- act(x), d <- act'(x)
__device__ __forceinline__ void act2_d(Pair x, int act, Pair &a, Pair &d) {
    if (act == MDN_ACT_NONE) {
        a = x;
        d = both(1.f);
        return;
    }
    const Pair s = sigmoid2(x), rest = fma2(s, both(-1.f), both(1.f));
    if (act == MDN_ACT_SILU) {
        a = mul2(x, s);
        d = mul2(s, fma2(x, rest, both(1.f)));
    } else {
        a = s;
        d = mul2(s, rest);
    }
}

// What centered elements d = x - mean become.
template <int V, bool GATE>
__device__ __forceinline__ Vals<V> forward_vals(const Vals<V> &d, const Vals<V> &g, float rstd, const Vals<V> &w,
                                                const Vals<V> &b, int act) {
    Vals<V> y;
    const Pair r = both(rstd);
#pragma unroll
    for (int i = 0; i < Vals<V>::N; ++i) {
        const Pair u = fma2(mul2(d.p[i], r), w.p[i], b.p[i]);
        y.p[i] = GATE ? mul2(u, act2(g.p[i], act)) : act2(u, act);
    }
    return y;
}
// x <- n, dy <- du, g <- dgate
template <int V, bool GATE>
__device__ __forceinline__ void backward_vals(Vals<V> &x, Vals<V> &g, Vals<V> &dy, float mean, float rstd, const Vals<V> &w,
                                              const Vals<V> &b, int act) {
    const Pair m = both(-mean), r = both(rstd);
#pragma unroll
    for (int i = 0; i < Vals<V>::N; ++i) {
        x.p[i] = mul2(add2(x.p[i], m), r);
        const Pair u = fma2(x.p[i], w.p[i], b.p[i]);
        Pair a, d;
        act2_d(GATE ? g.p[i] : u, act, a, d);
        if (GATE) g.p[i] = mul2(mul2(dy.p[i], u), d);
        dy.p[i] = mul2(dy.p[i], GATE ? a : d);
    }
}

// ----------------------------------------------------------- a token's groups

// The threads of a block that share a group, and what they take in turn.
struct TokenPlace {
    int tid;            // within the group
    long g;             // the group
    long row, step;     // its first token and the tokens between two of them
    int rounds;         // the same for the whole block
};
__device__ __forceinline__ TokenPlace token_place(const GroupNormProblem &p, int tpg) {
    TokenPlace t;
    const long ipb = blockDim.x / tpg, item0 = blockIdx.x * ipb, item = item0 + threadIdx.x / tpg;
    t.tid = threadIdx.x & (tpg - 1);
    t.row = item / p.G;
    t.g = item - t.row * p.G;
    t.step = gridDim.x * ipb / p.G;      // the grid is a whole number of tokens
    const long first = item0 / p.G;
    t.rounds = first < p.rows ? (int)((p.rows - first + t.step - 1) / t.step) : 0;
    return t;
}

// Threads of a block at most where each has NI packets of a group, as many as the
// registers leave.  Wider groups are taken by blocks of kThreadsWide in loops.
// (16384 tokens of one group of 2049 fp32 columns, gate: the forward 182 us, in
// loops 226; with the gradient 461 in loops, 945 with eight packets a thread.)
__host__ __device__ constexpr int most_threads(int NI, int V, bool bwd) {
    const int most = (V == 8 ? 2 : V == 4 ? 4 : 8) / (bwd && V < 8 ? 2 : 1);
    return NI > most ? 0 : bwd && V == 8 ? 256 : 512;
}
constexpr int kThreadsWide = 512;

// Q values from the first-th on, as fp32.
template <int Q, int V>
__device__ __forceinline__ Packet<float, Q> packet_of(const Vals<V> &r, int first) {
    float f[2 * Vals<V>::N];
#pragma unroll
    for (int i = 0; i < Vals<V>::N; ++i) split_pair(r.p[i], f[2 * i], f[2 * i + 1]);
    Packet<float, Q> q;
#pragma unroll
    for (int i = 0; i < Q; ++i) q.e[i] = f[first + i];
    return q;
}

// A thread keeps its weights, and asks for the next token's packets before it
// looks at this one's.
template <typename T, int V, int NI, bool GATE>
__global__ void __launch_bounds__(most_threads(NI, V, false)) token_fwd_kernel(GroupNormProblem p, int tpg) {
    __shared__ Sums<1> red[64];
    int turn = 0;
    const TokenPlace t = token_place(p, tpg);
    const int w = p.D / p.G;
    const long c0 = t.g * w;
    // this thread's packets of the next token to load, and of the one to store
    const T *x = static_cast<const T *>(p.x) + t.row * p.ld_x + c0 + t.tid * V;
    const T *gate = static_cast<const T *>(p.gate) + t.row * p.ld_gate + c0 + t.tid * V;
    T *y = static_cast<T *>(p.y) + t.row * p.D + c0 + t.tid * V;
    const long x_step = t.step * p.ld_x, gate_step = t.step * p.ld_gate, y_step = t.step * p.D;
    Vals<V> wt[NI], bs[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int c = (i * tpg + t.tid) * V;
        if (c < w) {
            wt[i] = load_weights<V>(p.weight, c0 + c, 1.f);
            bs[i] = load_weights<V>(p.bias, c0 + c, 0.f);
        }
    }
    Packet<T, V> px[NI], pg[GATE ? NI : 1];
    auto load = [&](long row) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            if (row < p.rows && (i * tpg + t.tid) * V < w) {
                px[i] = load_packet<T, V>(x + i * tpg * V);
                if (GATE) pg[i] = load_packet<T, V>(gate + i * tpg * V);
            }
        }
        x += x_step;
        if (GATE) gate += gate_step;
    };
    const float inv = 1.f / (float)w;
    long row = t.row;
    load(row);
    for (int k = 0; k < t.rounds; ++k, row += t.step) {
        const bool live = row < p.rows;
        Vals<V> d[NI], g[GATE ? NI : 1];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const bool in = live && (i * tpg + t.tid) * V < w;
            d[i] = in ? values<T, V>(px[i]) : zeros<V>();
            if (GATE) g[i] = values<T, V>(pg[i]);
        }
        load(row + t.step);
        float mean = 0.f;
        Sums<1> s;
        if (p.center) {
            s.v[0] = 0.f;
#pragma unroll
            for (int i = 0; i < NI; ++i) s.v[0] += sum_of<V>(d[i]);
            mean = group_sum(s, tpg, red, turn).v[0] * inv;
        }
        s.v[0] = 0.f;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const bool in = (i * tpg + t.tid) * V < w;
            Vals<V> q;
#pragma unroll
            for (int j = 0; j < Vals<V>::N; ++j) {
                d[i].p[j] = add2(d[i].p[j], both(-mean));
                q.p[j] = mul2(d[i].p[j], d[i].p[j]);
            }
            if (in) s.v[0] += sum_of<V>(q);
        }
        const float rstd = rsqrtf(fmaf(group_sum(s, tpg, red, turn).v[0], inv, p.eps));
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int c = (i * tpg + t.tid) * V;
            if (live && c < w) {
                store_packet<T, V>(y + i * tpg * V,
                                   packet<T, V>(forward_vals<V, GATE>(d[i], g[GATE ? i : 0], rstd, wt[i], bs[i], p.act)));
            }
        }
        if (p.stats && live && t.tid == 0)
            reinterpret_cast<float2 *>(p.stats)[row * p.G + t.g] = make_float2(mean, rstd);
        y += y_step;
    }
}

// The same for groups too wide for that: a block takes one at a time, in loops,
// and reads it again from the L1 cache for each of the sums and the result.
template <typename T, int V, bool GATE>
__global__ void __launch_bounds__(kThreadsWide, 2) wide_fwd_kernel(GroupNormProblem p) {
    __shared__ Sums<1> red[64];
    int turn = 0;
    const TokenPlace t = token_place(p, kThreadsWide);
    const int w = p.D / p.G;
    const long c0 = t.g * w;
    const float inv = 1.f / (float)w;
    for (long row = t.row; row < p.rows; row += t.step) {
        const T *x = static_cast<const T *>(p.x) + row * p.ld_x + c0, *gate = static_cast<const T *>(p.gate) + row * p.ld_gate + c0;
        T *y = static_cast<T *>(p.y) + row * p.D + c0;
        float mean = 0.f;
        Sums<1> s;
        if (p.center) {
            s.v[0] = 0.f;
#pragma unroll 4
            for (int c = t.tid * V; c < w; c += kThreadsWide * V) s.v[0] += sum_of<V>(values<T, V>(load_packet<T, V>(x + c)));
            mean = group_sum(s, kThreadsWide, red, turn).v[0] * inv;
        }
        auto centered = [&](int c) {
            Vals<V> d = values<T, V>(load_packet<T, V>(x + c));
#pragma unroll
            for (int j = 0; j < Vals<V>::N; ++j) d.p[j] = add2(d.p[j], both(-mean));
            return d;
        };
        s.v[0] = 0.f;
#pragma unroll 4
        for (int c = t.tid * V; c < w; c += kThreadsWide * V) {
            Vals<V> d = centered(c);
#pragma unroll
            for (int j = 0; j < Vals<V>::N; ++j) d.p[j] = mul2(d.p[j], d.p[j]);
            s.v[0] += sum_of<V>(d);
        }
        const float rstd = rsqrtf(fmaf(group_sum(s, kThreadsWide, red, turn).v[0], inv, p.eps));
#pragma unroll 2
        for (int c = t.tid * V; c < w; c += kThreadsWide * V) {
            Vals<V> g;
            if (GATE) g = values<T, V>(load_packet<T, V>(gate + c));
            store_packet<T, V>(y + c, packet<T, V>(forward_vals<V, GATE>(centered(c), g, rstd, load_weights<V>(p.weight, c0 + c, 1.f),
                                                                         load_weights<V>(p.bias, c0 + c, 0.f), p.act)));
        }
        if (p.stats && t.tid == 0) reinterpret_cast<float2 *>(p.stats)[row * p.G + t.g] = make_float2(mean, rstd);
    }
}

// part: [row lanes][2][D], one lane for every t.row of the first round.
template <typename T, int V, int NI, bool GATE>
__global__ void __launch_bounds__(most_threads(NI, V, true)) token_bwd_kernel(GroupNormProblem p, int tpg, float *part) {
    __shared__ Sums<2> red[64];
    grid_trigger();
    int turn = 0;
    const TokenPlace t = token_place(p, tpg);
    const int w = p.D / p.G;
    const long c0 = t.g * w;
    const T *x = static_cast<const T *>(p.x) + t.row * p.ld_x + c0 + t.tid * V;
    const T *gate = static_cast<const T *>(p.gate) + t.row * p.ld_gate + c0 + t.tid * V;
    const T *dyp = static_cast<const T *>(p.dy) + t.row * p.ld_dy + c0 + t.tid * V;
    T *dx = static_cast<T *>(p.dx) + t.row * p.D + c0 + t.tid * V, *dgate = static_cast<T *>(p.dgate) + t.row * p.D + c0 + t.tid * V;
    const float2 *stats = reinterpret_cast<const float2 *>(p.stats) + t.row * p.G + t.g;
    const long x_step = t.step * p.ld_x, gate_step = t.step * p.ld_gate, dy_step = t.step * p.ld_dy, out_step = t.step * p.D;
    Vals<V> wt[NI], bs[NI], dw[NI], db[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int c = (i * tpg + t.tid) * V;
        if (c < w) {
            wt[i] = load_weights<V>(p.weight, c0 + c, 1.f);
            bs[i] = load_weights<V>(p.bias, c0 + c, 0.f);
        }
        dw[i] = db[i] = zeros<V>();
    }
    Packet<T, V> px[NI], pd[NI], pg[GATE ? NI : 1];
    float2 st, next = make_float2(0.f, 0.f);
    auto load = [&](long row) {
        if (row >= p.rows) return;
        next = *stats;
#pragma unroll
        for (int i = 0; i < NI; ++i)
            if ((i * tpg + t.tid) * V < w) {
                px[i] = load_packet<T, V>(x + i * tpg * V);
                pd[i] = load_packet<T, V>(dyp + i * tpg * V);
                if (GATE) pg[i] = load_packet<T, V>(gate + i * tpg * V);
            }
        stats += t.step * p.G;
        x += x_step;
        dyp += dy_step;
        if (GATE) gate += gate_step;
    };
    const float inv = 1.f / (float)w;
    long row = t.row;
    load(row);
    for (int k = 0; k < t.rounds; ++k, row += t.step) {
        const bool live = row < p.rows;
        st = next;
        Vals<V> n[NI], d[NI], g[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            n[i] = values<T, V>(px[i]);
            d[i] = values<T, V>(pd[i]);
            if (GATE) g[i] = values<T, V>(pg[i]);
        }
        load(row + t.step);
        Sums<2> s;
        s.v[0] = s.v[1] = 0.f;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int c = (i * tpg + t.tid) * V;
            if (live && c < w) {
                backward_vals<V, GATE>(n[i], g[i], d[i], st.x, st.y, wt[i], bs[i], p.act);
                if (GATE) store_packet<T, V>(dgate + i * tpg * V, packet<T, V>(g[i]));
                Vals<V> dn, dnn;
#pragma unroll
                for (int j = 0; j < Vals<V>::N; ++j) {
                    dw[i].p[j] = fma2(d[i].p[j], n[i].p[j], dw[i].p[j]);
                    db[i].p[j] = add2(d[i].p[j], db[i].p[j]);
                    dn.p[j] = mul2(d[i].p[j], wt[i].p[j]);
                    dnn.p[j] = mul2(dn.p[j], n[i].p[j]);
                }
                s.v[0] += sum_of<V>(dn);
                s.v[1] += sum_of<V>(dnn);
            }
        }
        s = group_sum(s, tpg, red, turn);
        const Pair m1 = both(p.center ? -s.v[0] * inv : 0.f), m2 = both(-s.v[1] * inv), r = both(st.y);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int c = (i * tpg + t.tid) * V;
            if (live && c < w) {
                Vals<V> out;
#pragma unroll
                for (int j = 0; j < Vals<V>::N; ++j)
                    out.p[j] = mul2(r, fma2(n[i].p[j], m2, fma2(d[i].p[j], wt[i].p[j], m1)));
                store_packet<T, V>(dx + i * tpg * V, packet<T, V>(out));
            }
        }
        dx += out_step;
        if (GATE) dgate += out_step;
    }
    if (!part) return;
    float *out = part + t.row * 2 * p.D + c0;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int c = (i * tpg + t.tid) * V;
        if (c < w) {
            store_packet<float, V < 4 ? V : 4>(out + c, packet_of<V < 4 ? V : 4>(dw[i], 0));
            store_packet<float, V < 4 ? V : 4>(out + p.D + c, packet_of<V < 4 ? V : 4>(db[i], 0));
            if constexpr (V > 4) {
                store_packet<float, 4>(out + c + 4, packet_of<4>(dw[i], 4));
                store_packet<float, 4>(out + p.D + c + 4, packet_of<4>(db[i], 4));
            }
        }
    }
}

// The same for groups too wide for that, as wide_fwd_kernel: what the sums take
// is worked out again for dx; the parameters' sums are in shared memory, every
// thread its own columns'.
template <typename T, int V, bool GATE>
__global__ void __launch_bounds__(kThreadsWide, 2) wide_bwd_kernel(GroupNormProblem p, float *part) {
    __shared__ Sums<2> red[64];
    extern __shared__ __align__(16) unsigned char acc_raw[];
    grid_trigger();
    int turn = 0;
    const TokenPlace t = token_place(p, kThreadsWide);
    const int w = p.D / p.G;
    const long c0 = t.g * w;
    const float inv = 1.f / (float)w;
    using Acc = Packet<float, V < 4 ? V : 4>;
    constexpr int Q = V < 4 ? V : 4;
    float *dw = reinterpret_cast<float *>(acc_raw), *db = dw + w;
    if (part)
        for (int c = t.tid * V; c < w; c += kThreadsWide * V)
#pragma unroll
            for (int j = 0; j < V; ++j) dw[c + j] = db[c + j] = 0.f;
    for (long row = t.row; row < p.rows; row += t.step) {
        const T *x = static_cast<const T *>(p.x) + row * p.ld_x + c0, *gate = static_cast<const T *>(p.gate) + row * p.ld_gate + c0,
                *dy = static_cast<const T *>(p.dy) + row * p.ld_dy + c0;
        T *dx = static_cast<T *>(p.dx) + row * p.D + c0, *dgate = static_cast<T *>(p.dgate) + row * p.D + c0;
        const float2 st = reinterpret_cast<const float2 *>(p.stats)[row * p.G + t.g];
        Vals<V> n, d, g, wt;
        auto element = [&](int c) {
            n = values<T, V>(load_packet<T, V>(x + c));
            d = values<T, V>(load_packet<T, V>(dy + c));
            if (GATE) g = values<T, V>(load_packet<T, V>(gate + c));
            wt = load_weights<V>(p.weight, c0 + c, 1.f);
            backward_vals<V, GATE>(n, g, d, st.x, st.y, wt, load_weights<V>(p.bias, c0 + c, 0.f), p.act);
        };
        Sums<2> s;
        s.v[0] = s.v[1] = 0.f;
#pragma unroll 2
        for (int c = t.tid * V; c < w; c += kThreadsWide * V) {
            element(c);
            Vals<V> dn, dnn, du_n;
#pragma unroll
            for (int j = 0; j < Vals<V>::N; ++j) {
                du_n.p[j] = mul2(d.p[j], n.p[j]);
                dn.p[j] = mul2(d.p[j], wt.p[j]);
                dnn.p[j] = mul2(dn.p[j], n.p[j]);
            }
            s.v[0] += sum_of<V>(dn);
            s.v[1] += sum_of<V>(dnn);
            if (part)
#pragma unroll
                for (int q = 0; q < V; q += Q) {
                    Acc a = load_packet<float, Q>(dw + c + q), b = load_packet<float, Q>(db + c + q);
                    const Acc da = packet_of<Q>(du_n, q), dbb = packet_of<Q>(d, q);
#pragma unroll
                    for (int j = 0; j < Q; ++j) {
                        a.e[j] += da.e[j];
                        b.e[j] += dbb.e[j];
                    }
                    store_packet<float, Q>(dw + c + q, a);
                    store_packet<float, Q>(db + c + q, b);
                }
        }
        s = group_sum(s, kThreadsWide, red, turn);
        const Pair m1 = both(p.center ? -s.v[0] * inv : 0.f), m2 = both(-s.v[1] * inv), r = both(st.y);
#pragma unroll 2
        for (int c = t.tid * V; c < w; c += kThreadsWide * V) {
            element(c);
            Vals<V> out;
#pragma unroll
            for (int j = 0; j < Vals<V>::N; ++j)
                out.p[j] = mul2(r, fma2(n.p[j], m2, fma2(d.p[j], wt.p[j], m1)));
            if (GATE) store_packet<T, V>(dgate + c, packet<T, V>(g));
            store_packet<T, V>(dx + c, packet<T, V>(out));
        }
    }
    if (!part) return;
    float *out = part + t.row * 2 * p.D + c0;
    for (int c = t.tid * V; c < w; c += kThreadsWide * V)
#pragma unroll
        for (int q = 0; q < V; q += Q) {
            store_packet<float, Q>(out + c + q, load_packet<float, Q>(dw + c + q));
            store_packet<float, Q>(out + p.D + c + q, load_packet<float, Q>(db + c + q));
        }
}

// dw, dbias <- sums over the lanes of part, in a fixed order.
__global__ void __launch_bounds__(1024) param_kernel(const float *part, int lanes, int D, float *dw, float *dbias) {
    __shared__ float sums[32][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const long c = blockIdx.x * 32L + x;
    grid_wait();
    float s = 0.f;
    if (c < 2L * D) {
        const float *src = part + c;
#pragma unroll 8
        for (int l = y; l < lanes; l += 32) s += src[(long)l * 2 * D];
    }
    sums[y][x] = s;
    __syncthreads();
    // warp y adds up column y
    s = sums[x][y];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const long out = blockIdx.x * 32L + y;
    if (x || out >= 2L * D) return;
    if (out < D) {
        if (dw) dw[out] = s;
    } else if (dbias) {
        dbias[out - D] = s;
    }
}

// -------------------------------------------------------- a sequence's groups

// Whether cu_seqlens is well formed (whole CTA; uniform result): looked at by
// every block, or of many sequences once, by check_kernel.
constexpr int kManySequences = 1024;
__device__ __forceinline__ bool sequences_ok(const GroupNormProblem &p) {
    if (!p.cu) return true;
    if (p.ok) return *p.ok != 0;
    return cu_well_formed(p.cu, p.n_seq, (int)p.rows);
}
__global__ void __launch_bounds__(1024) check_kernel(GroupNormProblem p) {
    const bool ok = cu_well_formed(p.cu, p.n_seq, (int)p.rows);
    if (threadIdx.x) return;
    *p.ok = ok;
    if (!ok) atomicExch(p.status, MDN_ERR_INVALID_ARG);
}

// A tile of a sequence's tokens: `rows` of them at a time.  Tiles of sequence s
// begin at slot cu[s] / rows + s, which leaves room for the last, partial one.
struct Tile {
    int seq, k, len;    // k: which tile of the sequence; len: tokens of the sequence
    long start;         // its first token
    int n;              // tokens
};
__device__ __forceinline__ bool tile_of(const GroupNormProblem &p, int rows, int slot, Tile &t) {
    if (!p.cu) {
        const int per = (p.T + rows - 1) / rows;
        t.seq = slot / per;
        t.k = slot - t.seq * per;
        t.len = p.T;
        t.start = (long)t.seq * p.T + (long)t.k * rows;
    } else {
        int lo = 0, hi = p.n_seq;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.cu[mid] / rows + mid <= slot) lo = mid; else hi = mid;
        }
        t.seq = lo;
        t.k = slot - (p.cu[lo] / rows + lo);
        t.len = p.cu[lo + 1] - p.cu[lo];
        t.start = (long)p.cu[lo] + (long)t.k * rows;
    }
    t.n = min(rows, t.len - t.k * rows);
    return t.n > 0;
}
__device__ __forceinline__ long first_slot(const GroupNormProblem &p, int rows, int s) {
    return p.cu ? p.cu[s] / rows + s : (long)s * ((p.T + rows - 1) / rows);
}

// Which columns a block takes: whole groups, their packets over its threads and
// as many tokens at a time as fit.
struct Columns {
    int g0, groups;     // its groups
    int packets;        // of a token
    int lanes;          // tokens at a time
    int pc, lane;       // this thread's first packet and its lane (>= lanes: idle)
};
__device__ __forceinline__ Columns columns_of(const GroupNormProblem &p, int per_block, int V) {
    Columns c;
    const int w = p.D / p.G;
    c.g0 = blockIdx.y * per_block;
    c.groups = min(per_block, p.G - c.g0);
    c.packets = c.groups * (w / V);
    c.lanes = max(1, kThreads / c.packets);
    c.lane = c.packets >= kThreads ? 0 : (int)threadIdx.x / c.packets;
    c.pc = c.packets >= kThreads ? (int)threadIdx.x : (int)threadIdx.x - c.lane * c.packets;
    return c;
}

// take(g, packets of a group) for the block's groups g, one warp each.
template <typename F>
__device__ __forceinline__ void by_group(const Columns &c, F take) {
    const int warp = threadIdx.x >> 5, ppg = c.packets / c.groups;
    for (int g = warp; g < c.groups; g += kThreads / 32) take(g, ppg);
}

// Mean and sum of squared distances from it of parts with a mean, such a sum and
// a count each: sums of the means' distances c and of their squares, from a
// value that is near all of them (the first part's mean).
struct Join {
    float n, s1, s2;
};
__device__ __forceinline__ void join_part(Join &j, float center, float n, float mean, float m2) {
    const float d = mean - center;
    j.n += n;
    j.s1 = fmaf(n, d, j.s1);
    j.s2 += fmaf(n * d, d, m2);
}
__device__ __forceinline__ void join_warp(Join &j) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        j.n += __shfl_xor_sync(0xffffffffu, j.n, o);
        j.s1 += __shfl_xor_sync(0xffffffffu, j.s1, o);
        j.s2 += __shfl_xor_sync(0xffffffffu, j.s2, o);
    }
}
// (mean, sum of squared distances)
__device__ __forceinline__ float2 joined(const Join &j, float center) {
    const float d = j.s1 / j.n, m2 = j.s2 - j.s1 * d;
    return make_float2(center + d, m2 < 0.f ? 0.f : m2);      // (a NaN stays one)
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) seq_stats_kernel(GroupNormProblem p, int rows, int per_block, float2 *part) {
    __shared__ float mom[3][kThreads];
    grid_trigger();
    if (!sequences_ok(p)) {
        if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) atomicExch(p.status, MDN_ERR_INVALID_ARG);
        return;
    }
    Tile t;
    if (!tile_of(p, rows, blockIdx.x, t)) return;
    const Columns c = columns_of(p, per_block, V);
    const int w = p.D / p.G;
    float n = 0.f, mean = 0.f, m2 = 0.f;
    if (c.lane < c.lanes && c.lane < t.n)
        for (int pc = c.pc; pc < c.packets; pc += kThreads) {
            const T *x = static_cast<const T *>(p.x) + (t.start + c.lane) * p.ld_x + (long)c.g0 * w + pc * V;
            const long step = (long)c.lanes * p.ld_x;
            const int count = (t.n - c.lane + c.lanes - 1) / c.lanes;
            // sums about the mean of the first packet, so that they do not cancel
            const float shift = p.center ? sum_of<V>(values<T, V>(load_packet<T, V>(x))) * (1.f / V) : 0.f;
            Vals<V> s1 = zeros<V>(), s2 = zeros<V>();
            const Pair minus = both(-shift);
#pragma unroll 8
            for (int r = 0; r < count; ++r) {
                const Vals<V> f = values<T, V>(load_packet<T, V>(x + r * step));
#pragma unroll
                for (int j = 0; j < Vals<V>::N; ++j) {
                    const Pair d = add2(f.p[j], minus);
                    s1.p[j] = add2(s1.p[j], d);
                    s2.p[j] = fma2(d, d, s2.p[j]);
                }
            }
            Join j = {0.f, 0.f, 0.f};
            const float a = sum_of<V>(s1), b = sum_of<V>(s2), k = (float)count * V;
            const float mine = p.center ? shift + a / k : 0.f, m = p.center ? b - a * (a / k) : b;
            // (groups wider than the block: a thread's packets together)
            if (n > 0.f) join_part(j, mean, n, mean, m2);
            const float center = n > 0.f ? mean : mine;
            join_part(j, center, k, mine, m < 0.f ? 0.f : m);
            const float2 both_parts = joined(j, center);
            n = j.n;
            mean = p.center ? both_parts.x : 0.f;
            m2 = p.center ? both_parts.y : j.s2;
        }
    mom[0][threadIdx.x] = n;
    mom[1][threadIdx.x] = mean;
    mom[2][threadIdx.x] = m2;
    __syncthreads();
    by_group(c, [&](int g, int ppg) {
        const bool whole = c.packets >= kThreads && c.groups == 1;
        const int count = whole ? kThreads : ppg * c.lanes;
        const float center = mom[1][whole ? 0 : g * ppg];
        Join j = {0.f, 0.f, 0.f};
        for (int i = threadIdx.x & 31; i < count; i += 32) {
            const int lane = whole ? 0 : i / ppg, at = whole ? i : lane * c.packets + g * ppg + (i - lane * ppg);
            join_part(j, center, mom[0][at], mom[0][at] > 0.f ? mom[1][at] : center, mom[2][at]);
        }
        join_warp(j);
        if ((threadIdx.x & 31) == 0) part[(long)blockIdx.x * p.G + c.g0 + g] = p.center ? joined(j, center) : make_float2(0.f, j.s2);
    });
}

// One warp a group of a sequence: the statistics from the tiles'.
__global__ void __launch_bounds__(kThreads) seq_join_kernel(GroupNormProblem p, int rows, const float2 *part, float2 *stats) {
    const long i = blockIdx.x * (long)(kThreads / 32) + (threadIdx.x >> 5);
    const bool ok = sequences_ok(p);
    grid_trigger();
    grid_wait();
    if (i >= (long)p.n_seq * p.G) return;
    const int s = (int)(i / p.G), g = (int)(i - (long)s * p.G), w = p.D / p.G;
    const int len = !ok ? 0 : p.cu ? p.cu[s + 1] - p.cu[s] : p.T;
    const int tiles = (len + rows - 1) / rows;
    const float2 *src = part + (ok ? first_slot(p, rows, s) : 0) * p.G + g;
    const float center = tiles ? src[0].x : 0.f;
    Join j = {0.f, 0.f, 0.f};
#pragma unroll 4
    for (int k = threadIdx.x & 31; k < tiles; k += 32) {
        const float2 v = src[(long)k * p.G];
        join_part(j, center, (float)min(rows, len - k * rows) * w, v.x, v.y);
    }
    join_warp(j);
    if ((threadIdx.x & 31) == 0) {
        const float2 v = joined(j, center);
        stats[i] = len ? make_float2(p.center ? v.x : 0.f, rsqrtf((p.center ? v.y : j.s2) / j.n + p.eps)) : make_float2(0.f, 0.f);
    }
}

template <typename T, int V, bool GATE>
__global__ void __launch_bounds__(kThreads) seq_apply_kernel(GroupNormProblem p, int rows, int per_block, const float2 *stats) {
    const bool ok = sequences_ok(p);
    grid_trigger();
    grid_wait();
    Tile t;
    if (!ok || !tile_of(p, rows, blockIdx.x, t)) return;
    const Columns c = columns_of(p, per_block, V);
    if (c.lane >= c.lanes) return;
    const int w = p.D / p.G;
    for (int pc = c.pc; pc < c.packets; pc += kThreads) {
        const long col = (long)c.g0 * w + pc * V;
        const float2 st = stats[(long)t.seq * p.G + col / w];
        const Vals<V> wt = load_weights<V>(p.weight, col, 1.f), bs = load_weights<V>(p.bias, col, 0.f);
        const T *x = static_cast<const T *>(p.x) + t.start * p.ld_x + col;
        const T *gate = static_cast<const T *>(p.gate) + t.start * p.ld_gate + col;
        T *y = static_cast<T *>(p.y) + t.start * p.D + col;
        const Pair minus = both(-st.x);
#pragma unroll 4
        for (int r = c.lane; r < t.n; r += c.lanes) {
            Vals<V> f = values<T, V>(load_packet<T, V>(x + r * p.ld_x)), g;
            if (GATE) g = values<T, V>(load_packet<T, V>(gate + r * p.ld_gate));
#pragma unroll
            for (int j = 0; j < Vals<V>::N; ++j) f.p[j] = add2(f.p[j], minus);
            store_packet<T, V>(y + (long)r * p.D, packet<T, V>(forward_vals<V, GATE>(f, g, st.y, wt, bs, p.act)));
        }
    }
}

// Sums of dn and dn n of a tile's groups, and of du n and du of its columns.  Where
// there are more tiles than rows for the columns' sums, blocks take tiles in turn
// and add them up.
template <typename T, int V, bool GATE>
__global__ void __launch_bounds__(kThreads)
seq_sums_kernel(GroupNormProblem p, int rows, int per_block, int slots, float2 *part, float *params) {
    __shared__ float2 red[kThreads];
    __shared__ float cols[2][kThreads * V];
    grid_trigger();
    const bool ok = sequences_ok(p);
    if (!ok && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) atomicExch(p.status, MDN_ERR_INVALID_ARG);
    const Columns c = columns_of(p, per_block, V);
    const int w = p.D / p.G;
    float *out = params ? params + (long)blockIdx.x * 2 * p.D + (long)c.g0 * w : nullptr;
    for (int slot = blockIdx.x; slot < slots; slot += gridDim.x) {
        const bool first = slot == blockIdx.x;
        Tile t;
        const bool some = ok && tile_of(p, rows, slot, t);
        if (!some && !first) continue;
        if (!first) __syncthreads();       // (the last tile's sums have been read)
        float2 s = make_float2(0.f, 0.f);
        // whole rounds of packets, for the barriers; one round where lanes > 1
        for (int base = 0; base < c.packets; base += kThreads) {
            const int pc = base + c.pc;
            Vals<V> dw = zeros<V>(), db = zeros<V>();
            if (some && c.lane < c.lanes && pc < c.packets) {
                const long col = (long)c.g0 * w + pc * V;
                const float2 st = reinterpret_cast<const float2 *>(p.stats)[(long)t.seq * p.G + col / w];
                const Vals<V> wt = load_weights<V>(p.weight, col, 1.f), bs = load_weights<V>(p.bias, col, 0.f);
                const T *x = static_cast<const T *>(p.x) + t.start * p.ld_x + col;
                const T *gate = static_cast<const T *>(p.gate) + t.start * p.ld_gate + col;
                const T *dy = static_cast<const T *>(p.dy) + t.start * p.ld_dy + col;
#pragma unroll 4
                for (int r = c.lane; r < t.n; r += c.lanes) {
                    Vals<V> n = values<T, V>(load_packet<T, V>(x + r * p.ld_x)), g;
                    Vals<V> d = values<T, V>(load_packet<T, V>(dy + r * p.ld_dy));
                    if (GATE) g = values<T, V>(load_packet<T, V>(gate + r * p.ld_gate));
                    backward_vals<V, GATE>(n, g, d, st.x, st.y, wt, bs, p.act);
#pragma unroll
                    for (int j = 0; j < Vals<V>::N; ++j) {
                        dw.p[j] = fma2(d.p[j], n.p[j], dw.p[j]);
                        db.p[j] = add2(db.p[j], d.p[j]);
                    }
                }
                // the groups' sums follow from the columns'
                Vals<V> a, b;
#pragma unroll
                for (int j = 0; j < Vals<V>::N; ++j) {
                    a.p[j] = mul2(db.p[j], wt.p[j]);
                    b.p[j] = mul2(dw.p[j], wt.p[j]);
                }
                s.x += sum_of<V>(a);
                s.y += sum_of<V>(b);
            }
            if (!out) continue;
            float fw[2 * Vals<V>::N], fb[2 * Vals<V>::N];
#pragma unroll
            for (int j = 0; j < Vals<V>::N; ++j) {
                split_pair(dw.p[j], fw[2 * j], fw[2 * j + 1]);
                split_pair(db.p[j], fb[2 * j], fb[2 * j + 1]);
            }
            if (c.lanes == 1) {
                if (c.lane == 0 && pc < c.packets)
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        float *to = out + pc * V + v;
                        to[0] = first ? fw[v] : to[0] + fw[v];
                        to[p.D] = first ? fb[v] : to[p.D] + fb[v];
                    }
                continue;
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                cols[0][threadIdx.x * V + v] = fw[v];
                cols[1][threadIdx.x * V + v] = fb[v];
            }
            __syncthreads();
            const int n = c.packets * V;
            for (int i = threadIdx.x; i < 2 * n; i += kThreads) {
                const int which = i >= n, col = i - which * n;
                float sum = 0.f;
                for (int l = 0; l < c.lanes; ++l) sum += cols[which][l * n + col];
                float *to = out + which * p.D + col;
                *to = first ? sum : *to + sum;
            }
        }
        if (!some) continue;
        red[threadIdx.x] = s;
        __syncthreads();
        by_group(c, [&](int g, int ppg) {
            float2 a = make_float2(0.f, 0.f);
            const bool whole = c.packets >= kThreads && c.groups == 1;
            const int count = whole ? kThreads : ppg * c.lanes;
            for (int i = threadIdx.x & 31; i < count; i += 32) {
                const int lane = whole ? 0 : i / ppg;
                const float2 v = red[whole ? i : lane * c.packets + g * ppg + (i - lane * ppg)];
                a.x += v.x;
                a.y += v.y;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                a.x += __shfl_xor_sync(0xffffffffu, a.x, o);
                a.y += __shfl_xor_sync(0xffffffffu, a.y, o);
            }
            if ((threadIdx.x & 31) == 0) part[(long)slot * p.G + c.g0 + g] = a;
        });
    }
}

// One warp a group of a sequence: its means of dn and dn n.
__global__ void __launch_bounds__(kThreads) seq_means_kernel(GroupNormProblem p, int rows, const float2 *part, float2 *means) {
    const long i = blockIdx.x * (long)(kThreads / 32) + (threadIdx.x >> 5);
    const bool ok = sequences_ok(p);
    grid_trigger();
    grid_wait();
    if (!ok || i >= (long)p.n_seq * p.G) return;
    const int s = (int)(i / p.G), g = (int)(i - (long)s * p.G);
    const int len = p.cu ? p.cu[s + 1] - p.cu[s] : p.T, tiles = (len + rows - 1) / rows;
    const float2 *src = part + first_slot(p, rows, s) * p.G + g;
    float2 a = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int k = threadIdx.x & 31; k < tiles; k += 32) {
        const float2 v = src[(long)k * p.G];
        a.x += v.x;
        a.y += v.y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a.x += __shfl_xor_sync(0xffffffffu, a.x, o);
        a.y += __shfl_xor_sync(0xffffffffu, a.y, o);
    }
    if ((threadIdx.x & 31) == 0) {
        const float inv = len ? 1.f / ((float)len * (float)(p.D / p.G)) : 0.f;
        means[i] = make_float2(p.center ? a.x * inv : 0.f, a.y * inv);
    }
}

template <typename T, int V, bool GATE>
__global__ void __launch_bounds__(kThreads) seq_dx_kernel(GroupNormProblem p, int rows, int per_block, const float2 *means) {
    const bool ok = sequences_ok(p);
    grid_trigger();
    grid_wait();
    Tile t;
    if (!ok || !tile_of(p, rows, blockIdx.x, t)) return;
    const Columns c = columns_of(p, per_block, V);
    if (c.lane >= c.lanes) return;
    const int w = p.D / p.G;
    for (int pc = c.pc; pc < c.packets; pc += kThreads) {
        const long col = (long)c.g0 * w + pc * V;
        const float2 st = reinterpret_cast<const float2 *>(p.stats)[(long)t.seq * p.G + col / w];
        const float2 m = means[(long)t.seq * p.G + col / w];
        const Vals<V> wt = load_weights<V>(p.weight, col, 1.f), bs = load_weights<V>(p.bias, col, 0.f);
        const T *x = static_cast<const T *>(p.x) + t.start * p.ld_x + col;
        const T *gate = static_cast<const T *>(p.gate) + t.start * p.ld_gate + col;
        const T *dy = static_cast<const T *>(p.dy) + t.start * p.ld_dy + col;
        T *dx = static_cast<T *>(p.dx) + t.start * p.D + col, *dgate = static_cast<T *>(p.dgate) + t.start * p.D + col;
        const Pair m1 = both(-m.x), m2 = both(-m.y), rstd = both(st.y);
#pragma unroll 4
        for (int r = c.lane; r < t.n; r += c.lanes) {
            Vals<V> n = values<T, V>(load_packet<T, V>(x + r * p.ld_x)), g;
            Vals<V> d = values<T, V>(load_packet<T, V>(dy + r * p.ld_dy));
            if (GATE) g = values<T, V>(load_packet<T, V>(gate + r * p.ld_gate));
            backward_vals<V, GATE>(n, g, d, st.x, st.y, wt, bs, p.act);
            if (GATE) store_packet<T, V>(dgate + (long)r * p.D, packet<T, V>(g));
#pragma unroll
            for (int j = 0; j < Vals<V>::N; ++j)
                n.p[j] = mul2(rstd, fma2(n.p[j], m2, fma2(d.p[j], wt.p[j], m1)));
            store_packet<T, V>(dx + (long)r * p.D, packet<T, V>(n));
        }
    }
}

// ------------------------------------------------ ... in a cluster's shared memory
//
// A cluster of blocks takes neighbouring groups of one sequence, each block a run
// of its tokens.  Their packets are copied into shared memory at once, every
// thread its own (one column's, of every lanes-th token), and read from there
// for the sums and again for the results; the blocks' sums meet through the
// cluster's shared memory.  One launch and one reading instead of three and two.
// The gradient's clusters take sequences in turn where there are many, and add
// the columns' sums up: `walkers` of them to a column.

// Tokens of a block, for a sequence of len.
__device__ __forceinline__ int cluster_rows(int len, int blocks) { return (len + blocks - 1) / blocks; }

template <typename T, int V, bool GATE, bool BWD>
__global__ void __launch_bounds__(kThreads) seq_cluster_kernel(GroupNormProblem p, int per_block, int blocks, int walkers, float *params) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float mom[3][kThreads];
    __shared__ float cols[BWD ? 2 * kThreads * V : 1];
    __shared__ float3 own[kThreads], all[kThreads];     // of the block's groups
    if (BWD) grid_trigger();
    const int column_blocks = (p.G + per_block - 1) / per_block;
    const int rank = blockIdx.x % blocks, which = blockIdx.x / blocks, cb = which % column_blocks, walker = which / column_blocks;
    const bool ok = sequences_ok(p);
    if (!ok && blockIdx.x == 0 && threadIdx.x == 0) atomicExch(p.status, MDN_ERR_INVALID_ARG);
    int seq = walker;
    do {
        const int len = !ok ? 0 : p.cu ? p.cu[seq + 1] - p.cu[seq] : p.T;
        const long first = !ok ? 0 : p.cu ? p.cu[seq] : (long)seq * p.T;
        const int rows = cluster_rows(len, blocks), n = max(0, min(rows, len - rank * rows));
        const long start = first + (long)rank * rows;
        const int w = p.D / p.G, g0 = cb * per_block, groups = min(per_block, p.G - g0), ppg = w / V, packets = groups * ppg;
        const int lanes = kThreads / packets, lane = threadIdx.x / packets, pc = threadIdx.x - lane * packets;
        const int count = lane < lanes && lane < n ? (n - lane + lanes - 1) / lanes : 0;      // this thread's tokens
        const long col = (long)g0 * w + pc * V;
        constexpr int kArrays = BWD ? (GATE ? 3 : 2) : 1;
        using P = Packet<T, V>;
        P *tile = reinterpret_cast<P *>(smem) + threadIdx.x;        // [array][token of the thread][thread]
        const int depth = (rows + lanes - 1) / lanes;
        auto at = [&](int array, int r) -> P & { return tile[(array * depth + r) * kThreads]; };
        {
            const T *src[3] = {static_cast<const T *>(p.x), static_cast<const T *>(p.dy), static_cast<const T *>(p.gate)};
            const long ld[3] = {p.ld_x, p.ld_dy, p.ld_gate};
#pragma unroll
            for (int a = 0; a < kArrays; ++a) {
                const T *from = src[a] + (start + lane) * ld[a] + col;
                for (int r = 0; r < count; ++r) copy_packet<T, V>(&at(a, r), from + r * (lanes * ld[a]));
            }
            commit_copies();
        }
        const Vals<V> wt = count ? load_weights<V>(p.weight, col, 1.f) : zeros<V>();
        const Vals<V> bs = count ? load_weights<V>(p.bias, col, 0.f) : zeros<V>();
        float2 st = make_float2(0.f, 0.f);
        if (BWD && count) st = reinterpret_cast<const float2 *>(p.stats)[(long)seq * p.G + col / w];
        wait_copies<0>();
        float3 mine = make_float3(0.f, 0.f, 0.f);
        if constexpr (!BWD) {
            if (count) {
                // sums about the mean of the first packet, so that they do not cancel
                const float shift = p.center ? sum_of<V>(values<T, V>(at(0, 0))) * (1.f / V) : 0.f;
                Vals<V> s1 = zeros<V>(), s2 = zeros<V>();
                const Pair minus = both(-shift);
#pragma unroll 4
                for (int r = 0; r < count; ++r) {
                    const Vals<V> f = values<T, V>(at(0, r));
#pragma unroll
                    for (int j = 0; j < Vals<V>::N; ++j) {
                        const Pair d = add2(f.p[j], minus);
                        s1.p[j] = add2(s1.p[j], d);
                        s2.p[j] = fma2(d, d, s2.p[j]);
                    }
                }
                const float a = sum_of<V>(s1), b = sum_of<V>(s2), k = (float)count * V, m2 = p.center ? b - a * (a / k) : b;
                mine = make_float3(k, p.center ? shift + a / k : 0.f, m2 < 0.f ? 0.f : m2);
            }
        } else {
            Vals<V> dw = zeros<V>(), db = zeros<V>();
#pragma unroll 2
            for (int r = 0; r < count; ++r) {
                Vals<V> x = values<T, V>(at(0, r)), d = values<T, V>(at(1, r)), g;
                if (GATE) g = values<T, V>(at(kArrays - 1, r));
                backward_vals<V, GATE>(x, g, d, st.x, st.y, wt, bs, p.act);
#pragma unroll
                for (int j = 0; j < Vals<V>::N; ++j) {
                    dw.p[j] = fma2(d.p[j], x.p[j], dw.p[j]);
                    db.p[j] = add2(db.p[j], d.p[j]);
                }
            }
            Vals<V> a, b;
#pragma unroll
            for (int j = 0; j < Vals<V>::N; ++j) {
                a.p[j] = mul2(db.p[j], wt.p[j]);
                b.p[j] = mul2(dw.p[j], wt.p[j]);
            }
            mine = make_float3(0.f, sum_of<V>(a), sum_of<V>(b));
            if (params) {
                float fw[2 * Vals<V>::N], fb[2 * Vals<V>::N];
#pragma unroll
                for (int j = 0; j < Vals<V>::N; ++j) {
                    split_pair(dw.p[j], fw[2 * j], fw[2 * j + 1]);
                    split_pair(db.p[j], fb[2 * j], fb[2 * j + 1]);
                }
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    cols[threadIdx.x * V + v] = fw[v];
                    cols[(kThreads + threadIdx.x) * V + v] = fb[v];
                }
                __syncthreads();
                const int c = packets * V;
                float *out = params + ((long)walker * blocks + rank) * 2 * p.D + (long)g0 * w;
                for (int i = threadIdx.x; i < 2 * c; i += kThreads) {
                    const int k = i >= c, at_col = i - k * c;
                    float sum = 0.f;
                    for (int l = 0; l < lanes; ++l) sum += cols[k * kThreads * V + l * c + at_col];
                    float *to = out + k * p.D + at_col;
                    *to = seq == walker ? sum : *to + sum;
                }
            }
        }
        mom[0][threadIdx.x] = mine.x;
        mom[1][threadIdx.x] = mine.y;
        mom[2][threadIdx.x] = mine.z;
        __syncthreads();
        for (int g = threadIdx.x >> 5; g < groups; g += kThreads / 32) {
            const float center = BWD ? 0.f : mom[1][g * ppg];
            Join j = {0.f, 0.f, 0.f};
            for (int i = threadIdx.x & 31; i < ppg * lanes; i += 32) {
                const int l = i / ppg, k = l * packets + g * ppg + (i - l * ppg);
                if (BWD) {
                    j.s1 += mom[1][k];
                    j.s2 += mom[2][k];
                } else {
                    join_part(j, center, mom[0][k], mom[0][k] > 0.f ? mom[1][k] : center, mom[2][k]);
                }
            }
            join_warp(j);
            if ((threadIdx.x & 31) == 0) {
                float2 v = make_float2(j.s1, j.s2);
                if (!BWD) v = j.n > 0.f && p.center ? joined(j, center) : make_float2(0.f, j.s2);
                own[g] = make_float3(j.n, v.x, v.y);
            }
        }
        cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
        cluster.sync();
        // every block joins all blocks' sums, in their order
        for (int g = threadIdx.x; g < groups; g += kThreads) {
            const float center = BWD ? 0.f : cluster.map_shared_rank(own, 0)[g].y;      // (the first block has tokens)
            Join j = {0.f, 0.f, 0.f};
            for (int k = 0; k < blocks; ++k) {
                const float3 v = cluster.map_shared_rank(own, k)[g];
                if (BWD) {
                    j.s1 += v.y;
                    j.s2 += v.z;
                } else if (v.x > 0.f) {
                    join_part(j, center, v.x, v.y, v.z);
                }
            }
            if (BWD) {
                const float inv = len ? 1.f / ((float)len * (float)w) : 0.f;
                all[g] = make_float3(p.center ? j.s1 * inv : 0.f, j.s2 * inv, 0.f);
            } else {
                float2 v = make_float2(0.f, 0.f);
                if (len) {
                    const float2 m = joined(j, center);
                    v = make_float2(p.center ? m.x : 0.f, rsqrtf((p.center ? m.y : j.s2) / j.n + p.eps));
                }
                all[g] = make_float3(v.x, v.y, 0.f);
                if (p.stats && rank == 0) reinterpret_cast<float2 *>(p.stats)[(long)seq * p.G + g0 + g] = v;
            }
        }
        // (a block's sums stay until all have read them)
        cluster.sync();
        if (count) {
            const float3 got = all[pc / ppg];
            if constexpr (!BWD) {
                const T *gate = static_cast<const T *>(p.gate) + (start + lane) * p.ld_gate + col;
                T *y = static_cast<T *>(p.y) + (start + lane) * p.D + col;
                const Pair minus = both(-got.x);
#pragma unroll 4
                for (int r = 0; r < count; ++r) {
                    Vals<V> f = values<T, V>(at(0, r)), g;
                    if (GATE) g = values<T, V>(load_packet<T, V>(gate + r * (lanes * p.ld_gate)));
#pragma unroll
                    for (int j = 0; j < Vals<V>::N; ++j) f.p[j] = add2(f.p[j], minus);
                    store_packet<T, V>(y + (long)r * lanes * p.D, packet<T, V>(forward_vals<V, GATE>(f, g, got.y, wt, bs, p.act)));
                }
            } else {
                T *dx = static_cast<T *>(p.dx) + (start + lane) * p.D + col, *dgate = static_cast<T *>(p.dgate) + (start + lane) * p.D + col;
                const Pair m1 = both(-got.x), m2 = both(-got.y), rstd = both(st.y);
#pragma unroll 2
                for (int r = 0; r < count; ++r) {
                    Vals<V> x = values<T, V>(at(0, r)), d = values<T, V>(at(1, r)), g;
                    if (GATE) g = values<T, V>(at(kArrays - 1, r));
                    backward_vals<V, GATE>(x, g, d, st.x, st.y, wt, bs, p.act);
                    if (GATE) store_packet<T, V>(dgate + (long)r * lanes * p.D, packet<T, V>(g));
#pragma unroll
                    for (int j = 0; j < Vals<V>::N; ++j) x.p[j] = mul2(rstd, fma2(x.p[j], m2, fma2(d.p[j], wt.p[j], m1)));
                    store_packet<T, V>(dx + (long)r * lanes * p.D, packet<T, V>(x));
                }
            }
        }
        seq += walkers;
    } while (BWD && seq < p.n_seq);
}

// ------------------------------------------------------------------- host

int pow2_at_least(long x) {
    int r = 1;
    while (r < x) r *= 2;
    return r;
}

// Tokens of a tile: some 32768 elements, fewer where that leaves
// multiprocessors without one.
int tile_rows(long rows, int D) {
    int r = 512;
    while (r > 4 && (long)r * std::min(D, 2048) > 32768) r /= 2;
    while (r > 4 && rows / r * ((D + 2047) / 2048) < 608) r /= 2;
    return r;
}
long tile_slots(int n_seq, long rows, int D) { return rows / tile_rows(rows, D) + n_seq; }
// The gradient's rows of parameter sums: one for every block that takes tiles,
// for every cluster's blocks that take sequences, and no more for more sequences
// than leave no multiprocessor without work.  (Otherwise 32768 sequences of one
// token of 2048 bf16 columns would take 4.3 GB for 134 MB.)
long sum_blocks(int n_seq, long rows, int D) { return rows / tile_rows(rows, D) + std::min(n_seq, 512); }
int cluster_walkers(int n_seq, long blocks) { return (int)std::min<long>(n_seq, std::max(64L, 152 * 8 / blocks)); }

// How sequences are taken by clusters, if they are: neighbouring groups of 128
// bytes a token, and so many blocks that a thread's packets of the longest
// sequence there can be fit shared memory, three blocks to a multiprocessor where
// that goes.  (8 sequences of 2048 tokens of 2048 bf16 columns in 32 groups:
// 44 us; with two blocks to a multiprocessor 46, in tiles 62.  Forward and
// gradient of those 140, 142 and 203; of 1531 fp32 tokens of 330 columns in 6
// groups and 5 sequences 50, 56 and 62.)
struct ClusterShape {
    int per_block, blocks, smem;
};
int groups_per_cluster(int D, int G, int el) { return std::min(G, std::max(1, 128 / (D / G * el))); }
ClusterShape cluster_shape(const GroupNormProblem &p, int V, int el, bool bwd) {
    const int w = p.D / p.G, arrays = bwd ? (p.gate ? 3 : 2) : 1;
    ClusterShape c = {groups_per_cluster(p.D, p.G, el), 0, 0};
    const long packets = (long)c.per_block * (w / V), column_blocks = (p.G + c.per_block - 1) / c.per_block;
    if (packets > kThreads || p.n_seq * column_blocks * 8 > 0x7fffffffL) return c;
    const long lanes = kThreads / packets, longest = p.cu ? p.rows : p.T;
    for (int blocks = 1; blocks <= 8; blocks *= 2) {
        const long rows = (longest + blocks - 1) / blocks, bytes = (rows + lanes - 1) / lanes * kThreads * V * el * arrays;
        if (bytes > (blocks < 8 ? 56 : 176) * 1024) continue;
        c.blocks = blocks;
        c.smem = (int)bytes;
        break;
    }
    return c;
}

// Groups of a block that takes parts of sequences.
int groups_per_block(int D, int G, int V) { return std::max(1, std::min(G, kThreads * V / (D / G))); }

// How a call's tokens' groups are spread.
struct TokenShape {
    int tpg, NI, threads;
    long blocks, lanes;
};
long gcd(long a, long b) { return b ? gcd(b, a % b) : a; }

// Over `most` blocks at most.
void spread(const GroupNormProblem &p, TokenShape &t, long most) {
    const long ipb = t.threads / t.tpg, unit = p.G / gcd(ipb, p.G);
    const long blocks = std::min((p.rows * p.G + ipb - 1) / ipb, most) / unit * unit;
    t.blocks = std::max(blocks, unit);
    t.lanes = t.blocks * ipb / p.G;
}
// The gradient's blocks: two of 256 threads to a multiprocessor, as many as are
// there at once, since each lane of tokens leaves a row of the parameters' sums
// behind.  (16384 tokens of 16 groups of 128 bf16 columns, gate: forward and
// gradient 114 us; with one block 140, three 129, four 119.)
TokenShape token_shape(const GroupNormProblem &p, int V, bool bwd) {
    TokenShape t;
    const long P = (p.D / p.G) / V;
    // Two packets a thread, of small ones four, and more only where a block has no
    // more threads: more of them leave no registers for weights and the next token.
    // (32768 tokens of one group of 2048 bf16 columns, gate: one 110 us, two 86,
    // four 230; of four groups: 101, 79, 78.  16384 tokens of 1023 fp32 columns:
    // two 84, four 67.)
    for (int each = V < 4 ? 4 : 2;; each *= 2) {
        t.tpg = P <= 32 ? pow2_at_least(P) : std::max(32, pow2_at_least((P + each - 1) / each));
        t.NI = pow2_at_least((P + t.tpg - 1) / t.tpg);
        const int most = most_threads(t.NI, V, bwd);
        if (t.tpg <= most) break;
        if (most == 0) {
            t.tpg = t.threads = kThreadsWide;
            t.NI = 0;
            spread(p, t, 152L * 2);
            return t;
        }
    }
    t.threads = std::max(kThreads, t.tpg);
    spread(p, t, 152L * std::max(1, 2 * kThreads / t.threads));
    return t;
}
long token_lanes_most(long rows, int D, int G) {
    const long w = D / G;
    long most = 0;
    for (int V : {8, 4, 2, 1}) {
        if (w % V) continue;
        GroupNormProblem p = {};
        p.rows = rows;
        p.D = D;
        p.G = G;
        most = std::max(most, token_shape(p, V, true).lanes);
    }
    return most;
}

bool packets_fit(const GroupNormProblem &p, int el, int V, int bytes, bool bwd) {
    if ((p.D / p.G) % V) return false;
    if (!rows_aligned(p.x, p.ld_x, el, bytes) || (p.gate && !rows_aligned(p.gate, p.ld_gate, el, bytes))) return false;
    if (!bwd) return rows_aligned(p.y, p.D, el, bytes);
    return rows_aligned(p.dy, p.ld_dy, el, bytes) && rows_aligned(p.dx, p.D, el, bytes) &&
           rows_aligned(p.dgate, p.D, el, bytes);
}

template <typename T>
int width_of(const GroupNormProblem &p, bool bwd) {
    const int el = (int)sizeof(T);
    return packet_width(16 / el, el, [&](int V, int bytes) { return packets_fit(p, el, V, bytes, bwd); });
}

template <typename T, int V, int NI, bool GATE>
cudaError_t token_launch(const GroupNormProblem &p, TokenShape t, float *part, bool bwd, cudaStream_t st) {
    if (bwd) {
        if constexpr (most_threads(NI, V, true) > 0)
            token_bwd_kernel<T, V, NI, GATE><<<(unsigned)t.blocks, t.threads, 0, st>>>(p, t.tpg, part);
        return cudaGetLastError();
    }
    // The forward takes two whole waves: blocks end at different times, and the
    // second one's fill the gaps.  (32768 tokens of 16 groups of 128 columns,
    // gate.  bf16, three blocks to a multiprocessor at once: in all 5 92 us, 6 81,
    // 7 93, 8 89, 12 85; fp32, four: 5 167, 6 146, 7 137, 8 130, 12 132.)
    spread(p, t, 1L << 30);
    if (t.blocks > 152) {
        int resident = 1;
        const cudaError_t err =
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident, token_fwd_kernel<T, V, NI, GATE>, t.threads, 0);
        if (err != cudaSuccess) return err;
        spread(p, t, 152L * 2 * std::max(1, resident));
    }
    token_fwd_kernel<T, V, NI, GATE><<<(unsigned)t.blocks, t.threads, 0, st>>>(p, t.tpg);
    return cudaGetLastError();
}
template <typename T, int V, bool GATE>
cudaError_t wide_launch(const GroupNormProblem &p, const TokenShape &t, float *part, bool bwd, cudaStream_t st) {
    if (bwd) {
        const int smem = part ? 2 * (p.D / p.G) * (int)sizeof(float) : 0;
        // (the widest group's)
        const cudaError_t err = smem > 47 * 1024 ? allow_shared<wide_bwd_kernel<T, V, GATE>>(2 * 16384 * (int)sizeof(float)) : cudaSuccess;
        if (err != cudaSuccess) return err;
        wide_bwd_kernel<T, V, GATE><<<(unsigned)t.blocks, kThreadsWide, smem, st>>>(p, part);
    } else {
        wide_fwd_kernel<T, V, GATE><<<(unsigned)t.blocks, kThreadsWide, 0, st>>>(p);
    }
    return cudaGetLastError();
}
template <typename T, int V, bool GATE>
cudaError_t token_pick(const GroupNormProblem &p, const TokenShape &t, float *part, bool bwd, cudaStream_t st) {
    switch (t.NI) {
        case 0: return wide_launch<T, V, GATE>(p, t, part, bwd, st);
        case 1: return token_launch<T, V, 1, GATE>(p, t, part, bwd, st);
        case 2: return token_launch<T, V, 2, GATE>(p, t, part, bwd, st);
        case 4:
            if constexpr (V < 8) return token_launch<T, V, 4, GATE>(p, t, part, bwd, st);
            break;
        case 8:
            if constexpr (V < 4) return token_launch<T, V, 8, GATE>(p, t, part, bwd, st);
    }
    return cudaErrorInvalidValue;      // (token_shape gives no others)
}

cudaError_t params(const GroupNormProblem &p, const float *part, long lanes, cudaStream_t st) {
    if (!p.dw && !p.dbias) return cudaSuccess;
    return follow(param_kernel, dim3((2 * p.D + 31) / 32), 1024, st, part, (int)lanes, p.D, p.dw, p.dbias);
}

template <typename T, int V, bool GATE, bool BWD>
cudaError_t cluster_launch(const GroupNormProblem &p, const ClusterShape &c, int walkers, float *prm, cudaStream_t st) {
    const auto kernel = seq_cluster_kernel<T, V, GATE, BWD>;
    // (the largest of the shapes; below 48 KiB with the static arrays nothing need be asked)
    const cudaError_t err = allow_shared<seq_cluster_kernel<T, V, GATE, BWD>>(176 * 1024);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long)walkers * ((p.G + c.per_block - 1) / c.per_block) * c.blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = c.smem;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = c.blocks;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, c.per_block, c.blocks, walkers, prm);
}

template <typename T, int V, bool GATE>
cudaError_t run(const GroupNormProblem &p, bool bwd, cudaStream_t st) {
    cudaError_t err;
    if (!p.over_sequence) {
        const TokenShape t = token_shape(p, V, bwd);
        float *part = bwd && (p.dw || p.dbias) ? reinterpret_cast<float *>(p.ws) : nullptr;
        if ((err = token_pick<T, V, GATE>(p, t, part, bwd, st)) != cudaSuccess) return err;
        return bwd ? params(p, part, t.lanes, st) : cudaSuccess;
    }
    if (p.ok) {
        check_kernel<<<1, 1024, 0, st>>>(p);
        if ((err = cudaGetLastError()) != cudaSuccess) return err;
    }
    const ClusterShape c = cluster_shape(p, V, (int)sizeof(T), bwd);
    if (c.blocks) {
        float *prm = bwd && (p.dw || p.dbias) ? reinterpret_cast<float *>(p.ws) : nullptr;
        if (!bwd) return cluster_launch<T, V, GATE, false>(p, c, p.n_seq, prm, st);
        const int walkers = cluster_walkers(p.n_seq, (p.G + c.per_block - 1) / c.per_block * c.blocks);
        err = cluster_launch<T, V, GATE, true>(p, c, walkers, prm, st);
        return err == cudaSuccess ? params(p, prm, (long)walkers * c.blocks, st) : err;
    }
    const int rows = tile_rows(p.rows, p.D), gpb = groups_per_block(p.D, p.G, V);
    const long slots = p.cu ? tile_slots(p.n_seq, p.rows, p.D) : (long)p.n_seq * ((p.T + rows - 1) / rows);
    const long most = tile_slots(p.n_seq, p.rows, p.D);
    const dim3 grid((unsigned)slots, (p.G + gpb - 1) / gpb);
    const long groups = (long)p.n_seq * p.G;
    const unsigned joins = (unsigned)((groups + kThreads / 32 - 1) / (kThreads / 32));
    unsigned char *ws = p.ws;
    float2 *part = reinterpret_cast<float2 *>(ws);
    ws += round256(most * p.G * sizeof(float2));
    float2 *second = reinterpret_cast<float2 *>(ws);
    ws += round256(groups * sizeof(float2));
    if (!bwd) {
        float2 *stats = p.stats ? reinterpret_cast<float2 *>(p.stats) : second;
        seq_stats_kernel<T, V><<<grid, kThreads, 0, st>>>(p, rows, gpb, part);
        if ((err = cudaGetLastError()) != cudaSuccess) return err;
        if ((err = follow(seq_join_kernel, dim3(joins), kThreads, st, p, rows, part, stats)) != cudaSuccess) return err;
        return follow(seq_apply_kernel<T, V, GATE>, grid, kThreads, st, p, rows, gpb, stats);
    }
    float *prm = p.dw || p.dbias ? reinterpret_cast<float *>(ws) : nullptr;
    const long summed = std::min(slots, sum_blocks(p.n_seq, p.rows, p.D));
    seq_sums_kernel<T, V, GATE><<<dim3((unsigned)summed, grid.y), kThreads, 0, st>>>(p, rows, gpb, (int)slots, part, prm);
    if ((err = cudaGetLastError()) != cudaSuccess) return err;
    if ((err = follow(seq_means_kernel, dim3(joins), kThreads, st, p, rows, part, second)) != cudaSuccess) return err;
    if ((err = follow(seq_dx_kernel<T, V, GATE>, grid, kThreads, st, p, rows, gpb, second)) != cudaSuccess) return err;
    return params(p, prm, summed, st);
}

template <typename T, int V>
cudaError_t gated(const GroupNormProblem &p, bool bwd, cudaStream_t st) {
    return p.gate ? run<T, V, true>(p, bwd, st) : run<T, V, false>(p, bwd, st);
}

cudaError_t launch(const GroupNormProblem &given, bool bwd, cudaStream_t st) {
    GroupNormProblem p = given;
    if (p.cu && p.n_seq > kManySequences) {
        p.ok = reinterpret_cast<int *>(p.ws);
        p.ws += 256;
    }
    if (p.rows == 0) {
        cudaError_t err = cudaSuccess;
        if (!bwd && p.stats && p.over_sequence && p.n_seq)
            err = cudaMemsetAsync(p.stats, 0, (size_t)p.n_seq * p.G * sizeof(float2), st);
        if (bwd && p.dw) err = cudaMemsetAsync(p.dw, 0, p.D * sizeof(float), st);
        if (bwd && p.dbias && err == cudaSuccess) err = cudaMemsetAsync(p.dbias, 0, p.D * sizeof(float), st);
        return err;
    }
    if (p.dtype == MDN_BF16) {
        switch (width_of<__nv_bfloat16>(p, bwd)) {
            case 8: return gated<__nv_bfloat16, 8>(p, bwd, st);
            case 2: return gated<__nv_bfloat16, 2>(p, bwd, st);
            default: return gated<__nv_bfloat16, 1>(p, bwd, st);
        }
    }
    return width_of<float>(p, bwd) == 4 ? gated<float, 4>(p, bwd, st) : gated<float, 1>(p, bwd, st);
}

}  // namespace

cudaError_t launch_group_norm_fwd(const GroupNormProblem &p, cudaStream_t st) { return launch(p, false, st); }
cudaError_t launch_group_norm_bwd(const GroupNormProblem &p, cudaStream_t st) { return launch(p, true, st); }

size_t group_norm_fwd_workspace(int n_seq, long rows, int D, int G, bool over_sequence, mdn_dtype) {
    if (!over_sequence || rows == 0) return 0;
    // (256: check_kernel's flag)
    return 256 + round256(tile_slots(n_seq, rows, D) * G * sizeof(float2)) + round256((long)n_seq * G * sizeof(float2));
}
size_t group_norm_bwd_workspace(int n_seq, long rows, int D, int G, bool over_sequence, mdn_dtype dtype) {
    if (rows == 0) return 0;
    if (!over_sequence) return round256(token_lanes_most(rows, D, G) * 2 * D * sizeof(float));
    // (a cluster has eight blocks at most)
    const int per_block = groups_per_cluster(D, G, dtype == MDN_BF16 ? 2 : 4);
    long most = sum_blocks(n_seq, rows, D);
    for (long blocks = 1; blocks <= 8; blocks *= 2)
        most = std::max(most, cluster_walkers(n_seq, (G + per_block - 1) / per_block * blocks) * blocks);
    return group_norm_fwd_workspace(n_seq, rows, D, G, true, dtype) + round256(most * 2 * D * sizeof(float));
}

}  // namespace mdn
