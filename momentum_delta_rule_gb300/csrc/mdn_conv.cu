// Short causal depthwise convolution along the tokens: forward, gradient and
// the single-token step.
//
//   pre_t = bias + sum_{j<W} w_j x_{t-(W-1-j)},   y_t = act(pre_t)
//   dpre  = dy act'(pre);  dx_q = sum_k w_{W-1-k} dpre_{q+k};
//   dw_j  = sum_t dpre_t x_{t-(W-1-j)};  dbias = sum_t dpre_t
//
// Tokens before a sequence's first are its W - 1 initial-state rows.  Memory
// bound (2 W + 4 flops against 2 elements moved): a thread owns four
// neighbouring channels and a run of consecutive tokens, keeps the last W - 1
// inputs in registers, and copies the rows ahead of it asynchronously into
// shared memory that only it reads.  A batch of rows inside one sequence runs
// without a branch.  Runs are cut so that one wave of blocks covers the
// tokens: what a run starts with (weights, the rows before it, the search for
// its sequence) costs as much as a dozen tokens.
//
// Measured, bf16, SiLU, width 4: 32768 tokens of 2048 channels 49 us (5.5 TB/s
// over the 269 MB read and written once); 16384 tokens of 4096 channels 49 us
// forward and 90 us gradient (4.5 TB/s over 403 MB).  A copy of the same bytes
// takes 40, 40 and 59 us.  The forward is held by the latency at the ends of
// its one wave; the gradient also by issue: SiLU and its derivative beside the
// 4 W operations of an element.  256 sequences' single tokens at 2048
// channels: 3.5 us, the latency of one round of loads and stores.
#include <algorithm>

#include "mdn_ssm.cuh"

namespace mdn {
namespace {

constexpr int kConvThreads = 128;
// Blocks that an SM holds (the launch bounds give them the registers) and that
// one wave of the forward and of the gradient has on each.
constexpr int kFwdBlocks = 6, kBwdBlocks = 4;

// v <- act(v)
template <int V>
__device__ __forceinline__ void conv_act(float *v, int act) {
    if (act != MDN_CONV_SILU) return;
    float s[V];
    sigmoids<V>(v, s);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] *= s[i];
}
// v <- act'(v)
template <int V>
__device__ __forceinline__ void conv_dact(float *v, int act) {
    float s[V];
    if (act == MDN_CONV_SILU) sigmoids<V>(v, s);
#pragma unroll
    for (int i = 0; i < V; ++i)
        v[i] = act == MDN_CONV_SILU ? s[i] * fmaf(v[i], 1.f - s[i], 1.f) : 1.f;
}

// Walk over sequences: the one that holds the current token.
struct SeqWalk {
    int s;
    long start, end;
    __device__ __forceinline__ void find(const ConvProblem &p, long t) {
        if (p.cu) {
            s = seq_of_token(p.cu, p.n_seq, t);
            start = p.cu[s];
            end = p.cu[s + 1];
        } else {
            s = (int)(t / p.T);
            start = (long)s * p.T;
            end = start + p.T;
        }
    }
    // The next sequence with tokens.
    __device__ __forceinline__ void next(const ConvProblem &p) {
        do {
            ++s;
            start = end;
            end = p.cu ? (long)p.cu[s + 1] : start + p.T;
        } while (end == start);
    }
};

// The weights [tap][channel] and the bias of channels c .. c + V.
template <int V, int W>
__device__ __forceinline__ void load_weights(const ConvProblem &p, int c, float (*w)[V], float *bias) {
    float f[V * W];
    const float *src = p.w + (long)c * W;
    if constexpr (V == 4) {
#pragma unroll
        for (int i = 0; i < W; ++i) unpack<float, 4>(load_packet<float, 4>(src + 4 * i), f + 4 * i);
    } else {
#pragma unroll
        for (int i = 0; i < V * W; ++i) f[i] = src[i];
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][v] = f[v * W + j];
        bias[v] = p.bias ? p.bias[c + v] : 0.f;
    }
}

// Input at position `pos` of sequence w (pos >= start - (W - 1)): a token, an
// initial-state row or zero.
template <typename T, int V, int W>
__device__ __forceinline__ void conv_input(const ConvProblem &p, const SeqWalk &w, long pos, int c,
                                           float *f) {
    const T *src = nullptr;
    if (pos >= w.start)
        src = static_cast<const T *>(p.x) + pos * p.ld_x + c;
    else if (p.state0)
        src = static_cast<const T *>(p.state0) +
              ((long)w.s * (W - 1) + (W - 1) + (pos - w.start)) * p.D + c;
    if (src) {
        unpack<T, V>(load_packet<T, V>(src), f);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) f[v] = 0.f;
    }
}

// Copies state0's rows (or zeros) of sequence s to `out`.
template <typename T, int V, int W>
__device__ __forceinline__ void copy_state(const void *from, void *out, int s, int D, int c) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const long at = ((long)s * (W - 1) + j) * D + c;
        Packet<T, V> v;
        if (from) {
            v = load_packet<T, V>(static_cast<const T *>(from) + at);
        } else {
            float zero[V];
#pragma unroll
            for (int e = 0; e < V; ++e) zero[e] = 0.f;
            v = pack<T, V>(zero);
        }
        store_packet<T, V>(static_cast<T *>(out) + at, v);
    }
}

// Thread layout: cl lanes across channel packets (the fastest), the rest of
// the block across runs of tokens.
struct ConvGrid {
    int cl;            // channel lanes per block (a power of two)
    int ctiles;        // blocks across the channels
    int run;           // tokens per run
    long nruns;
};

// Rows of a batch: 64 bytes of a thread's packets, so that a block's copies
// ahead take as much shared memory in either type.
template <typename T, int V>
constexpr int kBatch = V * sizeof(T) == 16 ? 4 : 8;
constexpr int kConvAhead = 2;          // batches in flight

// This thread's rows ahead: batch k of a run in slot k % (kConvAhead + 1).
template <typename T, int V>
struct RowRing {
    static constexpr int kRows = kBatch<T, V>;
    Packet<T, V> (*at)[kRows][kConvThreads];
    const T *src;                      // the run's first row, this thread's channels
    long ld;
    Copies<T, V, kRows> copies;
    __device__ __forceinline__ RowRing(Packet<T, V> (*at_)[kRows][kConvThreads], const T *src_, long ld_)
        : at(at_), src(src_), ld(ld_) {
        copies.clear();
    }
    // Batch k, two ahead of the one in use: a copy that goes through registers
    // reaches shared memory with the next issue, still one ahead.
    __device__ __forceinline__ void issue(int k, long rows) {
        const int slot = k % (kConvAhead + 1);
        copies.put();
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            if (k * kRows + i < rows)
                copies.get(i, &at[slot][i][threadIdx.x], src + (long)(k * kRows + i) * ld);
    }
    __device__ __forceinline__ void row(int k, int i, float *f) const {
        unpack<T, V>(at[k % (kConvAhead + 1)][i][threadIdx.x], f);
    }
};

template <int V, int W>
__device__ __forceinline__ void conv_sum(const float (*w)[V], const float *bias, const float (*win)[V],
                                         const float *x, float *pre) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        pre[v] = fmaf(w[W - 1][v], x[v], bias[v]);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) pre[v] = fmaf(w[j][v], win[j][v], pre[v]);
    }
}
template <int V, int W>
__device__ __forceinline__ void push_row(float (*win)[V], const float *x) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) win[j][v] = j + 1 < W - 1 ? win[j + 1][v] : x[v];
}

template <typename T, int V, int W>
__global__ void __launch_bounds__(kConvThreads, kFwdBlocks) conv_fwd_kernel(ConvProblem p, ConvGrid g) {
    constexpr int kRows = kBatch<T, V>;
    __shared__ Packet<T, V> ring[kConvAhead + 1][kRows][kConvThreads];
    const int lane = threadIdx.x & (g.cl - 1);
    const int ct = blockIdx.x % g.ctiles;
    const long row = (long)(blockIdx.x / g.ctiles) * (kConvThreads / g.cl) + threadIdx.x / g.cl;
    const int c = (ct * g.cl + lane) * V;
    if (p.cu && !cu_well_formed(p.cu, p.n_seq, p.T_total)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicExch(p.status, (int)MDN_ERR_INVALID_ARG);
        if (p.state_T && c < p.D)
            for (long s = row; s < p.n_seq; s += g.nruns)
                copy_state<T, V, W>(p.state0, p.state_T, (int)s, p.D, c);
        return;
    }
    if (row >= g.nruns || c >= p.D) return;
    const long t0 = row * g.run;
    const long t1 = min(t0 + g.run, (long)p.T_total);
    RowRing<T, V> rx{ring, static_cast<const T *>(p.x) + t0 * p.ld_x + c, p.ld_x};
#pragma unroll
    for (int k = 0; k < kConvAhead; ++k) {
        rx.issue(k, t1 - t0);
        commit_copies();
    }
    T *yp = static_cast<T *>(p.y) + c;
    float w[W][V], bias[V];
    load_weights<V, W>(p, c, w, bias);
    SeqWalk q;
    q.find(p, t0);
    if (t0 == 0 && p.state_T)           // empty sequences before the first token
        for (int s = 0; s < q.s; ++s) copy_state<T, V, W>(p.state0, p.state_T, s, p.D, c);
    float win[W - 1][V];                // inputs t - (W - 1) .. t - 1
#pragma unroll
    for (int j = 0; j < W - 1; ++j) conv_input<T, V, W>(p, q, t0 - (W - 1) + j, c, win[j]);
    auto finish = [&]() {               // q ended: its state, and those of empty ones that follow
        if (!p.state_T) return;
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            store_packet<T, V>(static_cast<T *>(p.state_T) + ((long)q.s * (W - 1) + j) * p.D + c,
                               pack<T, V>(win[j]));
        if (p.cu)
            for (int s = q.s + 1; s < p.n_seq && p.cu[s + 1] == q.end; ++s)
                copy_state<T, V, W>(p.state0, p.state_T, s, p.D, c);
    };
    auto token = [&](long t, const float *x) {
        float o[V];
        conv_sum<V, W>(w, bias, win, x, o);
        conv_act<V>(o, p.act);
        store_packet<T, V>(yp + t * p.D, pack<T, V>(o));
        push_row<V, W>(win, x);
    };
    int k = 0;
    for (long tb = t0; tb < t1; tb += kRows, ++k) {
        rx.issue(k + kConvAhead, t1 - t0);
        commit_copies();
        wait_copies<kConvAhead>();
        if (tb + kRows <= t1 && tb + kRows <= q.end) {
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                float x[V];
                rx.row(k, i, x);
                token(tb + i, x);
            }
            if (tb + kRows == q.end) finish();
        } else {
#pragma unroll 1
            for (long t = tb; t < tb + kRows && t < t1; ++t) {
                if (t == q.end) {       // the next sequence with tokens
                    q.next(p);
#pragma unroll
                    for (int j = 0; j < W - 1; ++j)
                        conv_input<T, V, W>(p, q, t - (W - 1) + j, c, win[j]);
                }
                float x[V];
                rx.row(k, (int)(t - tb), x);
                token(t, x);
                if (t + 1 == q.end) finish();
            }
        }
        // a batch that begins a sequence starts from its state
        if (tb + kRows < t1 && tb + kRows == q.end) {
            q.next(p);
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
                conv_input<T, V, W>(p, q, q.start - (W - 1) + j, c, win[j]);
        }
    }
    wait_copies<0>();
}

// dx lags dpre by W - 1 tokens: at token t the output is position t - (W - 1).
// A run goes W - 1 tokens past its end (recomputing dpre there, the next run's
// first rows; zero behind a sequence's end), and where it holds a sequence's
// start it also produces the W - 1 positions before that, the gradient of the
// initial state.  dstate of a sequence without tokens is the adjoint of the
// state it hands on.
template <typename T, int V, int W>
__global__ void __launch_bounds__(kConvThreads, kBwdBlocks) conv_bwd_kernel(ConvProblem p, ConvGrid g) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    constexpr int kRows = kBatch<T, V>;
    using Ring = Packet<T, V>[kConvAhead + 1][kRows][kConvThreads];
    const int lane = threadIdx.x & (g.cl - 1);
    const int ct = blockIdx.x % g.ctiles;
    const long row = (long)(blockIdx.x / g.ctiles) * (kConvThreads / g.cl) + threadIdx.x / g.cl;
    const int c = (ct * g.cl + lane) * V;
    const bool ok = !p.cu || cu_well_formed(p.cu, p.n_seq, p.T_total);
    if (c >= p.D) return;
    float dw[W][V], db[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][v] = 0.f;
        db[v] = 0.f;
    }
    if (!ok) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicExch(p.status, (int)MDN_ERR_INVALID_ARG);
        if (p.dstate0)
            for (long s = row; s < p.n_seq; s += g.nruns)
                copy_state<T, V, W>(p.dstate_T, p.dstate0, (int)s, p.D, c);
    } else if (row < g.nruns) {
        const long t0 = row * g.run;
        const long t1 = min(t0 + g.run, (long)p.T_total);
        const T *xp = static_cast<const T *>(p.x) + c, *dyp = static_cast<const T *>(p.dy) + c;
        Ring *ring = reinterpret_cast<Ring *>(smem_raw);
        RowRing<T, V> rx{ring[0], xp + t0 * p.ld_x, p.ld_x};
        RowRing<T, V> ry{ring[1], dyp + t0 * p.ld_dy, p.ld_dy};
#pragma unroll
        for (int k = 0; k < kConvAhead; ++k) {
            rx.issue(k, t1 - t0);
            ry.issue(k, t1 - t0);
            commit_copies();
        }
        float w[W][V], bias[V];
        load_weights<V, W>(p, c, w, bias);
        SeqWalk q;
        q.find(p, t0);
        if (t0 == 0 && p.dstate0)
            for (int s = 0; s < q.s; ++s) copy_state<T, V, W>(p.dstate_T, p.dstate0, s, p.D, c);
        long a = t0;                     // first token of this run in sequence q
        float win[W - 1][V], dp[W - 1][V];     // inputs, and dpre, of the W - 1 tokens before t
        auto begin = [&]() {
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                conv_input<T, V, W>(p, q, a - (W - 1) + j, c, win[j]);
#pragma unroll
                for (int v = 0; v < V; ++v) dp[j][v] = 0.f;
            }
        };
        begin();
        // dpre of a token; its part of dw and db
        auto dpre = [&](const float *x, const float *d, bool mine, float *e) {
            conv_sum<V, W>(w, bias, win, x, e);
            conv_dact<V>(e, p.act);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                e[v] *= d[v];
                if (mine) {
                    db[v] += e[v];
                    dw[W - 1][v] = fmaf(e[v], x[v], dw[W - 1][v]);
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) dw[j][v] = fmaf(e[v], win[j][v], dw[j][v]);
                }
            }
            push_row<V, W>(win, x);
        };
        // dx of position t - (W - 1) once dpre_t is known
        auto back = [&](const float *e, float *o) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                o[v] = w[0][v] * e[v];
#pragma unroll
                for (int j = 0; j < W - 1; ++j) o[v] = fmaf(w[W - 1 - j][v], dp[j][v], o[v]);
            }
            push_row<V, W>(dp, e);
        };
        auto output = [&](long pos, float *o) {
            if (pos < a && !(a == q.start && p.dstate0)) return;
            if (p.dstate_T && pos >= q.end - (W - 1)) {
                float e[V];
                unpack<T, V>(load_packet<T, V>(static_cast<const T *>(p.dstate_T) +
                                               ((long)q.s * (W - 1) + (pos - (q.end - (W - 1)))) * p.D + c),
                             e);
#pragma unroll
                for (int v = 0; v < V; ++v) o[v] += e[v];
            }
            T *dst = pos >= a ? static_cast<T *>(p.dx) + pos * p.D + c
                              : static_cast<T *>(p.dstate0) +
                                    ((long)q.s * (W - 1) + (W - 1) + (pos - q.start)) * p.D + c;
            store_packet<T, V>(dst, pack<T, V>(o));
        };
        // the W - 1 positions still open at token t (the run's or q's end)
        auto drain = [&](long t) {
#pragma unroll 1
            for (int i = 0; i < W - 1; ++i, ++t) {
                float e[V], o[V];
                if (t < q.end) {
                    float x[V], d[V];
                    unpack<T, V>(load_packet<T, V>(xp + t * p.ld_x), x);
                    unpack<T, V>(load_packet<T, V>(dyp + t * p.ld_dy), d);
                    dpre(x, d, false, e);
                } else {
#pragma unroll
                    for (int v = 0; v < V; ++v) e[v] = 0.f;
                }
                back(e, o);
                output(t - (W - 1), o);
            }
            if (t >= q.end + (W - 1) && p.dstate0 && p.cu)      // empty sequences that follow
                for (int s = q.s + 1; s < p.n_seq && p.cu[s + 1] == q.end; ++s)
                    copy_state<T, V, W>(p.dstate_T, p.dstate0, s, p.D, c);
        };
        int k = 0;
        for (long tb = t0; tb < t1; tb += kRows, ++k) {
            rx.issue(k + kConvAhead, t1 - t0);
            ry.issue(k + kConvAhead, t1 - t0);
            commit_copies();
            wait_copies<kConvAhead>();
            if (tb >= a + W - 1 && tb + kRows <= t1 && tb + kRows <= q.end) {
                // all outputs are the run's own, and none is within
                // W - 1 of the sequence's end
                T *dst = static_cast<T *>(p.dx) + (tb - (W - 1)) * p.D + c;
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    float x[V], d[V], e[V], o[V];
                    rx.row(k, i, x);
                    ry.row(k, i, d);
                    dpre(x, d, true, e);
                    back(e, o);
                    store_packet<T, V>(dst + (long)i * p.D, pack<T, V>(o));
                }
            } else {
#pragma unroll 1
                for (long t = tb; t < tb + kRows && t < t1; ++t) {
                    if (t == q.end) {
                        drain(t);
                        q.next(p);
                        a = t;
                        begin();
                    }
                    float x[V], d[V], e[V], o[V];
                    rx.row(k, (int)(t - tb), x);
                    ry.row(k, (int)(t - tb), d);
                    dpre(x, d, true, e);
                    back(e, o);
                    output(t - (W - 1), o);
                }
            }
        }
        wait_copies<0>();
        drain(t1);
    }
    float *part = p.partial + row * (long)(W + 1) * p.D + c;
#pragma unroll
    for (int j = 0; j < W; ++j) store_packet<float, V>(part + (long)j * p.D, pack<float, V>(dw[j]));
    store_packet<float, V>(part + (long)W * p.D, pack<float, V>(db));
}

// Sums the rows' partial sums in order: 8 threads per column, a warp's 32
// columns side by side.
__global__ void __launch_bounds__(256)
conv_reduce_kernel(const float *partial, int rows, int D, int W, float *dw, float *dbias) {
    __shared__ float s[8][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const long cols = (long)(W + 1) * D;
    const long i = (long)blockIdx.x * 32 + tx;
    float a = 0.f;
    if (i < cols)
        for (int r = ty; r < rows; r += 8) a += partial[r * cols + i];
    s[ty][tx] = a;
    __syncthreads();
    if (ty != 0 || i >= cols) return;
#pragma unroll
    for (int k = 1; k < 8; ++k) a += s[k][tx];
    const int j = (int)(i / D);
    const int c = (int)(i - (long)j * D);
    if (j < W) dw[(long)c * W + j] = a;
    else if (dbias) dbias[c] = a;
}

template <typename T, int V, int W>
__global__ void __launch_bounds__(kConvThreads) conv_step_kernel(ConvProblem p, int packets) {
    const long idx = (long)blockIdx.x * kConvThreads + threadIdx.x;
    const long n = idx / packets;
    if (n >= p.n_seq) return;
    const int c = (int)(idx - n * packets) * V;
    const T *st = static_cast<const T *>(p.state0) + n * (W - 1) * p.D + c;
    T *so = static_cast<T *>(p.state_T) + n * (W - 1) * p.D + c;
    Packet<T, V> row[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) row[j] = load_packet<T, V>(st + (long)j * p.D);
    row[W - 1] = load_packet<T, V>(static_cast<const T *>(p.x) + n * p.ld_x + c);
    float w[W][V], o[V];
    load_weights<V, W>(p, c, w, o);
#pragma unroll
    for (int j = 0; j < W; ++j) {
        float x[V];
        unpack<T, V>(row[j], x);
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = fmaf(w[j][v], x[v], o[v]);
    }
    conv_act<V>(o, p.act);
    store_packet<T, V>(static_cast<T *>(p.y) + n * p.D + c, pack<T, V>(o));
#pragma unroll
    for (int j = 0; j < W - 1; ++j) store_packet<T, V>(so + (long)j * p.D, row[j + 1]);
}

// state_T <- state0 (or zero) for a call without tokens.
template <typename T>
__global__ void conv_copy_kernel(const T *from, T *to, long n) {
    for (long i = (long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long)gridDim.x * blockDim.x)
        to[i] = from ? from[i] : from_f32<T>(0.f);
}

template <typename T>
cudaError_t copy_states(const void *from, void *to, long n, cudaStream_t st) {
    if (!to || n == 0) return cudaSuccess;
    const long blocks = (n + 255) / 256;
    conv_copy_kernel<T><<<(unsigned)(blocks < 1216 ? blocks : 1216), 256, 0, st>>>(
        static_cast<const T *>(from), static_cast<T *>(to), n);
    return cudaGetLastError();
}

// Runs such that `blocks` blocks cover the tokens, of at least `least` tokens.
ConvGrid conv_grid(int D, int V, long T_total, long blocks, int least) {
    ConvGrid g;
    const int packets = (D + V - 1) / V;
    g.cl = 1;
    while (g.cl < packets && g.cl < kConvThreads) g.cl *= 2;
    g.ctiles = (packets + g.cl - 1) / g.cl;
    const long rows = std::max(1L, blocks / g.ctiles) * (kConvThreads / g.cl);
    g.run = (int)std::max<long>(least, (T_total + rows - 1) / rows);
    g.nruns = (T_total + g.run - 1) / g.run;
    return g;
}
// One wave on 152 SMs.  The gradient recomputes W - 1 tokens a run, so its
// shortest runs are longer; each run leaves one row of partial sums.  In us with
// half and twice these shortest runs, bf16: forward of 512 tokens of 2048
// channels 4.8 and 4.7 where this takes 4.3, of 4096 tokens of 512 channels 6.2
// and 5.5 for 5.2; gradient with its sums 10.2 and 13.1 for 11.0, and 15.6 and
// 13.7 for 13.3.
ConvGrid conv_fwd_grid(int D, int V, long T_total) { return conv_grid(D, V, T_total, 152L * kFwdBlocks, 8); }
ConvGrid conv_bwd_grid(int D, int V, long T_total) { return conv_grid(D, V, T_total, 152L * kBwdBlocks, 16); }
long conv_bwd_rows(const ConvGrid &g) {
    const int per = kConvThreads / g.cl;
    return std::max(1L, (g.nruns + per - 1) / per) * per;
}

template <typename T, int V, int W>
cudaError_t conv_fwd_t(const ConvProblem &p, cudaStream_t st) {
    const ConvGrid g = conv_fwd_grid(p.D, V, p.T_total);
    const long blocks = (g.nruns + kConvThreads / g.cl - 1) / (kConvThreads / g.cl) * g.ctiles;
    if (blocks > 0x7fffffffL) return cudaErrorInvalidConfiguration;
    conv_fwd_kernel<T, V, W><<<(unsigned)blocks, kConvThreads, 0, st>>>(p, g);
    return cudaGetLastError();
}
template <typename T, int V, int W>
cudaError_t conv_bwd_t(const ConvProblem &p, cudaStream_t st) {
    const ConvGrid g = conv_bwd_grid(p.D, V, p.T_total);
    const long rows = conv_bwd_rows(g);
    const long blocks = rows / (kConvThreads / g.cl) * g.ctiles;
    if (blocks > 0x7fffffffL) return cudaErrorInvalidConfiguration;
    constexpr int bytes = 2 * (kConvAhead + 1) * kBatch<T, V> * kConvThreads * (int)sizeof(Packet<T, V>);
    static_assert(bytes <= 48 * 1024, "four blocks an SM");
    conv_bwd_kernel<T, V, W><<<(unsigned)blocks, kConvThreads, bytes, st>>>(p, g);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    const long cols = (long)(W + 1) * p.D;
    conv_reduce_kernel<<<(unsigned)((cols + 31) / 32), 256, 0, st>>>(p.partial, (int)rows, p.D, W, p.dw,
                                                                     p.dbias);
    return cudaGetLastError();
}
template <typename T, int V, int W>
cudaError_t conv_step_t(const ConvProblem &p, cudaStream_t st) {
    const int packets = p.D / V;
    const long blocks = ((long)p.n_seq * packets + kConvThreads - 1) / kConvThreads;
    if (blocks > 0x7fffffffL) return cudaErrorInvalidConfiguration;
    conv_step_kernel<T, V, W><<<(unsigned)blocks, kConvThreads, 0, st>>>(p, packets);
    return cudaGetLastError();
}

enum class ConvKind { kFwd, kBwd, kStep };

template <ConvKind K, typename T, int V>
cudaError_t conv_width(const ConvProblem &p, cudaStream_t st) {
#define MDN_CONV_CASE(W)                                                     \
    case W:                                                                  \
        if constexpr (K == ConvKind::kFwd) return conv_fwd_t<T, V, W>(p, st); \
        if constexpr (K == ConvKind::kBwd) return conv_bwd_t<T, V, W>(p, st); \
        return conv_step_t<T, V, W>(p, st);
    switch (p.width) {
        MDN_CONV_CASE(2)
        MDN_CONV_CASE(3)
        MDN_CONV_CASE(4)
    }
#undef MDN_CONV_CASE
    return cudaErrorInvalidValue;
}

template <ConvKind K, typename T>
cudaError_t conv_dispatch(const ConvProblem &p, cudaStream_t st) {
    // packets of four channels (or two) where every row of every array starts
    // on a packet's boundary, single elements otherwise
    const int V = packet_width(4, sizeof(T), [&](int v, int bytes) {
        bool ok = p.D % v == 0 && rows_aligned(p.x, p.ld_x, sizeof(T), bytes) &&
                  rows_aligned(p.w, 4, 4, v == 4 ? 16 : 4);
        if (K == ConvKind::kBwd) ok = ok && rows_aligned(p.dy, p.ld_dy, sizeof(T), bytes);
        const void *dense[] = {p.state0, p.dstate_T, p.y, p.state_T, p.dx, p.dstate0};
        for (const void *ptr : dense) ok = ok && rows_aligned(ptr, p.D, sizeof(T), bytes);
        return ok;
    });
    if (V == 4) return conv_width<K, T, 4>(p, st);
    if constexpr (sizeof(T) == 2)
        if (V == 2) return conv_width<K, T, 2>(p, st);
    return conv_width<K, T, 1>(p, st);
}

}  // namespace

size_t conv_bwd_workspace(int T_total, int D, int width, mdn_dtype dtype) {
    size_t most = 0;
    for (int v : {4, 2, 1}) {
        const long rows = conv_bwd_rows(conv_bwd_grid(D, v, T_total));
        const size_t need = (size_t)rows * (width + 1) * D * sizeof(float);
        most = need > most ? need : most;
    }
    return round256(most);
}

cudaError_t launch_conv_fwd(const ConvProblem &p, cudaStream_t st) {
    if (p.T_total == 0) {
        const long n = (long)p.n_seq * (p.width - 1) * p.D;
        return p.dtype == MDN_BF16 ? copy_states<__nv_bfloat16>(p.state0, p.state_T, n, st)
                                   : copy_states<float>(p.state0, p.state_T, n, st);
    }
    return p.dtype == MDN_BF16 ? conv_dispatch<ConvKind::kFwd, __nv_bfloat16>(p, st)
                               : conv_dispatch<ConvKind::kFwd, float>(p, st);
}
cudaError_t launch_conv_bwd(const ConvProblem &p, cudaStream_t st) {
    if (p.T_total == 0) {
        cudaError_t err = cudaMemsetAsync(p.dw, 0, sizeof(float) * (size_t)p.D * p.width, st);
        if (err == cudaSuccess && p.dbias) err = cudaMemsetAsync(p.dbias, 0, sizeof(float) * (size_t)p.D, st);
        if (err != cudaSuccess) return err;
        const long n = (long)p.n_seq * (p.width - 1) * p.D;
        return p.dtype == MDN_BF16 ? copy_states<__nv_bfloat16>(p.dstate_T, p.dstate0, n, st)
                                   : copy_states<float>(p.dstate_T, p.dstate0, n, st);
    }
    return p.dtype == MDN_BF16 ? conv_dispatch<ConvKind::kBwd, __nv_bfloat16>(p, st)
                               : conv_dispatch<ConvKind::kBwd, float>(p, st);
}
cudaError_t launch_conv_step(const ConvProblem &p, cudaStream_t st) {
    if (p.n_seq == 0) return cudaSuccess;
    return p.dtype == MDN_BF16 ? conv_dispatch<ConvKind::kStep, __nv_bfloat16>(p, st)
                               : conv_dispatch<ConvKind::kStep, float>(p, st);
}

}  // namespace mdn
