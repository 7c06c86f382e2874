// Short causal depthwise convolution along the tokens: forward, gradient and
// the single-token step.
//
//   pre_t = bias + sum_{j<W} w_j x_{t-(W-1-j)},   y_t = act(pre_t)
//   dpre  = dy act'(pre);  dx_q = sum_k w_{W-1-k} dpre_{q+k};
//   dw_j  = sum_t dpre_t x_{t-(W-1-j)};  dbias = sum_t dpre_t
//
// Tokens before a sequence's first are its W - 1 initial-state rows.  Memory
// bound (2 W + 4 flops against 2 elements moved): a thread owns a packet of
// channels and a run of consecutive tokens, keeps the last W - 1 inputs in
// registers, and issues several rows' loads before it uses the first.
#include "mdn_ssm.cuh"

namespace mdn {
namespace {

constexpr int kConvThreads = 256;

__device__ __forceinline__ float conv_act(float v, int act) {
    return act == MDN_CONV_SILU ? v * sigmoid_f(v) : v;
}
__device__ __forceinline__ float conv_dact(float v, int act) {
    if (act != MDN_CONV_SILU) return 1.f;
    const float s = sigmoid_f(v);
    return s * fmaf(v, 1.f - s, 1.f);
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
};

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

template <typename T, int V, int W>
__global__ void __launch_bounds__(kConvThreads) conv_fwd_kernel(ConvProblem p, ConvGrid g) {
    constexpr int UN = 8;          // rows loaded ahead
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
    float w[W][V], bias[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][v] = p.w[(long)(c + v) * W + j];
        bias[v] = p.bias ? p.bias[c + v] : 0.f;
    }
    SeqWalk q;
    q.find(p, t0);
    if (t0 == 0 && p.state_T)           // empty sequences before the first token
        for (int s = 0; s < q.s; ++s) copy_state<T, V, W>(p.state0, p.state_T, s, p.D, c);
    float win[W - 1][V];                // inputs t - (W - 1) .. t - 1
#pragma unroll
    for (int j = 0; j < W - 1; ++j) conv_input<T, V, W>(p, q, t0 - (W - 1) + j, c, win[j]);
    const T *xp = static_cast<const T *>(p.x) + c;
    T *yp = static_cast<T *>(p.y) + c;
    for (long tb = t0; tb < t1; tb += UN) {
        Packet<T, V> in[UN];
#pragma unroll
        for (int i = 0; i < UN; ++i)
            if (tb + i < t1) in[i] = load_packet<T, V>(xp + (tb + i) * p.ld_x);
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const long t = tb + i;
            if (t >= t1) break;
            if (t == q.end) {           // the next sequence with tokens
                do {
                    ++q.s;
                    q.start = q.end;
                    q.end = p.cu ? (long)p.cu[q.s + 1] : q.start + p.T;
                } while (q.end == q.start);
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
                    conv_input<T, V, W>(p, q, t - (W - 1) + j, c, win[j]);
            }
            float x[V], o[V];
            unpack<T, V>(in[i], x);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float a = fmaf(w[W - 1][v], x[v], bias[v]);
#pragma unroll
                for (int j = 0; j < W - 1; ++j) a = fmaf(w[j][v], win[j][v], a);
                o[v] = conv_act(a, p.act);
            }
            store_packet<T, V>(yp + t * p.D, pack<T, V>(o));
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) win[j][v] = j + 1 < W - 1 ? win[j + 1][v] : x[v];
            if (p.state_T && t == q.end - 1) {
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
                    store_packet<T, V>(static_cast<T *>(p.state_T) +
                                           ((long)q.s * (W - 1) + j) * p.D + c,
                                       pack<T, V>(win[j]));
                if (p.cu)               // empty sequences that follow
                    for (int s = q.s + 1; s < p.n_seq && p.cu[s + 1] == q.end; ++s)
                        copy_state<T, V, W>(p.state0, p.state_T, s, p.D, c);
            }
        }
    }
}

// dstate of a sequence without tokens is the adjoint of the state it hands on.
// dx of positions [a - (W - 1), ..] lags dpre by W - 1 tokens: the loop runs
// W - 1 tokens past the run (recomputing dpre there, the next run's first
// rows) and a run that holds a sequence's start also produces the W - 1
// positions before it, the initial state's gradient.
template <typename T, int V, int W>
__global__ void __launch_bounds__(kConvThreads) conv_bwd_kernel(ConvProblem p, ConvGrid g, long rows) {
    constexpr int UN = 4;
    const int lane = threadIdx.x & (g.cl - 1);
    const int ct = blockIdx.x % g.ctiles;
    const long row = (long)(blockIdx.x / g.ctiles) * (kConvThreads / g.cl) + threadIdx.x / g.cl;
    const int c = (ct * g.cl + lane) * V;
    const bool ok = !p.cu || cu_well_formed(p.cu, p.n_seq, p.T_total);
    if (row >= rows || c >= p.D) return;
    float w[W][V], bias[V], dw[W][V], db[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int j = 0; j < W; ++j) {
            w[j][v] = p.w[(long)(c + v) * W + j];
            dw[j][v] = 0.f;
        }
        bias[v] = p.bias ? p.bias[c + v] : 0.f;
        db[v] = 0.f;
    }
    if (!ok) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicExch(p.status, (int)MDN_ERR_INVALID_ARG);
        if (p.dstate0)
            for (long s = row; s < p.n_seq; s += rows)
                copy_state<T, V, W>(p.dstate_T, p.dstate0, (int)s, p.D, c);
    }
    const T *xp = static_cast<const T *>(p.x) + c;
    const T *dyp = static_cast<const T *>(p.dy) + c;
    for (long r = row; ok && r < g.nruns; r += rows) {
        const long t0 = r * g.run;
        const long t1 = min(t0 + g.run, (long)p.T_total);
        SeqWalk q;
        q.find(p, t0);
        if (t0 == 0 && p.dstate0)
            for (int s = 0; s < q.s; ++s) copy_state<T, V, W>(p.dstate_T, p.dstate0, s, p.D, c);
        long a = t0;                    // first token of the piece
        while (a < t1) {
            const long b = min(t1, q.end);
            const bool at_start = a == q.start;
            float win[W - 1][V], dp[W][V];    // dp[k]: dpre_{t-(W-1)+k}
#pragma unroll
            for (int j = 0; j < W - 1; ++j) conv_input<T, V, W>(p, q, a - (W - 1) + j, c, win[j]);
#pragma unroll
            for (int k = 0; k < W; ++k)
#pragma unroll
                for (int v = 0; v < V; ++v) dp[k][v] = 0.f;
            const long stop = b + W - 1;
            for (long tb = a; tb < stop; tb += UN) {
                Packet<T, V> in[UN], dn[UN];
#pragma unroll
                for (int i = 0; i < UN; ++i)
                    if (tb + i < stop && tb + i < q.end) {
                        in[i] = load_packet<T, V>(xp + (tb + i) * p.ld_x);
                        dn[i] = load_packet<T, V>(dyp + (tb + i) * p.ld_dy);
                    }
#pragma unroll
                for (int i = 0; i < UN; ++i) {
                    const long t = tb + i;
                    if (t >= stop) break;
#pragma unroll
                    for (int k = 0; k < W - 1; ++k)
#pragma unroll
                        for (int v = 0; v < V; ++v) dp[k][v] = dp[k + 1][v];
                    if (t < q.end) {
                        float x[V], d[V];
                        unpack<T, V>(in[i], x);
                        unpack<T, V>(dn[i], d);
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            float pre = fmaf(w[W - 1][v], x[v], bias[v]);
#pragma unroll
                            for (int j = 0; j < W - 1; ++j) pre = fmaf(w[j][v], win[j][v], pre);
                            const float e = d[v] * conv_dact(pre, p.act);
                            dp[W - 1][v] = e;
                            if (t < b) {
                                db[v] += e;
                                dw[W - 1][v] = fmaf(e, x[v], dw[W - 1][v]);
#pragma unroll
                                for (int j = 0; j < W - 1; ++j)
                                    dw[j][v] = fmaf(e, win[j][v], dw[j][v]);
                            }
                        }
#pragma unroll
                        for (int j = 0; j < W - 1; ++j)
#pragma unroll
                            for (int v = 0; v < V; ++v)
                                win[j][v] = j + 1 < W - 1 ? win[j + 1][v] : x[v];
                    } else {
#pragma unroll
                        for (int v = 0; v < V; ++v) dp[W - 1][v] = 0.f;
                    }
                    const long pos = t - (W - 1);
                    if (pos < a && !(at_start && p.dstate0)) continue;
                    float o[V];
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        o[v] = 0.f;
#pragma unroll
                        for (int k = 0; k < W; ++k) o[v] = fmaf(w[W - 1 - k][v], dp[k][v], o[v]);
                    }
                    if (p.dstate_T && pos >= q.end - (W - 1)) {
                        float e[V];
                        unpack<T, V>(load_packet<T, V>(
                                         static_cast<const T *>(p.dstate_T) +
                                         ((long)q.s * (W - 1) + (pos - (q.end - (W - 1)))) * p.D + c),
                                     e);
#pragma unroll
                        for (int v = 0; v < V; ++v) o[v] += e[v];
                    }
                    T *dst = pos >= a ? static_cast<T *>(p.dx) + pos * p.D + c
                                      : static_cast<T *>(p.dstate0) +
                                            ((long)q.s * (W - 1) + (W - 1) + (pos - q.start)) * p.D + c;
                    store_packet<T, V>(dst, pack<T, V>(o));
                }
            }
            if (b == q.end && p.dstate0 && p.cu)
                for (int s = q.s + 1; s < p.n_seq && p.cu[s + 1] == q.end; ++s)
                    copy_state<T, V, W>(p.dstate_T, p.dstate0, s, p.D, c);
            a = b;
            if (a < t1) q.find(p, a);
        }
    }
    float *part = p.partial + row * (long)(W + 1) * p.D + c;
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int j = 0; j < W; ++j) part[(long)j * p.D + v] = dw[j][v];
        part[(long)W * p.D + v] = db[v];
    }
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
    float o[V];
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = p.bias ? p.bias[c + v] : 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) {
        float x[V];
        unpack<T, V>(row[j], x);
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = fmaf(p.w[(long)(c + v) * W + j], x[v], o[v]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = conv_act(o[v], p.act);
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

ConvGrid conv_grid(int D, int V, int run, long T_total) {
    ConvGrid g;
    const int packets = (D + V - 1) / V;
    g.cl = 1;
    while (g.cl < packets && g.cl < kConvThreads) g.cl *= 2;
    g.ctiles = (packets + g.cl - 1) / g.cl;
    g.run = run;
    g.nruns = (T_total + run - 1) / run;
    return g;
}

// Rows of partial sums of the gradient: enough token runs in flight to fill
// the device (two blocks of 256 threads on each of 152 SMs), no more than the
// tokens need.
constexpr int kBwdRun = 32;
long conv_bwd_rows(const ConvGrid &g) {
    const int per = kConvThreads / g.cl;
    long blocks = (152L * 2 + g.ctiles - 1) / g.ctiles;
    if (blocks < 1) blocks = 1;
    long rows = blocks * per;
    const long most = (g.nruns + per - 1) / per * per;
    return rows < most ? rows : (most > 0 ? most : per);
}

template <typename T, int V, int W>
cudaError_t conv_fwd_t(const ConvProblem &p, cudaStream_t st) {
    const ConvGrid g = conv_grid(p.D, V, 16, p.T_total);
    const long blocks = (g.nruns + kConvThreads / g.cl - 1) / (kConvThreads / g.cl) * g.ctiles;
    if (blocks > 0x7fffffffL) return cudaErrorInvalidConfiguration;
    conv_fwd_kernel<T, V, W><<<(unsigned)blocks, kConvThreads, 0, st>>>(p, g);
    return cudaGetLastError();
}
template <typename T, int V, int W>
cudaError_t conv_bwd_t(const ConvProblem &p, cudaStream_t st) {
    const ConvGrid g = conv_grid(p.D, V, kBwdRun, p.T_total);
    const long rows = conv_bwd_rows(g);
    const long blocks = rows / (kConvThreads / g.cl) * g.ctiles;
    conv_bwd_kernel<T, V, W><<<(unsigned)blocks, kConvThreads, 0, st>>>(p, g, rows);
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
    // 16-byte packets where every row of every array starts on a 16-byte
    // boundary, single elements otherwise
    constexpr int V = 16 / (int)sizeof(T);
    bool wide = p.D % V == 0 && rows_aligned(p.x, p.ld_x, sizeof(T), 16);
    if (K == ConvKind::kBwd) wide = wide && rows_aligned(p.dy, p.ld_dy, sizeof(T), 16);
    const void *dense[] = {p.state0, p.dstate_T, p.y, p.state_T, p.dx, p.dstate0};
    for (const void *ptr : dense) wide = wide && rows_aligned(ptr, p.D, sizeof(T), 16);
    return wide ? conv_width<K, T, V>(p, st) : conv_width<K, T, 1>(p, st);
}

}  // namespace

size_t conv_bwd_workspace(int T_total, int D, int width, mdn_dtype dtype) {
    const int V = dtype == MDN_BF16 ? 8 : 4;
    size_t most = 0;
    for (int v : {V, 1}) {
        const long rows = conv_bwd_rows(conv_grid(D, v, kBwdRun, T_total));
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
