// The norm after a block, its gate, the scaled residual sum and the norm
// before the next block, in one pass over the rows; and the gradient.
//
//   r1 = (mean(y^2) + eps)^(-1/2);  n = y r1 w_post;  b = n act(gate)
//   X  = x + scale b;  r2 = (mean(X^2) + eps)^(-1/2);  h = X r2 w_pre
//
//   dX     = dx_out + r2 (w_pre dh - X r2^2 mean(dh w_pre X));   dx = dX
//   db     = dX scale;  dgate = db n act'(gate);  dn = db act(gate)
//   dy     = r1 (w_post dn - y r1^2 mean(dn w_post y))
//   dw_pre = sum dh X r2;  dscale = sum dX b;  dw_post = sum dn y r1
//
// Memory bound: a row's elements stay in registers (of the widest rows in shared
// memory or the caches) between its reductions, so every array is read from or
// written to memory once.  Blocks take rows in turn, and every thread copies
// its packets of the rows ahead into shared memory that only it reads, so that
// the reductions of one row do not hold up the loads of the next.  The gradient
// keeps the columns' parameter sums in registers.
//
// Measured, bf16: 32768 rows of 2048, no gate, 82 us (537 MB, 6.5 TB/s, 96 % of
// a copy's rate); 16384 rows of 2048 with a gate 51 us (336 MB, 6.5 TB/s), its
// gradient 122 us (537 MB, 4.4 TB/s) and 6 us for the parameters' partial rows.
// The gradient is bound by issue: 64 % of the slots, with 16 warps an SM at
// 128 registers a thread.  64 rows of 1001 in fp32: 3.3 us, the latency of a
// row's loads and its two sums.
#include <algorithm>

#include "mdn_ssm.cuh"

namespace mdn {
namespace {

// Sum over the threads of a row: `tpr` threads (a power of two, 32 or more),
// blockDim.x / tpr rows a block.  Every thread gets the sum.  Calls alternate
// between the two halves of `red` (`turn`), so that one barrier a call is
// enough: a half is written again only after the barrier of the call between.
__device__ __forceinline__ float row_sum(float v, int tpr, float *red, int &turn) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (tpr == 32) return v;
    float *r = red + turn;
    turn ^= 32;
    if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
    __syncthreads();
    // the row's warps: lane j takes warp j's sum, of tpr / 32 that repeat
    const int wpr = tpr >> 5;
    v = r[((threadIdx.x >> 5) & ~(wpr - 1)) + (threadIdx.x & (wpr - 1))];
    for (int o = wpr >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// a <- act(g), d <- act'(g)
template <int V>
__device__ __forceinline__ void gate_acts(const float *g, int act, float *a) {
    sigmoids<V>(g, a);
    if (act == MDN_GATE_SILU)
#pragma unroll
        for (int v = 0; v < V; ++v) a[v] *= g[v];
}
template <int V>
__device__ __forceinline__ void gate_acts_d(const float *g, int act, float *a, float *d) {
    float s[V];
    sigmoids<V>(g, s);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const bool silu = act == MDN_GATE_SILU;
        a[v] = silu ? g[v] * s[v] : s[v];
        d[v] = silu ? s[v] * fmaf(g[v], 1.f - s[v], 1.f) : s[v] * (1.f - s[v]);
    }
}

// V weights from column c on, in packets of 16 bytes where V has them; `none`
// where there are no weights or no such column.
template <int V>
__device__ __forceinline__ void load_cols(const float *w, int c, int D, float none, float *f) {
    constexpr int P = V < 4 ? V : 4;
    if (w && c < D) {
#pragma unroll
        for (int i = 0; i < V; i += P) unpack<float, P>(load_packet<float, P>(w + c + i), f + i);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = none;
    }
}

// Rows ahead by the bytes of a thread's packets of one array, so that 512
// threads of the forward and `threads` of the gradient fit their copies (its
// five arrays' in 160 KB); negative: the rows are read where they are used.
// So are packets that a copy would hold in registers (`held`) where a thread
// has many.
__host__ __device__ constexpr int fwd_ahead(int bytes, bool held) {
    return held ? -1 : bytes <= 32 ? 2 : bytes <= 64 ? 1 : 0;
}
__host__ __device__ constexpr int bwd_ahead(int bytes, int threads, bool held) {
    if (held) return -1;
    return bytes * threads <= 16 * 1024 ? 1 : bytes * threads <= 32 * 1024 ? 0 : -1;
}

// (us in place and copied ahead, bf16: 2048 rows of 12001 240 and 438, but 4096
// rows of 6001 320 and 180.)
__host__ __device__ constexpr bool fwd_held(int NI, int V, int el) { return V * el < 4 && NI >= 32; }

// This thread's packets of one array: of its rows in turn, copied AHEAD rows
// early into AHEAD + 1 slots of shared memory that only it reads.
template <typename T, int V, int NI, int AHEAD>
struct RowStream {
    const T *next;                    // the next row to copy (AHEAD < 0: to read)
    long step;                        // elements to the row after
    Packet<T, V> *ring;               // [AHEAD + 1][NI][blockDim.x], this thread's
    int D, tpr, tid;
    Copies<T, V, AHEAD < 0 ? 1 : NI> copies;

    __device__ __forceinline__ RowStream(const void *src, long ld, long row, long rows_step, unsigned char *smem,
                                         int which, int D_, int tpr_, int tid_)
        : next(static_cast<const T *>(src) + row * ld + tid_ * V), step(rows_step * ld),
          ring(reinterpret_cast<Packet<T, V> *>(smem) + which * (AHEAD + 1) * NI * blockDim.x + threadIdx.x),
          D(D_), tpr(tpr_), tid(tid_) {
        copies.clear();
    }
    __device__ __forceinline__ bool in(int i) const { return (i * tpr + tid) * V < D; }
    // Copies the next row into `slot` (not past the last row).  A copy that goes
    // through registers reaches shared memory with the next one.
    __device__ __forceinline__ void issue(int slot, bool live) {
        if constexpr (AHEAD >= 0) {
            copies.put();
            if (live) {
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    if (in(i)) copies.get(i, &ring[(slot * NI + i) * blockDim.x], next + i * tpr * V);
            }
            if (AHEAD == 0) copies.put();
            next += step;
        }
    }
    // Packet i of the row in `slot` (zeros past the row's end).
    __device__ __forceinline__ void get(int slot, int i, bool live, float *f) const {
        if (live && in(i)) {
            if constexpr (AHEAD >= 0) unpack<T, V>(ring[(slot * NI + i) * blockDim.x], f);
            else unpack<T, V>(load_packet<T, V>(next + i * tpr * V), f);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) f[v] = 0.f;
        }
    }
    __device__ __forceinline__ void done() {
        if constexpr (AHEAD < 0) next += step;
    }
};

// One row at a time per group of tpr threads; the columns' weights stay in
// registers (w_post and scale meet as one factor).
template <typename T, int V, int NI, bool GATE>
__global__ void __launch_bounds__(512) norm_fwd_kernel(NormProblem p, int tpr) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float red[64];
    constexpr int AHEAD = fwd_ahead(NI * V * (int)sizeof(T), fwd_held(NI, V, (int)sizeof(T)));
    int turn = 0;
    const int tid = threadIdx.x & (tpr - 1), mine = threadIdx.x / tpr;
    const long rpb = blockDim.x / tpr, step = gridDim.x * rpb;
    long row = blockIdx.x * rpb + mine;
    using Stream = RowStream<T, V, NI, AHEAD>;
    Stream sy(p.y, p.ld_y, row, step, smem, 0, p.D, tpr, tid);
    Stream sx(p.x, p.ld_x, row, step, smem, 1, p.D, tpr, tid);
    Stream sg(p.gate, p.ld_gate, row, step, smem, 2, p.D, tpr, tid);
    auto issue = [&](int slot, bool live) {
        sy.issue(slot, live);
        sx.issue(slot, live);
        if (GATE) sg.issue(slot, live);
        commit_copies();
    };
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) issue(k, row + k * step < p.rows);
    float ws[NI][V], wpre[NI][V];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int c = (i * tpr + tid) * V;
        float sc[V];
        load_cols<V>(p.w_post, c, p.D, 1.f, ws[i]);
        load_cols<V>(p.scale, c, p.D, 1.f, sc);
        load_cols<V>(p.w_pre, c, p.D, 0.f, wpre[i]);
#pragma unroll
        for (int v = 0; v < V; ++v) ws[i][v] *= sc[v];
    }
    T *xo = static_cast<T *>(p.x_out) + row * p.D + tid * V;
    T *ho = static_cast<T *>(p.h) + row * p.D + tid * V;
    const long out_step = step * p.D;
    const float inv_d = 1.f / (float)p.D;
    // every thread of a block makes the same number of rounds (the sums wait
    // for the whole block)
    int get = 0, put = AHEAD < 0 ? 0 : AHEAD;
    for (long base = blockIdx.x * rpb; base < p.rows; base += step) {
        const bool live = row < p.rows;
        issue(put, row + AHEAD * step < p.rows);
        wait_copies<(AHEAD < 0 ? 0 : AHEAD)>();
        float y[NI][V], x[NI][V];
        float r1 = 1.f, r2 = 1.f, ss = 0.f;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            sy.get(get, i, live, y[i]);
#pragma unroll
            for (int v = 0; v < V; ++v) ss = fmaf(y[i][v], y[i][v], ss);
        }
        if (p.w_post) r1 = rsqrtf(fmaf(row_sum(ss, tpr, red, turn), inv_d, p.eps));
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            float g[V], act[V];
            sx.get(get, i, live, x[i]);
            if (GATE) {
                sg.get(get, i, live, g);
                gate_acts<V>(g, p.gate_act, act);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float b = y[i][v] * r1;
                if (GATE) b *= act[v];
                x[i][v] = fmaf(b, ws[i][v], x[i][v]);
                ss = fmaf(x[i][v], x[i][v], ss);
            }
            if (live && sy.in(i)) store_packet<T, V>(xo + i * tpr * V, pack<T, V>(x[i]));
        }
        if (p.w_pre) {
            r2 = rsqrtf(fmaf(row_sum(ss, tpr, red, turn), inv_d, p.eps));
#pragma unroll
            for (int i = 0; i < NI; ++i) {
#pragma unroll
                for (int v = 0; v < V; ++v) x[i][v] *= r2 * wpre[i][v];
                if (live && sy.in(i)) store_packet<T, V>(ho + i * tpr * V, pack<T, V>(x[i]));
            }
        }
        if (p.stats && live && tid == 0)
            *reinterpret_cast<float2 *>(p.stats + 2 * row) = make_float2(r1, r2);
        row += step;
        xo += out_step;
        ho += out_step;
        get = AHEAD <= 0 || get == AHEAD ? 0 : get + 1;
        put = AHEAD <= 0 || put == AHEAD ? 0 : put + 1;
        sy.done(); sx.done(); sg.done();
    }
    wait_copies<0>();
}

// Values of a row that a thread of the gradient has at most.
constexpr int kBwdValues = 16;

// A thread keeps its row's elements in registers, but not for rows that give
// it kBwdValues (or half as many single two-byte ones): it reads those again
// for each of the steps, and the weights with them, since seven arrays, three
// weights and three sums of 16 values do not fit 128 registers.  In us with
// both, 67 M bf16 values: rows of 8192 299 and 488, with a gate 405 and 571;
// 33 M values, rows of 16384 248 and 417; 25 M in rows of 3001 530 and 694.
__host__ __device__ constexpr bool bwd_lean(int NI, int V, int el) {
    return NI * V == kBwdValues || (V * el < 4 && 2 * NI * V == kBwdValues);
}

template <typename T, int V, int NI, bool GATE, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_bwd_kernel(NormProblem p, int tpr) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float red[64];
    constexpr bool LEAN = bwd_lean(NI, V, (int)sizeof(T));
    constexpr int AHEAD = bwd_ahead(NI * V * (int)sizeof(T), MAXT, LEAN && V * sizeof(T) < 4);
    int turn = 0;
    const int tid = threadIdx.x & (tpr - 1), mine = threadIdx.x / tpr;
    const long rpb = blockDim.x / tpr, step = gridDim.x * rpb;
    const long first = blockIdx.x * rpb + mine;
    long row = first;
    using Stream = RowStream<T, V, NI, AHEAD>;
    Stream sy(p.y, p.ld_y, row, step, smem, 0, p.D, tpr, tid);
    Stream sx(p.x, p.ld_x, row, step, smem, 1, p.D, tpr, tid);
    Stream sd(p.dx_out, p.ld_dx_out, row, step, smem, 2, p.D, tpr, tid);
    Stream sh(p.dh, p.ld_dh, row, step, smem, 3, p.D, tpr, tid);
    Stream sg(p.gate, p.ld_gate, row, step, smem, 4, p.D, tpr, tid);
    const bool pre = p.w_pre != nullptr;
    auto issue = [&](int slot, bool live) {
        sy.issue(slot, live);
        sx.issue(slot, live);
        sd.issue(slot, live);
        sh.issue(slot, live && pre);
        if (GATE) sg.issue(slot, live);
        commit_copies();
    };
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) issue(k, row + k * step < p.rows);
    auto load_weights = [&](int i, float *post, float *scale, float *before) {
        const int c = (i * tpr + tid) * V;
        load_cols<V>(p.w_post, c, p.D, 1.f, post);
        load_cols<V>(p.scale, c, p.D, 1.f, scale);
        load_cols<V>(p.w_pre, c, p.D, 0.f, before);
    };
    float wpost[LEAN ? 1 : NI][V], wpre[LEAN ? 1 : NI][V], sc[LEAN ? 1 : NI][V];
    float a_post[NI][V], a_pre[NI][V], a_scale[NI][V];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        if (!LEAN) load_weights(i, wpost[LEAN ? 0 : i], sc[LEAN ? 0 : i], wpre[LEAN ? 0 : i]);
#pragma unroll
        for (int v = 0; v < V; ++v) a_post[i][v] = a_pre[i][v] = a_scale[i][v] = 0.f;
    }
    long at = row * p.D + tid * V;
    const float inv_d = 1.f / (float)p.D;
    int get = 0, put = AHEAD < 0 ? 0 : AHEAD;
    for (long base = blockIdx.x * rpb; base < p.rows; base += step) {
        const bool live = row < p.rows;
        const float r1 = live ? p.stats[2 * row] : 0.f;
        const float r2 = live ? p.stats[2 * row + 1] : 0.f;
        issue(put, row + AHEAD * step < p.rows);
        wait_copies<(AHEAD < 0 ? 0 : AHEAD)>();
        // packet i: its elements, X again and dh w_pre
        constexpr int K = LEAN ? 1 : NI;
        float y[K][V], X[K][V], act[K][V], dact[K][V], dh[K][V], dX[NI][V];
        auto read = [&](int i, float *dx, bool sums) {
            const int k = LEAN ? 0 : i;
            if (LEAN) load_weights(i, wpost[k], sc[k], wpre[k]);
            sy.get(get, i, live, y[k]);
            sx.get(get, i, live, X[k]);
            sd.get(get, i, live, dx);
            sh.get(get, i, live && pre, dh[k]);
            if (GATE) {
                float g[V];
                sg.get(get, i, live, g);
                gate_acts_d<V>(g, p.gate_act, act[k], dact[k]);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float b = y[k][v] * (r1 * wpost[k][v]);
                if (GATE) b *= act[k][v];
                X[k][v] = fmaf(sc[k][v], b, X[k][v]);
                if (sums) a_pre[i][v] = fmaf(dh[k][v] * r2, X[k][v], a_pre[i][v]);
                dh[k][v] *= wpre[k][v];
            }
        };
        // mean(dh w_pre X)
        float s2 = 0.f;
        if (!LEAN || pre) {
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int k = LEAN ? 0 : i;
                read(i, dX[i], true);
#pragma unroll
                for (int v = 0; v < V; ++v) s2 = fmaf(dh[k][v], X[k][v], s2);
            }
        }
        const float m2 = pre ? row_sum(s2, tpr, red, turn) * inv_d * r2 * r2 : 0.f;
        // through the residual sum, the scale and the gate; mean(dn w_post y)
        float s1 = 0.f;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const bool here = live && sy.in(i);
            const long o = at + i * tpr * V;
            const int k = LEAN ? 0 : i;
            if (LEAN) read(i, dX[i], false);
            if (pre)
#pragma unroll
                for (int v = 0; v < V; ++v) dX[i][v] = fmaf(r2, fmaf(-m2, X[k][v], dh[k][v]), dX[i][v]);
            if (here) store_packet<T, V>(static_cast<T *>(p.dx) + o, pack<T, V>(dX[i]));
            float dg[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float n = y[k][v] * (r1 * wpost[k][v]);
                const float ga = GATE ? act[k][v] : 1.f;
                a_scale[i][v] = fmaf(dX[i][v], n * ga, a_scale[i][v]);
                const float db = dX[i][v] * sc[k][v];
                if (GATE) dg[v] = db * n * dact[k][v];
                const float dn = db * ga;
                a_post[i][v] = fmaf(dn * r1, y[k][v], a_post[i][v]);
                dX[i][v] = dn * wpost[k][v];
                s1 = fmaf(dX[i][v], y[k][v], s1);
            }
            if (GATE && here) store_packet<T, V>(static_cast<T *>(p.dgate) + o, pack<T, V>(dg));
        }
        // without w_post r1 is 1 and y passes on as it is
        const float m = p.w_post ? row_sum(s1, tpr, red, turn) * inv_d * r1 * r1 : 0.f;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int k = LEAN ? 0 : i;
            if (LEAN) sy.get(get, i, live, y[k]);
#pragma unroll
            for (int v = 0; v < V; ++v) dX[i][v] = r1 * fmaf(-m, y[k][v], dX[i][v]);
            if (live && sy.in(i))
                store_packet<T, V>(static_cast<T *>(p.dy) + at + i * tpr * V, pack<T, V>(dX[i]));
        }
        row += step;
        at += step * p.D;
        get = AHEAD <= 0 || get == AHEAD ? 0 : get + 1;
        put = AHEAD <= 0 || put == AHEAD ? 0 : put + 1;
        sy.done(); sx.done(); sd.done(); sh.done(); sg.done();
    }
    wait_copies<0>();
    float *part = p.partial + first * 3L * p.D + tid * V;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        if (!sy.in(i)) continue;
        constexpr int P = V < 4 ? V : 4;
#pragma unroll
        for (int v = 0; v < V; v += P) {
            float *o = part + i * tpr * V + v;
            store_packet<float, P>(o, pack<float, P>(a_post[i] + v));
            store_packet<float, P>(o + p.D, pack<float, P>(a_pre[i] + v));
            store_packet<float, P>(o + 2L * p.D, pack<float, P>(a_scale[i] + v));
        }
    }
}

// Sums the partial rows in order: 8 threads per column.
__global__ void __launch_bounds__(256)
norm_reduce_kernel(const float *partial, int rows, int D, float *dw_post, float *dw_pre,
                   float *dscale) {
    __shared__ float s[8][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const long cols = 3L * D;
    const long i = (long)blockIdx.x * 32 + tx;
    float a = 0.f;
    if (i < cols)
        for (int r = ty; r < rows; r += 8) a += partial[r * cols + i];
    s[ty][tx] = a;
    __syncthreads();
    if (ty != 0 || i >= cols) return;
#pragma unroll
    for (int k = 1; k < 8; ++k) a += s[k][tx];
    const int which = (int)(i / D);
    const int c = (int)(i - (long)which * D);
    float *out = which == 0 ? dw_post : which == 1 ? dw_pre : dscale;
    if (out) out[c] = a;
}

struct NormShape {
    int tpr, ni, threads;
};
// Threads per row and packets per thread.  A row takes up to 128 threads
// first, then `soft` values a thread, then up to `most` threads, then `hard`
// values, then 1024 threads.
NormShape norm_shape(int D, int V, int soft, int most, int hard) {
    const int packets = (D + V - 1) / V;
    NormShape s;
    s.tpr = 32;
    s.ni = 1;
    while (s.tpr * s.ni < packets) {
        if (s.tpr < 128) s.tpr *= 2;
        else if (s.ni * V < soft) s.ni *= 2;
        else if (s.tpr < most) s.tpr *= 2;
        else if (s.ni * V < hard) s.ni *= 2;
        else s.tpr *= 2;
    }
    s.threads = s.tpr < 128 ? 128 : s.tpr;
    return s;
}
// The forward holds two arrays of a row and their weights: 32 values and 512
// threads reach D = 16384.  Few rows (at most one for each SM) take more
// threads and fewer values: their time is the latency of one row.  In us with
// the one shape and the other, bf16: 152 rows of 2048 3.1 and 3.3, of 4096 3.7
// and 3.8; but 303 rows of 4096 5.1 and 4.6, 1000 rows 10.3 and 9.1.
NormShape norm_fwd_shape(int rows, int D, int V) {
    return rows <= 152 ? norm_shape(D, V, V, 512, 32) : norm_shape(D, V, V < 4 ? 4 * V : 2 * V, 512, 32);
}
// The gradient holds seven arrays, weights and sums: 16 values and 512
// threads, and 1024 above D = 8192 (8192 rows of 8192, no gate: 299 us; with
// 8 values and 1024 threads, in registers, 582 us).
NormShape norm_bwd_shape(int D, int V) { return norm_shape(D, V, V < 4 ? 4 * V : 8, 512, kBwdValues); }
// Blocks that share the rows: as many threads on each of 152 SMs as their
// registers allow, where there are rows for them.
int norm_blocks(int rows, const NormShape &s, int threads) {
    const long rpb = s.threads / s.tpr, most = (rows + rpb - 1) / rpb;
    return (int)std::min(most, 152L * std::max(1, threads / s.threads));
}
// (16384 rows of 2048 bf16, no gate: 41 us with 640 threads an SM, 43 with 512;
// with a gate, or 32 values a thread, no more than 512 fit.)
int fwd_threads(const NormShape &s, int V, bool gate) { return s.ni * V <= 16 && !gate ? 640 : 512; }
constexpr int kBwdThreads = 512;

// Launches a kernel of at most MAXT threads that keeps `each` bytes a thread.
template <auto Kernel, int MAXT>
cudaError_t norm_run(const NormProblem &p, const NormShape &s, int blocks, int each, cudaStream_t st) {
    const cudaError_t err = allow_shared<Kernel>(each * MAXT);
    if (err != cudaSuccess) return err;
    Kernel<<<blocks, s.threads, each * s.threads, st>>>(p, s.tpr);
    return cudaGetLastError();
}

template <bool BWD, typename T, int V, int NI>
cudaError_t norm_launch(const NormProblem &p, const NormShape &s, cudaStream_t st) {
    const int blocks = norm_blocks(p.rows, s, BWD ? kBwdThreads : fwd_threads(s, V, p.gate != nullptr));
    constexpr int each = NI * V * (int)sizeof(T);
    const bool gate = p.gate != nullptr;
    if constexpr (BWD) {
        constexpr bool held = bwd_lean(NI, V, (int)sizeof(T)) && V * sizeof(T) < 4;
        cudaError_t err = cudaErrorInvalidValue;
        if (s.threads <= 512) {
            constexpr int bytes = 5 * (bwd_ahead(each, 512, held) + 1) * each;
            err = gate ? norm_run<norm_bwd_kernel<T, V, NI, true, 512>, 512>(p, s, blocks, bytes, st)
                       : norm_run<norm_bwd_kernel<T, V, NI, false, 512>, 512>(p, s, blocks, bytes, st);
        }
        if constexpr (NI * V == kBwdValues)
            if (s.threads > 512) {
                constexpr int bytes = 5 * (bwd_ahead(each, 1024, held) + 1) * each;
                err = gate ? norm_run<norm_bwd_kernel<T, V, NI, true, 1024>, 1024>(p, s, blocks, bytes, st)
                           : norm_run<norm_bwd_kernel<T, V, NI, false, 1024>, 1024>(p, s, blocks, bytes, st);
            }
        if (err != cudaSuccess) return err;
        norm_reduce_kernel<<<(3 * p.D + 31) / 32, 256, 0, st>>>(
            p.partial, blocks * (s.threads / s.tpr), p.D, p.dw_post, p.dw_pre, p.dscale);
        return cudaGetLastError();
    } else {
        constexpr int bytes = 3 * (fwd_ahead(each, fwd_held(NI, V, (int)sizeof(T))) + 1) * each;
        return gate ? norm_run<norm_fwd_kernel<T, V, NI, true>, 512>(p, s, blocks, bytes, st)
                    : norm_run<norm_fwd_kernel<T, V, NI, false>, 512>(p, s, blocks, bytes, st);
    }
}

template <bool BWD, typename T, int V>
cudaError_t norm_items(const NormProblem &p, cudaStream_t st) {
    const NormShape s = BWD ? norm_bwd_shape(p.D, V) : norm_fwd_shape(p.rows, p.D, V);
    constexpr int kMost = (BWD ? kBwdValues : 32) / V;      // D = 16384
    if (s.ni == 1) return norm_launch<BWD, T, V, 1>(p, s, st);
    if (s.ni == 2) return norm_launch<BWD, T, V, 2>(p, s, st);
    if constexpr (kMost >= 4)
        if (s.ni == 4) return norm_launch<BWD, T, V, 4>(p, s, st);
    if constexpr (kMost >= 8)
        if (s.ni == 8) return norm_launch<BWD, T, V, 8>(p, s, st);
    if constexpr (kMost >= 16)
        if (s.ni == 16) return norm_launch<BWD, T, V, 16>(p, s, st);
    if constexpr (kMost >= 32)
        if (s.ni == 32) return norm_launch<BWD, T, V, 32>(p, s, st);
    return cudaErrorInvalidValue;
}

template <bool BWD, typename T>
cudaError_t norm_dispatch(const NormProblem &p, cudaStream_t st) {
    constexpr int MOST = 16 / (int)sizeof(T);
    const int V = packet_width(MOST, sizeof(T), [&](int v, int bytes) {
        bool ok = p.D % v == 0 && rows_aligned(p.y, p.ld_y, sizeof(T), bytes) &&
                  rows_aligned(p.x, p.ld_x, sizeof(T), bytes) &&
                  rows_aligned(p.gate, p.ld_gate, sizeof(T), bytes);
        if (BWD)
            ok = ok && rows_aligned(p.dx_out, p.ld_dx_out, sizeof(T), bytes) &&
                 rows_aligned(p.dh, p.ld_dh, sizeof(T), bytes);
        for (const float *w : {p.w_post, p.w_pre, p.scale}) ok = ok && rows_aligned(w, 0, 4, v >= 4 ? 16 : 4 * v);
        const void *dense[] = {p.x_out, p.h, p.dy, p.dx, p.dgate};
        for (const void *ptr : dense) ok = ok && rows_aligned(ptr, p.D, sizeof(T), bytes);
        return ok;
    });
    if (V == MOST) return norm_items<BWD, T, MOST>(p, st);
    if constexpr (sizeof(T) == 2)
        if (V == 2) return norm_items<BWD, T, 2>(p, st);
    return norm_items<BWD, T, 1>(p, st);
}

}  // namespace

size_t norm_bwd_workspace(int rows, int D, mdn_dtype dtype) {
    size_t most = 0;
    for (int v : {dtype == MDN_BF16 ? 8 : 4, 2, 1}) {
        const NormShape s = norm_bwd_shape(D, v);
        const size_t need =
            (size_t)norm_blocks(rows, s, kBwdThreads) * (s.threads / s.tpr) * 3 * D * sizeof(float);
        most = need > most ? need : most;
    }
    return round256(most);
}

cudaError_t launch_norm_fwd(const NormProblem &p, cudaStream_t st) {
    if (p.rows == 0) return cudaSuccess;
    return p.dtype == MDN_BF16 ? norm_dispatch<false, __nv_bfloat16>(p, st)
                               : norm_dispatch<false, float>(p, st);
}
cudaError_t launch_norm_bwd(const NormProblem &p, cudaStream_t st) {
    if (p.rows == 0) {
        float *out[] = {p.dw_post, p.dw_pre, p.dscale};
        for (float *o : out)
            if (o) {
                cudaError_t err = cudaMemsetAsync(o, 0, sizeof(float) * (size_t)p.D, st);
                if (err != cudaSuccess) return err;
            }
        return cudaSuccess;
    }
    return p.dtype == MDN_BF16 ? norm_dispatch<true, __nv_bfloat16>(p, st)
                               : norm_dispatch<true, float>(p, st);
}

}  // namespace mdn
