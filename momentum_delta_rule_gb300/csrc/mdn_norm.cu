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
// Memory bound: a row's elements stay in registers between its reductions, so
// every array is read or written once.  The gradient's blocks each take many
// rows and keep the columns' parameter sums in registers.
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
    float *r = red + turn * 32;
    turn ^= 1;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) r[warp] = v;
    __syncthreads();
    const int wpr = tpr >> 5, first = warp / wpr * wpr;
    v = 0.f;
    for (int w = 0; w < wpr; ++w) v += r[first + w];
    return v;
}

__device__ __forceinline__ float gate_act(float g, int act) {
    const float s = sigmoid_f(g);
    return act == MDN_GATE_SILU ? g * s : s;
}
__device__ __forceinline__ void gate_act_d(float g, int act, float &a, float &d) {
    const float s = sigmoid_f(g);
    if (act == MDN_GATE_SILU) {
        a = g * s;
        d = s * fmaf(g, 1.f - s, 1.f);
    } else {
        a = s;
        d = s * (1.f - s);
    }
}

template <typename T, int V, int NI>
__global__ void __launch_bounds__(512) norm_fwd_kernel(NormProblem p, int tpr) {
    __shared__ float red[64];
    int turn = 0;
    const int tid = threadIdx.x & (tpr - 1);
    const long row = (long)blockIdx.x * (blockDim.x / tpr) + threadIdx.x / tpr;
    const bool live = row < p.rows;
    float y[NI][V], x[NI][V], g[NI][V];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int c = (i * tpr + tid) * V;
        if (live && c < p.D) {
            const auto py = load_packet<T, V>(static_cast<const T *>(p.y) + row * p.ld_y + c);
            const auto px = load_packet<T, V>(static_cast<const T *>(p.x) + row * p.ld_x + c);
            if (p.gate)
                unpack<T, V>(load_packet<T, V>(static_cast<const T *>(p.gate) + row * p.ld_gate + c), g[i]);
            unpack<T, V>(py, y[i]);
            unpack<T, V>(px, x[i]);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) y[i][v] = x[i][v] = g[i][v] = 0.f;
        }
    }
    const float inv_d = 1.f / (float)p.D;
    float r1 = 1.f, r2 = 1.f;
    if (p.w_post) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) ss = fmaf(y[i][v], y[i][v], ss);
        r1 = rsqrtf(fmaf(row_sum(ss, tpr, red, turn), inv_d, p.eps));
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int c = (i * tpr + tid) * V;
        if (c >= p.D) continue;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float b = y[i][v];
            if (p.w_post) b *= r1 * p.w_post[c + v];
            if (p.gate) b *= gate_act(g[i][v], p.gate_act);
            const float X = p.scale ? fmaf(p.scale[c + v], b, x[i][v]) : x[i][v] + b;
            x[i][v] = X;
            ss = fmaf(X, X, ss);
        }
        if (live)
            store_packet<T, V>(static_cast<T *>(p.x_out) + row * p.D + c, pack<T, V>(x[i]));
    }
    if (p.w_pre) {
        r2 = rsqrtf(fmaf(row_sum(ss, tpr, red, turn), inv_d, p.eps));
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int c = (i * tpr + tid) * V;
            if (!live || c >= p.D) continue;
#pragma unroll
            for (int v = 0; v < V; ++v) x[i][v] *= r2 * p.w_pre[c + v];
            store_packet<T, V>(static_cast<T *>(p.h) + row * p.D + c, pack<T, V>(x[i]));
        }
    }
    if (p.stats && live && tid == 0)
        *reinterpret_cast<float2 *>(p.stats + 2 * row) = make_float2(r1, r2);
}

template <typename T, int V, int NI, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_bwd_kernel(NormProblem p, int tpr) {
    __shared__ float red[64];
    int turn = 0;
    const int tid = threadIdx.x & (tpr - 1);
    const int rpb = blockDim.x / tpr;
    const long first = (long)blockIdx.x * rpb + threadIdx.x / tpr;
    const float inv_d = 1.f / (float)p.D;
    float a_post[NI][V], a_pre[NI][V], a_scale[NI][V];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) a_post[i][v] = a_pre[i][v] = a_scale[i][v] = 0.f;
    // every thread of a block makes the same number of rounds (the sums below
    // wait for the whole block)
    for (long base = (long)blockIdx.x * rpb; base < p.rows; base += (long)gridDim.x * rpb) {
        const long row = base + threadIdx.x / tpr;
        const bool live = row < p.rows;
        const float r1 = live ? p.stats[2 * row] : 0.f;
        const float r2 = live ? p.stats[2 * row + 1] : 0.f;
        float y[NI][V], X[NI][V], g[NI][V], dX[NI][V], dh[NI][V];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int c = (i * tpr + tid) * V;
            if (live && c < p.D) {
                const auto py = load_packet<T, V>(static_cast<const T *>(p.y) + row * p.ld_y + c);
                const auto px = load_packet<T, V>(static_cast<const T *>(p.x) + row * p.ld_x + c);
                const auto pd =
                    load_packet<T, V>(static_cast<const T *>(p.dx_out) + row * p.ld_dx_out + c);
                if (p.gate)
                    unpack<T, V>(load_packet<T, V>(static_cast<const T *>(p.gate) + row * p.ld_gate + c), g[i]);
                if (p.w_pre)
                    unpack<T, V>(load_packet<T, V>(static_cast<const T *>(p.dh) + row * p.ld_dh + c), dh[i]);
                unpack<T, V>(py, y[i]);
                unpack<T, V>(px, X[i]);
                unpack<T, V>(pd, dX[i]);
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) y[i][v] = X[i][v] = g[i][v] = dX[i][v] = dh[i][v] = 0.f;
            }
        }
        // X again, and mean(dh w_pre X)
        float s2 = 0.f;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int c = (i * tpr + tid) * V;
            if (c >= p.D) continue;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float b = y[i][v];
                if (p.w_post) b *= r1 * p.w_post[c + v];
                if (p.gate) b *= gate_act(g[i][v], p.gate_act);
                X[i][v] = p.scale ? fmaf(p.scale[c + v], b, X[i][v]) : X[i][v] + b;
                if (p.w_pre) {
                    a_pre[i][v] = fmaf(dh[i][v] * r2, X[i][v], a_pre[i][v]);
                    dh[i][v] *= p.w_pre[c + v];
                    s2 = fmaf(dh[i][v], X[i][v], s2);
                }
            }
        }
        if (p.w_pre) {
            const float k = row_sum(s2, tpr, red, turn) * inv_d * r2 * r2;
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    dX[i][v] = fmaf(r2, fmaf(-k, X[i][v], dh[i][v]), dX[i][v]);
        }
        // through the residual sum, the scale and the gate; mean(dn w_post y)
        float s1 = 0.f;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int c = (i * tpr + tid) * V;
            if (c >= p.D) continue;
            float dg[V];
            if (live)
                store_packet<T, V>(static_cast<T *>(p.dx) + row * p.D + c, pack<T, V>(dX[i]));
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float n = p.w_post ? y[i][v] * r1 * p.w_post[c + v] : y[i][v];
                float act = 1.f, dact = 0.f;
                if (p.gate) gate_act_d(g[i][v], p.gate_act, act, dact);
                float db = dX[i][v];
                if (p.scale) {
                    a_scale[i][v] = fmaf(db, n * act, a_scale[i][v]);
                    db *= p.scale[c + v];
                }
                dg[v] = db * n * dact;
                float dn = db * act;
                if (p.w_post) {
                    a_post[i][v] = fmaf(dn * r1, y[i][v], a_post[i][v]);
                    dn *= p.w_post[c + v];
                    s1 = fmaf(dn, y[i][v], s1);
                }
                dX[i][v] = dn;
            }
            if (p.gate && live)
                store_packet<T, V>(static_cast<T *>(p.dgate) + row * p.D + c, pack<T, V>(dg));
        }
        const float k = p.w_post ? row_sum(s1, tpr, red, turn) * inv_d * r1 * r1 : 0.f;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int c = (i * tpr + tid) * V;
            if (!live || c >= p.D) continue;
            if (p.w_post) {
#pragma unroll
                for (int v = 0; v < V; ++v) dX[i][v] = r1 * fmaf(-k, y[i][v], dX[i][v]);
            }
            store_packet<T, V>(static_cast<T *>(p.dy) + row * p.D + c, pack<T, V>(dX[i]));
        }
    }
    float *part = p.partial + first * 3L * p.D;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int c = (i * tpr + tid) * V;
        if (c >= p.D) continue;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            part[c + v] = a_post[i][v];
            part[p.D + c + v] = a_pre[i][v];
            part[2L * p.D + c + v] = a_scale[i][v];
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
// first, then `soft` values a thread, then up to `most` threads, then more
// values.
NormShape norm_shape(int D, int V, int soft, int most) {
    const int packets = (D + V - 1) / V;
    NormShape s;
    s.tpr = 32;
    s.ni = 1;
    while (s.tpr * s.ni < packets) {
        if (s.tpr < 128) s.tpr *= 2;
        else if (s.ni * V < soft) s.ni *= 2;
        else if (s.tpr < most) s.tpr *= 2;
        else s.ni *= 2;
    }
    s.threads = s.tpr < 128 ? 128 : s.tpr;
    return s;
}
// The forward holds three arrays of a row, the gradient five and three sums.
NormShape norm_fwd_shape(int D, int V) { return norm_shape(D, V, 16, 512); }
NormShape norm_bwd_shape(int D, int V) { return norm_shape(D, V, 8, 1024); }
int norm_bwd_blocks(int rows, const NormShape &s) {
    const int rpb = s.threads / s.tpr;
    const long most = ((long)rows + rpb - 1) / rpb;
    const long want = 152L * (s.threads >= 512 ? 1 : 512 / s.threads);
    return (int)(most < want ? most : want);
}

template <bool BWD, typename T, int V, int NI>
cudaError_t norm_launch(const NormProblem &p, const NormShape &s, cudaStream_t st) {
    if constexpr (BWD) {
        const int blocks = norm_bwd_blocks(p.rows, s);
        if (s.threads <= 512)
            norm_bwd_kernel<T, V, NI, 512><<<blocks, s.threads, 0, st>>>(p, s.tpr);
        else
            norm_bwd_kernel<T, V, NI, 1024><<<blocks, s.threads, 0, st>>>(p, s.tpr);
        cudaError_t err = cudaGetLastError();
        if (err != cudaSuccess) return err;
        norm_reduce_kernel<<<(3 * p.D + 31) / 32, 256, 0, st>>>(
            p.partial, blocks * (s.threads / s.tpr), p.D, p.dw_post, p.dw_pre, p.dscale);
    } else {
        const int rpb = s.threads / s.tpr;
        norm_fwd_kernel<T, V, NI><<<(p.rows + rpb - 1) / rpb, s.threads, 0, st>>>(p, s.tpr);
    }
    return cudaGetLastError();
}

template <bool BWD, typename T, int V>
cudaError_t norm_items(const NormProblem &p, cudaStream_t st) {
    const NormShape s = BWD ? norm_bwd_shape(p.D, V) : norm_fwd_shape(p.D, V);
    constexpr int kMost = (BWD ? 16 : 32) / V;      // D = 16384
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
    constexpr int V = 16 / (int)sizeof(T);
    bool wide = p.D % V == 0 && rows_aligned(p.y, p.ld_y, sizeof(T), 16) &&
                rows_aligned(p.x, p.ld_x, sizeof(T), 16) &&
                rows_aligned(p.gate, p.ld_gate, sizeof(T), 16);
    if (BWD)
        wide = wide && rows_aligned(p.dx_out, p.ld_dx_out, sizeof(T), 16) &&
               rows_aligned(p.dh, p.ld_dh, sizeof(T), 16);
    const void *dense[] = {p.x_out, p.h, p.dy, p.dx, p.dgate};
    for (const void *ptr : dense) wide = wide && rows_aligned(ptr, p.D, sizeof(T), 16);
    return wide ? norm_items<BWD, T, V>(p, st) : norm_items<BWD, T, 1>(p, st);
}

}  // namespace

size_t norm_bwd_workspace(int rows, int D, mdn_dtype dtype) {
    size_t most = 0;
    for (int v : {dtype == MDN_BF16 ? 8 : 4, 1}) {
        const NormShape s = norm_bwd_shape(D, v);
        const size_t need =
            (size_t)norm_bwd_blocks(rows, s) * (s.threads / s.tpr) * 3 * D * sizeof(float);
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
