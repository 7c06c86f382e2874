// Selective state-space scan: forward over whole sequences, and the
// single-token step.
//
//   delta_t = softplus(dt_t + dt_bias);   a_t[n] = exp(delta_t A[n])
//   h_t[n]  = a_t[n] h_{t-1}[n] + delta_t u_t B_t[n]
//   y_t     = (sum_n C_t[n] h_t[n] + D_skip u_t) silu(z_t)
#include "mdn_scan.cuh"

namespace mdn {
namespace scan {
namespace {

// ------------------------------------------------------------------ layout

// One block: checks cu_seqlens, writes the slot offsets (chunks of kTokens
// from each sequence's own start) and the sequences longest first (for up to
// kMaxOrdered of them).  A malformed array sets the status word and leaves
// every sequence without slots.
constexpr int kMaxOrdered = 1024;

__global__ void __launch_bounds__(1024)
layout_kernel(const int32_t *cu, int n_seq, int T_total, int32_t *off, int32_t *order, int *status) {
    __shared__ int32_t part[32];
    if (!cu_well_formed(cu, n_seq, T_total)) {
        for (int s = threadIdx.x; s <= n_seq; s += blockDim.x) {
            off[s] = 0;
            if (s < n_seq) order[s] = s;
        }
        if (threadIdx.x == 0) atomicExch(status, (int)MDN_ERR_INVALID_ARG);
        return;
    }
    for (int s = threadIdx.x; s < n_seq; s += blockDim.x) {
        int rank = s;
        if (n_seq <= kMaxOrdered) {
            const int mine = cu[s + 1] - cu[s];
            rank = 0;
            for (int o = 0; o < n_seq; ++o) {
                const int len = cu[o + 1] - cu[o];
                rank += len > mine || (len == mine && o < s);
            }
        }
        order[rank] = s;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t carry = 0;
    for (int base = 0; base < n_seq; base += 1024) {
        const int s = base + threadIdx.x;
        int32_t mine = s < n_seq ? (cu[s + 1] - cu[s] + kTokens - 1) / kTokens : 0;
        int32_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) part[warp] = incl;
        __syncthreads();
        int32_t before = carry, total = 0;
        for (int w = 0; w < 32; ++w) {
            if (w < warp) before += part[w];
            total += part[w];
        }
        if (s < n_seq) off[s] = before + incl - mine;
        carry += total;
        __syncthreads();
    }
    if (threadIdx.x == 0) off[n_seq] = carry;
}

// ----------------------------------------------------------------- forward

template <typename S>
struct FwdSmem {
    float delta[kTokens][S::CB];      // delta, later unused
    float du[kTokens][S::CB];         // delta u
    float y[kTokens][S::CB];
    float B[kTokens][S::NP], C[kTokens][S::NP];
};

// One block takes CB channels of one group through one whole sequence, in
// stages of kTokens tokens: every thread turns its share of the stage's u and
// dt into fp32 delta and delta u in shared memory, the warps run the
// recurrence, and the threads that hold u finish y.
template <typename T, typename S, int V>
__global__ void __launch_bounds__(S::NT) scan_fwd_kernel(ScanProblem p, Layout l, int tiles) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    FwdSmem<S> &sm = *reinterpret_cast<FwdSmem<S> *>(smem_raw);
    constexpr int QC = S::CB / V;                    // column packets per token
    constexpr int PS = (kTokens * QC + S::NT - 1) / S::NT;
    const int Dg = p.D / p.G;
    const int gtiles = tiles / p.G;
    const int tile = blockIdx.x % tiles;
    const int seq = p.cu ? l.order[blockIdx.x / tiles] : blockIdx.x / tiles;
    const int g = tile / gtiles;
    const int c0 = (tile % gtiles) * S::CB;          // first channel, within the group
    const long d0 = (long)g * Dg + c0;
    long t0, slot0;
    int len;
    sequence(p, l, seq, t0, len, slot0);

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nl = lane % S::NL;
    const int cw = warp * S::WC + lane / S::NL * S::CPT;     // lane's first channel in the block
    float a2[S::CPT][kStates], h[S::CPT][kStates];
#pragma unroll
    for (int c = 0; c < S::CPT; ++c) {
        const bool live = c0 + cw + c < Dg && nl * kStates < p.N;
#pragma unroll
        for (int i = 0; i < kStates; ++i) a2[c][i] = h[c][i] = 0.f;
        if (live) {
            load_states(p.A, d0 + cw + c, nl * kStates, p.N, a2[c]);
            if (p.h0) load_states(p.h0 + (long)seq * p.D * p.N, d0 + cw + c, nl * kStates, p.N, h[c]);
        }
#pragma unroll
        for (int i = 0; i < kStates; ++i) a2[c][i] *= kLog2e;
    }
    // the thread's column packet of the stage
    const int qc = threadIdx.x % QC;
    const bool qlive = c0 + qc * V < Dg;
    float bias[V], skip[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        bias[v] = qlive && p.dt_bias ? p.dt_bias[d0 + qc * V + v] : 0.f;
        skip[v] = qlive && p.D_skip ? p.D_skip[d0 + qc * V + v] : 0.f;
    }
    for (int tb = 0; tb < len; tb += kTokens) {
        const int n = min(kTokens, len - tb);
        Packet<T, V> u[PS];
#pragma unroll
        for (int i = 0; i < PS; ++i) {
            const int t = (i * S::NT + threadIdx.x) / QC;
            if (t >= n) continue;
            float uf[V], df[V];
#pragma unroll
            for (int v = 0; v < V; ++v) uf[v] = df[v] = 0.f;
            if (qlive) {
                const long row = t0 + tb + t, col = d0 + qc * V;
                u[i] = load_packet<T, V>(static_cast<const T *>(p.u) + row * p.ld_u + col);
                unpack<T, V>(u[i], uf);
                unpack<T, V>(load_packet<T, V>(static_cast<const T *>(p.dt) + row * p.ld_dt + col), df);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    df[v] += bias[v];
                    if (p.softplus) df[v] = softplus_rel(df[v]);
                }
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                sm.delta[t][qc * V + v] = df[v];
                sm.du[t][qc * V + v] = df[v] * uf[v];
            }
        }
        stage_bc<T, S::NP>(p, t0 + tb, n, g, &sm.B[0][0], &sm.C[0][0]);
        __syncthreads();
        if (p.h_chunks) {
            float *hc = p.h_chunks + (slot0 + tb / kTokens) * p.D * p.N;
#pragma unroll
            for (int c = 0; c < S::CPT; ++c)
                if (c0 + cw + c < Dg && nl * kStates < p.N)
                    store_states(hc, d0 + cw + c, nl * kStates, p.N, h[c]);
        }
#pragma unroll 4
        for (int t = 0; t < n; ++t) {
            const float4 Bv = *reinterpret_cast<const float4 *>(&sm.B[t][nl * kStates]);
            const float4 Cv = *reinterpret_cast<const float4 *>(&sm.C[t][nl * kStates]);
            const float bv[kStates] = {Bv.x, Bv.y, Bv.z, Bv.w};
            const float cv[kStates] = {Cv.x, Cv.y, Cv.z, Cv.w};
            float acc[S::CPT];
#pragma unroll
            for (int c = 0; c < S::CPT; ++c) {
                const float delta = sm.delta[t][cw + c], du = sm.du[t][cw + c];
                acc[c] = 0.f;
#pragma unroll
                for (int i = 0; i < kStates; ++i) {
                    h[c][i] = fmaf(ex2(delta * a2[c][i]), h[c][i], du * bv[i]);
                    acc[c] = fmaf(h[c][i], cv[i], acc[c]);
                }
#pragma unroll
                for (int o = S::NL / 2; o > 0; o >>= 1)
                    acc[c] += __shfl_xor_sync(0xffffffffu, acc[c], o);
            }
            if (nl == 0)
#pragma unroll
                for (int c = 0; c < S::CPT; ++c) sm.y[t][cw + c] = acc[c];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < PS; ++i) {
            const int t = (i * S::NT + threadIdx.x) / QC;
            if (t >= n || !qlive) continue;
            const long row = t0 + tb + t, col = d0 + qc * V;
            float uf[V], o[V], z[V];
            unpack<T, V>(u[i], uf);
            if (p.z) unpack<T, V>(load_packet<T, V>(static_cast<const T *>(p.z) + row * p.ld_z + col), z);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                o[v] = fmaf(skip[v], uf[v], sm.y[t][qc * V + v]);
                if (p.z) o[v] *= z[v] * sigmoid_f(z[v]);
            }
            store_packet<T, V>(static_cast<T *>(p.y) + row * p.D + col, pack<T, V>(o));
        }
        // the next stage writes delta and du, which every warp has read, and y
        // only after the barrier that follows that
    }
    if (p.h_T)
#pragma unroll
        for (int c = 0; c < S::CPT; ++c)
            if (c0 + cw + c < Dg && nl * kStates < p.N)
                store_states(p.h_T + (long)seq * p.D * p.N, d0 + cw + c, nl * kStates, p.N, h[c]);
}

template <typename T, typename S, int V>
cudaError_t fwd_t(const ScanProblem &p, const Layout &l, cudaStream_t st) {
    const int Dg = p.D / p.G;
    const long tiles = (long)p.G * ((Dg + S::CB - 1) / S::CB);
    const long blocks = tiles * p.n_seq;
    if (blocks > 0x7fffffffL) return cudaErrorInvalidConfiguration;
    auto k = scan_fwd_kernel<T, S, V>;
    cudaError_t err = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           (int)sizeof(FwdSmem<S>));
    if (err != cudaSuccess) return err;
    k<<<(unsigned)blocks, S::NT, sizeof(FwdSmem<S>), st>>>(p, l, (int)tiles);
    return cudaGetLastError();
}

template <typename T>
cudaError_t fwd_dispatch(const ScanProblem &p, const Layout &l, cudaStream_t st) {
    constexpr int V = 4;
    const int bytes = V * (int)sizeof(T);
    const bool wide = (p.D / p.G) % V == 0 && rows_aligned(p.u, p.ld_u, sizeof(T), bytes) &&
                      rows_aligned(p.dt, p.ld_dt, sizeof(T), bytes) &&
                      rows_aligned(p.z, p.ld_z, sizeof(T), bytes) &&
                      rows_aligned(p.y, p.D, sizeof(T), bytes);
#define MDN_SCAN_CASE(NL)                                       \
    case NL:                                                    \
        return wide ? fwd_t<T, Shape<NL, 2>, V>(p, l, st)       \
                    : fwd_t<T, Shape<NL, 2>, 1>(p, l, st);
    switch (lanes_of_states(p.N)) {
        MDN_SCAN_CASE(2)
        MDN_SCAN_CASE(4)
        MDN_SCAN_CASE(8)
        MDN_SCAN_CASE(16)
        MDN_SCAN_CASE(32)
    }
#undef MDN_SCAN_CASE
    return cudaErrorInvalidValue;
}

// -------------------------------------------------------------------- step

// Memory bound by the states (read and written once, in order): a thread
// holds four states of one channel.
template <typename T, int NL>
__global__ void __launch_bounds__(256) scan_step_kernel(ScanProblem p) {
    const long idx = ((long)blockIdx.x * 256 + threadIdx.x);
    const long ch = idx / NL;                        // sequence * D + channel
    const int n0 = (int)(idx % NL) * kStates;
    const bool live = ch < (long)p.n_seq * p.D;
    const long s = live ? ch / p.D : 0;
    const int d = live ? (int)(ch - s * p.D) : 0;
    const bool mine = live && n0 < p.N;
    float a[kStates], h[kStates], acc = 0.f, u = 0.f;
    if (mine) {
        load_states(p.A, d, n0, p.N, a);
        if (p.N % kStates == 0) {
            const float4 v = *reinterpret_cast<const float4 *>(p.h0 + ch * p.N + n0);
            h[0] = v.x; h[1] = v.y; h[2] = v.z; h[3] = v.w;
        } else {
            load_states(p.h0, ch, n0, p.N, h);
        }
        u = to_f32(static_cast<const T *>(p.u)[s * p.ld_u + d]);
        float delta = to_f32(static_cast<const T *>(p.dt)[s * p.ld_dt + d]);
        if (p.dt_bias) delta += p.dt_bias[d];
        if (p.softplus) delta = softplus_rel(delta);
        const long gb = (long)(d / (p.D / p.G)) * p.N + n0;
        const T *Bp = static_cast<const T *>(p.Bm) + s * p.ld_B + gb;
        const T *Cp = static_cast<const T *>(p.Cm) + s * p.ld_C + gb;
#pragma unroll
        for (int i = 0; i < kStates; ++i) {
            const bool in = n0 + i < p.N;
            const float b = in ? to_f32(Bp[i]) : 0.f, c = in ? to_f32(Cp[i]) : 0.f;
            h[i] = fmaf(ex2(delta * (a[i] * kLog2e)), h[i], delta * u * b);
            acc = fmaf(h[i], c, acc);
        }
        store_states(p.h_T, ch, n0, p.N, h);
    }
#pragma unroll
    for (int o = NL / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (live && n0 == 0) {
        if (p.D_skip) acc = fmaf(p.D_skip[d], u, acc);
        if (p.z) {
            const float z = to_f32(static_cast<const T *>(p.z)[s * p.ld_z + d]);
            acc *= z * sigmoid_f(z);
        }
        static_cast<T *>(p.y)[ch] = from_f32<T>(acc);
    }
}

template <typename T>
cudaError_t step_dispatch(const ScanProblem &p, cudaStream_t st) {
    const int nl = lanes_of_states(p.N);
    const long blocks = ((long)p.n_seq * p.D * nl + 255) / 256;
    if (blocks > 0x7fffffffL) return cudaErrorInvalidConfiguration;
    switch (nl) {
        case 2: scan_step_kernel<T, 2><<<(unsigned)blocks, 256, 0, st>>>(p); break;
        case 4: scan_step_kernel<T, 4><<<(unsigned)blocks, 256, 0, st>>>(p); break;
        case 8: scan_step_kernel<T, 8><<<(unsigned)blocks, 256, 0, st>>>(p); break;
        case 16: scan_step_kernel<T, 16><<<(unsigned)blocks, 256, 0, st>>>(p); break;
        case 32: scan_step_kernel<T, 32><<<(unsigned)blocks, 256, 0, st>>>(p); break;
        default: return cudaErrorInvalidValue;
    }
    return cudaGetLastError();
}

// to <- from, or zero (the states of a call without tokens).
__global__ void states_copy_kernel(const float *from, float *to, long n) {
    for (long i = (long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long)gridDim.x * blockDim.x)
        to[i] = from ? from[i] : 0.f;
}

}  // namespace

cudaError_t launch_layout(const ScanProblem &p, Layout &l, cudaStream_t st) {
    l.slot_off = l.order = nullptr;
    if (!p.cu) return cudaSuccess;
    int32_t *off = reinterpret_cast<int32_t *>(p.ws);
    int32_t *order = reinterpret_cast<int32_t *>(p.ws + layout_bytes(p.n_seq) / 2);
    l.slot_off = off;
    l.order = order;
    layout_kernel<<<1, 1024, 0, st>>>(p.cu, p.n_seq, p.T_total, off, order, p.status);
    return cudaGetLastError();
}

cudaError_t launch_states_copy(const float *from, float *to, long n, cudaStream_t st) {
    if (!to || n == 0 || from == to) return cudaSuccess;
    const long blocks = (n + 255) / 256;
    states_copy_kernel<<<(unsigned)(blocks < 1216 ? blocks : 1216), 256, 0, st>>>(from, to, n);
    return cudaGetLastError();
}

}  // namespace scan

size_t scan_fwd_workspace(int n_seq, int T_total, int D, int G, int N, mdn_dtype dtype) {
    return scan::layout_bytes(n_seq);
}

cudaError_t launch_scan_fwd(const ScanProblem &p, cudaStream_t st) {
    if (p.n_seq == 0) return cudaSuccess;
    if (p.T_total == 0) return scan::launch_states_copy(p.h0, p.h_T, (long)p.n_seq * p.D * p.N, st);
    scan::Layout l;
    const cudaError_t err = scan::launch_layout(p, l, st);
    if (err != cudaSuccess) return err;
    return p.dtype == MDN_BF16 ? scan::fwd_dispatch<__nv_bfloat16>(p, l, st)
                               : scan::fwd_dispatch<float>(p, l, st);
}

cudaError_t launch_scan_step(const ScanProblem &p, cudaStream_t st) {
    if (p.n_seq == 0) return cudaSuccess;
    return p.dtype == MDN_BF16 ? scan::step_dispatch<__nv_bfloat16>(p, st)
                               : scan::step_dispatch<float>(p, st);
}

}  // namespace mdn
