// Gradient of the selective state-space scan.
//
// With a_t = exp(delta_t A), h_t = a_t h_{t-1} + delta_t u_t B_t and e_t the
// adjoint of y before its gate (dy silu(z)), the adjoint of h_t is
//   g_t = C_t e_t + a_{t+1} g_{t+1}
// and, with w_t = a_t g_t h_{t-1},
//   du_t   = delta_t sum_n g_t B_t + D_skip e_t
//   ddelta = sum_n A w_t + u_t sum_n g_t B_t
//   dA     = sum_t delta_t w_t;   dB_t = sum_d g_t delta_t u_t;   dC_t = sum_d e_t h_t
// (sums over the channels d of the group), ddt = ddelta softplus'(dt).
//
// The recurrence cannot be run backwards (h_{t-1} = (h_t - ..) / a_t blows up
// for small a), so every chunk of 32 tokens starts from the state the forward
// saved: one pass forward keeps the state before every fourth token in shared
// memory, then each group of four tokens, last first, is run forward again
// with its states and decays in registers and walked back.
#include "mdn_scan.cuh"

namespace mdn {
namespace scan {
namespace {

constexpr int kSub = 4;                       // tokens walked back at a time
constexpr int kSubs = kTokens / kSub;

template <typename S>
struct BwdSmem {
    float delta[kTokens][S::CB];      // delta; then ddelta
    float u[kTokens][S::CB];          // u; then du
    float e[kTokens][S::CB];          // e; then y before the gate
    float B[kTokens][S::NP], C[kTokens][S::NP];
    float4 sub[kSubs][S::CPT][S::NT];         // state before every fourth token
    float bc[2][S::NW][kSub][2][S::NP];       // the warps' dB, dC of four tokens
};

struct BwdPartials {
    float *bc;        // [tile of the group][T_total][G][2][N]
    float *A;         // [slot][D][N]
    float *D, *bias;  // [slot][D]
    int slots;        // blocks that share a tile's sequences
};

template <typename T, typename S, int V>
__global__ void __launch_bounds__(S::NT) scan_bwd_kernel(ScanProblem p, Layout l, BwdPartials w, int tiles) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    BwdSmem<S> &sm = *reinterpret_cast<BwdSmem<S> *>(smem_raw);
    constexpr int QC = S::CB / V;
    constexpr int RS = S::NT / QC;                   // token rows per pass
    static_assert(S::NT % QC == 0, "a thread keeps its columns");
    const int Dg = p.D / p.G;
    const int gtiles = tiles / p.G;
    const int tile = blockIdx.x % tiles;
    const int slot = blockIdx.x / tiles;
    const int g = tile / gtiles;
    const int c0 = (tile % gtiles) * S::CB;
    const long d0 = (long)g * Dg + c0;

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nl = lane % S::NL;
    const int n0 = nl * kStates;
    const int cw = warp * S::WC + lane / S::NL * S::CPT;
    float a2[S::CPT][kStates], dA[S::CPT][kStates], skip[S::CPT];
    bool live[S::CPT];
#pragma unroll
    for (int c = 0; c < S::CPT; ++c) {
        live[c] = c0 + cw + c < Dg && n0 < p.N;
        skip[c] = c0 + cw + c < Dg && p.D_skip ? p.D_skip[d0 + cw + c] : 0.f;
#pragma unroll
        for (int i = 0; i < kStates; ++i) a2[c][i] = dA[c][i] = 0.f;
        if (live[c]) load_states(p.A, d0 + cw + c, n0, p.N, a2[c]);
#pragma unroll
        for (int i = 0; i < kStates; ++i) a2[c][i] *= kLog2e;
    }
    const int qc = threadIdx.x % QC, qrow = threadIdx.x / QC;
    const bool qlive = c0 + qc * V < Dg;
    const long col = d0 + qc * V;
    float bias[V], dD[V], dbias[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        bias[v] = qlive && p.dt_bias ? p.dt_bias[col + v] : 0.f;
        dD[v] = dbias[v] = 0.f;
    }

    for (int k = slot; k < l.items; k += w.slots) {
        Item it;
        long t0, slot0;
        if (!find_item(p, l, k, false, it, t0, slot0)) break;
        const int seq = it.seq, len = it.len;
        const long sbase = (long)seq * p.D * p.N;
        float gc[S::CPT][kStates];                   // a_{t+1} g_{t+1}
#pragma unroll
        for (int c = 0; c < S::CPT; ++c) {
#pragma unroll
            for (int i = 0; i < kStates; ++i) gc[c][i] = 0.f;
            if (live[c] && p.dh_T) load_states(p.dh_T + sbase, d0 + cw + c, n0, p.N, gc[c]);
        }
        for (int chunk = (len + kTokens - 1) / kTokens - 1; chunk >= 0; --chunk) {
            const int tb = chunk * kTokens;
            const int n = min(kTokens, len - tb);
            const int n4 = (n + kSub - 1) / kSub * kSub;
            // stage the chunk; tokens n .. n4 are zero and change nothing
            for (int t = qrow; t < n4; t += RS) {
                float df[V], uf[V], ef[V];
#pragma unroll
                for (int v = 0; v < V; ++v) df[v] = uf[v] = ef[v] = 0.f;
                if (t < n && qlive) {
                    const long row = t0 + tb + t;
                    unpack<T, V>(load_packet<T, V>(static_cast<const T *>(p.u) + row * p.ld_u + col), uf);
                    unpack<T, V>(load_packet<T, V>(static_cast<const T *>(p.dt) + row * p.ld_dt + col), df);
                    unpack<T, V>(load_packet<T, V>(static_cast<const T *>(p.dy) + row * p.ld_dy + col), ef);
                    if (p.z) {
                        float z[V];
                        unpack<T, V>(load_packet<T, V>(static_cast<const T *>(p.z) + row * p.ld_z + col), z);
#pragma unroll
                        for (int v = 0; v < V; ++v) ef[v] *= z[v] * sigmoid_f(z[v]);
                    }
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        df[v] += bias[v];
                        if (p.softplus) df[v] = softplus_rel(df[v]);
                        dD[v] = fmaf(ef[v], uf[v], dD[v]);
                    }
                }
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    sm.delta[t][qc * V + v] = df[v];
                    sm.u[t][qc * V + v] = uf[v];
                    sm.e[t][qc * V + v] = ef[v];
                }
            }
            stage_bc<T, S::NP, true, true>(p, t0 + tb, n, n4, g, threadIdx.x, S::NT, &sm.B[0][0], &sm.C[0][0]);
            __syncthreads();
            // forward: the state before every fourth token
            {
                const float *hc = p.h_chunks + (slot0 + chunk) * p.D * p.N;
                float h[S::CPT][kStates];
#pragma unroll
                for (int c = 0; c < S::CPT; ++c) {
#pragma unroll
                    for (int i = 0; i < kStates; ++i) h[c][i] = 0.f;
                    if (live[c]) load_states(hc, d0 + cw + c, n0, p.N, h[c]);
                }
                for (int s = 0; s < n4 / kSub; ++s) {
#pragma unroll
                    for (int c = 0; c < S::CPT; ++c)
                        sm.sub[s][c][threadIdx.x] = make_float4(h[c][0], h[c][1], h[c][2], h[c][3]);
                    if (s == n4 / kSub - 1) break;
#pragma unroll
                    for (int j = 0; j < kSub; ++j) {
                        const int t = s * kSub + j;
                        const float4 Bv = *reinterpret_cast<const float4 *>(&sm.B[t][n0]);
                        const float bv[kStates] = {Bv.x, Bv.y, Bv.z, Bv.w};
#pragma unroll
                        for (int c = 0; c < S::CPT; ++c) {
                            const float delta = sm.delta[t][cw + c];
                            const float du = delta * sm.u[t][cw + c];
#pragma unroll
                            for (int i = 0; i < kStates; ++i)
                                h[c][i] = fmaf(ex2(delta * a2[c][i]), h[c][i], du * bv[i]);
                        }
                    }
                }
            }
            float dAc[S::CPT][kStates];              // this chunk's dA
#pragma unroll
            for (int c = 0; c < S::CPT; ++c)
#pragma unroll
                for (int i = 0; i < kStates; ++i) dAc[c][i] = 0.f;
            for (int s = n4 / kSub - 1; s >= 0; --s) {
                float h[kSub + 1][S::CPT][kStates], a[kSub][S::CPT][kStates];
#pragma unroll
                for (int c = 0; c < S::CPT; ++c) {
                    const float4 v = sm.sub[s][c][threadIdx.x];
                    h[0][c][0] = v.x; h[0][c][1] = v.y; h[0][c][2] = v.z; h[0][c][3] = v.w;
                }
#pragma unroll
                for (int j = 0; j < kSub; ++j) {
                    const int t = s * kSub + j;
                    const float4 Bv = *reinterpret_cast<const float4 *>(&sm.B[t][n0]);
                    const float bv[kStates] = {Bv.x, Bv.y, Bv.z, Bv.w};
#pragma unroll
                    for (int c = 0; c < S::CPT; ++c) {
                        const float delta = sm.delta[t][cw + c];
                        const float du = delta * sm.u[t][cw + c];
#pragma unroll
                        for (int i = 0; i < kStates; ++i) {
                            a[j][c][i] = ex2(delta * a2[c][i]);
                            h[j + 1][c][i] = fmaf(a[j][c][i], h[j][c][i], du * bv[i]);
                        }
                    }
                }
#pragma unroll
                for (int j = kSub - 1; j >= 0; --j) {
                    const int t = s * kSub + j;
                    const float4 Bv = *reinterpret_cast<const float4 *>(&sm.B[t][n0]);
                    const float4 Cv = *reinterpret_cast<const float4 *>(&sm.C[t][n0]);
                    const float bv[kStates] = {Bv.x, Bv.y, Bv.z, Bv.w};
                    const float cv[kStates] = {Cv.x, Cv.y, Cv.z, Cv.w};
                    float dB[kStates], dC[kStates];
#pragma unroll
                    for (int i = 0; i < kStates; ++i) dB[i] = dC[i] = 0.f;
#pragma unroll
                    for (int c = 0; c < S::CPT; ++c) {
                        const float delta = sm.delta[t][cw + c], u = sm.u[t][cw + c];
                        const float e = sm.e[t][cw + c], du = delta * u;
                        float s1 = 0.f, s2 = 0.f, y = 0.f;
#pragma unroll
                        for (int i = 0; i < kStates; ++i) {
                            const float gg = fmaf(cv[i], e, gc[c][i]);
                            dB[i] = fmaf(gg, du, dB[i]);
                            dC[i] = fmaf(e, h[j + 1][c][i], dC[i]);
                            y = fmaf(cv[i], h[j + 1][c][i], y);
                            s1 = fmaf(gg, bv[i], s1);
                            gc[c][i] = a[j][c][i] * gg;
                            const float wv = gc[c][i] * h[j][c][i];
                            s2 = fmaf(a2[c][i], wv, s2);
                            dAc[c][i] = fmaf(delta, wv, dAc[c][i]);
                        }
#pragma unroll
                        for (int o = S::NL / 2; o > 0; o >>= 1) {
                            s1 += __shfl_xor_sync(0xffffffffu, s1, o);
                            s2 += __shfl_xor_sync(0xffffffffu, s2, o);
                            y += __shfl_xor_sync(0xffffffffu, y, o);
                        }
                        __syncwarp();
                        if (nl == 0) {
                            sm.delta[t][cw + c] = fmaf(u, s1, s2 * (1.f / kLog2e));
                            sm.u[t][cw + c] = fmaf(delta, s1, skip[c] * e);
                            sm.e[t][cw + c] = fmaf(skip[c], u, y);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < kStates; ++i)
#pragma unroll
                        for (int o = S::NL; o < 32; o <<= 1) {
                            dB[i] += __shfl_xor_sync(0xffffffffu, dB[i], o);
                            dC[i] += __shfl_xor_sync(0xffffffffu, dC[i], o);
                        }
                    if (lane < S::NL)
#pragma unroll
                        for (int i = 0; i < kStates; ++i) {
                            sm.bc[s & 1][warp][j][0][n0 + i] = dB[i];
                            sm.bc[s & 1][warp][j][1][n0 + i] = dC[i];
                        }
                }
                __syncthreads();
                // the block's dB, dC of the four tokens
                for (int i = threadIdx.x; i < kSub * 2 * S::NP; i += S::NT) {
                    const int j = i / (2 * S::NP), which = i / S::NP % 2, m = i % S::NP;
                    const int t = s * kSub + j;
                    if (t >= n || m >= p.N) continue;
                    float v = 0.f;
#pragma unroll
                    for (int q = 0; q < S::NW; ++q) v += sm.bc[s & 1][q][j][which][m];
                    w.bc[((((long)(tile % gtiles) * p.T_total + t0 + tb + t) * p.G + g) * 2 + which) * p.N + m] = v;
                }
            }
#pragma unroll
            for (int c = 0; c < S::CPT; ++c)
#pragma unroll
                for (int i = 0; i < kStates; ++i) dA[c][i] += dAc[c][i];
            // the last barrier above stands between the results in shared
            // memory and here
            for (int t = qrow; t < n && qlive; t += RS) {
                const long row = t0 + tb + t;
                float o[V], x[V];
#pragma unroll
                for (int v = 0; v < V; ++v) o[v] = sm.u[t][qc * V + v];
                store_packet<T, V>(static_cast<T *>(p.du) + row * p.D + col, pack<T, V>(o));
                unpack<T, V>(load_packet<T, V>(static_cast<const T *>(p.dt) + row * p.ld_dt + col), x);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    o[v] = sm.delta[t][qc * V + v];
                    if (p.softplus) o[v] *= sigmoid_f(x[v] + bias[v]);
                    dbias[v] += o[v];
                }
                store_packet<T, V>(static_cast<T *>(p.ddt) + row * p.D + col, pack<T, V>(o));
                if (p.z) {
                    float z[V];
                    unpack<T, V>(load_packet<T, V>(static_cast<const T *>(p.dy) + row * p.ld_dy + col), x);
                    unpack<T, V>(load_packet<T, V>(static_cast<const T *>(p.z) + row * p.ld_z + col), z);
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const float sg = sigmoid_f(z[v]);
                        o[v] = x[v] * sm.e[t][qc * V + v] * sg * fmaf(z[v], 1.f - sg, 1.f);
                    }
                    store_packet<T, V>(static_cast<T *>(p.dz) + row * p.D + col, pack<T, V>(o));
                }
            }
            __syncthreads();
        }
        if (p.dh0)
#pragma unroll
            for (int c = 0; c < S::CPT; ++c)
                if (live[c]) store_states(p.dh0 + sbase, d0 + cw + c, n0, p.N, gc[c]);
    }
    const long pbase = (long)slot * p.D;
#pragma unroll
    for (int c = 0; c < S::CPT; ++c)
        if (live[c]) store_states(w.A + pbase * p.N, d0 + cw + c, n0, p.N, dA[c]);
    // the threads of a column packet add up in order
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (qrow < kTokens) {                        // later rows hold no token
            sm.delta[qrow][qc * V + v] = dD[v];
            sm.u[qrow][qc * V + v] = dbias[v];
        }
    __syncthreads();
    for (int c = threadIdx.x; c < S::CB; c += S::NT) {
        if (c0 + c >= Dg) continue;
        float x = 0.f, y = 0.f;
        for (int r = 0; r < RS && r < kTokens; ++r) {
            x += sm.delta[r][c];
            y += sm.u[r][c];
        }
        w.D[pbase + d0 + c] = x;
        w.bias[pbase + d0 + c] = y;
    }
}

// dB, dC [T_total, G, N]: the tiles' partial sums, in order.  Nothing is
// written where malformed packed offsets left no slots (total_slots 0).
template <typename T>
__global__ void __launch_bounds__(256)
scan_reduce_bc_kernel(const int32_t *total_slots, const float *part, int gtiles, long rows, int N, T *dB, T *dC) {
    if (total_slots && *total_slots == 0) return;
    const long per = rows * 2 * N;
    for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < per; i += (long)gridDim.x * 256) {
        float v = 0.f;
        for (int k = 0; k < gtiles; ++k) v += part[k * per + i];
        const long row = i / (2 * N);
        const int m = (int)(i - row * 2 * N);
        if (m < N) dB[row * N + m] = from_f32<T>(v);
        else dC[row * N + m - N] = from_f32<T>(v);
    }
}

// out[i] = sum over the slots, in order, of part[slot][i].
__global__ void __launch_bounds__(256)
scan_reduce_params_kernel(BwdPartials w, long dn, int D, float *dA, float *dD, float *dbias) {
    const long total = dn + 2L * D;
    for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < total; i += (long)gridDim.x * 256) {
        const float *src = i < dn ? w.A + i : i < dn + D ? w.D + (i - dn) : w.bias + (i - dn - D);
        const long step = i < dn ? dn : D;
        float *out = i < dn ? dA + i : i < dn + D ? dD : dbias;
        if (!out) continue;
        float v = 0.f;
        for (int s = 0; s < w.slots; ++s) v += src[s * step];
        if (i < dn) *out = v;
        else out[i < dn + D ? i - dn : i - dn - D] = v;
    }
}

int bwd_block_channels(int N) {
    switch (lanes_of_states(N)) {
        case 2: return Shape<2, 2, 4, 0>::CB;
        case 4: return Shape<4, 2, 4, 0>::CB;
        case 8: return Shape<8, 2, 4, 0>::CB;
        case 16: return Shape<16, 2, 8, 0>::CB;
        default: return Shape<32, 2, 8, 0>::CB;
    }
}

struct BwdPlan {
    long tiles, gtiles;
    int slots;
    size_t bc, A, D, bytes;       // float offsets; bytes of the whole workspace
    size_t base;
};
BwdPlan bwd_plan(int n_seq, int T_total, int D, int G, int N) {
    BwdPlan b;
    const int Dg = D / G, CB = bwd_block_channels(N);
    b.gtiles = (Dg + CB - 1) / CB;
    b.tiles = b.gtiles * G;
    const long want = (152L * 4 + b.tiles - 1) / b.tiles;
    b.slots = (int)(n_seq < want ? n_seq : want);
    if (b.slots < 1) b.slots = 1;
    b.base = layout_bytes(n_seq, T_total, D, N);
    b.bc = round256((size_t)b.gtiles * T_total * G * 2 * N * sizeof(float));
    b.A = round256((size_t)b.slots * D * N * sizeof(float));
    b.D = round256((size_t)b.slots * D * sizeof(float));
    b.bytes = b.base + b.bc + b.A + 2 * b.D;
    return b;
}

template <typename T, typename S, int V>
cudaError_t bwd_t(const ScanProblem &p, const Layout &l, const BwdPartials &w, const BwdPlan &b,
                  cudaStream_t st) {
    const long blocks = b.tiles * w.slots;
    if (blocks > 0x7fffffffL) return cudaErrorInvalidConfiguration;
    auto k = scan_bwd_kernel<T, S, V>;
    cudaError_t err = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           (int)sizeof(BwdSmem<S>));
    if (err != cudaSuccess) return err;
    k<<<(unsigned)blocks, S::NT, sizeof(BwdSmem<S>), st>>>(p, l, w, (int)b.tiles);
    return cudaGetLastError();
}

template <typename T>
cudaError_t bwd_dispatch(const ScanProblem &p, const Layout &l, const BwdPartials &w,
                         const BwdPlan &b, cudaStream_t st) {
    constexpr int V = 4;
    const int bytes = V * (int)sizeof(T);
    bool wide = (p.D / p.G) % V == 0 && rows_aligned(p.u, p.ld_u, sizeof(T), bytes) &&
                rows_aligned(p.dt, p.ld_dt, sizeof(T), bytes) &&
                rows_aligned(p.z, p.ld_z, sizeof(T), bytes) &&
                rows_aligned(p.dy, p.ld_dy, sizeof(T), bytes);
    const void *dense[] = {p.du, p.ddt, p.dz};
    for (const void *ptr : dense) wide = wide && rows_aligned(ptr, p.D, sizeof(T), bytes);
    cudaError_t err = cudaErrorInvalidValue;
#define MDN_SCAN_CASE(NL, NW)                                          \
    case NL:                                                           \
        err = wide ? bwd_t<T, Shape<NL, 2, NW, 0>, V>(p, l, w, b, st)     \
                   : bwd_t<T, Shape<NL, 2, NW, 0>, 1>(p, l, w, b, st);    \
        break;
    switch (lanes_of_states(p.N)) {
        MDN_SCAN_CASE(2, 4)
        MDN_SCAN_CASE(4, 4)
        MDN_SCAN_CASE(8, 4)
        MDN_SCAN_CASE(16, 8)
        MDN_SCAN_CASE(32, 8)
    }
#undef MDN_SCAN_CASE
    if (err != cudaSuccess) return err;
    const long rows = (long)p.T_total * p.G, per = rows * 2 * p.N;
    const long blocks = (per + 255) / 256;
    scan_reduce_bc_kernel<T><<<(unsigned)(blocks < 152 * 8 ? blocks : 152 * 8), 256, 0, st>>>(
        l.slot_off ? l.slot_off + p.n_seq : nullptr, w.bc, (int)b.gtiles, rows, p.N, static_cast<T *>(p.dB), static_cast<T *>(p.dC));
    err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    const long dn = (long)p.D * p.N;
    const long pb = (dn + 2L * p.D + 255) / 256;
    scan_reduce_params_kernel<<<(unsigned)(pb < 152 * 8 ? pb : 152 * 8), 256, 0, st>>>(w, dn, p.D, p.dA, p.dD,
                                                                                  p.ddt_bias);
    return cudaGetLastError();
}

}  // namespace
}  // namespace scan

size_t scan_bwd_workspace(int n_seq, int T_total, int D, int G, int N, mdn_dtype dtype) {
    return scan::bwd_plan(n_seq, T_total, D, G, N).bytes;
}

cudaError_t launch_scan_bwd(const ScanProblem &p, cudaStream_t st) {
    if (p.T_total == 0 || p.n_seq == 0) {
        const size_t n[] = {(size_t)p.D * p.N, (size_t)p.D, (size_t)p.D};
        float *out[] = {p.dA, p.dD, p.ddt_bias};
        for (int i = 0; i < 3; ++i)
            if (out[i]) {
                const cudaError_t err = cudaMemsetAsync(out[i], 0, n[i] * sizeof(float), st);
                if (err != cudaSuccess) return err;
            }
        return scan::launch_states_copy(p.dh_T, p.dh0, (long)p.n_seq * p.D * p.N, st);
    }
    scan::Layout l;
    const cudaError_t err = scan::make_layout(p, l, st, false);
    if (err != cudaSuccess) return err;
    const scan::BwdPlan b = scan::bwd_plan(p.n_seq, p.T_total, p.D, p.G, p.N);
    scan::BwdPartials w;
    unsigned char *at = p.ws + b.base;
    w.bc = reinterpret_cast<float *>(at);
    w.A = reinterpret_cast<float *>(at + b.bc);
    w.D = reinterpret_cast<float *>(at + b.bc + b.A);
    w.bias = reinterpret_cast<float *>(at + b.bc + b.A + b.D);
    w.slots = b.slots;
    return p.dtype == MDN_BF16 ? scan::bwd_dispatch<__nv_bfloat16>(p, l, w, b, st)
                               : scan::bwd_dispatch<float>(p, l, w, b, st);
}

}  // namespace mdn
