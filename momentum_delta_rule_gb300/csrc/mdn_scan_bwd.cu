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
//
// Measured, bf16, 16 states, 16384 tokens of 2048 channels: 641 to 651 us, and
// 26 us for the adjoints of the cut parts and 19 us for the partial sums; in
// fp32 785 us.  A token, channel and state
// takes two exponentials and about 15 other operations with its share of the
// exchanges, 537 M of them: the exponentials alone are 113 us, the bytes (u,
// dt, B, C, z, dy and the saved states in, five gradients out) 80 us.  Bound
// by the latency of dependent steps: 230 registers a thread and 100 KB of shared
// memory hold an SM to eight warps, which fill 55 % of the issue slots and 60 %
// of the shared-memory pipe.  Tried: helper warps as in the
// forward (987 us where this took 903), the same with registers moved from the
// helpers to the rest (1215 us), channels instead of states in pairs (665 us).
#include <algorithm>

#include "mdn_scan.cuh"

namespace mdn {
namespace scan {
namespace {

constexpr int kSub = 4;                       // tokens walked back at a time
constexpr int kSubs = kTokens / kSub;

template <typename T, typename S, int V>
struct BwdSmem {
    static constexpr int QC = S::CB / V;                             // packets per token
    static constexpr int PS = (kTokens * QC + S::NT - 1) / S::NT;    // packets per thread
    static constexpr int QB = S::NP / 4;
    static constexpr int PB = (kTokens * QB + S::NT - 1) / S::NT;    // of B, of C
    static_assert(S::NT % QC == 0, "a thread keeps its columns");
    float delta[kTokens][S::CB];      // delta; then ddelta
    float u[kTokens][S::CB];          // u; then du
    float e[kTokens][S::CB];          // e; then y before the gate
    float B[kTokens][S::NP], C[kTokens][S::NP];
    float4 sub[kSubs - 1][S::CPT][S::NT];     // state before every fourth token but the first
    float4 entry[2][S::CPT][S::NT];           // saved states: of this chunk and the next
    float bc[2][S::NW][kSub][2][S::NP];       // the warps' dB, dC of four tokens
    // the inputs as they are, one place for each thread's packets: the next
    // chunk's, and with two slots this one's until its gradients are out (in
    // fp32 that would leave an SM with one block; there they are read again)
    static constexpr int kSlots = sizeof(T) == 2 ? 2 : 1;
    Packet<T, V> in_u[PS][S::NT];
    Packet<T, V> in_dt[kSlots][PS][S::NT], in_dy[kSlots][PS][S::NT], in_z[kSlots][PS][S::NT];
    Packet<T, 4> in_b[PB][S::NT], in_c[PB][S::NT];
};

struct BwdPartials {
    float *bc;        // [tile of the group][T_total][G][2][N]
    float *A;         // [slot][D][N]
    float *D, *bias;  // [slot][D]
    int slots;        // blocks that share a tile's items
};

// The values a lane adds up over the NL lanes of its channels: per token and
// channel sum_n g B, sum_n A w, sum_n C h (in that order).  Lanes exchange
// halves while the count stays whole and leave the rest in every lane.
template <int NL, int M>
__device__ __forceinline__ int reduce_triples(float *v, int nl) {
    int left = M, at = 0;
#pragma unroll
    for (int o = 1; o < NL; o <<= 1) {
        if (left % 6 == 0) {
            left /= 2;
            const bool up = nl & o;
            if (up) at += left;
#pragma unroll
            for (int i = 0; i < M / 2; ++i) {
                if (i < left) {
                    const float send = up ? v[i] : v[i + left];
                    const float keep = up ? v[i + left] : v[i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 3; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        }
    }
    return at / 3;                    // first (token, channel) of this lane's
}

// One block takes CB channels of one group through its items, each item's
// chunks last first.  A lane's two channels are held as two pairs of states
// each: pair i has channel i / 2, states 2 (i % 2) and the next.
template <typename T, typename S, int V, Pad PAD>
__global__ void __launch_bounds__(S::NT, S::NT <= 128 ? 2 : 1)
scan_bwd_kernel(ScanProblem p, Layout l, BwdPartials w, int tiles) {
    using Sm = BwdSmem<T, S, V>;
    static_assert(S::CPT == 2 && kStates == 4, "four pairs a lane");
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Sm &sm = *reinterpret_cast<Sm *>(smem_raw);
    constexpr int RS = S::NT / Sm::QC;               // tokens between a thread's packets
    const int tid = threadIdx.x;
    const int Dg = p.D / p.G;
    const int gtiles = tiles / p.G;
    const int tile = blockIdx.x % tiles;
    const int slot = blockIdx.x / tiles;
    const int g = tile / gtiles;
    const int c0 = (tile % gtiles) * S::CB;
    const long d0 = (long)g * Dg + c0;

    const int lane = tid & 31, warp = tid >> 5;
    const int nl = lane % S::NL, n0 = nl * kStates;
    const int cw = warp * S::WC + lane / S::NL * 2;  // the lane's first channel in the block
    const bool live0 = c0 + cw < Dg && n0 < p.N, live1 = c0 + cw + 1 < Dg && n0 < p.N;
    bool in[kStates];                                // of the lane's states, the real ones
#pragma unroll
    for (int i = 0; i < kStates; ++i) in[i] = n0 + i < p.N;
    auto real = [&](Pair v, int i) {                 // pair i without padded states
        return PAD == Pad::kStates ? real_states(v, in[i % 2 * 2], in[i % 2 * 2 + 1]) : v;
    };
    const float skip0 = c0 + cw < Dg && p.D_skip ? p.D_skip[d0 + cw] : 0.f;
    const float skip1 = c0 + cw + 1 < Dg && p.D_skip ? p.D_skip[d0 + cw + 1] : 0.f;
    auto load_pairs = [&](const float *base, Pair *out) {
        float x[kStates] = {0.f, 0.f, 0.f, 0.f}, y[kStates] = {0.f, 0.f, 0.f, 0.f};
        if (live0) load_states(base, d0 + cw, n0, p.N, x);
        if (live1) load_states(base, d0 + cw + 1, n0, p.N, y);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            out[i] = make_pair(x[2 * i], x[2 * i + 1]);
            out[2 + i] = make_pair(y[2 * i], y[2 * i + 1]);
        }
    };
    auto store_pairs = [&](float *base, const Pair *v) {
        float x[kStates], y[kStates];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            split_pair(v[i], x[2 * i], x[2 * i + 1]);
            split_pair(v[2 + i], y[2 * i], y[2 * i + 1]);
        }
        if (live0) store_states(base, d0 + cw, n0, p.N, x);
        if (live1) store_states(base, d0 + cw + 1, n0, p.N, y);
    };
    Pair a2[kStates], dA[kStates];
    load_pairs(p.A, a2);
#pragma unroll
    for (int i = 0; i < kStates; ++i) {
        float x, y;
        split_pair(a2[i], x, y);
        a2[i] = make_pair(decay_rate(x), decay_rate(y));
        dA[i] = make_pair(0.f, 0.f);
    }
    const int row = tid / Sm::QC, qcol = tid % Sm::QC * V;
    const bool qlive = c0 + qcol < Dg;
    const long col = d0 + qcol;
    float bias[V], dD[V], dbias[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        bias[v] = qlive && p.dt_bias ? p.dt_bias[col + v] : 0.f;
        dD[v] = dbias[v] = 0.f;
    }
    // copies tokens t0 .. t0 + n of the chunk whose saved states lie at hc, this
    // thread's packets
    auto issue = [&](long t0, int n, const float *hc, int chunk) {
        const int r = chunk % Sm::kSlots;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float4 *dst = &sm.entry[chunk & 1][c][tid];
            if (!(c ? live1 : live0)) {
                *dst = make_float4(0.f, 0.f, 0.f, 0.f);
            } else if (p.N % kStates == 0) {
                copy_packet<float, 4>(reinterpret_cast<Packet<float, 4> *>(dst), hc + (d0 + cw + c) * p.N + n0);
            } else {
                float f[kStates];
                load_states(hc, d0 + cw + c, n0, p.N, f);
                *dst = make_float4(f[0], f[1], f[2], f[3]);
            }
        }
#pragma unroll
        for (int i = 0; i < Sm::PS; ++i) {
            const int t = i * RS + row;
            if (t >= n || !qlive) break;
            copy_packet<T, V>(&sm.in_u[i][tid], static_cast<const T *>(p.u) + (t0 + t) * p.ld_u + col);
            copy_packet<T, V>(&sm.in_dt[r][i][tid], static_cast<const T *>(p.dt) + (t0 + t) * p.ld_dt + col);
            copy_packet<T, V>(&sm.in_dy[r][i][tid], static_cast<const T *>(p.dy) + (t0 + t) * p.ld_dy + col);
            if (p.z)
                copy_packet<T, V>(&sm.in_z[r][i][tid], static_cast<const T *>(p.z) + (t0 + t) * p.ld_z + col);
        }
#pragma unroll
        for (int i = 0; i < Sm::PB; ++i) {
            const int j = i * S::NT + tid, t = j / Sm::QB, m = j % Sm::QB * 4;
            if (t >= n || m >= p.N) continue;
            const T *bp = static_cast<const T *>(p.Bm) + (t0 + t) * p.ld_B + (long)g * p.N + m;
            const T *cp = static_cast<const T *>(p.Cm) + (t0 + t) * p.ld_C + (long)g * p.N + m;
            if (p.bc_wide) {
                copy_packet<T, 4>(&sm.in_b[i][tid], bp);
                copy_packet<T, 4>(&sm.in_c[i][tid], cp);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    sm.in_b[i][tid].e[e] = m + e < p.N ? bp[e] : from_f32<T>(0.f);
                    sm.in_c[i][tid].e[e] = m + e < p.N ? cp[e] : from_f32<T>(0.f);
                }
            }
        }
        commit_copies();
    };

    for (int k = slot; k < l.items; k += w.slots) {
        Item it;
        long t0, slot0;
        if (!find_item<false, false>(p, l, k, it, t0, slot0)) break;
        const long sbase = (long)it.seq * p.D * p.N;
        const int seq_len = p.cu ? p.cu[it.seq + 1] - p.cu[it.seq] : p.T;
        const int chunks = (it.len + kTokens - 1) / kTokens;
        const long hstep = (long)p.D * p.N;
        const float *hc = p.h_chunks + slot0 * hstep;
        if (chunks > 0)
            issue(t0 + (chunks - 1) * kTokens, it.len - (chunks - 1) * kTokens,
                  hc + (chunks - 1) * hstep, chunks - 1);
        Pair gc[kStates];                            // a_{t+1} g_{t+1}
        if (p.dh_T) {
            load_pairs(p.dh_T + sbase, gc);
        } else {
#pragma unroll
            for (int i = 0; i < kStates; ++i) gc[i] = make_pair(0.f, 0.f);
        }
        // the adjoint behind this segment, through those that follow it
        const int segs = it.len > 0 ? segments_of(seq_len, l.cut, l.trigger) : 1;
        for (int q = segs - 1; q > it.tok0 / l.cut; --q) {
            const long at = it.pre + q - 1;
            Pair r[kStates];
            load_pairs(l.pre_h + at * p.D * p.N, r);
            const float s0 = live0 ? l.pre_sum[at * p.D + d0 + cw] : 0.f;
            const float s1 = live1 ? l.pre_sum[at * p.D + d0 + cw + 1] : 0.f;
#pragma unroll
            for (int i = 0; i < kStates; ++i) {
                float x, y, gx, gy, rx, ry;
                const float sc = i < 2 ? s0 : s1;
                split_pair(mul2(make_pair(sc, sc), a2[i]), x, y);
                split_pair(gc[i], gx, gy);
                split_pair(r[i], rx, ry);
                gc[i] = make_pair(through_segment(x, gx, rx), through_segment(y, gy, ry));
            }
        }
        for (int chunk = chunks - 1; chunk >= 0; --chunk) {
            const int tb = chunk * kTokens;
            const int n = min(kTokens, it.len - tb);
            const int n4 = (n + kSub - 1) / kSub * kSub;
            // this chunk's inputs to fp32 (tokens n .. n4 are zero and change
            // nothing), then the copies of the one before it
            const int r = chunk % Sm::kSlots;
            wait_copies<0>();
#pragma unroll
            for (int i = 0; i < Sm::PS; ++i) {
                const int t = i * RS + row;
                if (t >= n4) break;
                float df[V], uf[V], ef[V];
#pragma unroll
                for (int v = 0; v < V; ++v) df[v] = uf[v] = ef[v] = 0.f;
                if (t < n && qlive) {
                    unpack<T, V>(sm.in_u[i][tid], uf);
                    unpack<T, V>(sm.in_dt[r][i][tid], df);
                    unpack<T, V>(sm.in_dy[r][i][tid], ef);
                    if (p.z) {
                        float z[V];
                        unpack<T, V>(sm.in_z[r][i][tid], z);
                        apply_gate<V>(ef, z);
                    }
                    step_sizes<V>(df, bias, p.softplus);
#pragma unroll
                    for (int v = 0; v < V; ++v) dD[v] = fmaf(ef[v], uf[v], dD[v]);
                }
                store_packet<float, V>(&sm.delta[t][qcol], pack<float, V>(df));
                store_packet<float, V>(&sm.u[t][qcol], pack<float, V>(uf));
                store_packet<float, V>(&sm.e[t][qcol], pack<float, V>(ef));
            }
#pragma unroll
            for (int i = 0; i < Sm::PB; ++i) {
                const int j = i * S::NT + tid, t = j / Sm::QB, m = j % Sm::QB * 4;
                if (t >= n4) break;
                float b[4] = {0.f, 0.f, 0.f, 0.f}, c[4] = {0.f, 0.f, 0.f, 0.f};
                if (t < n && m < p.N) {
                    unpack<T, 4>(sm.in_b[i][tid], b);
                    unpack<T, 4>(sm.in_c[i][tid], c);
                }
                store_packet<float, 4>(&sm.B[t][m], pack<float, 4>(b));
                store_packet<float, 4>(&sm.C[t][m], pack<float, 4>(c));
            }
            if (chunk > 0) issue(t0 + tb - kTokens, kTokens, hc + (chunk - 1) * hstep, chunk - 1);
            __syncthreads();
            // a lane's saved states (its own copies), or those of sub s
            auto load_sub = [&](const float4 (*from)[S::NT], Pair *h) {
                const float4 x = from[0][tid], y = from[1][tid];
                h[0] = make_pair(x.x, x.y); h[1] = make_pair(x.z, x.w);
                h[2] = make_pair(y.x, y.y); h[3] = make_pair(y.z, y.w);
            };
            auto state_pair = [](const Packet<float, kStates> &q, int i) {
                return make_pair(q.e[i % 2 * 2], q.e[i % 2 * 2 + 1]);
            };
            // forward: the state before every fourth token
            {
                Pair h[kStates];
                load_sub(sm.entry[chunk & 1], h);
#pragma unroll 1
                for (int s = 0; s < n4 / kSub - 1; ++s) {
#pragma unroll
                    for (int j = 0; j < kSub; ++j) {
                        const int t = s * kSub + j;
                        const auto bv = load_packet<float, kStates>(&sm.B[t][n0]);
                        const auto dl = load_packet<float, 2>(&sm.delta[t][cw]);
                        const auto uv = load_packet<float, 2>(&sm.u[t][cw]);
                        const float x0 = dl.e[0] * uv.e[0], x1 = dl.e[1] * uv.e[1];
#pragma unroll
                        for (int i = 0; i < kStates; ++i) {
                            const float d = dl.e[i / 2], x = i < 2 ? x0 : x1;
                            float e0, e1;
                            split_pair(fma2(make_pair(d, d), a2[i], make_pair(kDecayBias, kDecayBias)), e0, e1);
                            h[i] = real(fma2(make_pair(ex2(e0), ex2(e1)), h[i], mul2(make_pair(x, x), state_pair(bv, i))), i);
                        }
                    }
                    float x[kStates], y[kStates];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        split_pair(h[i], x[2 * i], x[2 * i + 1]);
                        split_pair(h[2 + i], y[2 * i], y[2 * i + 1]);
                    }
                    sm.sub[s][0][tid] = make_float4(x[0], x[1], x[2], x[3]);
                    sm.sub[s][1][tid] = make_float4(y[0], y[1], y[2], y[3]);
                }
            }
            Pair dAc[kStates];                       // this chunk's dA
#pragma unroll
            for (int i = 0; i < kStates; ++i) dAc[i] = make_pair(0.f, 0.f);
            // four tokens forward again, and back; LAST: some are behind the end
            auto walk = [&](int s, auto last) {
                constexpr bool LAST = decltype(last)::value;
                Pair h[kSub + 1][kStates], a[kSub][kStates];
                load_sub(s > 0 ? sm.sub[s - 1] : sm.entry[chunk & 1], h[0]);
#pragma unroll
                for (int j = 0; j < kSub; ++j) {
                    const int t = s * kSub + j;
                    const auto bv = load_packet<float, kStates>(&sm.B[t][n0]);
                    const auto dl = load_packet<float, 2>(&sm.delta[t][cw]);
                    const auto uv = load_packet<float, 2>(&sm.u[t][cw]);
                    const float x0 = dl.e[0] * uv.e[0], x1 = dl.e[1] * uv.e[1];
#pragma unroll
                    for (int i = 0; i < kStates; ++i) {
                        const float d = dl.e[i / 2], x = i < 2 ? x0 : x1;
                        float e0, e1;
                        split_pair(fma2(make_pair(d, d), a2[i], make_pair(kDecayBias, kDecayBias)), e0, e1);
                        a[j][i] = real(make_pair(ex2(e0), ex2(e1)), i);
                        h[j + 1][i] = real(fma2(a[j][i], h[j][i], mul2(make_pair(x, x), state_pair(bv, i))), i);
                    }
                }
                float tri[kSub * 6], bc[kSub * 2 * kStates];
#pragma unroll
                for (int j = kSub - 1; j >= 0; --j) {
                    const int t = s * kSub + j;
                    const auto bv = load_packet<float, kStates>(&sm.B[t][n0]);
                    const auto cv = load_packet<float, kStates>(&sm.C[t][n0]);
                    const auto dl = load_packet<float, 2>(&sm.delta[t][cw]);
                    const auto uv = load_packet<float, 2>(&sm.u[t][cw]);
                    const auto ev = load_packet<float, 2>(&sm.e[t][cw]);
                    Pair db[2], dc[2];               // dB, dC of the lane's states
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float xc = dl.e[c] * uv.e[c];
                        const Pair x = make_pair(xc, xc), e = make_pair(ev.e[c], ev.e[c]);
                        const Pair d = make_pair(dl.e[c], dl.e[c]);
                        Pair s1, s2, y;
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int i = 2 * c + k;
                            const Pair b = state_pair(bv, i), cc = state_pair(cv, i), ht = h[j + 1][i];
                            const Pair gt = real(fma2(cc, e, gc[i]), i);
                            db[k] = c ? fma2(gt, x, db[k]) : mul2(gt, x);
                            dc[k] = c ? fma2(ht, e, dc[k]) : mul2(ht, e);
                            y = k ? fma2(cc, ht, y) : mul2(cc, ht);
                            s1 = k ? fma2(gt, b, s1) : mul2(gt, b);
                            gc[i] = mul2(a[j][i], gt);
                            const Pair wv = mul2(gc[i], h[j][i]);
                            s2 = k ? fma2(a2[i], wv, s2) : mul2(a2[i], wv);
                            dAc[i] = fma2(d, wv, dAc[i]);
                            // a token behind the end has d = 0, but may
                            // meet an infinite or NaN state
                            if (LAST && s * kSub + j >= n) dAc[i] = make_pair(0.f, 0.f);
                        }
                        auto both = [&](Pair v) {
                            float lo, hi;
                            split_pair(v, lo, hi);
                            return PAD != Pad::kLanes || in[0] ? lo + hi : 0.f;
                        };
                        tri[j * 6 + 3 * c] = both(s1);
                        tri[j * 6 + 3 * c + 1] = both(s2);
                        tri[j * 6 + 3 * c + 2] = both(y);
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float *o = bc + j * 2 * kStates + 2 * k;
                        split_pair(db[k], o[0], o[1]);
                        split_pair(dc[k], o[kStates], o[kStates + 1]);
                    }
                }
                // a lane ends with R (token, channel) triples and finishes them
                // where it owns them; the row's readers are all past it
                {
                    constexpr int M = kSub * 2, R = M > S::NL ? M / S::NL : 1;
                    const int first = reduce_triples<S::NL, kSub * 6>(tri, nl);
                    __syncwarp();
                    if (S::NL <= M || nl < M)
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            const int t = s * kSub + (first + r) / 2, c = (first + r) & 1;
                            const float dl = sm.delta[t][cw + c], u = sm.u[t][cw + c], e = sm.e[t][cw + c];
                            const float skip = c ? skip1 : skip0;
                            sm.delta[t][cw + c] = fmaf(u, tri[3 * r], tri[3 * r + 1] * (1.f / kLog2e));
                            sm.u[t][cw + c] = fmaf(dl, tri[3 * r], skip * e);
                            sm.e[t][cw + c] = fmaf(skip, u, tri[3 * r + 2]);
                        }
                }
                // the same over the lanes of other channels, for dB and dC
                {
                    constexpr int CL = 32 / S::NL, M = kSub * 2 * kStates, R = M / CL;
                    const int cl = lane / S::NL;
                    reduce_lanes<CL, M, S::NL>(bc, cl);
                    const int first = reduced_first<CL, M>(cl);
                    float *dst = &sm.bc[s & 1][warp][0][0][0];
#pragma unroll
                    for (int r = 0; r < R; r += R < 4 ? R : 4) {
                        constexpr int P = R < 4 ? R : 4;
                        const int at = first + r;
                        store_packet<float, P>(dst + at / kStates * S::NP + n0 + at % kStates,
                                               pack<float, P>(bc + r));
                    }
                }
                __syncthreads();
                for (int i = tid; i < kSub * 2 * S::NP; i += S::NT) {
                    const int j = i / (2 * S::NP), which = i / S::NP % 2, m = i % S::NP;
                    const int t = s * kSub + j;
                    if (t >= n || m >= p.N) continue;
                    float v = 0.f;
#pragma unroll
                    for (int q = 0; q < S::NW; ++q) v += sm.bc[s & 1][q][j][which][m];
                    w.bc[((((long)(tile % gtiles) * p.T_total + t0 + tb + t) * p.G + g) * 2 + which) * p.N + m] = v;
                }
            };
            int sub = n4 / kSub - 1;
            if (n < n4) walk(sub--, std::true_type());
#pragma unroll 1
            for (; sub >= 0; --sub) walk(sub, std::false_type());
#pragma unroll
            for (int i = 0; i < kStates; ++i) dA[i] = fma2(dAc[i], make_pair(1.f, 1.f), dA[i]);
            // the last barrier above stands between the results in shared
            // memory and here
            if (qlive)
#pragma unroll
                for (int i = 0; i < Sm::PS; ++i) {
                    const int t = i * RS + row;
                    if (t >= n) break;
                    const long tok = t0 + tb + t;
                    float o[V], x[V];
                    auto q = load_packet<float, V>(&sm.u[t][qcol]);
                    unpack<float, V>(q, o);
                    store_packet<T, V>(static_cast<T *>(p.du) + tok * p.D + col, pack<T, V>(o));
                    q = load_packet<float, V>(&sm.delta[t][qcol]);
                    unpack<T, V>(Sm::kSlots == 2 ? sm.in_dt[r][i][tid]
                                                 : load_packet<T, V>(static_cast<const T *>(p.dt) + tok * p.ld_dt + col), x);
                    float sg[V];
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        o[v] = q.e[v];
                        x[v] += bias[v];
                    }
                    if (p.softplus) {
                        sigmoids<V>(x, sg);
#pragma unroll
                        for (int v = 0; v < V; ++v) o[v] *= sg[v];
                    }
#pragma unroll
                    for (int v = 0; v < V; ++v) dbias[v] += o[v];
                    store_packet<T, V>(static_cast<T *>(p.ddt) + tok * p.D + col, pack<T, V>(o));
                    if (p.z) {
                        float z[V];
                        q = load_packet<float, V>(&sm.e[t][qcol]);
                        unpack<T, V>(Sm::kSlots == 2 ? sm.in_dy[r][i][tid]
                                                     : load_packet<T, V>(static_cast<const T *>(p.dy) + tok * p.ld_dy + col), x);
                        unpack<T, V>(Sm::kSlots == 2 ? sm.in_z[r][i][tid]
                                                     : load_packet<T, V>(static_cast<const T *>(p.z) + tok * p.ld_z + col), z);
                        sigmoids<V>(z, sg);
#pragma unroll
                        for (int v = 0; v < V; ++v)
                            o[v] = x[v] * q.e[v] * (sg[v] * fmaf(z[v], 1.f - sg[v], 1.f));
                        store_packet<T, V>(static_cast<T *>(p.dz) + tok * p.D + col, pack<T, V>(o));
                    }
                }
            __syncthreads();
        }
        if (p.dh0 && it.tok0 == 0) store_pairs(p.dh0 + sbase, gc);
    }
    const long pbase = (long)slot * p.D;
    store_pairs(w.A + pbase * p.N, dA);
    // the threads of a column packet add up in order
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (row < kTokens) {                         // later rows hold no token
            sm.delta[row][qcol + v] = dD[v];
            sm.u[row][qcol + v] = dbias[v];
        }
    __syncthreads();
    for (int c = tid; c < S::CB; c += S::NT) {
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

// Sums what the blocks left, in order: dB, dC [rows, N] over the group's tiles
// (rows = T_total * G; nothing is written where malformed packed offsets left
// no slots, total_slots 0), then dA, dD_skip and ddt_bias over the blocks that
// shared a tile.
template <typename T>
__global__ void __launch_bounds__(256)
scan_reduce_kernel(const int32_t *total_slots, BwdPartials w, int gtiles, long rows, int D, int N,
                   T *dB, T *dC, float *dA, float *dD, float *dbias) {
    const long per = rows * 2 * N, dn = (long)D * N;
    const bool tokens = !total_slots || *total_slots != 0;
    for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < per + dn + 2L * D; i += (long)gridDim.x * 256) {
        float v = 0.f;
        if (i < per) {
            if (!tokens) continue;
#pragma unroll 4
            for (int k = 0; k < gtiles; ++k) v += w.bc[k * per + i];
            const long row = i / (2 * N);
            const int m = (int)(i - row * 2 * N);
            if (m < N) dB[row * N + m] = from_f32<T>(v);
            else dC[row * N + m - N] = from_f32<T>(v);
            continue;
        }
        const long q = i - per;
        const float *src = q < dn ? w.A + q : q < dn + D ? w.D + (q - dn) : w.bias + (q - dn - D);
        float *out = q < dn ? dA + q : q < dn + D ? dD : dbias;
        if (!out) continue;
        for (int s = 0; s < w.slots; ++s) v += src[s * (q < dn ? dn : D)];
        if (q < dn) *out = v;
        else out[q < dn + D ? q - dn : q - dn - D] = v;
    }
}

// The shapes by lanes per channel: 64 channels a block while eight warps allow.
template <int NL> struct BwdShape;
template <> struct BwdShape<2> { using S = Shape<2, 2, 2, 0>; };
template <> struct BwdShape<4> { using S = Shape<4, 2, 4, 0>; };
template <> struct BwdShape<8> { using S = Shape<8, 2, 4, 0>; };
template <> struct BwdShape<16> { using S = Shape<16, 2, 8, 0>; };
template <> struct BwdShape<32> { using S = Shape<32, 2, 8, 0>; };

int bwd_block_channels(int N) {
    switch (lanes_of_states(N)) {
        case 2: return BwdShape<2>::S::CB;
        case 4: return BwdShape<4>::S::CB;
        case 8: return BwdShape<8>::S::CB;
        case 16: return BwdShape<16>::S::CB;
        default: return BwdShape<32>::S::CB;
    }
}

int bwd_block_warps(int N) { return lanes_of_states(N) == 2 ? 2 : lanes_of_states(N) <= 8 ? 4 : 8; }

struct BwdPlan {
    long tiles, gtiles;
    int slots;
    Cut cut;
    size_t base, bc, A, D, bytes; // bytes of each part, and of the whole workspace
};
BwdPlan bwd_plan(int n_seq, int T_total, int D, int G, int N, bool packed) {
    BwdPlan b;
    const int Dg = D / G, CB = bwd_block_channels(N);
    b.gtiles = (Dg + CB - 1) / CB;
    b.tiles = b.gtiles * G;
    // an SM holds eight warps of any shape
    const long held = 152L * (8 / bwd_block_warps(N));
    b.cut = packed ? choose_cut(T_total, D, N)
                   : choose_even_cut(n_seq ? T_total / n_seq : 0, b.tiles * n_seq, held);
    const long items = packed ? n_seq + (T_total > b.cut.trigger ? T_total / b.cut.cut : 0)
                              : (long)n_seq * (n_seq ? segments_of(T_total / n_seq, b.cut.cut, b.cut.trigger) : 0);
    // a block for every item, as far as two waves of blocks go: every block
    // leaves partial sums.  In us with those, with two waves and with eight:
    // 2048 sequences of 64 tokens, 256 channels, 668 and 706; 100 packed ones of
    // 16000 tokens, 1024 channels, 330 and 340; 32 of 12000, 2048, 480 and 493
    b.slots = (int)std::max(1L, std::min(items, (2 * held + b.tiles - 1) / b.tiles));
    b.base = layout_bytes(n_seq, T_total, D, N, b.cut, packed, false);
    b.bc = round256((size_t)b.gtiles * T_total * G * 2 * N * sizeof(float));
    b.A = round256((size_t)b.slots * D * N * sizeof(float));
    b.D = round256((size_t)b.slots * D * sizeof(float));
    b.bytes = b.base + b.bc + b.A + 2 * b.D;
    return b;
}

template <typename T, typename S, int V, Pad PAD>
cudaError_t bwd_launch(const ScanProblem &p, const Layout &l, const BwdPartials &w, const BwdPlan &b,
                       cudaStream_t st) {
    const long blocks = b.tiles * w.slots;
    if (blocks > 0x7fffffffL) return cudaErrorInvalidConfiguration;
    constexpr int bytes = (int)sizeof(BwdSmem<T, S, V>);
    const cudaError_t err = allow_shared<scan_bwd_kernel<T, S, V, PAD>>(bytes);
    if (err != cudaSuccess) return err;
    scan_bwd_kernel<T, S, V, PAD><<<(unsigned)blocks, S::NT, bytes, st>>>(p, l, w, (int)b.tiles);
    return cudaGetLastError();
}
template <typename T, typename S, int V>
cudaError_t bwd_t(const ScanProblem &p, const Layout &l, const BwdPartials &w, const BwdPlan &b,
                  cudaStream_t st) {
    switch (pad_of(p.N)) {
        case Pad::kNone: return bwd_launch<T, S, V, Pad::kNone>(p, l, w, b, st);
        case Pad::kLanes: return bwd_launch<T, S, V, Pad::kLanes>(p, l, w, b, st);
        default: return bwd_launch<T, S, V, Pad::kStates>(p, l, w, b, st);
    }
}

template <typename T>
cudaError_t bwd_dispatch(const ScanProblem &p, const Layout &l, const BwdPartials &w,
                         const BwdPlan &b, cudaStream_t st) {
    constexpr int MOST = 16 / (int)sizeof(T);
    const int V = packet_width(MOST, sizeof(T), [&](int v, int bytes) {
        bool ok = (p.D / p.G) % v == 0 && rows_aligned(p.u, p.ld_u, sizeof(T), bytes) &&
                  rows_aligned(p.dt, p.ld_dt, sizeof(T), bytes) &&
                  rows_aligned(p.z, p.ld_z, sizeof(T), bytes) &&
                  rows_aligned(p.dy, p.ld_dy, sizeof(T), bytes);
        const void *dense[] = {p.du, p.ddt, p.dz};
        for (const void *ptr : dense) ok = ok && rows_aligned(ptr, p.D, sizeof(T), bytes);
        return ok;
    });
    cudaError_t err = cudaErrorInvalidValue;
#define MDN_SCAN_CASE(NL)                                                    \
    case NL:                                                                 \
        if (V == MOST) err = bwd_t<T, BwdShape<NL>::S, MOST>(p, l, w, b, st); \
        else if (V == 2) err = bwd_t<T, BwdShape<NL>::S, sizeof(T) == 2 ? 2 : 1>(p, l, w, b, st); \
        else err = bwd_t<T, BwdShape<NL>::S, 1>(p, l, w, b, st);             \
        break;
    switch (lanes_of_states(p.N)) {
        MDN_SCAN_CASE(2)
        MDN_SCAN_CASE(4)
        MDN_SCAN_CASE(8)
        MDN_SCAN_CASE(16)
        MDN_SCAN_CASE(32)
    }
#undef MDN_SCAN_CASE
    if (err != cudaSuccess) return err;
    const long rows = (long)p.T_total * p.G;
    const long blocks = (rows * 2 * p.N + (long)p.D * (p.N + 2) + 255) / 256;
    scan_reduce_kernel<T><<<(unsigned)std::min(blocks, 152L * 8), 256, 0, st>>>(
        l.slot_off ? l.slot_off + p.n_seq : nullptr, w, (int)b.gtiles, rows, p.D, p.N,
        static_cast<T *>(p.dB), static_cast<T *>(p.dC), p.dA, p.dD, p.ddt_bias);
    return cudaGetLastError();
}

}  // namespace
}  // namespace scan

size_t scan_bwd_workspace(int n_seq, int T_total, int D, int G, int N, mdn_dtype dtype) {
    // which of the two a call is, its sizes do not tell
    return std::max(scan::bwd_plan(n_seq, T_total, D, G, N, true).bytes,
                    scan::bwd_plan(n_seq, T_total, D, G, N, false).bytes);
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
    const scan::BwdPlan b = scan::bwd_plan(p.n_seq, p.T_total, p.D, p.G, p.N, p.cu != nullptr);
    scan::Layout l;
    cudaError_t err = scan::make_layout(p, b.cut, l, st);
    if (err == cudaSuccess) err = scan::launch_adjoint_ends(p, l, st);
    if (err != cudaSuccess) return err;
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
