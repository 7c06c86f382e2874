// Selective state-space scan: forward over whole sequences, and the
// single-token step.
//
//   delta_t = softplus(dt_t + dt_bias);   a_t[n] = exp(delta_t A[n])
//   h_t[n]  = a_t[n] h_{t-1}[n] + delta_t u_t B_t[n]
//   y_t     = (sum_n C_t[n] h_t[n] + D_skip u_t) silu(z_t)
//
// A depends on channel and state, so the decays a_t[n] do not factor into
// products of matrices: each (token, channel, state) takes one exponential and
// four multiplications or fma on the CUDA cores.  At 16 states that is more
// time than the bytes: 32768 tokens of 2048 channels cost 1.07 G exponentials,
// 113 us at the measured 62 a nanosecond and SM, against 80 us for 541 MB.
//
// Measured, bf16, 16 states: 32768 packed tokens of 2048 channels 357 us
// (3.0 T exponentials a second, 0.31 of that rate); one sequence of 16384
// tokens 176 us and 107 us for its first pass.  Bound by issue (70 % of the
// slots) and the shared-memory pipe (75 %): delta, delta u, B and C come from
// there for every token.  Four channels a lane instead of two read B and C
// half as often but leave fewer warps: 365 us, and 190 to 215 for 176.
#include <algorithm>

#include "mdn_scan.cuh"

namespace mdn {
namespace scan {
namespace {

// ------------------------------------------------------------------ layout

// One block: checks cu_seqlens, writes the first saved-state slot of each
// sequence (chunks of kTokens from its own start) and the tables of items,
// sequences longest first (for up to kMaxOrdered of them).  A malformed array
// sets the status word and leaves one empty item per sequence.
constexpr int kMaxOrdered = 1024;

__device__ __forceinline__ int block_scan(int mine, int32_t *part, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    int before = 0;
    total = 0;
    for (int w = 0; w < (int)blockDim.x >> 5; ++w) {
        if (w < warp) before += part[w];
        total += part[w];
    }
    __syncthreads();
    return before + incl - mine;
}

__global__ void __launch_bounds__(1024)
layout_kernel(const int32_t *cu, int n_seq, int T_total, int cut, int trigger, int32_t *off,
              int32_t *order, Item *item, Item *pre_item, int32_t *count, int *status) {
    __shared__ int32_t part[32];
    if (!cu_well_formed(cu, n_seq, T_total)) {
        for (int s = threadIdx.x; s <= n_seq; s += blockDim.x) {
            off[s] = 0;
            if (s < n_seq) item[s] = Item{s, 0, 0, 0};
        }
        if (threadIdx.x == 0) {
            count[0] = n_seq;
            count[1] = 0;
            atomicExch(status, (int)MDN_ERR_INVALID_ARG);
        }
        return;
    }
    int slots = 0;
    for (int base = 0; base < n_seq; base += blockDim.x) {
        const int s = base + threadIdx.x;
        int total;
        const int at = block_scan(s < n_seq ? (cu[s + 1] - cu[s] + kTokens - 1) / kTokens : 0, part, total);
        if (s < n_seq) {
            off[s] = slots + at;
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
        slots += total;
    }
    if (threadIdx.x == 0) off[n_seq] = slots;
    __syncthreads();
    int items = 0, pres = 0;
    for (int base = 0; base < n_seq; base += blockDim.x) {
        const int r = base + threadIdx.x;
        int s = 0, len = 0, segs = 0, total, pre_total;
        if (r < n_seq) {
            s = order[r];
            len = cu[s + 1] - cu[s];
            segs = segments_of(len, cut, trigger);
        }
        const int at = items + block_scan(segs, part, total);
        const int pre = pres + block_scan(segs > 0 ? segs - 1 : 0, part, pre_total);
        for (int k = 0; k < segs; ++k) {
            const Item it{s, k * cut, segs == 1 ? len : min(cut, len - k * cut), pre};
            item[at + k] = it;
            if (k < segs - 1) pre_item[pre + k] = it;
        }
        items += total;
        pres += pre_total;
    }
    if (threadIdx.x == 0) {
        count[0] = items;
        count[1] = pres;
    }
}

// ----------------------------------------------------------------- forward

constexpr int kStage = 16;            // tokens per stage
enum class Pass { kMain, kEnds, kAdjoint };
constexpr int kAhead = 1;             // stages whose copies are in flight
constexpr int kRing = kAhead + 3;     // staged, in flight, and waiting for their outputs

template <typename T, typename S, int V>
struct FwdSmem {
    static constexpr int QC = S::CB / V;                                   // packets per token
    static constexpr int PS = (kStage * QC + S::HT - 1) / S::HT;           // packets per helper
    static constexpr int QB = S::NP / 4;
    static constexpr int PB = (kStage * QB + S::HT - 1) / S::HT;           // of B, of C
    static_assert(S::HT % QC == 0, "a helper keeps its columns");
    float delta[2][kStage][S::CB];
    float du[2][kStage][S::CB];       // delta u, then sum_n C h of the same token
    float B[2][kStage][S::NP], C[2][kStage][S::NP];
    // the inputs as they are, one place for each packet of each helper
    Slot<T, V> u[kRing][PS][S::HT], dt[kRing][PS][S::HT], z[kRing][PS][S::HT];
    Packet<T, 4> b[kRing][PB][S::HT], c[kRing][PB][S::HT];
};

// One block takes CB channels of one group through one item, in stages of
// kStage tokens with two buffers: while the recurrence warps run a stage, the
// helper warps finish the outputs of the stage before and turn the inputs of
// the next into fp32 delta and delta u.  A helper copies the packets it will
// use itself, kAhead stages early, so that only it has to wait for them.
// kEnds: the first pass over a cut segment, whose end state and sum of delta are
// all it leaves.  kAdjoint: the same for the gradient's adjoint of the state,
// which runs through the tokens last first, r <- a_t (r + C_t e_t).  Neither adds
// up states, so neither cares for PAD.
template <typename T, typename S, int V, Pass PASS, Pad PAD>
__global__ void __launch_bounds__(S::NT + S::HT, S::NT + S::HT <= 256 ? 3 : 2)
scan_fwd_kernel(ScanProblem p, Layout l, int tiles) {
    using Sm = FwdSmem<T, S, V>;
    constexpr bool PRE = PASS != Pass::kMain, REV = PASS == Pass::kAdjoint;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Sm &sm = *reinterpret_cast<Sm *>(smem_raw);
    const int Dg = p.D / p.G;
    const int gtiles = tiles / p.G;
    const int tile = blockIdx.x % tiles;
    const int g = tile / gtiles;
    const int c0 = (tile % gtiles) * S::CB;          // first channel, within the group
    const long d0 = (long)g * Dg + c0;
    Item it;
    long t0, slot0;
    if (!find_item<PASS != Pass::kMain, REV>(p, l, blockIdx.x / tiles, it, t0, slot0)) return;
    const int stages = (it.len + kStage - 1) / kStage;

    if (threadIdx.x >= S::NT) {
        // ---------------------------------------------------------- helpers
        const int hid = threadIdx.x - S::NT;
        const int row = hid / Sm::QC, col = hid % Sm::QC * V;
        constexpr int RS = S::HT / Sm::QC;               // tokens between a helper's packets
        const bool qlive = c0 + col < Dg;
        // the adjoint has dy and C where the state has u and B
        const long ld_u = REV ? p.ld_dy : p.ld_u, ld_B = REV ? p.ld_C : p.ld_B;
        const T *up = static_cast<const T *>(REV ? p.dy : p.u) + t0 * ld_u + d0 + col;
        const T *dp = static_cast<const T *>(p.dt) + t0 * p.ld_dt + d0 + col;
        const T *zp = p.z ? static_cast<const T *>(p.z) + t0 * p.ld_z + d0 + col : nullptr;
        const T *Bp = static_cast<const T *>(REV ? p.Cm : p.Bm) + t0 * ld_B + (long)g * p.N;
        const T *Cp = static_cast<const T *>(p.Cm) + t0 * p.ld_C + (long)g * p.N;
        T *yp = static_cast<T *>(p.y) + t0 * p.D + d0 + col;
        float bias[V], skip[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            bias[v] = qlive && p.dt_bias ? p.dt_bias[d0 + col + v] : 0.f;
            skip[v] = qlive && p.D_skip ? p.D_skip[d0 + col + v] : 0.f;
        }
        const Span<T> us = span_of<T>(REV ? p.dy : p.u, p.T_total, ld_u, p.D);
        const Span<T> ds = span_of<T>(p.dt, p.T_total, p.ld_dt, p.D);
        const Span<T> zs = span_of<T>(p.z, p.T_total, p.ld_z, p.D);
        auto issue = [&](int k) {
            const int tk = (REV ? stages - 1 - k : k) * kStage, n = it.len - tk, r = k % kRing;
            if (k < stages) {
#pragma unroll
                for (int i = 0; i < Sm::PS; ++i) {
                    const int t = i * RS + row;
                    if (t < n && t < kStage && qlive) {
                        copy_slot<T, V>(&sm.u[r][i][hid], up + (long)(tk + t) * ld_u, us);
                        copy_slot<T, V>(&sm.dt[r][i][hid], dp + (long)(tk + t) * p.ld_dt, ds);
                        if ((!PRE || REV) && zp)
                            copy_slot<T, V>(&sm.z[r][i][hid], zp + (long)(tk + t) * p.ld_z, zs);
                    }
                }
#pragma unroll
                for (int i = 0; i < Sm::PB; ++i) {
                    const int j = i * S::HT + hid, t = j / Sm::QB, m = j % Sm::QB * 4;
                    if (t >= n || t >= kStage || m >= p.N) continue;
                    const T *bp = Bp + (long)(tk + t) * ld_B + m, *cp = Cp + (long)(tk + t) * p.ld_C + m;
                    if (p.bc_wide) {
                        copy_packet<T, 4>(&sm.b[r][i][hid], bp);
                        if (!PRE) copy_packet<T, 4>(&sm.c[r][i][hid], cp);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            sm.b[r][i][hid].e[e] = m + e < p.N ? bp[e] : from_f32<T>(0.f);
                            if (!PRE) sm.c[r][i][hid].e[e] = m + e < p.N ? cp[e] : from_f32<T>(0.f);
                        }
                    }
                }
            }
            commit_copies();
        };
#pragma unroll
        for (int k = 0; k < kAhead; ++k) issue(k);
        // round -1 only stages stage 0, round `stages` only finishes the last
        for (int k = -1; k <= stages; ++k) {
            issue(k + 1 + kAhead);
            const int nb = (k + 1) & 1;                      // the next stage's buffer
            if (!PRE && k >= 1 && qlive) {
                const int tk = (k - 1) * kStage, n = min(kStage, it.len - tk), r = (k - 1) % kRing;
#pragma unroll
                for (int i = 0; i < Sm::PS; ++i) {
                    const int t = i * RS + row;
                    if (t >= n) break;
                    float u[V], z[V], o[V];
                    unpack_slot<T, V>(sm.u[r][i][hid], up + (long)(tk + t) * ld_u, u);
                    if (zp) unpack_slot<T, V>(sm.z[r][i][hid], zp + (long)(tk + t) * p.ld_z, z);
                    const auto sum = load_packet<float, V>(&sm.du[nb][t][col]);
#pragma unroll
                    for (int v = 0; v < V; ++v) o[v] = fmaf(skip[v], u[v], sum.e[v]);
                    if (zp) apply_gate<V>(o, z);
                    store_packet<T, V>(yp + (long)(tk + t) * p.D, pack<T, V>(o));
                }
            }
            wait_copies<kAhead>();
            if (k + 1 < stages) {
                const int tk = (REV ? stages - 2 - k : k + 1) * kStage;
                const int n = min(kStage, it.len - tk), r = (k + 1) % kRing;
                const int n_zero = (n + S::TB - 1) / S::TB * S::TB;     // zeros up to a whole batch
#pragma unroll
                for (int i = 0; i < Sm::PS; ++i) {
                    const int t = i * RS + row;
                    if (t >= n_zero) break;
                    float u[V], d[V];
#pragma unroll
                    for (int v = 0; v < V; ++v) u[v] = d[v] = 0.f;
                    if (qlive && t < n) {
                        unpack_slot<T, V>(sm.u[r][i][hid], up + (long)(tk + t) * ld_u, u);
                        unpack_slot<T, V>(sm.dt[r][i][hid], dp + (long)(tk + t) * p.ld_dt, d);
                        step_sizes<V>(d, bias, p.softplus);
                        if (!REV) {
#pragma unroll
                            for (int v = 0; v < V; ++v) u[v] *= d[v];
                        } else if (zp) {
                            float z[V];
                            unpack_slot<T, V>(sm.z[r][i][hid], zp + (long)(tk + t) * p.ld_z, z);
                            apply_gate<V>(u, z);
                        }
                    }
                    store_packet<float, V>(&sm.delta[nb][t][col], pack<float, V>(d));
                    store_packet<float, V>(&sm.du[nb][t][col], pack<float, V>(u));
                }
#pragma unroll
                for (int i = 0; i < Sm::PB; ++i) {
                    const int j = i * S::HT + hid, t = j / Sm::QB, m = j % Sm::QB * 4;
                    if (t >= n_zero) break;
                    const bool in = t < n && m < p.N;
                    float f[4] = {0.f, 0.f, 0.f, 0.f};
                    if (in) unpack<T, 4>(sm.b[r][i][hid], f);
                    store_packet<float, 4>(&sm.B[nb][t][m], pack<float, 4>(f));
                    if (PRE) continue;
                    if (in) unpack<T, 4>(sm.c[r][i][hid], f);
                    store_packet<float, 4>(&sm.C[nb][t][m], pack<float, 4>(f));
                }
            }
            if (k < stages) __syncthreads();
        }
        wait_copies<0>();
        return;
    }
    // ------------------------------------------------------------ recurrence
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nl = lane % S::NL, n0 = nl * kStates;
    const int cw = warp * S::WC + lane / S::NL * S::CPT;     // lane's first channel in the block
    // two neighbouring states to a pair (two channels instead, whose B and C
    // are scalars, cost 110 us where this costs 107, in the first pass)
    Pair a2[S::CPT][kStates / 2], h[S::CPT][kStates / 2];
    float sum[S::CPT];
    bool live[S::CPT];
    bool in[kStates];                    // of the lane's states, the real ones
#pragma unroll
    for (int i = 0; i < kStates; ++i) in[i] = n0 + i < p.N;
    {
        // a cut sequence's initial state, if its final state takes its place
        float *kept = l.pre_h0 + (long)it.pre * p.D * p.N;
        const bool cut = !PRE && l.pre_h0 && it.len > 0 &&
                         it.len < (p.cu ? p.cu[it.seq + 1] - p.cu[it.seq] : p.T);
        const float *h0 = cut ? kept : p.h0 + (long)it.seq * p.D * p.N;
        float a[S::CPT][kStates], s0[S::CPT][kStates];
#pragma unroll
        for (int c = 0; c < S::CPT; ++c) {
            live[c] = c0 + cw + c < Dg && n0 < p.N;
            sum[c] = 0.f;
#pragma unroll
            for (int i = 0; i < kStates; ++i) a[c][i] = s0[c][i] = 0.f;
            if (live[c]) {
                load_states(p.A, d0 + cw + c, n0, p.N, a[c]);
                if (!PRE && p.h0) load_states(h0, d0 + cw + c, n0, p.N, s0[c]);
                if (PASS == Pass::kEnds && l.pre_h0 && it.tok0 == 0) {
                    float keep[kStates];
                    load_states(h0, d0 + cw + c, n0, p.N, keep);
                    store_states(kept, d0 + cw + c, n0, p.N, keep);
                }
            }
#pragma unroll
            for (int i = 0; i < kStates; ++i) a[c][i] = decay_rate(a[c][i]);
            if (!PRE && live[c]) {
                // the state before this segment, through those before it
                const int before = it.tok0 / l.cut;
#pragma unroll 4
                for (int k = 0; k < before; ++k) {
                    float end[kStates];
                    load_states(l.pre_h + (long)(it.pre + k) * p.D * p.N, d0 + cw + c, n0, p.N, end);
                    const float s = l.pre_sum[(long)(it.pre + k) * p.D + d0 + cw + c];
#pragma unroll
                    for (int i = 0; i < kStates; ++i) s0[c][i] = through_segment(s * a[c][i], s0[c][i], end[i]);
                }
            }
        }
#pragma unroll
        for (int c = 0; c < S::CPT; ++c)
#pragma unroll
            for (int i = 0; i < kStates / 2; ++i) {
                a2[c][i] = make_pair(a[c][2 * i], a[c][2 * i + 1]);
                h[c][i] = make_pair(s0[c][2 * i], s0[c][2 * i + 1]);
            }
    }
    auto store_h = [&](float *base) {
#pragma unroll
        for (int c = 0; c < S::CPT; ++c) {
            float x[kStates];
#pragma unroll
            for (int i = 0; i < kStates / 2; ++i) split_pair(h[c][i], x[2 * i], x[2 * i + 1]);
            if (live[c]) store_states(base, d0 + cw + c, n0, p.N, x);
        }
    };
    __syncthreads();
    for (int k = 0; k < stages; ++k) {
        const int buf = k & 1;
        const int n = min(kStage, it.len - (REV ? stages - 1 - k : k) * kStage);
        if (!PRE && p.h_chunks && k * kStage % kTokens == 0)
            store_h(p.h_chunks + (slot0 + k * kStage / kTokens) * p.D * p.N);
        // tokens past n are zero and change nothing
#pragma unroll 1
        for (int step = 0; step < n; step += S::TB) {
            const int t = REV ? (n - 1) / S::TB * S::TB - step : step;
            // every input of the batch first: the sums go back into du, which
            // would hold up loads of later tokens behind them
            Packet<float, kStates> bv[S::TB], cv[S::TB];
            Packet<float, S::CPT> dl[S::TB], du[S::TB];
#pragma unroll
            for (int j = 0; j < S::TB; ++j) {
                bv[j] = load_packet<float, kStates>(&sm.B[buf][t + j][n0]);
                if (!PRE) cv[j] = load_packet<float, kStates>(&sm.C[buf][t + j][n0]);
                dl[j] = load_packet<float, S::CPT>(&sm.delta[buf][t + j][cw]);
                du[j] = load_packet<float, S::CPT>(&sm.du[buf][t + j][cw]);
            }
            float acc[S::TB * S::CPT];
#pragma unroll
            for (int jj = 0; jj < S::TB; ++jj) {
                const int j = REV ? S::TB - 1 - jj : jj;
#pragma unroll
                for (int c = 0; c < S::CPT; ++c) {
                    const float dc = dl[j].e[c], duc = du[j].e[c];
                    if (PRE) sum[c] += dc;
                    Pair y;
#pragma unroll
                    for (int i = 0; i < kStates / 2; ++i) {
                        const Pair b = make_pair(bv[j].e[2 * i], bv[j].e[2 * i + 1]);
                        float e0, e1;
                        split_pair(fma2(make_pair(dc, dc), a2[c][i], make_pair(kDecayBias, kDecayBias)), e0, e1);
                        const Pair a = make_pair(ex2(e0), ex2(e1));
                        if (REV) {
                            h[c][i] = mul2(a, fma2(make_pair(duc, duc), b, h[c][i]));
                            continue;
                        }
                        h[c][i] = fma2(a, h[c][i], mul2(make_pair(duc, duc), b));
                        if (PAD == Pad::kStates) h[c][i] = real_states(h[c][i], in[2 * i], in[2 * i + 1]);
                        if (!PRE) {
                            const Pair cc = make_pair(cv[j].e[2 * i], cv[j].e[2 * i + 1]);
                            y = i ? fma2(h[c][i], cc, y) : mul2(h[c][i], cc);
                        }
                    }
                    if (PRE) continue;
                    float y0, y1;
                    split_pair(y, y0, y1);
                    acc[j * S::CPT + c] = PAD != Pad::kLanes || in[0] ? y0 + y1 : 0.f;
                }
            }
            if (!PRE) {
                constexpr int M = S::TB * S::CPT, R = M > S::NL ? M / S::NL : 1;
                static_assert(R <= S::CPT, "a lane's sums belong to one token");
                reduce_lanes<S::NL, M>(acc, nl);
                const int first = reduced_first<S::NL, M>(nl);
                if (S::NL <= M || nl < M)
                    store_packet<float, R>(&sm.du[buf][t + first / S::CPT][cw + first % S::CPT],
                                           pack<float, R>(acc));
            }
        }
        __syncthreads();
    }
    // a first pass's slot: segments 0 .. of the states, 1 .. of the adjoints
    const long pre_slot = (long)it.pre + it.tok0 / l.cut - (REV ? 1 : 0);
    float *out = PRE ? l.pre_h + pre_slot * p.D * p.N
                     : p.h_T + (long)it.seq * p.D * p.N;
    // only the item that ends the sequence knows its final state
    const int seq_len = p.cu ? p.cu[it.seq + 1] - p.cu[it.seq] : p.T;
    if (PRE || (p.h_T && (it.len == 0 || it.tok0 + it.len == seq_len))) store_h(out);
    if (PRE && nl == 0)
#pragma unroll
        for (int c = 0; c < S::CPT; ++c)
            if (c0 + cw + c < Dg)
                l.pre_sum[pre_slot * p.D + d0 + cw + c] = sum[c];
}

template <typename T, typename S, int V, Pass PASS, Pad PAD = Pad::kNone>
cudaError_t fwd_launch(const ScanProblem &p, const Layout &l, int blocks_per_tile, cudaStream_t st) {
    if (blocks_per_tile == 0) return cudaSuccess;
    const int Dg = p.D / p.G;
    const long tiles = (long)p.G * ((Dg + S::CB - 1) / S::CB);
    if (tiles * blocks_per_tile > 0x7fffffffL) return cudaErrorInvalidConfiguration;
    constexpr int bytes = (int)sizeof(FwdSmem<T, S, V>);
    const cudaError_t err = allow_shared<scan_fwd_kernel<T, S, V, PASS, PAD>>(bytes);
    if (err != cudaSuccess) return err;
    scan_fwd_kernel<T, S, V, PASS, PAD>
        <<<(unsigned)(tiles * blocks_per_tile), S::NT + S::HT, bytes, st>>>(p, l, (int)tiles);
    return cudaGetLastError();
}

template <typename T, typename S, int V>
cudaError_t fwd_t(const ScanProblem &p, const Layout &l, Pass pass, cudaStream_t st) {
    if (pass == Pass::kAdjoint) return fwd_launch<T, S, V, Pass::kAdjoint>(p, l, l.pres, st);
    const cudaError_t err = fwd_launch<T, S, V, Pass::kEnds>(p, l, l.pres, st);
    if (err != cudaSuccess) return err;
    switch (pad_of(p.N)) {
        case Pad::kNone: return fwd_launch<T, S, V, Pass::kMain, Pad::kNone>(p, l, l.items, st);
        case Pad::kLanes: return fwd_launch<T, S, V, Pass::kMain, Pad::kLanes>(p, l, l.items, st);
        default: return fwd_launch<T, S, V, Pass::kMain, Pad::kStates>(p, l, l.items, st);
    }
}

template <typename T>
cudaError_t fwd_dispatch(const ScanProblem &p, const Layout &l, Pass pass, cudaStream_t st) {
    // 16-byte packets (or pairs of two-byte elements) where every row starts on
    // a packet's boundary, single elements otherwise
    constexpr int MOST = 16 / (int)sizeof(T);
    const int V = packet_width(MOST, sizeof(T), [&](int v, int bytes) {
        return (p.D / p.G) % v == 0 && rows_aligned(p.u, p.ld_u, sizeof(T), bytes) &&
               rows_aligned(p.dt, p.ld_dt, sizeof(T), bytes) &&
               rows_aligned(p.z, p.ld_z, sizeof(T), bytes) &&
               rows_aligned(p.y, p.D, sizeof(T), bytes) && rows_aligned(p.dy, p.ld_dy, sizeof(T), bytes);
    });
    // Four channels a lane above 32 states.  Forward in us with those and with
    // two, bf16: 8192 tokens of 2048 channels, 64 states 292 and 335, 128 states
    // 581 and 599 (fp32 661 and 739).  Where blocks are few, two are the better
    // ones: 2048 tokens of 256 channels, 40 and 37, 93 and 63.
#define MDN_SCAN_CASE(NL, CPT, NW, HW)                                \
    case NL:                                                          \
        if (V == MOST) return fwd_t<T, Shape<NL, CPT, NW, HW>, MOST>(p, l, pass, st); \
        if constexpr (sizeof(T) == 2)                                 \
            if (V == 2) return fwd_t<T, Shape<NL, CPT, NW, HW>, 2>(p, l, pass, st); \
        return fwd_t<T, Shape<NL, CPT, NW, HW>, 1>(p, l, pass, st);
    switch (lanes_of_states(p.N)) {
        MDN_SCAN_CASE(2, 2, 2, 4)
        MDN_SCAN_CASE(4, 2, 4, 4)
        MDN_SCAN_CASE(8, 2, 8, 4)
        MDN_SCAN_CASE(16, 4, 8, 4)
        MDN_SCAN_CASE(32, 4, 8, 4)
    }
#undef MDN_SCAN_CASE
    return cudaErrorInvalidValue;
}

// -------------------------------------------------------------------- step

constexpr int kStepWarps = 4;

// Memory bound by the states, read and written once.  A warp takes 32
// channels of one group and sequence: lane j prepares channel j's delta and
// delta u once, the states then pass in steps of 32 / NL channels (whole
// lines), K of them in flight, and the exchange that adds up a channel's
// states leaves each owner lane one channel's output to finish.  The first K
// steps' states are asked for before anything else and every other input with
// them, so that a warp waits for memory once.  256 sequences of 2048 channels
// and 16 states: 12.7 us, 71 MB at 5.6 TB/s (10.5 us at a copy's rate); 15.5 us
// with the states behind the deltas and the gates behind the sums.  Warps that
// took several sequences one after another took 20 to 34 us.
template <typename T, int NL, Pad PAD>
__global__ void __launch_bounds__(32 * kStepWarps) scan_step_kernel(ScanProblem p, int tiles) {
    constexpr int CL = 32 / NL, K = NL < 4 ? NL : 4, STEPS = NL;
    const int lane = threadIdx.x & 31;
    const int tile = blockIdx.x * kStepWarps + (threadIdx.x >> 5);
    if (tile >= tiles) return;
    const int Dg = p.D / p.G, gtiles = tiles / p.G;
    const int g = p.G == 1 ? 0 : tile / gtiles;
    const int c0 = (tile - g * gtiles) * 32;         // first channel, within the group
    const int d0 = g * Dg + c0;
    const long s = blockIdx.y;
    const int nl = lane % NL, cl = lane / NL, n0 = nl * kStates;
    constexpr bool whole = PAD != Pad::kStates;
    const T *up = static_cast<const T *>(p.u) + s * p.ld_u + d0;
    const T *zp = static_cast<const T *>(p.z) + s * p.ld_z + d0;
    const float *hp = p.h0 + (s * p.D + d0) * p.N, *ap = p.A + (long)d0 * p.N;
    float *ho = p.h_T + (s * p.D + d0) * p.N;
    // the states of the K steps from st on
    float h[K][kStates], a[K][kStates];
    auto load = [&](int st) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int ch = (st + k) * CL + cl;
#pragma unroll
            for (int i = 0; i < kStates; ++i) h[k][i] = a[k][i] = 0.f;
            if (c0 + ch >= Dg || n0 >= p.N) continue;
            if (whole) {
                const float4 v = __ldcs(reinterpret_cast<const float4 *>(hp + ch * p.N + n0));
                h[k][0] = v.x; h[k][1] = v.y; h[k][2] = v.z; h[k][3] = v.w;
                unpack<float, kStates>(load_packet<float, kStates>(ap + ch * p.N + n0), a[k]);
            } else {
                load_states(hp, ch, n0, p.N, h[k]);
                load_states(ap, ch, n0, p.N, a[k]);
            }
        }
    };
    load(0);
    // lane j's channel c0 + j
    float delta = 0.f, du = 0.f, u = 0.f, skip = 0.f, gate = 0.f;
    if (c0 + lane < Dg) {
        u = to_f32(up[lane]);
        delta = to_f32(static_cast<const T *>(p.dt)[s * p.ld_dt + d0 + lane]);
        if (p.D_skip) skip = p.D_skip[d0 + lane];
        if (p.z) gate = to_f32(zp[lane]);
        if (p.dt_bias) delta += p.dt_bias[d0 + lane];
    }
    float b[kStates] = {0.f, 0.f, 0.f, 0.f}, c[kStates] = {0.f, 0.f, 0.f, 0.f};
    if (n0 < p.N) {
        const T *bp = static_cast<const T *>(p.Bm) + s * p.ld_B + g * p.N + n0;
        const T *cp = static_cast<const T *>(p.Cm) + s * p.ld_C + g * p.N + n0;
        if (p.bc_wide) {
            unpack<T, kStates>(load_packet<T, kStates>(bp), b);
            unpack<T, kStates>(load_packet<T, kStates>(cp), c);
        } else {
#pragma unroll
            for (int i = 0; i < kStates; ++i)
                if (n0 + i < p.N) {
                    b[i] = to_f32(bp[i]);
                    c[i] = to_f32(cp[i]);
                }
        }
    }
    if (p.softplus) delta = softplus_rel(delta);
    du = delta * u;
    gate *= sigmoid_f(gate);
#pragma unroll 1
    for (int st = 0; st < STEPS; st += K) {
        float acc[K];
        if (st > 0) load(st);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int ch = (st + k) * CL + cl;
            const float dk = __shfl_sync(0xffffffffu, delta, ch), duk = __shfl_sync(0xffffffffu, du, ch);
            acc[k] = 0.f;
#pragma unroll
            for (int i = 0; i < kStates; ++i) {
                h[k][i] = fmaf(ex2(fmaf(dk, decay_rate(a[k][i]), kDecayBias)), h[k][i], duk * b[i]);
                if (PAD != Pad::kStates || n0 + i < p.N) acc[k] = fmaf(h[k][i], c[i], acc[k]);
            }
            if (PAD == Pad::kLanes && n0 >= p.N) acc[k] = 0.f;
            if (c0 + ch >= Dg || n0 >= p.N) continue;
            if (whole) __stcs(reinterpret_cast<float4 *>(ho + ch * p.N + n0), make_float4(h[k][0], h[k][1], h[k][2], h[k][3]));
            else store_states(ho, ch, n0, p.N, h[k]);
        }
        reduce_lanes<NL, K>(acc, nl);
        const int ch = (st + reduced_first<NL, K>(nl)) * CL + cl;
        float y = acc[0];
        const float su = __shfl_sync(0xffffffffu, u, ch), sd = __shfl_sync(0xffffffffu, skip, ch);
        const float sg = __shfl_sync(0xffffffffu, gate, ch);
        if (p.D_skip) y = fmaf(sd, su, y);
        if (p.z) y *= sg;
        if (nl < K && c0 + ch < Dg) static_cast<T *>(p.y)[s * p.D + d0 + ch] = from_f32<T>(y);
    }
}

template <typename T, int NL>
cudaError_t step_t(const ScanProblem &p, cudaStream_t st) {
    const int tiles = p.G * ((p.D / p.G + 31) / 32);
    const unsigned blocks = (unsigned)((tiles + kStepWarps - 1) / kStepWarps);
    // the grid's second dimension ends at 65535
    for (long s0 = 0; s0 < p.n_seq; s0 += 65535L) {
        ScanProblem q = p;
        auto rows = [&](const void *x, long ld) -> const void * {
            return x ? static_cast<const T *>(x) + s0 * ld : nullptr;
        };
        q.u = rows(p.u, p.ld_u);
        q.dt = rows(p.dt, p.ld_dt);
        q.z = rows(p.z, p.ld_z);
        q.Bm = rows(p.Bm, p.ld_B);
        q.Cm = rows(p.Cm, p.ld_C);
        q.y = const_cast<void *>(rows(p.y, p.D));
        q.h0 = p.h0 + s0 * p.D * p.N;
        q.h_T = p.h_T + s0 * p.D * p.N;
        const dim3 grid(blocks, (unsigned)std::min(65535L, p.n_seq - s0));
        switch (pad_of(p.N)) {
            case Pad::kNone: scan_step_kernel<T, NL, Pad::kNone><<<grid, 32 * kStepWarps, 0, st>>>(q, tiles); break;
            case Pad::kLanes: scan_step_kernel<T, NL, Pad::kLanes><<<grid, 32 * kStepWarps, 0, st>>>(q, tiles); break;
            default: scan_step_kernel<T, NL, Pad::kStates><<<grid, 32 * kStepWarps, 0, st>>>(q, tiles);
        }
        const cudaError_t err = cudaGetLastError();
        if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
}

template <typename T>
cudaError_t step_dispatch(const ScanProblem &p, cudaStream_t st) {
    switch (lanes_of_states(p.N)) {
        case 2: return step_t<T, 2>(p, st);
        case 4: return step_t<T, 4>(p, st);
        case 8: return step_t<T, 8>(p, st);
        case 16: return step_t<T, 16>(p, st);
        case 32: return step_t<T, 32>(p, st);
    }
    return cudaErrorInvalidValue;
}

// to <- from, or zero (the states of a call without tokens).
__global__ void states_copy_kernel(const float *from, float *to, long n) {
    for (long i = (long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long)gridDim.x * blockDim.x)
        to[i] = from ? from[i] : 0.f;
}

}  // namespace

// Warps of the recurrence that one item of `D` channels keeps busy, and the
// warp schedulers of the device (152 SMs of four).  A sequence is worth cutting,
// at the price of running its cut part twice, where it is longer than 1.3 times
// the tokens that each scheduler has of the whole batch's work; one warp alone
// takes a token in about 1.3 times the issue time its work needs, so it alone
// would outlast the batch spread over the device 1.7 times.  It is then cut so
// that three warps meet on each scheduler.  Both passes in us, 2048
// channels: one sequence of 16384 tokens 287, uncut 1063, with two warps a
// scheduler 364, with four 287; one of 1024 tokens 31, uncut 69; four of 512,
// which the rule leaves whole, 36, cut 45.
constexpr long kSchedulers = 152 * 4;

Cut choose_cut(int T_total, int D, int N) {
    const long warps = std::max(1L, (long)D * lanes_of_states(N) / 64);
    const long most = std::max(128L, 13L * T_total * warps / (10 * kSchedulers));
    long len = std::max(64L, T_total * warps / (3 * kSchedulers));
    len = (len + kTokens - 1) / kTokens * kTokens;
    return Cut{(int)std::min<long>(len, 1 << 30), (int)std::min<long>(std::max(most, len), 0x7fffffff)};
}

// Blocks come in waves of `held`; where the last one leaves more than a tenth
// of the device idle, the sequences are cut so that their first parts fill
// whole waves and the rest, a first pass of a seventh of its cost, the gaps.
// (8 x 2048 tokens, 2048 channels: 256 blocks of 304, 732 us whole, 671 + 27 us
// cut.)
Cut choose_even_cut(int T, long whole, long held) {
    const long waves = (whole + held - 1) / held;
    if (whole == 0 || 10 * whole >= 9 * waves * held) return Cut{kTokens, 0x7fffffff};
    long len = std::max(64L, T * whole / (waves * held));
    len = (len + kTokens - 1) / kTokens * kTokens;
    return Cut{(int)std::min<long>(len, 1 << 30), (int)std::min<long>(len, 1 << 30)};
}

namespace {

struct LayoutBytes {
    size_t off, order, item, pre_item, count, pre_h, pre_sum, pre_h0, total;
    long items, pres;
};
LayoutBytes layout_plan(int n_seq, int T_total, int D, int N, Cut cut, bool packed, bool h0) {
    LayoutBytes b;
    size_t at = 0;
    auto take = [&](size_t bytes) { const size_t o = at; at += round256(bytes); return o; };
    if (packed) {
        // every segment but a sequence's last holds `cut` tokens
        b.pres = T_total > cut.trigger ? T_total / cut.cut : 0;
        b.items = n_seq + b.pres;
    } else {
        const int segs = n_seq ? segments_of(T_total / n_seq, cut.cut, cut.trigger) : 0;
        b.items = (long)n_seq * segs;
        b.pres = n_seq ? (long)n_seq * (segs - 1) : 0;
    }
    const size_t n = packed ? (size_t)n_seq : 0;
    b.off = take(n ? sizeof(int32_t) * (n + 1) : 0);
    b.order = take(sizeof(int32_t) * n);
    b.item = take(n ? sizeof(Item) * (size_t)b.items : 0);
    b.pre_item = take(n ? sizeof(Item) * (size_t)b.pres : 0);
    b.count = take(n ? 2 * sizeof(int32_t) : 0);
    b.pre_h = take(sizeof(float) * (size_t)b.pres * D * N);
    b.pre_sum = take(sizeof(float) * (size_t)b.pres * D);
    b.pre_h0 = take(h0 ? sizeof(float) * (size_t)b.pres * D * N : 0);
    b.total = at;
    return b;
}

}  // namespace

size_t layout_bytes(int n_seq, int T_total, int D, int N, Cut cut, bool packed, bool h0) {
    return layout_plan(n_seq, T_total, D, N, cut, packed, h0).total;
}

cudaError_t make_layout(const ScanProblem &p, Cut cut, Layout &l, cudaStream_t st) {
    l.cut = cut.cut;
    l.trigger = cut.trigger;
    // the gradient has no h0
    const bool replaced = p.h0 && p.h0 == p.h_T;
    const LayoutBytes b = layout_plan(p.n_seq, p.T_total, p.D, p.N, cut, p.cu != nullptr, replaced);
    l.items = (int)b.items;
    l.pres = (int)b.pres;
    l.pre_h = reinterpret_cast<float *>(p.ws + b.pre_h);
    l.pre_sum = reinterpret_cast<float *>(p.ws + b.pre_sum);
    l.pre_h0 = replaced ? reinterpret_cast<float *>(p.ws + b.pre_h0) : nullptr;
    l.slot_off = l.count = nullptr;
    l.item = l.pre_item = nullptr;
    if (!p.cu) return cudaSuccess;
    int32_t *off = reinterpret_cast<int32_t *>(p.ws + b.off);
    int32_t *count = reinterpret_cast<int32_t *>(p.ws + b.count);
    Item *item = reinterpret_cast<Item *>(p.ws + b.item);
    Item *pre_item = reinterpret_cast<Item *>(p.ws + b.pre_item);
    l.slot_off = off;
    l.count = count;
    l.item = item;
    l.pre_item = pre_item;
    const int threads = std::min(1024, (p.n_seq + 31) / 32 * 32);
    layout_kernel<<<1, threads, 0, st>>>(p.cu, p.n_seq, p.T_total, l.cut, l.trigger, off,
                                         reinterpret_cast<int32_t *>(p.ws + b.order), item, pre_item,
                                         count, p.status);
    return cudaGetLastError();
}

cudaError_t launch_adjoint_ends(const ScanProblem &p, const Layout &l, cudaStream_t st) {
    return p.dtype == MDN_BF16 ? fwd_dispatch<__nv_bfloat16>(p, l, Pass::kAdjoint, st)
                               : fwd_dispatch<float>(p, l, Pass::kAdjoint, st);
}

cudaError_t launch_states_copy(const float *from, float *to, long n, cudaStream_t st) {
    if (!to || n == 0 || from == to) return cudaSuccess;
    const long blocks = (n + 255) / 256;
    states_copy_kernel<<<(unsigned)(blocks < 1216 ? blocks : 1216), 256, 0, st>>>(from, to, n);
    return cudaGetLastError();
}

}  // namespace scan

size_t scan_fwd_workspace(int n_seq, int T_total, int D, int G, int N, mdn_dtype dtype) {
    // which of the two a call is, its sizes do not tell
    const scan::Cut cut = scan::choose_cut(T_total, D, N);
    return std::max(scan::layout_bytes(n_seq, T_total, D, N, cut, true, true),
                    scan::layout_bytes(n_seq, T_total, D, N, cut, false, true));
}

cudaError_t launch_scan_fwd(const ScanProblem &p, cudaStream_t st) {
    if (p.n_seq == 0) return cudaSuccess;
    if (p.T_total == 0) return scan::launch_states_copy(p.h0, p.h_T, (long)p.n_seq * p.D * p.N, st);
    scan::Layout l;
    const cudaError_t err = scan::make_layout(p, scan::choose_cut(p.T_total, p.D, p.N), l, st);
    if (err != cudaSuccess) return err;
    return p.dtype == MDN_BF16 ? scan::fwd_dispatch<__nv_bfloat16>(p, l, scan::Pass::kMain, st)
                               : scan::fwd_dispatch<float>(p, l, scan::Pass::kMain, st);
}

cudaError_t launch_scan_step(const ScanProblem &p, cudaStream_t st) {
    if (p.n_seq == 0) return cudaSuccess;
    return p.dtype == MDN_BF16 ? scan::step_dispatch<__nv_bfloat16>(p, st)
                               : scan::step_dispatch<float>(p, st);
}

}  // namespace mdn
