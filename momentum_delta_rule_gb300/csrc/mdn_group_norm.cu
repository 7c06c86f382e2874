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
// token, so that weights and the parameters' sums stay in registers too.  The
// groups of a sequence take two readings, the second one after the sums of
// tiles of its tokens have been joined; a sequence batch that fits the L2 cache
// is read from memory once.
#include <algorithm>

#include "mdn_attn.cuh"

namespace mdn {
namespace {

constexpr int kThreads = 256;

// Sum over the threads of a group: tpg threads (a power of two).  The halves of
// `red` alternate, as one barrier a call then is enough.
__device__ __forceinline__ float2 group_sum(float2 v, int tpg, float2 *red, int &turn) {
    for (int o = min(tpg, 32) >> 1; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    if (tpg <= 32) return v;
    float2 *r = red + turn;
    turn ^= 32;
    if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
    __syncthreads();
    const int wpg = tpg >> 5;
    v = r[((threadIdx.x >> 5) & ~(wpg - 1)) + (threadIdx.x & (wpg - 1))];
    for (int o = wpg >> 1; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    return v;
}

template <int V>
__device__ __forceinline__ void activate(const float *x, int act, float *a) {
    if (act == MDN_ACT_NONE) {
#pragma unroll
        for (int v = 0; v < V; ++v) a[v] = x[v];
        return;
    }
    sigmoids<V>(x, a);
    if (act == MDN_ACT_SILU)
#pragma unroll
        for (int v = 0; v < V; ++v) a[v] *= x[v];
}
template <int V>
__device__ __forceinline__ void activate_d(const float *x, int act, float *a, float *d) {
    if (act == MDN_ACT_NONE) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            a[v] = x[v];
            d[v] = 1.f;
        }
        return;
    }
    float s[V];
    sigmoids<V>(x, s);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const bool silu = act == MDN_ACT_SILU;
        a[v] = silu ? x[v] * s[v] : s[v];
        d[v] = silu ? s[v] * fmaf(x[v], 1.f - s[v], 1.f) : s[v] * (1.f - s[v]);
    }
}

template <int V>
__device__ __forceinline__ void load_weights(const float *w, long c, float none, float *f) {
#pragma unroll
    for (int v = 0; v < V; ++v) f[v] = w ? __ldg(w + c + v) : none;
}

// What a group's elements become, and their gradient.
template <int V, bool GATE>
__device__ __forceinline__ void forward_packet(float *x, const float *g, float mean, float rstd, const float *w,
                                               const float *b, int act) {
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = fmaf((x[v] - mean) * rstd, w[v], b[v]);
    float a[V];
    activate<V>(GATE ? g : x, act, a);
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = GATE ? x[v] * a[v] : a[v];
}
// x <- n, dy <- du, g <- dgate
template <int V, bool GATE>
__device__ __forceinline__ void backward_packet(float *x, float *g, float *dy, float mean, float rstd, const float *w,
                                                const float *b, int act) {
    float u[V], a[V], d[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        x[v] = (x[v] - mean) * rstd;
        u[v] = fmaf(x[v], w[v], b[v]);
    }
    activate_d<V>(GATE ? g : u, act, a, d);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (GATE) g[v] = dy[v] * u[v] * d[v];
        dy[v] *= GATE ? a[v] : d[v];
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

// Threads of a block at most: of groups that take more than four packets a
// thread, as many as the widest group (16384 columns) needs.
__host__ __device__ constexpr int most_threads(int NI, int V) { return NI <= 4 || V >= 8 ? 256 : V == 4 ? 512 : 1024; }

template <typename T, int V, int NI, bool GATE>
__global__ void __launch_bounds__(most_threads(NI, V)) token_fwd_kernel(GroupNormProblem p, int tpg) {
    __shared__ float2 red[64];
    constexpr bool HOLD = NI * V <= 16;
    int turn = 0;
    const TokenPlace t = token_place(p, tpg);
    const int w = p.D / p.G;
    const long c0 = t.g * w;
    const T *x = static_cast<const T *>(p.x) + c0, *gate = static_cast<const T *>(p.gate) + c0;
    T *y = static_cast<T *>(p.y) + c0;
    float wt[HOLD ? NI : 1][V], bs[HOLD ? NI : 1][V];
    auto weights = [&](int i, int c) {
        load_weights<V>(p.weight, c0 + c, 1.f, wt[HOLD ? i : 0]);
        load_weights<V>(p.bias, c0 + c, 0.f, bs[HOLD ? i : 0]);
    };
    if (HOLD)
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int c = (i * tpg + t.tid) * V;
            if (c < w) weights(i, c);
        }
    const float inv = 1.f / (float)w;
    long row = t.row;
    for (int k = 0; k < t.rounds; ++k, row += t.step) {
        const bool live = row < p.rows;
        Packet<T, V> px[NI], pg[GATE ? NI : 1];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int c = (i * tpg + t.tid) * V;
            if (live && c < w) {
                px[i] = load_packet<T, V>(x + row * p.ld_x + c);
                if (GATE) pg[i] = load_packet<T, V>(gate + row * p.ld_gate + c);
            }
        }
        float mean = 0.f;
        if (p.center) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                float f[V];
                if (live && (i * tpg + t.tid) * V < w) {
                    unpack<T, V>(px[i], f);
#pragma unroll
                    for (int v = 0; v < V; ++v) s += f[v];
                }
            }
            mean = group_sum(make_float2(s, 0.f), tpg, red, turn).x * inv;
        }
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            float f[V];
            if (live && (i * tpg + t.tid) * V < w) {
                unpack<T, V>(px[i], f);
#pragma unroll
                for (int v = 0; v < V; ++v) s = fmaf(f[v] - mean, f[v] - mean, s);
            }
        }
        const float rstd = rsqrtf(fmaf(group_sum(make_float2(s, 0.f), tpg, red, turn).x, inv, p.eps));
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int c = (i * tpg + t.tid) * V;
            if (live && c < w) {
                float f[V], g[V];
                if (!HOLD) weights(i, c);
                unpack<T, V>(px[i], f);
                if (GATE) unpack<T, V>(pg[i], g);
                forward_packet<V, GATE>(f, g, mean, rstd, wt[HOLD ? i : 0], bs[HOLD ? i : 0], p.act);
                store_packet<T, V>(y + row * p.D + c, pack<T, V>(f));
            }
        }
        if (p.stats && live && t.tid == 0)
            reinterpret_cast<float2 *>(p.stats)[row * p.G + t.g] = make_float2(mean, rstd);
    }
}

// part: [row lanes][2][D], one lane for every t.row of the first round.
template <typename T, int V, int NI, bool GATE>
__global__ void __launch_bounds__(most_threads(NI, V))
token_bwd_kernel(GroupNormProblem p, int tpg, float *part) {
    __shared__ float2 red[64];
    int turn = 0;
    const TokenPlace t = token_place(p, tpg);
    const int w = p.D / p.G;
    const long c0 = t.g * w;
    const T *x = static_cast<const T *>(p.x) + c0, *gate = static_cast<const T *>(p.gate) + c0;
    const T *dyp = static_cast<const T *>(p.dy) + c0;
    T *dx = static_cast<T *>(p.dx) + c0, *dgate = static_cast<T *>(p.dgate) + c0;
    constexpr bool HOLD = NI * V <= 16;
    float wt[HOLD ? NI : 1][V], bs[HOLD ? NI : 1][V], dw[NI][V], db[NI][V];
    auto weights = [&](int i, int c) {
        load_weights<V>(p.weight, c0 + c, 1.f, wt[HOLD ? i : 0]);
        load_weights<V>(p.bias, c0 + c, 0.f, bs[HOLD ? i : 0]);
    };
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int c = (i * tpg + t.tid) * V;
        if (HOLD && c < w) weights(i, c);
#pragma unroll
        for (int v = 0; v < V; ++v) dw[i][v] = db[i][v] = 0.f;
    }
    const float inv = 1.f / (float)w;
    long row = t.row;
    for (int k = 0; k < t.rounds; ++k, row += t.step) {
        const bool live = row < p.rows;
        Packet<T, V> px[NI], pd[NI], pg[GATE ? NI : 1];
        float2 st = make_float2(0.f, 0.f), s = make_float2(0.f, 0.f);
        if (live) st = reinterpret_cast<const float2 *>(p.stats)[row * p.G + t.g];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int c = (i * tpg + t.tid) * V;
            if (live && c < w) {
                px[i] = load_packet<T, V>(x + row * p.ld_x + c);
                pd[i] = load_packet<T, V>(dyp + row * p.ld_dy + c);
                if (GATE) pg[i] = load_packet<T, V>(gate + row * p.ld_gate + c);
            }
        }
        // the elements are taken apart twice, as keeping n and dn of all of
        // them takes twice the registers
        auto element = [&](int i, int c, float *n, float *d, float *g) {
            if (!HOLD) weights(i, c);
            unpack<T, V>(px[i], n);
            unpack<T, V>(pd[i], d);
            if (GATE) unpack<T, V>(pg[i], g);
            backward_packet<V, GATE>(n, g, d, st.x, st.y, wt[HOLD ? i : 0], bs[HOLD ? i : 0], p.act);
        };
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int c = (i * tpg + t.tid) * V;
            if (live && c < w) {
                float n[V], d[V], g[V];
                element(i, c, n, d, g);
                if (GATE) store_packet<T, V>(dgate + row * p.D + c, pack<T, V>(g));
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    dw[i][v] = fmaf(d[v], n[v], dw[i][v]);
                    db[i][v] += d[v];
                    const float dn = d[v] * wt[HOLD ? i : 0][v];
                    s.x += dn;
                    s.y = fmaf(dn, n[v], s.y);
                }
            }
        }
        s = group_sum(s, tpg, red, turn);
        const float m1 = p.center ? s.x * inv : 0.f, m2 = s.y * inv;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int c = (i * tpg + t.tid) * V;
            if (live && c < w) {
                float n[V], d[V], g[V];
                element(i, c, n, d, g);
#pragma unroll
                for (int v = 0; v < V; ++v) n[v] = st.y * (fmaf(d[v], wt[HOLD ? i : 0][v], -m1) - n[v] * m2);
                store_packet<T, V>(dx + row * p.D + c, pack<T, V>(n));
            }
        }
    }
    if (!part) return;
    float *out = part + t.row * 2 * p.D + c0;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int c = (i * tpg + t.tid) * V;
        if (c < w)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                out[c + v] = dw[i][v];
                out[p.D + c + v] = db[i][v];
            }
    }
}

// dw, dbias <- sums over the lanes of part, in their order.
__global__ void __launch_bounds__(kThreads) param_kernel(const float *part, int lanes, int D, float *dw, float *dbias) {
    __shared__ float sums[8][32];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const long c = blockIdx.x * 32L + x;
    float s = 0.f;
    if (c < 2L * D) {
        const float *src = part + c;
#pragma unroll 8
        for (int l = y; l < lanes; l += 8) s += src[(long)l * 2 * D];
    }
    sums[y][x] = s;
    __syncthreads();
    if (y || c >= 2L * D) return;
    for (int k = 1; k < 8; ++k) s += sums[k][x];
    if (c < D) {
        if (dw) dw[c] = s;
    } else if (dbias) {
        dbias[c - D] = s;
    }
}

// -------------------------------------------------------- a sequence's groups

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

// Count, mean and sum of squared distances from it, of two parts together.
struct Moments {
    float n, mean, m2;
};
__device__ __forceinline__ Moments join(const Moments &a, const Moments &b) {
    Moments r;
    r.n = a.n + b.n;
    const float f = r.n > 0.f ? b.n / r.n : 0.f, d = b.mean - a.mean;
    r.mean = b.n > 0.f ? fmaf(d, f, a.mean) : a.mean;
    r.m2 = b.n > 0.f ? a.m2 + b.m2 + (a.n > 0.f ? d * d * a.n * f : 0.f) : a.m2;
    if (a.n <= 0.f) r = b;
    return r;
}
__device__ __forceinline__ Moments join_warp(Moments a) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        Moments b;
        b.n = __shfl_xor_sync(0xffffffffu, a.n, o);
        b.mean = __shfl_xor_sync(0xffffffffu, a.mean, o);
        b.m2 = __shfl_xor_sync(0xffffffffu, a.m2, o);
        // the same order of the two in both lanes
        a = (threadIdx.x & o) ? join(b, a) : join(a, b);
    }
    return a;
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

// Sums or moments of the block's threads, group by group.  Every thread brings
// the value of its packets, all of one group but in blocks of one group only.
template <typename F>
__device__ __forceinline__ void by_group(const GroupNormProblem &p, const Columns &c, int V, F take) {
    const int warp = threadIdx.x >> 5, ppg = c.packets / c.groups;
    for (int g = warp; g < c.groups; g += kThreads / 32) take(g, ppg);
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) seq_stats_kernel(GroupNormProblem p, int rows, int per_block, float2 *part) {
    __shared__ Moments mom[kThreads];
    if (p.cu && !cu_well_formed(p.cu, p.n_seq, (int)p.rows)) {
        if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) atomicExch(p.status, MDN_ERR_INVALID_ARG);
        return;
    }
    Tile t;
    if (!tile_of(p, rows, blockIdx.x, t)) return;
    const Columns c = columns_of(p, per_block, V);
    const int w = p.D / p.G;
    Moments m = {0.f, 0.f, 0.f};
    if (c.lane < c.lanes)
        for (int pc = c.pc; pc < c.packets; pc += kThreads) {
            const T *x = static_cast<const T *>(p.x) + t.start * p.ld_x + (long)c.g0 * w + pc * V;
            // sums about the mean of the first packet, so that they do not cancel
            float shift = 0.f, s1 = 0.f, s2 = 0.f;
            int count = 0;
#pragma unroll 8
            for (int r = c.lane; r < t.n; r += c.lanes, ++count) {
                float f[V];
                unpack<T, V>(load_packet<T, V>(x + r * p.ld_x), f);
                if (r == c.lane && p.center) {
#pragma unroll
                    for (int v = 0; v < V; ++v) shift += f[v] * (1.f / V);
                }
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float d = f[v] - shift;
                    s1 += d;
                    s2 = fmaf(d, d, s2);
                }
            }
            const float n = (float)count * V, mean = count ? s1 / n : 0.f;
            Moments one;
            one.n = n;
            one.mean = p.center ? shift + mean : 0.f;
            one.m2 = p.center ? fmaxf(s2 - s1 * mean, 0.f) : s2;
            if (s2 != s2) one.m2 = s2;                   // fmaxf drops a NaN
            m = join(m, one);
        }
    mom[threadIdx.x] = m;
    __syncthreads();
    by_group(p, c, V, [&](int g, int ppg) {
        Moments a = {0.f, 0.f, 0.f};
        if (c.packets >= kThreads && c.groups == 1) {
            for (int i = threadIdx.x & 31; i < kThreads; i += 32) a = join(a, mom[i]);
        } else {
            for (int i = threadIdx.x & 31; i < ppg * c.lanes; i += 32) {
                const int lane = i / ppg;
                a = join(a, mom[lane * c.packets + g * ppg + (i - lane * ppg)]);
            }
        }
        a = join_warp(a);
        if ((threadIdx.x & 31) == 0) part[(long)blockIdx.x * p.G + c.g0 + g] = make_float2(a.mean, a.m2);
    });
}

// One warp a group of a sequence: the statistics from the tiles'.
__global__ void __launch_bounds__(kThreads) seq_join_kernel(GroupNormProblem p, int rows, const float2 *part, float2 *stats) {
    const long i = blockIdx.x * (long)(kThreads / 32) + (threadIdx.x >> 5);
    const bool ok = !p.cu || cu_well_formed(p.cu, p.n_seq, (int)p.rows);
    if (i >= (long)p.n_seq * p.G) return;
    const int s = (int)(i / p.G), g = (int)(i - (long)s * p.G), w = p.D / p.G;
    const int len = !ok ? 0 : p.cu ? p.cu[s + 1] - p.cu[s] : p.T;
    const int tiles = (len + rows - 1) / rows;
    const long slot = ok ? first_slot(p, rows, s) : 0;
    Moments a = {0.f, 0.f, 0.f};
    for (int k = threadIdx.x & 31; k < tiles; k += 32) {
        const float2 v = part[(slot + k) * p.G + g];
        Moments one = {(float)min(rows, len - k * rows) * w, v.x, v.y};
        a = join(a, one);
    }
    a = join_warp(a);
    if ((threadIdx.x & 31) == 0)
        stats[i] = len ? make_float2(a.mean, rsqrtf(a.m2 / a.n + p.eps)) : make_float2(0.f, 0.f);
}

template <typename T, int V, bool GATE>
__global__ void __launch_bounds__(kThreads) seq_apply_kernel(GroupNormProblem p, int rows, int per_block, const float2 *stats) {
    if (p.cu && !cu_well_formed(p.cu, p.n_seq, (int)p.rows)) return;
    Tile t;
    if (!tile_of(p, rows, blockIdx.x, t)) return;
    const Columns c = columns_of(p, per_block, V);
    if (c.lane >= c.lanes) return;
    const int w = p.D / p.G;
    for (int pc = c.pc; pc < c.packets; pc += kThreads) {
        const long col = (long)c.g0 * w + pc * V;
        const float2 st = stats[(long)t.seq * p.G + col / w];
        float wt[V], bs[V];
        load_weights<V>(p.weight, col, 1.f, wt);
        load_weights<V>(p.bias, col, 0.f, bs);
        const T *x = static_cast<const T *>(p.x) + t.start * p.ld_x + col;
        const T *gate = static_cast<const T *>(p.gate) + t.start * p.ld_gate + col;
        T *y = static_cast<T *>(p.y) + t.start * p.D + col;
#pragma unroll 4
        for (int r = c.lane; r < t.n; r += c.lanes) {
            float f[V], g[V];
            unpack<T, V>(load_packet<T, V>(x + r * p.ld_x), f);
            if (GATE) unpack<T, V>(load_packet<T, V>(gate + r * p.ld_gate), g);
            forward_packet<V, GATE>(f, g, st.x, st.y, wt, bs, p.act);
            store_packet<T, V>(y + (long)r * p.D, pack<T, V>(f));
        }
    }
}

// Sums of dn and dn n of a tile's groups, and of du n and du of its columns.
template <typename T, int V, bool GATE>
__global__ void __launch_bounds__(kThreads)
seq_sums_kernel(GroupNormProblem p, int rows, int per_block, float2 *part, float *params) {
    __shared__ float2 red[kThreads];
    __shared__ float cols[2][kThreads * V];
    const bool ok = !p.cu || cu_well_formed(p.cu, p.n_seq, (int)p.rows);
    if (!ok && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) atomicExch(p.status, MDN_ERR_INVALID_ARG);
    Tile t;
    const bool some = ok && tile_of(p, rows, blockIdx.x, t);
    const Columns c = columns_of(p, per_block, V);
    const int w = p.D / p.G;
    float2 s = make_float2(0.f, 0.f);
    float *out = params ? params + (long)blockIdx.x * 2 * p.D + (long)c.g0 * w : nullptr;
    // whole rounds of packets, for the barriers; one round where lanes > 1
    for (int base = 0; base < c.packets; base += kThreads) {
        const int pc = base + c.pc;
        float dw[V], db[V];
#pragma unroll
        for (int v = 0; v < V; ++v) dw[v] = db[v] = 0.f;
        if (some && c.lane < c.lanes && pc < c.packets) {
            const long col = (long)c.g0 * w + pc * V;
            const float2 st = reinterpret_cast<const float2 *>(p.stats)[(long)t.seq * p.G + col / w];
            float wt[V], bs[V];
            load_weights<V>(p.weight, col, 1.f, wt);
            load_weights<V>(p.bias, col, 0.f, bs);
            const T *x = static_cast<const T *>(p.x) + t.start * p.ld_x + col;
            const T *gate = static_cast<const T *>(p.gate) + t.start * p.ld_gate + col;
            const T *dy = static_cast<const T *>(p.dy) + t.start * p.ld_dy + col;
#pragma unroll 4
            for (int r = c.lane; r < t.n; r += c.lanes) {
                float n[V], d[V], g[V];
                unpack<T, V>(load_packet<T, V>(x + r * p.ld_x), n);
                unpack<T, V>(load_packet<T, V>(dy + r * p.ld_dy), d);
                if (GATE) unpack<T, V>(load_packet<T, V>(gate + r * p.ld_gate), g);
                backward_packet<V, GATE>(n, g, d, st.x, st.y, wt, bs, p.act);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    dw[v] = fmaf(d[v], n[v], dw[v]);
                    db[v] += d[v];
                }
            }
            // the groups' sums follow from the columns'
#pragma unroll
            for (int v = 0; v < V; ++v) {
                s.x = fmaf(db[v], wt[v], s.x);
                s.y = fmaf(dw[v], wt[v], s.y);
            }
        }
        if (!out) continue;
        if (c.lanes == 1) {
            if (c.lane == 0 && pc < c.packets)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    out[pc * V + v] = dw[v];
                    out[p.D + pc * V + v] = db[v];
                }
            continue;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            cols[0][threadIdx.x * V + v] = dw[v];
            cols[1][threadIdx.x * V + v] = db[v];
        }
        __syncthreads();
        const int n = c.packets * V;
        for (int i = threadIdx.x; i < 2 * n; i += kThreads) {
            const int which = i >= n, col = i - which * n;
            float sum = 0.f;
            for (int l = 0; l < c.lanes; ++l) sum += cols[which][l * n + col];
            out[which * p.D + col] = sum;
        }
    }
    if (!some) return;
    red[threadIdx.x] = s;
    __syncthreads();
    by_group(p, c, V, [&](int g, int ppg) {
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
        if ((threadIdx.x & 31) == 0) part[(long)blockIdx.x * p.G + c.g0 + g] = a;
    });
}

// One warp a group of a sequence: its means of dn and dn n.
__global__ void __launch_bounds__(kThreads) seq_means_kernel(GroupNormProblem p, int rows, const float2 *part, float2 *means) {
    const long i = blockIdx.x * (long)(kThreads / 32) + (threadIdx.x >> 5);
    const bool ok = !p.cu || cu_well_formed(p.cu, p.n_seq, (int)p.rows);
    if (!ok || i >= (long)p.n_seq * p.G) return;
    const int s = (int)(i / p.G), g = (int)(i - (long)s * p.G);
    const int len = p.cu ? p.cu[s + 1] - p.cu[s] : p.T, tiles = (len + rows - 1) / rows;
    const long slot = first_slot(p, rows, s);
    float2 a = make_float2(0.f, 0.f);
    for (int k = threadIdx.x & 31; k < tiles; k += 32) {
        const float2 v = part[(slot + k) * p.G + g];
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
    if (p.cu && !cu_well_formed(p.cu, p.n_seq, (int)p.rows)) return;
    Tile t;
    if (!tile_of(p, rows, blockIdx.x, t)) return;
    const Columns c = columns_of(p, per_block, V);
    if (c.lane >= c.lanes) return;
    const int w = p.D / p.G;
    for (int pc = c.pc; pc < c.packets; pc += kThreads) {
        const long col = (long)c.g0 * w + pc * V;
        const float2 st = reinterpret_cast<const float2 *>(p.stats)[(long)t.seq * p.G + col / w];
        const float2 m = means[(long)t.seq * p.G + col / w];
        float wt[V], bs[V];
        load_weights<V>(p.weight, col, 1.f, wt);
        load_weights<V>(p.bias, col, 0.f, bs);
        const T *x = static_cast<const T *>(p.x) + t.start * p.ld_x + col;
        const T *gate = static_cast<const T *>(p.gate) + t.start * p.ld_gate + col;
        const T *dy = static_cast<const T *>(p.dy) + t.start * p.ld_dy + col;
        T *dx = static_cast<T *>(p.dx) + t.start * p.D + col, *dgate = static_cast<T *>(p.dgate) + t.start * p.D + col;
#pragma unroll 4
        for (int r = c.lane; r < t.n; r += c.lanes) {
            float n[V], d[V], g[V];
            unpack<T, V>(load_packet<T, V>(x + r * p.ld_x), n);
            unpack<T, V>(load_packet<T, V>(dy + r * p.ld_dy), d);
            if (GATE) unpack<T, V>(load_packet<T, V>(gate + r * p.ld_gate), g);
            backward_packet<V, GATE>(n, g, d, st.x, st.y, wt, bs, p.act);
            if (GATE) store_packet<T, V>(dgate + (long)r * p.D, pack<T, V>(g));
#pragma unroll
            for (int v = 0; v < V; ++v) n[v] = st.y * (fmaf(d[v], wt[v], -m.x) - n[v] * m.y);
            store_packet<T, V>(dx + (long)r * p.D, pack<T, V>(n));
        }
    }
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

// Groups of a block that takes parts of sequences.
int groups_per_block(int D, int G, int V) { return std::max(1, std::min(G, kThreads * V / (D / G))); }

// How a call's tokens' groups are spread.
struct TokenShape {
    int tpg, NI, threads;
    long blocks, lanes;
};
long gcd(long a, long b) { return b ? gcd(b, a % b) : a; }

TokenShape token_shape(const GroupNormProblem &p, int V, int per_sm) {
    TokenShape t;
    const long P = (p.D / p.G) / V;
    // up to eight packets a thread before a group takes several warps
    t.tpg = P <= 32 ? pow2_at_least(P) : std::max(32, pow2_at_least((P + 7) / 8));
    t.NI = (int)((P + t.tpg - 1) / t.tpg);
    if (t.tpg > 1024) {
        t.tpg = 1024;
        t.NI = (int)((P + 1023) / 1024);
    }
    t.NI = pow2_at_least(t.NI);
    t.threads = std::max(kThreads, t.tpg);
    const long ipb = t.threads / t.tpg, unit = p.G / gcd(ipb, p.G);
    const long need = (p.rows * p.G + ipb - 1) / ipb, most = 152L * std::max(1, per_sm * kThreads / t.threads);
    long blocks = std::min(need, most);
    blocks = blocks / unit * unit;
    t.blocks = std::max(blocks, unit);
    t.lanes = t.blocks * ipb / p.G;
    return t;
}

// The gradient's blocks: each lane of tokens leaves a row of the parameters'
// sums behind, which are read again.
constexpr int kFwdPerSM = 8, kBwdPerSM = 4;
long token_lanes_most(long rows, int D, int G) {
    // for any packet width: at most 152 * 4 * 256 threads, and one unit more
    const long w = D / G;
    long most = 0;
    for (int V : {8, 4, 2, 1}) {
        if (w % V) continue;
        GroupNormProblem p = {};
        p.rows = rows;
        p.D = D;
        p.G = G;
        most = std::max(most, token_shape(p, V, kBwdPerSM).lanes);
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
cudaError_t token_launch(const GroupNormProblem &p, const TokenShape &t, float *part, bool bwd, cudaStream_t st) {
    if (bwd) token_bwd_kernel<T, V, NI, GATE><<<(unsigned)t.blocks, t.threads, 0, st>>>(p, t.tpg, part);
    else token_fwd_kernel<T, V, NI, GATE><<<(unsigned)t.blocks, t.threads, 0, st>>>(p, t.tpg);
    return cudaGetLastError();
}
template <typename T, int V, bool GATE>
cudaError_t token_pick(const GroupNormProblem &p, const TokenShape &t, float *part, bool bwd, cudaStream_t st) {
    switch (t.NI) {
        case 1: return token_launch<T, V, 1, GATE>(p, t, part, bwd, st);
        case 2: return token_launch<T, V, 2, GATE>(p, t, part, bwd, st);
        case 4: return token_launch<T, V, 4, GATE>(p, t, part, bwd, st);
        case 8: return token_launch<T, V, 8, GATE>(p, t, part, bwd, st);
        default: return token_launch<T, V, 16, GATE>(p, t, part, bwd, st);
    }
}

cudaError_t params(const GroupNormProblem &p, const float *part, long lanes, cudaStream_t st) {
    if (!p.dw && !p.dbias) return cudaSuccess;
    param_kernel<<<(2 * p.D + 31) / 32, kThreads, 0, st>>>(part, (int)lanes, p.D, p.dw, p.dbias);
    return cudaGetLastError();
}

template <typename T, int V, bool GATE>
cudaError_t run(const GroupNormProblem &p, bool bwd, cudaStream_t st) {
    cudaError_t err;
    if (!p.over_sequence) {
        const TokenShape t = token_shape(p, V, bwd ? kBwdPerSM : kFwdPerSM);
        float *part = bwd && (p.dw || p.dbias) ? reinterpret_cast<float *>(p.ws) : nullptr;
        if ((err = token_pick<T, V, GATE>(p, t, part, bwd, st)) != cudaSuccess) return err;
        return bwd ? params(p, part, t.lanes, st) : cudaSuccess;
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
        seq_join_kernel<<<joins, kThreads, 0, st>>>(p, rows, part, stats);
        seq_apply_kernel<T, V, GATE><<<grid, kThreads, 0, st>>>(p, rows, gpb, stats);
        return cudaGetLastError();
    }
    float *prm = p.dw || p.dbias ? reinterpret_cast<float *>(ws) : nullptr;
    seq_sums_kernel<T, V, GATE><<<grid, kThreads, 0, st>>>(p, rows, gpb, part, prm);
    seq_means_kernel<<<joins, kThreads, 0, st>>>(p, rows, part, second);
    seq_dx_kernel<T, V, GATE><<<grid, kThreads, 0, st>>>(p, rows, gpb, second);
    if ((err = cudaGetLastError()) != cudaSuccess) return err;
    return params(p, prm, slots, st);
}

template <typename T, int V>
cudaError_t gated(const GroupNormProblem &p, bool bwd, cudaStream_t st) {
    return p.gate ? run<T, V, true>(p, bwd, st) : run<T, V, false>(p, bwd, st);
}

cudaError_t launch(const GroupNormProblem &p, bool bwd, cudaStream_t st) {
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
    return round256(tile_slots(n_seq, rows, D) * G * sizeof(float2)) + round256((long)n_seq * G * sizeof(float2));
}
size_t group_norm_bwd_workspace(int n_seq, long rows, int D, int G, bool over_sequence, mdn_dtype dtype) {
    if (rows == 0) return 0;
    if (!over_sequence) return round256(token_lanes_most(rows, D, G) * 2 * D * sizeof(float));
    return group_norm_fwd_workspace(n_seq, rows, D, G, true, dtype) +
           round256(tile_slots(n_seq, rows, D) * 2 * D * sizeof(float));
}

}  // namespace mdn
