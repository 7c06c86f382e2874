// Pieces shared by the selective scan's forward and gradient kernels.
#pragma once

#include "mdn_ssm.cuh"

namespace mdn {
namespace scan {

constexpr int kTokens = MDN_SSM_CHUNK;    // tokens between saved states, a chunk of the gradient
constexpr int kStates = 4;                // states a lane holds of each of its channels

// How a block covers channels and states.  A channel's (padded) states lie
// across NL lanes, four each; the other lanes of a warp take other channels,
// CPT neighbouring ones each.  Padded states have A = B = C = 0 and stay 0.
// NW warps run the recurrence; HW more stage their inputs and finish their
// outputs.
template <int NL_, int CPT_, int NW_, int HW_>
struct Shape {
    static constexpr int NL = NL_, CPT = CPT_, NW = NW_, HW = HW_;
    static constexpr int NP = NL * kStates;              // padded states
    static constexpr int WC = 32 / NL * CPT;             // channels per warp
    static constexpr int CB = WC * NW;                   // channels per block
    static constexpr int NT = NW * 32;                   // recurrence threads
    static constexpr int HT = HW * 32;                   // helper threads
    // tokens whose inputs are read and whose sums are exchanged together
    static constexpr int TB = NL < 4 ? NL : 4;
};

inline int lanes_of_states(int N) {
    int nl = 2;
    while (nl * kStates < N) nl *= 2;
    return nl;
}

// Which of a channel's padded states a kernel meets: none, whole lanes of them,
// or some beside others in a lane.  An infinite delta u makes NaN of a padded
// state (inf times B = 0), which must not reach a sum over states.  The first
// kind needs no instruction for that, the second one a channel and token of the
// forward, the third one a state.
enum class Pad { kNone, kLanes, kStates };
inline Pad pad_of(int N) {
    return N % kStates ? Pad::kStates : lanes_of_states(N) * kStates > N ? Pad::kLanes : Pad::kNone;
}

// A stretch of one sequence's tokens that a block runs on its own: the whole
// sequence, or one of the segments a long sequence is cut into.
struct Item {
    int seq, tok0, len;       // tokens tok0 .. tok0 + len of the sequence
    int pre;                  // first slot of the sequence's cut segments
};

// The work, as the kernels see it.  Sequences longer than `trigger` tokens
// run as segments of `cut` tokens: a first pass takes every segment but the
// last from a zero state and leaves its end state and its sum of delta in the
// sequence's slots; the main pass chains those (h <- exp(A sum delta) h + end)
// up to its own segment.  Shorter sequences have one item and no first pass.
struct Layout {
    int cut, trigger;
    int items, pres;                  // launch bounds; the packed arrays say how many there are
    const int32_t *slot_off;          // packed: [n_seq + 1] first saved state of each sequence
    const Item *item, *pre_item;      // packed: tables
    const int32_t *count;             // packed: items, pre items
    float *pre_h, *pre_sum;           // [slot][D][N], [slot][D]
    // h0 of the cut sequences at their first slots, where the final states
    // replace it: the last segment may end before the others have read theirs.
    // Null where nothing does.
    float *pre_h0;
};

// Where sequences are cut.  For packed sequences a function of the totals alone
// (no lengths on the host).
struct Cut {
    int cut, trigger;
};
Cut choose_cut(int T_total, int D, int N);
// The gradient of equal lengths: `whole` blocks for the uncut sequences, of
// which the device holds `held` at once.
Cut choose_even_cut(int T, long whole, long held);
// Bytes of the workspace that make_layout fills with these cuts.
// `h0`: with room for copies of the initial states.
size_t layout_bytes(int n_seq, int T_total, int D, int N, Cut cut, bool packed, bool h0);
// Describes the work of p in its workspace (packed: one small kernel).
cudaError_t make_layout(const ScanProblem &p, Cut cut, Layout &l, cudaStream_t st);
// The gradient's first pass over cut segments: what each segment but the first
// hands back to the one before it, from a zero adjoint.
cudaError_t launch_adjoint_ends(const ScanProblem &p, const Layout &l, cudaStream_t st);
// to <- from, or zero where from is null.
cudaError_t launch_states_copy(const float *from, float *to, long n, cudaStream_t st);

__host__ __device__ inline int segments_of(int len, int cut, int trigger) {
    return len > trigger ? (len + cut - 1) / cut : 1;
}

// Item i of the main pass, or of a first pass (every segment but the last, or
// of the adjoints but the first); false past the end.
template <bool PRE, bool REV>
__device__ __forceinline__ bool find_item(const ScanProblem &p, const Layout &l, int i, Item &it,
                                          long &t0, long &slot0) {
    int len = p.T;                    // of the whole sequence
    if (p.cu) {
        if (i >= l.count[PRE]) return false;
        it = PRE ? l.pre_item[i] : l.item[i];
        t0 = p.cu[it.seq];
        slot0 = l.slot_off[it.seq];
        if (REV) len = p.cu[it.seq + 1] - (int)t0;
    } else {
        const int all = segments_of(p.T, l.cut, l.trigger), segs = PRE ? all - 1 : all;
        // first segments first: the last ones are the shorter ones
        const int k = i / p.n_seq;
        if (k >= segs) return false;
        it.seq = i - k * p.n_seq;
        it.tok0 = k * l.cut;
        it.len = all == 1 ? p.T : min(l.cut, p.T - it.tok0);
        it.pre = it.seq * (all - 1);
        t0 = (long)it.seq * p.T;
        slot0 = (long)it.seq * ((p.T + kTokens - 1) / kTokens);
    }
    if (REV) {
        it.tok0 += l.cut;
        it.len = min(l.cut, len - it.tok0);
    }
    t0 += it.tok0;
    slot0 += it.tok0 / kTokens;
    return true;
}

// A log2 e, the decays' exponent a unit of delta, kept above -infinity: a token
// behind a sequence's end has delta = 0 and must change nothing, which 0 times
// -infinity would.  Any delta above 1e-36 still gives 2^-huge = 0.
__device__ __forceinline__ float decay_rate(float a) {
    float x = a * kLog2e;
    asm("max.NaN.f32 %0, %0, 0fFF7FFFFF;" : "+f"(x));        // -FLT_MAX; NaN stays
    return x;
}

// The state behind a segment, `end` where it began from zero, that began from x
// and decayed by 2^e.  An infinite x stays: the segment's decay may be zero where
// none of its tokens' is.
__device__ __forceinline__ float through_segment(float e, float x, float end) {
    return fabsf(x) == INFINITY ? x + end : fmaf(ex2(e), x, end);
}

// A lane's A, states or gradients of one channel (four of N): [D, N] row d.
__device__ __forceinline__ void load_states(const float *base, long d, int n, int N, float *f) {
#pragma unroll
    for (int i = 0; i < kStates; ++i) f[i] = n + i < N ? base[d * N + n + i] : 0.f;
}
__device__ __forceinline__ void store_states(float *base, long d, int n, int N, const float *f) {
    if (N % kStates == 0) {
        *reinterpret_cast<float4 *>(base + d * N + n) = make_float4(f[0], f[1], f[2], f[3]);
        return;
    }
#pragma unroll
    for (int i = 0; i < kStates; ++i)
        if (n + i < N) base[d * N + n + i] = f[i];
}

// A pair of states without the padded ones.
__device__ __forceinline__ Pair real_states(Pair v, bool lo, bool hi) {
    float x, y;
    split_pair(v, x, y);
    return make_pair(lo ? x : 0.f, hi ? y : 0.f);
}

// Sums v[0 .. M) over NL lanes, halving the values a lane carries at each
// exchange: lane nl ends with the M / NL (at least one) values from
// reduced_first(nl) on, in v[0 ..]; where NL > M only lanes nl < M own theirs.
// The lanes lie STEP apart in the warp.
template <int NL, int M, int STEP = 1>
__device__ __forceinline__ void reduce_lanes(float *v, int nl) {
    int left = M;
#pragma unroll
    for (int o = 1; o < NL; o <<= 1) {
        if (left > 1) {
            left /= 2;
            const bool up = nl & o;
#pragma unroll
            for (int i = 0; i < M / 2; ++i) {
                if (i < left) {
                    const float send = up ? v[i] : v[i + left];
                    const float keep = up ? v[i + left] : v[i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o * STEP);
                }
            }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], o * STEP);
        }
    }
}
template <int NL, int M>
__device__ __forceinline__ int reduced_first(int nl) {
    int at = 0, left = M;
#pragma unroll
    for (int o = 1; o < NL; o <<= 1) {
        if (left == 1) break;
        left /= 2;
        if (nl & o) at += left;
    }
    return at;
}

}  // namespace scan
}  // namespace mdn
