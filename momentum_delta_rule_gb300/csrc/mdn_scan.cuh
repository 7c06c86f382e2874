// Pieces shared by the selective scan's forward and gradient kernels.
#pragma once

#include "mdn_ssm.cuh"

namespace mdn {
namespace scan {

constexpr int kTokens = MDN_SSM_CHUNK;    // tokens per stage, and between saved states
constexpr int kStates = 4;                // states a lane holds of each of its channels

// How a block covers channels and states.  A channel's (padded) states lie
// across NL lanes, four each; the other lanes of a warp take other channels,
// CPT neighbouring ones each.  Padded states have A = B = C = 0 and stay 0.
template <int NL_, int CPT_>
struct Shape {
    static constexpr int NL = NL_, CPT = CPT_;
    static constexpr int NP = NL * kStates;              // padded states
    static constexpr int WC = 32 / NL * CPT;             // channels per warp
    static constexpr int NW = NL >= 16 ? 8 : 4;          // warps per block
    static constexpr int NT = NW * 32;
    static constexpr int CB = WC * NW;                   // channels per block
};

inline int lanes_of_states(int N) {
    int nl = 2;
    while (nl * kStates < N) nl *= 2;
    return nl;
}

// Device arrays that describe the work: where each sequence's saved states
// begin, and the sequences longest first.
struct Layout {
    const int32_t *slot_off;      // [n_seq + 1], packed sequences only
    const int32_t *order;         // [n_seq]
};
inline size_t layout_bytes(int n_seq) {
    return 2 * round256(sizeof(int32_t) * ((size_t)n_seq + 1));
}
// Fills them (packed sequences; one block).
cudaError_t launch_layout(const ScanProblem &p, Layout &l, cudaStream_t st);
// to <- from, or zero where from is null.
cudaError_t launch_states_copy(const float *from, float *to, long n, cudaStream_t st);

// The tokens of sequence s and its first slot.  Malformed packed offsets left
// every sequence without slots: it then has no tokens.
__device__ __forceinline__ void sequence(const ScanProblem &p, const Layout &l, int s, long &t0,
                                         int &len, long &slot0) {
    if (!p.cu) {
        t0 = (long)s * p.T;
        len = p.T;
        slot0 = (long)s * ((p.T + kTokens - 1) / kTokens);
    } else {
        t0 = p.cu[s];
        slot0 = l.slot_off[s];
        len = max(0, min(p.cu[s + 1] - (int)t0, (l.slot_off[s + 1] - (int)slot0) * kTokens));
    }
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

// Stages the B and C rows of tokens t0 .. t0 + n (group g) as fp32 [token][NP].
template <typename T, int NP>
__device__ __forceinline__ void stage_bc(const ScanProblem &p, long t0, int n, int g, float *Bs,
                                         float *Cs) {
    for (int i = threadIdx.x; i < n * NP; i += blockDim.x) {
        const int t = i / NP, k = i % NP;
        float b = 0.f, c = 0.f;
        if (k < p.N) {
            b = to_f32(static_cast<const T *>(p.Bm)[(t0 + t) * p.ld_B + (long)g * p.N + k]);
            c = to_f32(static_cast<const T *>(p.Cm)[(t0 + t) * p.ld_C + (long)g * p.N + k]);
        }
        Bs[i] = b;
        Cs[i] = c;
    }
}

}  // namespace scan
}  // namespace mdn
