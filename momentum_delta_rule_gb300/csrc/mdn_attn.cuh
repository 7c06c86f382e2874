// Declarations shared by the translation units of linear attention with a
// decay for each head and of the group norm.
#pragma once

#include "mdn_ssm.cuh"

namespace mdn {

// Everything here is one computation with different roles.  A pass takes rows
// X, Y (kd wide) and W (vd wide) and a state Z [kd, vd], and computes along the
// tokens, with the decay l of the head,
//   out_i = out_scale (sum_{j <= i} l^(i-j) w_scale (X_i . Y_j) W_j + l^(i+1) Z^T X_i)
//   Z    <- l^n Z + sum_j l^(n-1-j) w_scale Y_j W_j^T
// or, reversed, with j >= i, l^(j-i), and the state that the last token sees:
//   out_i = ... + l^(n-1-i) Z^T X_i,    Z <- l^n Z + sum_j l^(j+1) w_scale Y_j W_j^T.
//   forward   X = q,  Y = k,  W = v,  Z = S
//   dq        X = do, Y = v,  W = k,  Z = S^T
//   dk        X = v,  Y = do, W = q,  Z = dS^T, reversed
//   dv        X = k,  Y = q,  W = do, Z = dS,   reversed
struct AttnPass {
    const void *X, *Y, *W;
    long ld_x, ld_y, ld_w;          // elements between tokens
    int sx, sy, sw;                 // query heads that share a head of X, Y, W
    int kd, vd;
    bool reversed;
    float out_scale, w_scale;
    void *out;                      // [tokens, H, vd], dense; or nullptr (states only)
    bool out_f32;                   // fp32 whatever the dtype
    const float *init;              // [n_seq, H, ...] states the sequences start from, or nullptr
    const float *seg_init;          // [slot, H, ...] the segments' own states, or nullptr
    bool combined;                  // ... or already the states they start from
    bool init_t;                    // those lie transposed, [vd, kd]
    float *fin;                     // [n_seq, H, kd, vd] or nullptr
    float *seg_out;                 // states only: [slot, H, kd, vd] of the segments alone
};

// A run of tokens of one sequence that one block takes.
struct AttnItem {
    int start, len, seq, slot;
    int k, n;                       // which segment of the sequence, of how many
    int tail;                       // tokens of the last one
    int pad;

    __host__ __device__ bool first() const { return k == 0; }
    __host__ __device__ bool last() const { return k == n - 1; }
};

struct AttnProblem {
    AttnPass pass[3];
    int n_pass;
    const float *log_decay;
    int H, n_seq, T, T_total;
    int seg;                        // tokens of a segment (a multiple of 64), 0: whole sequences
    int slots;                      // items, for packed sequences at most
    const int32_t *cu;              // device, or nullptr for equal lengths
    AttnItem *items;                // packed: slots items, longest first, or nullptr (attn_item)
    int32_t *seg_off;               // packed: [n_seq + 1] slots of the sequences; [n_seq + 1] more: whether cu is well formed
    mdn_dtype dtype;
    int *status;
};

struct AttnStepProblem {
    const void *q, *k, *v;
    const float *log_decay, *S;
    float *S_out;
    void *o;
    int n, H, shared, dk, dv;       // shared: query heads of a key and value head
    float scale;
    long ld_q, ld_k, ld_v;
    mdn_dtype dtype;
};

struct GroupNormProblem {
    const void *x, *gate, *dy;
    const float *weight, *bias;
    void *y, *dx, *dgate;
    float *stats, *dw, *dbias;
    const int32_t *cu;
    int n_seq, T;                   // sequences (over_sequence) and their length when equal
    long rows;
    int D, G, act;
    bool over_sequence, center;
    float eps;
    long ld_x, ld_gate, ld_dy;
    mdn_dtype dtype;
    unsigned char *ws;
    int *ok;                        // whether cu is well formed, or nullptr
    int *status;
};

// Tokens of a segment (0: none), and the most slots they take.
int attn_segment(int n_seq, long T_total, int H, int passes, mdn_dtype dtype);
long attn_slots(int n_seq, long T_total, int seg);

cudaError_t launch_attn_layout(const AttnProblem &p, cudaStream_t st);
cudaError_t launch_attn(const AttnProblem &p, cudaStream_t st);
cudaError_t launch_attn_tc(const AttnProblem &p, cudaStream_t st);      // bf16 rows
cudaError_t launch_attn_tc32(const AttnProblem &p, cudaStream_t st);    // fp32 rows
// Segments' own states [slot, H, size] (the second: reversed, or nullptr) -> the
// states they start from.
cudaError_t launch_attn_combine(const AttnProblem &p, float *seg, float *seg_reversed, int size, cudaStream_t st);
// out [tokens, H / shared, d] <- sums over the heads that share, of fp32 rows.
cudaError_t launch_attn_reduce(const AttnProblem &p, const float *part, void *out, int d, int shared,
                               cudaStream_t st);
cudaError_t launch_attn_step(const AttnStepProblem &p, cudaStream_t st);

cudaError_t launch_group_norm_fwd(const GroupNormProblem &p, cudaStream_t st);
cudaError_t launch_group_norm_bwd(const GroupNormProblem &p, cudaStream_t st);
size_t group_norm_fwd_workspace(int n_seq, long rows, int D, int G, bool over_sequence, mdn_dtype dtype);
size_t group_norm_bwd_workspace(int n_seq, long rows, int D, int G, bool over_sequence, mdn_dtype dtype);

// ---------------------------------------------------------------- device

// The head's decay as a power of two: l^e = 2^(e * log2_decay).  A decay of
// zero (-inf) becomes a finite number, so that l^0 is 1.
__device__ __forceinline__ float log2_decay(const float *log_decay, int h) {
    const float l = log_decay[h] * kLog2e;
    return l < -1e30f ? -1e30f : l;
}

// The item of block i (whole CTA; uniform result).  Few packed sequences that
// are not cut order themselves, longest first: a kernel that does it costs 5 us
// and its launch.  scratch: kAttnOrdered + 8 ints of shared memory.
constexpr int kAttnOrdered = 256;
__device__ __forceinline__ bool attn_item(const AttnProblem &p, int i, AttnItem &it, int *scratch) {
    if (p.cu && p.items) {
        it = p.items[i];
        return it.slot >= 0;
    }
    if (p.cu) {
        const int tid = threadIdx.x;
        const bool ok = cu_well_formed(p.cu, p.n_seq, p.T_total);
        if (tid == 0 && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) {
            if (!ok) atomicExch(p.status, MDN_ERR_INVALID_ARG);
            p.seg_off[p.n_seq + 1] = ok;
        }
        int *lens = scratch + 8;
        int start = 0, len = 0;
        if (tid < p.n_seq) {
            if (ok) {
                start = p.cu[tid];
                len = p.cu[tid + 1] - start;
            }
            lens[tid] = len;
        }
        __syncthreads();
        if (tid < p.n_seq) {
            int place = 0;
            for (int j = 0; j < p.n_seq; ++j) place += lens[j] > len || (lens[j] == len && j < tid);
            if (place == i) {
                scratch[0] = start;
                scratch[1] = len;
                scratch[2] = tid;
            }
        }
        __syncthreads();
        it.start = scratch[0];
        it.len = scratch[1];
        it.seq = it.slot = scratch[2];
        it.k = 0;
        it.n = 1;
        it.tail = it.len;
        __syncthreads();
        return true;
    }
    const int per = p.seg ? max(1, (p.T + p.seg - 1) / p.seg) : 1;
    const int s = i / per, k = i - s * per;
    it.seq = s;
    it.slot = i;
    it.start = s * p.T + k * p.seg;
    it.len = p.seg ? min(p.seg, p.T - k * p.seg) : p.T;
    it.k = k;
    it.n = per;
    it.tail = p.T - (per - 1) * p.seg;
    return true;
}

// Where sequences are cut, the last segment of a pass's order leaves no state to
// another: its place keeps the state that its sequence starts from, which may
// be overwritten by the time a later block asks for it (final states may replace
// the initial ones).
__device__ __forceinline__ void attn_keep_initial(const AttnProblem &p, const AttnPass &a, const AttnItem &it, int h) {
    const long size = (long)a.kd * a.vd;
    const float *src = a.init ? a.init + ((long)it.seq * p.H + h) * size : nullptr;
    float *dst = a.seg_out + ((long)it.slot * p.H + h) * size;
    for (int i = threadIdx.x; i < size; i += blockDim.x) dst[i] = src ? src[i] : 0.f;
}

// The state a run of tokens starts from: elements [0, N) of a thread, `step`
// apart from element `at` of a state [kd, vd] or its transpose on, of which `take`
// are there.  Where sequences are cut: the sequence's initial state and the
// segments' own ones before this run's (behind it, reversed), in their order,
// unless a kernel of its own has joined them.
template <int N>
__device__ __forceinline__ void attn_initial(const AttnProblem &p, const AttnPass &a, const AttnItem &it, int h, long at, long step,
                                             int take, float *z) {
    const long size = (long)a.kd * a.vd, next = (a.reversed ? -1 : 1) * (long)p.H * size;
    const int before = a.reversed ? it.n - 1 - it.k : it.k;      // segments of the sequence
    const float *src = nullptr;
    if (a.out != nullptr && a.seg_init)
        src = a.seg_init + ((long)(a.combined ? it.slot : a.reversed ? it.slot - it.k : it.slot + (it.n - 1 - it.k)) * p.H + h) * size + at;
    else if (a.out != nullptr && a.init)
        src = a.init + ((long)it.seq * p.H + h) * size + at;
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = src && i < take ? src[i * step] : 0.f;
    if (a.out == nullptr || !a.seg_init || a.combined) return;
    const float l2 = log2_decay(p.log_decay, h), full = exp2f((float)p.seg * l2), tail = exp2f((float)it.tail * l2);
    src = a.seg_init + ((long)(a.reversed ? it.slot + before : it.slot - before) * p.H + h) * size + at;
    for (int j = 0; j < before; ++j, src += next) {
        const float f = a.reversed && j == 0 ? tail : full;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < take) z[i] = fmaf(f, z[i], src[i * step]);
    }
}

}  // namespace mdn
