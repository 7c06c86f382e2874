// Linear attention with a decay for each head: how sequences are cut and laid
// out, the segments' states joined, shared heads' gradients summed.  (The passes
// and their roles: mdn_attn.cuh; their kernels: mdn_attn_tc.cu, mdn_attn_tc32.cu.)
#include "mdn_attn.cuh"

namespace mdn {

// A segment's states cost a second reading of Y and W and their own products,
// so sequences are cut only where whole ones leave multiprocessors idle.  In
// units of the time a block takes for a chunk (1.7 us for bf16 rows, 6 for fp32):
// the blocks of a launch run in waves of 152, each of which fills its pipeline
// once; a chunk's states alone take 0.55, a segment reads the states of those
// before it, and the launch more costs what it costs.  (16384 tokens of 16 heads of
// 128 bf16 columns: 108 us cut in 9, 116 in 8, 446 whole.  Forward and gradients of
// 1531 fp32 tokens in 5 sequences, 6 heads on 3, 40 and 72 columns: 114, 135 whole.)
int attn_segment(int n_seq, long T_total, int H, int passes, mdn_dtype dtype) {
    if (n_seq == 0 || T_total == 0) return 0;
    const bool wide = dtype == MDN_F32;
    const double fill = wide ? 0.5 : 2.5, more = wide ? 1.0 : 3.0, read = wide ? 0.1 : 0.3;
    const long lines = (long)n_seq * H, mean = (T_total + n_seq - 1) / n_seq, chunks = (mean + 63) / 64;
    auto waves = [](long blocks) { return (blocks + 151) / 152; };
    const int states = passes > 1 ? 2 : 1;
    double best = waves(lines * passes) * (chunks + fill);
    long best_chunks = 0;
    for (long parts = 2; parts <= 64 && parts <= chunks; ++parts) {
        const long per = (chunks + parts - 1) / parts, n = (chunks + per - 1) / per;
        const double t = waves(lines * states * (n - 1)) * (per * 0.55 + fill) + more +
                         waves(lines * passes * n) * (per + fill + read * n);
        if (t < best) {
            best = t;
            best_chunks = per;
        }
    }
    return (int)(best_chunks * 64);
}

long attn_slots(int n_seq, long T_total, int seg) {
    return n_seq + (seg ? T_total / seg : 0);
}

namespace {

// Packed sequences: every sequence's slots, and the items, longest first.
__global__ void __launch_bounds__(1024) attn_layout_kernel(AttnProblem p) {
    __shared__ int sums[32];
    __shared__ int base;
    const bool ok = cu_well_formed(p.cu, p.n_seq, p.T_total);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        base = 0;
        if (!ok) atomicExch(p.status, MDN_ERR_INVALID_ARG);
        p.seg_off[p.n_seq + 1] = ok;
    }
    __syncthreads();
    for (int s0 = 0; s0 < p.n_seq; s0 += 1024) {
        const int s = s0 + tid;
        int len = 0, start = 0, n = 0;
        if (s < p.n_seq) {
            if (ok) {
                start = p.cu[s];
                len = p.cu[s + 1] - start;
            }
            n = p.seg ? max(1, (len + p.seg - 1) / p.seg) : 1;
        }
        int at = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, at, o);
            if (lane >= o) at += v;
        }
        if (lane == 31) sums[warp] = at;
        __syncthreads();
        if (warp == 0) {
            int v = sums[lane];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += u;
            }
            sums[lane] = v;
        }
        __syncthreads();
        at += base + (warp ? sums[warp - 1] : 0) - n;
        if (s < p.n_seq) {
            p.seg_off[s] = at;
            // whole sequences are ordered by their length (n_seq^2 / 1024
            // comparisons a thread, where that is quick)
            int place = at;
            if (!p.seg && ok && p.n_seq <= 2048) {
                place = 0;
                for (int j = 0; j < p.n_seq; ++j) {
                    const int other = p.cu[j + 1] - p.cu[j];
                    place += other > len || (other == len && j < s);
                }
            }
            for (int k = 0; k < n; ++k) {
                AttnItem it;
                it.start = start + k * p.seg;
                it.len = p.seg ? min(p.seg, len - k * p.seg) : len;
                it.seq = s;
                it.slot = at + k;
                it.k = k;
                it.n = n;
                it.tail = len - (n - 1) * p.seg;
                it.pad = 0;
                p.items[place + k] = it;
            }
        }
        __syncthreads();
        if (tid == 0) base += sums[31];
        __syncthreads();
    }
    if (tid == 0) p.seg_off[p.n_seq] = base;
    for (int i = base + tid; i < p.slots; i += 1024) p.items[i].slot = -1;
}

// Turns the segments' own states into the states they start from: V neighbouring
// elements of a state a thread, eight segments asked for at a time.  One thread
// of a block works out the decays: thousands of blocks of which every warp reads
// the head's own make the one sector that holds them the bottleneck (107 us
// instead of 8).
template <int V>
__global__ void __launch_bounds__(256) attn_combine_kernel(AttnProblem p, float *seg0, float *seg1, int size) {
    __shared__ float full, tail;
    __shared__ int s_n, s_off;
    const int s = blockIdx.x / p.H, h = blockIdx.x % p.H;
    const bool reversed = blockIdx.z != 0;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (threadIdx.x == 0) {
        int off, n;
        long len;
        if (p.cu) {
            off = p.seg_off[s];
            n = p.seg_off[s + 1] - off;
            len = p.seg_off[p.n_seq + 1] ? p.cu[s + 1] - p.cu[s] : 0;
        } else {
            n = max(1, (p.T + p.seg - 1) / p.seg);
            off = s * n;
            len = p.T;
        }
        const float l2 = log2_decay(p.log_decay, h);
        full = exp2f((float)p.seg * l2);
        tail = exp2f((float)(len - (long)(n - 1) * p.seg) * l2);
        s_n = n;
        s_off = off;
    }
    __syncthreads();
    const int e = (blockIdx.y * 256 + threadIdx.x) * V, n = s_n;
    if (e >= size) return;
    const float f = full;
    const long stride = (long)p.H * size, step = reversed ? -stride : stride;
    float *at = (reversed ? seg1 : seg0) + ((long)s_off * p.H + h) * size + e + (reversed ? (n - 1) * stride : 0);
    Packet<float, V> z = load_packet<float, V>(at + (n - 1) * step);       // (attn_keep_initial)
    for (int k0 = 0; k0 < n; k0 += 8) {
        Packet<float, V> own[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k0 + k < n - 1) own[k] = load_packet<float, V>(at + k * step);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k0 + k < n) {
                store_packet<float, V>(at + k * step, z);
                // (reversed, the sequence's short segment is the first)
                const float g = reversed && k0 + k == 0 ? tail : f;
                if (k0 + k < n - 1)
#pragma unroll
                    for (int v = 0; v < V; ++v) z.e[v] = fmaf(g, z.e[v], own[k].e[v]);
            }
        at += 8 * step;
    }
}

template <typename T>
__global__ void __launch_bounds__(256) attn_reduce_kernel(const float *part, T *out, const int32_t *ok, long rows, int d,
                                                          int shared) {
    if (ok && !*ok) return;
    const long total = rows * d;
    for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < total; i += (long)gridDim.x * 256) {
        const long r = i / d;
        const float *src = part + r * shared * d + (i - r * d);
        float s = src[0];
        for (int k = 1; k < shared; ++k) s += src[(long)k * d];
        out[i] = from_f32<T>(s);
    }
}

}  // namespace

cudaError_t launch_attn_layout(const AttnProblem &p, cudaStream_t st) {
    attn_layout_kernel<<<1, 1024, 0, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_attn(const AttnProblem &p, cudaStream_t st) {
    if (p.slots == 0) return cudaSuccess;
    return p.dtype == MDN_BF16 ? launch_attn_tc(p, st) : launch_attn_tc32(p, st);
}

cudaError_t launch_attn_combine(const AttnProblem &p, float *seg, float *seg_reversed, int size, cudaStream_t st) {
    const int V = size % 4 ? 1 : 4;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long)p.n_seq * p.H), (size / V + 255) / 256, seg_reversed ? 2 : 1);
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return V == 4 ? cudaLaunchKernelEx(&cfg, attn_combine_kernel<4>, p, seg, seg_reversed, size)
                  : cudaLaunchKernelEx(&cfg, attn_combine_kernel<1>, p, seg, seg_reversed, size);
}

cudaError_t launch_attn_reduce(const AttnProblem &p, const float *part, void *out, int d, int shared, cudaStream_t st) {
    const long rows = (long)p.T_total * (p.H / shared), total = rows * d;
    if (total == 0) return cudaSuccess;
    const long blocks = (total + 255) / 256;
    const unsigned grid = (unsigned)(blocks < 152 * 16 ? blocks : 152 * 16);
    const int32_t *ok = p.cu ? p.seg_off + p.n_seq + 1 : nullptr;
    if (p.dtype == MDN_BF16)
        attn_reduce_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(part, static_cast<__nv_bfloat16 *>(out), ok, rows, d, shared);
    else
        attn_reduce_kernel<float><<<grid, 256, 0, st>>>(part, static_cast<float *>(out), ok, rows, d, shared);
    return cudaGetLastError();
}

}  // namespace mdn
