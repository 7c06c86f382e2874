// Linear attention with a decay for each head, in chunks of 64 tokens, on the
// CUDA cores: fp32 rows, any head widths up to 128, any alignment.  (The passes and their roles: mdn_attn.cuh.)
//
// Per chunk of n tokens with the state Z before it:
//   A_ij  = l^(i-j) w_scale X_i . Y_j  (j <= i, else 0)
//   out   = out_scale (A W + diag(l^(i+1)) X Z)
//   Z     = l^n Z + (diag(w_scale l^(n-1-j)) Y)^T W
// One block takes a run of a sequence's tokens, one head and 64 columns of W;
// every matrix is staged in shared memory in fp32 and multiplied in 4 x 4
// register tiles.
#include "mdn_attn.cuh"

namespace mdn {

// A segment's states cost a second reading of Y and W and their own products,
// so sequences are cut only where whole ones leave multiprocessors idle.  In
// units of the time a block takes for a chunk: the blocks of a launch run in
// waves of 152, each of which fills its pipeline once (2.5); a chunk's states
// alone take 0.45, and the two launches more that segments need 5.
int attn_segment(int n_seq, long T_total, int H, int passes) {
    if (n_seq == 0 || T_total == 0) return 0;
    const long lines = (long)n_seq * H, mean = (T_total + n_seq - 1) / n_seq, chunks = (mean + 63) / 64;
    auto waves = [](long blocks) { return (blocks + 151) / 152; };
    const int states = passes > 1 ? 2 : 1;
    double best = waves(lines * passes) * (chunks + 2.5);
    long best_chunks = 0;
    for (long parts = 2; parts <= 64 && parts * 4 <= chunks; ++parts) {
        const long per = (chunks + parts - 1) / parts, n = (chunks + per - 1) / per;
        const double t = waves(lines * states * (n - 1)) * (per * 0.45 + 2.5) + 5 + waves(lines * passes * n) * (per + 2.5);
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

constexpr int kC = 64;              // tokens of a chunk
constexpr int kV = 64;              // columns of W a block takes
constexpr int kPitch = kV + 4;

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
                it.first = k == 0;
                it.last = k == n - 1;
                it.pad0 = it.pad1 = 0;
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

__global__ void __launch_bounds__(256) attn_kernel(AttnProblem p) {
    extern __shared__ __align__(16) float smem[];
    __shared__ float lam[kC + 1];
    const AttnPass &a = p.pass[blockIdx.y];
    const int h = blockIdx.x % p.H, c0 = blockIdx.z * kV;
    AttnItem it;
    if (!attn_item(p, blockIdx.x / p.H, it, reinterpret_cast<int *>(smem)) || c0 >= a.vd) return;
    const bool states_only = a.out == nullptr;
    const bool closes = a.reversed ? it.first : it.last;      // the sequence's last run in the pass's order
    if (states_only && closes) return;                        // no run starts from that state
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int KR = (a.kd + 7) & ~7, KS = KR + 4, cols = min(kV, a.vd - c0);
    float *Xs = smem, *Ys = Xs + kC * KS, *Ws = Ys + kC * KS, *As = Ws + kC * kPitch, *Zs = As + kC * kPitch;
    const float l2 = log2_decay(p.log_decay, h);
    if (tid <= kC) lam[tid] = exp2f((float)tid * l2);

    // the state: rows 8 ty .., columns 4 tx ..
    float z[8][4];
    {
        const bool opens = a.reversed ? it.last : it.first;
        const float *src = nullptr;
        if (!states_only) {
            if (a.seg_init) src = a.seg_init + ((long)it.slot * p.H + h) * a.kd * a.vd;
            else if (a.init && opens) src = a.init + ((long)it.seq * p.H + h) * a.kd * a.vd;
        }
#pragma unroll
        for (int r = 0; r < 8; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int k = ty * 8 + r, col = c0 + tx * 4 + c;
                z[r][c] = src && k < a.kd && col < a.vd
                              ? src[a.init_t ? (long)col * a.kd + k : (long)k * a.vd + col] : 0.f;
            }
    }
    auto put_state = [&]() {
        if (ty * 8 < KR)
#pragma unroll
            for (int r = 0; r < 8; ++r)
                *reinterpret_cast<float4 *>(Zs + (ty * 8 + r) * kPitch + tx * 4) = make_float4(z[r][0], z[r][1], z[r][2], z[r][3]);
    };
    put_state();

    const float *X = static_cast<const float *>(a.X) + (long)(h / a.sx) * a.kd;
    const float *Y = static_cast<const float *>(a.Y) + (long)(h / a.sy) * a.kd;
    const float *W = static_cast<const float *>(a.W) + (long)(h / a.sw) * a.vd + c0;
    const int chunks = (it.len + kC - 1) / kC;
    for (int c = 0; c < chunks; ++c) {
        const int at = (a.reversed ? chunks - 1 - c : c) * kC, n = min(kC, it.len - at);
        const long t0 = it.start + at;
        __syncthreads();                                      // the last chunk's readers are done
        for (int i = tid; i < kC * KR; i += 256) {
            const int r = i / KR, k = i - r * KR;
            const bool in = r < n && k < a.kd;
            if (!states_only) Xs[r * KS + k] = in ? X[(t0 + r) * a.ld_x + k] : 0.f;
            Ys[r * KS + k] = in ? Y[(t0 + r) * a.ld_y + k] : 0.f;
        }
        for (int i = tid; i < kC * kV; i += 256) {
            const int r = i / kV, k = i - r * kV;
            Ws[r * kPitch + k] = r < n && k < cols ? W[(t0 + r) * a.ld_w + k] * a.w_scale : 0.f;
        }
        __syncthreads();
        if (!states_only) {
            float s[4][4] = {};
            for (int k = 0; k < KR; k += 4) {
                float4 x[4], y[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    x[r] = *reinterpret_cast<const float4 *>(Xs + (ty + 16 * r) * KS + k);
                    y[r] = *reinterpret_cast<const float4 *>(Ys + (tx + 16 * r) * KS + k);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        s[r][q] = fmaf(x[r].x, y[q].x, s[r][q]);
                        s[r][q] = fmaf(x[r].y, y[q].y, s[r][q]);
                        s[r][q] = fmaf(x[r].z, y[q].z, s[r][q]);
                        s[r][q] = fmaf(x[r].w, y[q].w, s[r][q]);
                    }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int i = ty + 16 * r, j = tx + 16 * q, e = a.reversed ? j - i : i - j;
                    As[i * kPitch + j] = e < 0 ? 0.f : s[r][q] * lam[e];
                }
            __syncthreads();
            float o[4][4] = {};
            for (int k = 0; k < KR; k += 4) {
                float4 x[4], zr[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    x[r] = *reinterpret_cast<const float4 *>(Xs + (ty + 16 * r) * KS + k);
                    zr[r] = *reinterpret_cast<const float4 *>(Zs + (k + r) * kPitch + tx * 4);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float xs[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        o[r][0] = fmaf(xs[q], zr[q].x, o[r][0]);
                        o[r][1] = fmaf(xs[q], zr[q].y, o[r][1]);
                        o[r][2] = fmaf(xs[q], zr[q].z, o[r][2]);
                        o[r][3] = fmaf(xs[q], zr[q].w, o[r][3]);
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = ty + 16 * r;
                const float f = i < n ? lam[a.reversed ? n - 1 - i : i + 1] : 0.f;
#pragma unroll
                for (int q = 0; q < 4; ++q) o[r][q] *= f;
            }
            for (int j = 0; j < n; j += 4) {
                float4 s4[4], w[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    s4[r] = *reinterpret_cast<const float4 *>(As + (ty + 16 * r) * kPitch + j);
                    w[r] = *reinterpret_cast<const float4 *>(Ws + (j + r) * kPitch + tx * 4);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float sr[4] = {s4[r].x, s4[r].y, s4[r].z, s4[r].w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        o[r][0] = fmaf(sr[q], w[q].x, o[r][0]);
                        o[r][1] = fmaf(sr[q], w[q].y, o[r][1]);
                        o[r][2] = fmaf(sr[q], w[q].z, o[r][2]);
                        o[r][3] = fmaf(sr[q], w[q].w, o[r][3]);
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = ty + 16 * r;
                if (i >= n) continue;
                const long row = ((t0 + i) * p.H + h) * a.vd + c0;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int col = tx * 4 + q;
                    if (col >= cols) continue;
                    static_cast<float *>(a.out)[row + col] = o[r][q] * a.out_scale;
                }
            }
        }
        if (ty * 8 < KR) {
            const float f = lam[n];
#pragma unroll
            for (int r = 0; r < 8; ++r)
#pragma unroll
                for (int q = 0; q < 4; ++q) z[r][q] *= f;
            for (int j = 0; j < n; ++j) {
                const float d = lam[a.reversed ? j + 1 : n - 1 - j];
                float4 w = *reinterpret_cast<const float4 *>(Ws + j * kPitch + tx * 4);
                w.x *= d; w.y *= d; w.z *= d; w.w *= d;
                const float4 y0 = *reinterpret_cast<const float4 *>(Ys + j * KS + ty * 8);
                const float4 y1 = *reinterpret_cast<const float4 *>(Ys + j * KS + ty * 8 + 4);
                const float y[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    z[r][0] = fmaf(y[r], w.x, z[r][0]);
                    z[r][1] = fmaf(y[r], w.y, z[r][1]);
                    z[r][2] = fmaf(y[r], w.z, z[r][2]);
                    z[r][3] = fmaf(y[r], w.w, z[r][3]);
                }
            }
        }
        __syncthreads();                                      // Zs has been read
        put_state();
    }
    float *dst = nullptr;
    if (states_only) dst = a.seg_out + ((long)it.slot * p.H + h) * a.kd * a.vd;
    else if (a.fin && closes) dst = a.fin + ((long)it.seq * p.H + h) * a.kd * a.vd;
    if (!dst) return;
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int k = ty * 8 + r, col = c0 + tx * 4 + c;
            if (k < a.kd && col < a.vd) dst[(long)k * a.vd + col] = z[r][c];
        }
}

// Four neighbouring elements of a state a thread, along the segments of their
// sequence, eight of which it asks for at a time.  One thread of a block works
// out the decays: 64 x 64 blocks of which every warp reads the head's own make
// the one sector that holds them the bottleneck (107 us instead of 8).
template <int V>
__global__ void __launch_bounds__(256) attn_combine_kernel(AttnProblem p, AttnCombine c) {
    __shared__ float full, tail;
    __shared__ int s_n, s_off;
    const int s = blockIdx.x / p.H, h = blockIdx.x % p.H;
    const bool reversed = blockIdx.z != 0;
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
    if (e >= c.size) return;
    const float f = full;
    const float *init = c.init[reversed];
    const long stride = (long)p.H * c.size, step = reversed ? -stride : stride;
    float *at = c.seg[reversed] + ((long)s_off * p.H + h) * c.size + e + (reversed ? (n - 1) * stride : 0);
    Packet<float, V> z;
#pragma unroll
    for (int v = 0; v < V; ++v) z.e[v] = 0.f;
    if (init) z = load_packet<float, V>(init + ((long)s * p.H + h) * c.size + e);
    for (int k0 = 0; k0 < n; k0 += 8) {
        Packet<float, V> own[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k0 + k < n - 1) own[k] = load_packet<float, V>(at + k * step);    // the last one's leads nowhere
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

int attn_smem(int kd) {
    const int KR = (kd + 7) & ~7, KS = KR + 4;
    return (2 * kC * KS + 2 * kC * kPitch + KR * kPitch) * (int)sizeof(float);
}

}  // namespace

cudaError_t launch_attn_layout(const AttnProblem &p, cudaStream_t st) {
    attn_layout_kernel<<<1, 1024, 0, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_attn(const AttnProblem &p, cudaStream_t st) {
    if (p.slots == 0) return cudaSuccess;
    if (p.dtype == MDN_BF16) return launch_attn_tc(p, st);
    int kd = 0, vd = 0;
    for (int i = 0; i < p.n_pass; ++i) {
        kd = kd > p.pass[i].kd ? kd : p.pass[i].kd;
        vd = vd > p.pass[i].vd ? vd : p.pass[i].vd;
    }
    const dim3 grid((unsigned)(p.slots * (long)p.H), p.n_pass, (vd + kV - 1) / kV);
    const int smem = attn_smem(kd);
    const cudaError_t err = allow_shared<attn_kernel>(attn_smem(128));
    if (err != cudaSuccess) return err;
    attn_kernel<<<grid, 256, smem, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_attn_combine(const AttnProblem &p, const AttnCombine &c, cudaStream_t st) {
    const int V = c.size % 4 ? 1 : 4;
    const dim3 grid((unsigned)((long)p.n_seq * p.H), (c.size / V + 255) / 256, c.seg[1] ? 2 : 1);
    if (V == 4) attn_combine_kernel<4><<<grid, 256, 0, st>>>(p, c);
    else attn_combine_kernel<1><<<grid, 256, 0, st>>>(p, c);
    return cudaGetLastError();
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
