// Linear attention with a decay for each head, fp32 rows, on the 5th-generation
// tensor cores: head widths up to 128, any alignment.  (The passes and their
// roles: mdn_attn.cuh; the chunk's products: mdn_attn_tc.cu.)
//
// Every operand is a sum of three bf16 parts (8 bits each, 24 together), and a
// product of operands the six products of parts that reach 2^-24 of it:
//   (3,1) (2,2) (1,3) (2,1) (1,2) (1,1)
// with fp32 sums, so results are nearly as fp32 arithmetic gives them.  Each MMA
// cuts the sum it adds to short; in this order most sums are still small then
// (the other way round the gradients over 1531 tokens are off by 1.5e-6, not
// 1.9e-7).  X, Y, W, D W and P are split on their way into shared memory, Z on
// its way into TMEM.
//
// One CTA of 16 warps takes a run of a sequence's tokens and one head, and goes
// through a chunk in steps that all warps share; the products of a chunk,
// 9.2 thousand cycles of the tensor pipe at widths of 128, overlap the steps
// between them:
//   split X, Y, W, D W | A, dZ, O1 issued | A -> P | O2 issued | Z | outputs
// Packed prompts of 32768 tokens, 16 heads of 128: 0.70 ms, bound by the splits
// and the steps between them; 5.9 ms on the CUDA cores in 4 x 4 register tiles.
#include "mdn_attn_tc.cuh"

namespace mdn {
namespace {

using namespace attn_tc;

constexpr int kThreads = 512;
constexpr uint32_t kOperand = 3 * kTile;          // three parts
constexpr uint32_t kOffX = 0, kOffY = kOperand, kOffW = 2 * kOperand, kOffD = 3 * kOperand;
constexpr uint32_t kOffP = 4 * kOperand;          // three parts of 64 x 64
constexpr uint32_t kOffBars = kOffP + 3 * kBlock;
constexpr uint32_t kBarsBytes = 1536;
constexpr uint32_t kSmem = kOffBars + kBarsBytes;
static_assert(kSmem <= 232448, "shared memory of one CTA");

// TMEM columns
constexpr uint32_t kColA = 0, kColO1 = 64, kColO2 = 128, kColD = 192, kColZ = 320 /* three of 64 */;
constexpr uint32_t kTmemCols = 512;

struct Bars {
    uint64_t a, d, o1, o2, drain;
    uint32_t tmem_base;
    int abort;
    float lam[kC + 1];                // l^e
    float enter[2][kC], leave[2][kC]; // as in mdn_attn_tc.cu: of whole chunks, of the partial one
};
static_assert(sizeof(Bars) <= kBarsBytes, "barrier block");

// Eight columns of a row as the operand's 16-byte packets.
__device__ __forceinline__ void put_parts(unsigned char *operand, uint32_t part_bytes, uint32_t at, const float *f) {
    uint32_t r[4][3];
#pragma unroll
    for (int q = 0; q < 4; ++q) split_parts<3>(f[2 * q], f[2 * q + 1], r[q]);
#pragma unroll
    for (int i = 0; i < 3; ++i)
        *reinterpret_cast<uint4 *>(operand + i * part_bytes + at) = make_uint4(r[0][i], r[1][i], r[2][i], r[3][i]);
}

// Columns [c, c + 8) of a row of `width`, zeros behind it.
template <int V>
__device__ __forceinline__ void load8(const float *row, int c, int width, float *f) {
    if (V == 4) {
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c + i < width) v = *reinterpret_cast<const float4 *>(row + c + i);
            f[i] = v.x;
            f[i + 1] = v.y;
            f[i + 2] = v.z;
            f[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = c + i < width ? row[c + i] : 0.f;
    }
}

__device__ __forceinline__ void prefetch_l2(const void *at) { asm volatile("prefetch.global.L2 [%0];" ::"l"(at)); }

// The six products of parts (counted from 0), the smallest first.
__device__ __forceinline__ void parts_of(int i, int &a, int &b) {
    a = i == 0 ? 2 : i == 1 || i == 3 ? 1 : 0;
    b = i == 2 ? 2 : i == 1 || i == 4 ? 1 : 0;
}

// V: 4 where all rows move 16 bytes at a time, else 1.
template <int V>
__global__ void __launch_bounds__(kThreads, 1) attn_tc32_kernel(const __grid_constant__ AttnProblem p) {
    extern __shared__ __align__(1024) unsigned char smem[];      // (the only shared memory: at its start)
    Bars *bars = reinterpret_cast<Bars *>(smem + kOffBars);
    volatile int *abort = &bars->abort;
    const AttnPass &a = p.pass[blockIdx.y];
    const int h = blockIdx.x % p.H;
    AttnItem it;
    grid_launch_dependents();
    grid_dependency_wait();
    if (!attn_item(p, blockIdx.x / p.H, it, reinterpret_cast<int *>(smem))) return;
    const bool states_only = a.out == nullptr;
    const bool closes = a.reversed ? it.first() : it.last();  // the sequence's last run in the pass's order
    if (states_only && closes) {
        attn_keep_initial(p, a, it, h);
        return;
    }
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int kd = a.kd, vd = a.vd, ksteps = (kd + 15) / 16;
    const int chunks = (it.len + kC - 1) / kC;
    const bool rev = a.reversed;

    if (tid == 0) {
        mbar_init(&bars->a, 1);
        mbar_init(&bars->d, 1);
        mbar_init(&bars->o1, 1);
        mbar_init(&bars->o2, 1);
        mbar_init(&bars->drain, 1);
        bars->abort = 0;
        fence_mbar_init();
    }
    if (tid < 2 * kC) {
        const float l2 = log2_decay(p.log_decay, h);
        const int i = tid & (kC - 1), n = tid < kC ? kC : it.len & (kC - 1);
        const float up = exp2f((float)(i + 1) * l2), down = i < n ? exp2f((float)(n - 1 - i) * l2) : 0.f;
        bars->enter[tid >> 6][i] = rev ? down : up;
        bars->leave[tid >> 6][i] = rev ? up : down;
        if (tid < kC) bars->lam[kC - 1 - i] = down;
        if (tid == kC - 1) bars->lam[kC] = up;
    }
    if (warp == 0) {
        tmem_alloc(&bars->tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    const float *lam = bars->lam;
    const int quad = warp & 3, group = warp >> 2;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    // the state: row `col` of Z^T, columns k0 .. k0 + 31
    const int col = quad * 32 + lane, k0 = group * 32;
    const bool mine = k0 < kd;
    float z[32];
    attn_initial<32>(p, a, it, h, a.init_t ? (long)col * kd + k0 : (long)k0 * vd + col, a.init_t ? 1 : vd,
                     col < vd ? kd - k0 : 0, z);
    auto put_state = [&]() {
        if (!mine) return;
        float part[3][16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            uint32_t r[3];
            split_parts<3>(z[2 * k], z[2 * k + 1], r);
#pragma unroll
            for (int i = 0; i < 3; ++i) part[i][k] = __uint_as_float(r[i]);
        }
#pragma unroll
        for (int i = 0; i < 3; ++i) tmem_st16(lanes + kColZ + i * 64 + k0 / 2, part[i]);
        tmem_st_wait();
    };
    if (!states_only) put_state();

    const float *X = static_cast<const float *>(a.X) + (long)(h / a.sx) * kd;
    const float *Y = static_cast<const float *>(a.Y) + (long)(h / a.sy) * kd;
    const float *W = static_cast<const float *>(a.W) + (long)(h / a.sw) * vd;
    const int kper = ksteps * 2, wper = (vd + 7) / 8;         // 16-byte packets of a row
    const uint32_t base = smem_u32(smem);
    const long step = (long)p.H * vd;
    bool fine = true;
    for (int c = 0; c < chunks && fine; ++c) {
        const int at = (rev ? chunks - 1 - c : c) * kC, n = min(kC, it.len - at);
        const long t0 = it.start + at;
        // ---- X, Y, W and D W into shared memory
        for (int i = tid; i < kC * kper; i += kThreads) {
            const int r = i / kper, ch = i - r * kper;
            const uint32_t to = (ch >> 3) * kBlock + sw128_offset(r, ch & 7);
            float f[8] = {}, g[8] = {};
            if (r < n) {
                if (!states_only) load8<V>(X + (t0 + r) * a.ld_x, ch * 8, kd, f);
                load8<V>(Y + (t0 + r) * a.ld_y, ch * 8, kd, g);
            }
            if (!states_only) put_parts(smem + kOffX, kTile, to, f);
            put_parts(smem + kOffY, kTile, to, g);
        }
        for (int i = tid; i < kC * wper; i += kThreads) {
            const int r = i / wper, ch = i - r * wper;
            const uint32_t to = (ch >> 3) * kBlock + sw128_offset(r, ch & 7);
            float f[8] = {};
            if (r < n) load8<V>(W + (t0 + r) * a.ld_w, ch * 8, vd, f);
#pragma unroll
            for (int q = 0; q < 8; ++q) f[q] *= a.w_scale;
            if (!states_only) put_parts(smem + kOffW, kTile, to, f);
            const float d = bars->leave[n < kC][r];
#pragma unroll
            for (int q = 0; q < 8; ++q) f[q] *= d;
            put_parts(smem + kOffD, kTile, to, f);
        }
        fence_proxy_async();
        tc_fence_before();
        __syncthreads();
        // ---- the products that need nothing else
        if (warp == 0) {
            tc_fence_after();
            if (elect_one()) {
                const uint32_t idesc_a = idesc_bf16(64, 64, false, false), idesc_d = idesc_bf16(128, ksteps * 16, true, true);
                const uint32_t idesc_o1 = idesc_bf16(128, 64, false, false);
                const uint64_t x0 = sdesc_sw128(base + kOffX, 16, 1024), y0 = sdesc_sw128(base + kOffY, 16, 1024);
                const uint64_t yt0 = sdesc_sw128(base + kOffY, kBlock, 1024), d0 = sdesc_sw128(base + kOffD, kBlock, 1024);
                auto along_k = [](int k) { return (uint32_t)((k >> 2) * (kBlock / 16) + (k & 3) * 2); };
                if (!states_only) {
#pragma unroll 1
                    for (int i = 0; i < 6; ++i) {
                        int pa, pb;
                        parts_of(i, pa, pb);
#pragma unroll 1
                        for (int k = 0; k < ksteps; ++k)
                            mma_bf16(tmem + kColA, x0 + pa * (kTile / 16) + along_k(k), y0 + pb * (kTile / 16) + along_k(k),
                                     idesc_a, (i | k) != 0);
                    }
                    mma_commit(&bars->a);
                }
#pragma unroll 1
                for (int i = 0; i < 6; ++i) {
                    int pa, pb;
                    parts_of(i, pa, pb);
#pragma unroll 1
                    for (int k = 0; k < 4; ++k)
                        mma_bf16(tmem + kColD, d0 + pa * (kTile / 16) + (uint32_t)(k * 128),
                                 yt0 + pb * (kTile / 16) + (uint32_t)(k * 128), idesc_d, (i | k) != 0);
                }
                mma_commit(&bars->d);
                if (!states_only) {
#pragma unroll 1
                    for (int i = 0; i < 6; ++i) {
                        int pa, pb;
                        parts_of(i, pa, pb);
#pragma unroll 1
                        for (int k = 0; k < ksteps; ++k)
                            mma_bf16_ta(tmem + kColO1, tmem + kColZ + pa * 64 + k * 8, x0 + pb * (kTile / 16) + along_k(k),
                                        idesc_o1, (i | k) != 0);
                    }
                    mma_commit(&bars->o1);
                }
            }
            __syncwarp();
        }
        // ---- the next chunk's rows into L2
        if (c + 1 < chunks) {
            const int at2 = (rev ? chunks - 2 - c : c + 1) * kC, n2 = min(kC, it.len - at2), r = tid >> 3, part = tid & 7;
            if (r < n2) {
                const long t = it.start + at2 + r;
                for (int k = part * 32; k < kd; k += 256) {
                    if (!states_only) prefetch_l2(X + t * a.ld_x + k);
                    prefetch_l2(Y + t * a.ld_y + k);
                }
                for (int k = part * 32; k < vd; k += 256) prefetch_l2(W + t * a.ld_w + k);
            }
        }
        // ---- A -> P: thread t and t + 16 of a warp take eight columns each of
        // 16, of row 16 quad + t % 16
        if (!states_only) {
            fine = warp_wait(&bars->a, c & 1, abort);
            tc_fence_after();
            const int i = quad * 16 + (lane & 15), j0 = group * 16 + (lane >> 4) * 8;
            float s[8];
            tmem_ld_16x2x8(lanes + kColA + group * 16, s);
            tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const int e = rev ? j0 + q - i : i - j0 - q;
                s[q] = e < 0 ? 0.f : s[q] * lam[max(e, 0)];
            }
            put_parts(smem + kOffP, kBlock, sw128_offset(i, j0 >> 3), s);
            fence_proxy_async();
            tc_fence_before();
            __syncthreads();
            if (warp == 0) {
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t idesc_o2 = idesc_bf16(128, 64, true, false);
                    const uint64_t w0 = sdesc_sw128(base + kOffW, kBlock, 1024), p0 = sdesc_sw128(base + kOffP, 16, 1024);
#pragma unroll 1
                    for (int q = 0; q < 6; ++q) {
                        int pa, pb;
                        parts_of(q, pa, pb);
#pragma unroll 1
                        for (int k = 0; k < 4; ++k)
                            mma_bf16(tmem + kColO2, w0 + pa * (kTile / 16) + (uint32_t)(k * 128),
                                     p0 + pb * (kBlock / 16) + (uint32_t)(k * 2), idesc_o2, (q | k) != 0);
                    }
                    mma_commit(&bars->o2);
                }
                __syncwarp();
            }
        }
        // ---- the state behind the chunk
        fine = warp_wait(&bars->d, c & 1, abort) && fine;
        tc_fence_after();
        const float f = lam[n];
        if (mine)
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                float d[16];
                tmem_ld16(lanes + kColD + k0 + m * 16, d);
                tmem_ld_wait();
#pragma unroll
                for (int q = 0; q < 16; ++q) z[m * 16 + q] = fmaf(f, z[m * 16 + q], d[q]);
            }
        if (!states_only) {
            fine = warp_wait(&bars->o1, c & 1, abort) && fine;
            tc_fence_after();
            if (c + 1 < chunks) put_state();
            // ---- outputs: 16 tokens of the warp's 32 columns
            fine = warp_wait(&bars->o2, c & 1, abort) && fine;
            tc_fence_after();
            float o1[16], o2[16];
            tmem_ld16(lanes + kColO1 + group * 16, o1);
            tmem_ld16(lanes + kColO2 + group * 16, o2);
            tmem_ld_wait();
            float *out = static_cast<float *>(a.out) + ((t0 + group * 16) * p.H + h) * vd + col;
            const float *enter = bars->enter[n < kC] + group * 16;
#pragma unroll
            for (int q = 0; q < 16; ++q, out += step)
                if (col < vd && group * 16 + q < n) *out = fmaf(enter[q], o1[q], o2[q]) * a.out_scale;
        }
        tc_fence_before();
        // (a wait that ran out ends the loop for all warps)
        fine = !__syncthreads_or(!fine);
        tc_fence_after();
    }
    if (!fine && warp == 0) {
        // whatever was issued completes before TMEM is freed
        if (elect_one()) {
            mma_commit(&bars->drain);
            int dummy = 0;
            mbar_wait(&bars->drain, 0, &dummy);
        }
        __syncwarp();
    }
    float *dst = nullptr;
    if (states_only) dst = a.seg_out + ((long)it.slot * p.H + h) * kd * vd;
    else if (a.fin && closes) dst = a.fin + ((long)it.seq * p.H + h) * kd * vd;
    if (dst && fine && col < vd)
#pragma unroll
        for (int k = 0; k < 32; ++k)
            if (k0 + k < kd) dst[(k0 + k) * vd + col] = z[k];
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && bars->abort) atomicExch(p.status, MDN_ERR_DEVICE_TIMEOUT);
    if (warp == 0) tmem_dealloc(tmem, kTmemCols);
}

template <int V>
cudaError_t launch(const AttnProblem &p, cudaStream_t st) {
    const cudaError_t err = allow_shared<attn_tc32_kernel<V>>(kSmem);
    if (err != cudaSuccess) return err;
    return launch_after(attn_tc32_kernel<V>, p, kThreads, kSmem, st, p);
}

}  // namespace

cudaError_t launch_attn_tc32(const AttnProblem &p, cudaStream_t st) {
    bool wide = true;
    for (int i = 0; i < p.n_pass; ++i) {
        const AttnPass &a = p.pass[i];
        wide = wide && a.kd % 4 == 0 && a.vd % 4 == 0 && rows_aligned(a.X, a.ld_x, 4, 16) && rows_aligned(a.Y, a.ld_y, 4, 16) &&
               rows_aligned(a.W, a.ld_w, 4, 16);
    }
    return wide ? launch<4>(p, st) : launch<1>(p, st);
}

}  // namespace mdn
