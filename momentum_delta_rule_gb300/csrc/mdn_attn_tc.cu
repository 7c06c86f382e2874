// Linear attention with a decay for each head on the 5th-generation tensor
// cores: bf16 rows, head widths up to 128.  (The passes and their roles:
// mdn_attn.cuh.)
//
// Per chunk of n <= 64 tokens, with the state Z before it and everything
// transposed, so that every large product has 128 rows (columns of W) whatever
// the chunk's length:
//   MMA1  A    = X Y^T                    M 64 tokens, N 64, K kd
//   MMA2  O1^T = Z^T X^T                  M vd, N 64, K kd; Z^T as two bf16 parts from TMEM
//   MMA3  O2^T = W^T P^T                  M vd, N 64, K 64;  P_ij = l^(i-j) w_scale A_ij as two bf16 parts
//   MMA4  dZ^T = (D W)^T Y                M vd, N kd, K 64;  D_j = w_scale l^(n-1-j)
//   out^T = out_scale (l^(i+1) O1^T + O2^T),   Z = l^n Z + dZ
//
// The decays l^(i+1) of O1 are applied to the fp32 result and the state is kept
// in fp32 registers.  A term of out passes one operand that is not bf16 as it
// comes, P or Z: in two parts (2^-17 of it), so that out is rounded once, to its
// type.  D W comes in three parts, all 24 bits of an fp32 product, and Y is bf16, so
// that states are as exact as fp32 has them: off by 2e-7.  (One part of P and Z
// and two of D W: outputs off by 2.3e-3 instead of 1.7e-3, states by 4e-6, and
// the prompts below take 104 us instead of 134.)
//
// One CTA takes a run of a sequence's tokens and one head.  Warps: 0 and 1 copy
// X, Y and W into the 128-byte-swizzled operand layout; 2 issues MMA1 and MMA4,
// 3 owns TMEM and issues MMA2 and MMA3; 4..7 turn A into P; 8..11 write the
// outputs; 12..27 keep Z, 32 columns each of their TMEM quadrant's 32 rows, and
// split the next chunk's D W (for states alone warps 4..11 do).  The only chain
// along the tokens is MMA4 -> Z -> MMA2.  TMEM is full: A lies in the buffer of the
// O2 that it leads to, which is written when A has been read.
//
// Rows on 16-byte boundaries come by TMA, others with cp.async or plain loads.
// In a sequence's last, partial chunk the tokens behind its end are zeros and
// not the next sequence's.  (Outputs staged in the chunk's X tile by stmatrix
// and stored by TMA took fewer instructions, but kept the tile from the next
// load.)
//
// What it is made for is few instructions: 28 warps of six roles share four
// schedulers and an instruction cache, so that every instruction saved shortens
// all the handovers; the roles' loops are kept short (straight code that each
// warp runs once a chunk waits for its instructions).  The issuers' are not: what
// is added to a descriptor is known, two instructions an MMA (in loops the same
// products took 154 us, up to 150 cycles an MMA).  Packed prompts of 32768 tokens in
// 21 sequences, 16 heads of 128: 134 us, calls one behind another (537 MB, 0.59 of
// the copy rate).  A sixth of that is fill and uneven ends; in between a chunk takes
// some 3600 cycles.  No unit is full then (tensor pipe 43 % of the cycles, issue slots
// 63 %, DRAM 49 %): its products are 3040 cycles where each runs by itself (MMA1 58 a
// step, MMA2 43, MMA3 77, MMA4 106) but two issuers' are in turns and slower, a
// barrier that is already complete takes 200 to 400 cycles to see, and the state's
// warps do one thing after another: split, dZ, Z.  Tried: four warps that do nothing
// but split 133 (one long prompt 112 instead of 109, training 191 instead of 187);
// the split behind dZ, in one buffer, 145; one issuer in a fixed order 159; MMA3
// without the blocks that are zero 138.
// Every wait is bounded (1 s); on expiry the CTA records MDN_ERR_DEVICE_TIMEOUT,
// drains its copies and MMAs, frees TMEM and returns.
#include "mdn_attn_tc.cuh"

namespace mdn {
namespace {

using namespace attn_tc;

constexpr int kThreads = 896;
// Places for chunks: two of X and Y, three of W, which is split a chunk ahead.
constexpr int kStages = 2, kStagesW = 3;
constexpr uint32_t kStage = 2 * kTile;                                // X, Y
constexpr uint32_t kOffW = kStages * kStage;
constexpr uint32_t kOffParts = kOffW + kStagesW * kTile;              // two buffers of D W in three parts
constexpr uint32_t kOffP = kOffParts + 6 * kTile;                     // two parts of P
constexpr uint32_t kOffBars = kOffP + 2 * kBlock;
constexpr uint32_t kBarsBytes = 2560;
constexpr uint32_t kSmem = kOffBars + kBarsBytes;
static_assert(kSmem <= 232448, "shared memory of one CTA");

// TMEM columns
constexpr uint32_t kColO = 0 /* two of O1, O2: 64 each */, kColA = 64 /* in O2, read before it is written */;
constexpr uint32_t kColD = 256, kColZ = 384 /* two parts of 64 */;
constexpr uint32_t kTmemCols = 512;

struct Bars {
    uint64_t full[kStages], empty[kStages], full_w[kStagesW], empty_w[kStagesW];
    // What one side may do twice before the other looks has a barrier for each
    // buffer: a wait sees no more than the last completion.
    uint64_t o1_done, d_ready, d_free, z_ready, p_ready, partial, drain[2];
    uint64_t a_ready[2], parts_ready[2], parts_free[2], o_ready[2], o_free[2];
    uint32_t tmem_base;
    int abort;
    float lam[kC + 1];                // l^e
    float within[kC];                 // l^e w_scale out_scale: the decays of A
    // what enters with the state decays by l^(i+1) out_scale, what leaves with it
    // by l^(n-1-i) w_scale; reversed, the other way round.  [0]: whole chunks,
    // [1]: the run's partial one.
    alignas(16) float enter[2][kC], leave[2][kC];
};
static_assert(sizeof(Bars) <= kBarsBytes, "barrier block");

// Arrives on `bar` when all of this thread's cp.async so far have landed.
__device__ __forceinline__ void copies_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// 4 bytes, or zeros.
__device__ __forceinline__ void cp_async_or_zero(uint32_t dst, const void *src, bool take) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(take ? 4 : 0) : "memory");
}

// Without TMA: one warp copies rows [from, to) of `width` columns into a tile
// (zeros from the n-th on), V elements (one or two) at a time.
template <int V>
__device__ __forceinline__ void copy_tile(uint32_t tile, const __nv_bfloat16 *src, long ld, int width, int n, int from,
                                          int to) {
    const int lane = threadIdx.x & 31;
    const int per = width / V;
    if constexpr (V == 1) {
        const int total = to * per;
        for (int base = from * per; base < total; base += 32 * 8) {
            unsigned short v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int i = base + u * 32 + lane, r = i / per;
                v[u] = i < total && r < n ? *reinterpret_cast<const unsigned short *>(src + r * ld + (i - r * per)) : 0;
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int i = base + u * 32 + lane, r = i / per, c = i - r * per;
                if (i < total)
                    asm volatile("st.shared.b16 [%0], %1;" ::"r"(tile + (c >> 6) * kBlock + sw128_offset(r, (c & 63) >> 3) +
                                                                 (c & 7) * 2),
                                 "h"(v[u])
                                 : "memory");
            }
        }
    } else {
        const int total = to * per;
        for (int i = from * per + lane; i < total; i += 32) {
            const int r = i / per, c = (i - r * per) * V;
            cp_async_or_zero(tile + (c >> 6) * kBlock + sw128_offset(r, (c & 63) >> 3) + (c & 7) * 2,
                             r < n ? src + r * ld + c : src, r < n);
        }
    }
}

// V: elements that X, Y and W move at a time; 8: by TMA.
struct Maps {
    CUtensorMap x, y, w;
};
struct AllMaps {
    Maps pass[3];
};

template <int V>
__global__ void __launch_bounds__(kThreads, 1)
attn_tc_kernel(const __grid_constant__ AttnProblem p, const __grid_constant__ AllMaps maps) {
    constexpr bool kTma = V == 8;
    extern __shared__ __align__(1024) unsigned char smem_raw[];    // (the only shared memory: at its start)
    unsigned char *smem = smem_raw;
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
    auto chunk_at = [&](int c) { return (rev ? chunks - 1 - c : c) * kC; };
    auto chunk_len = [&](int c) { return min(kC, it.len - chunk_at(c)); };

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bars->full[i], kTma ? 1 : 64);
            mbar_init(&bars->empty[i], states_only ? 1 : 2);   // MMA4, MMA2
        }
        for (int i = 0; i < kStagesW; ++i) {
            mbar_init(&bars->full_w[i], kTma ? 1 : 64);
            mbar_init(&bars->empty_w[i], 1);                   // MMA3, or for states alone MMA4
        }
        mbar_init(&bars->o1_done, 1);
        mbar_init(&bars->d_ready, 1);
        mbar_init(&bars->d_free, 16);
        mbar_init(&bars->z_ready, 16);
        mbar_init(&bars->p_ready, 4);
        mbar_init(&bars->partial, 2);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->drain[i], 1);
            mbar_init(&bars->a_ready[i], 1);
            mbar_init(&bars->parts_ready[i], states_only ? 8 : 16);
            mbar_init(&bars->parts_free[i], 1);
            mbar_init(&bars->o_ready[i], 1);
            mbar_init(&bars->o_free[i], 4);
        }
        bars->abort = 0;
        fence_mbar_init();
    }
    if (tid < 2 * kC) {
        const float l2 = log2_decay(p.log_decay, h);
        const int i = tid & (kC - 1), n = tid < kC ? kC : it.len & (kC - 1);
        const float up = exp2f((float)(i + 1) * l2), down = i < n ? exp2f((float)(n - 1 - i) * l2) : 0.f;
        bars->enter[tid >> 6][i] = (rev ? down : up) * a.out_scale;
        bars->leave[tid >> 6][i] = (rev ? up : down) * a.w_scale;
        if (tid < kC) {
            bars->lam[kC - 1 - i] = down;
            bars->within[kC - 1 - i] = down * (a.w_scale * a.out_scale);
            if (i == kC - 1) bars->lam[kC] = up;
        }
    }
    // P's masked halves stay zero
    for (uint32_t i = tid; i < 2 * kBlock / 16; i += kThreads)
        *reinterpret_cast<uint4 *>(smem + kOffP + i * 16) = make_uint4(0, 0, 0, 0);
    if (!kTma && (kd & 15))    // the products' last step reads up to the next 16 columns of X and Y
        for (uint32_t i = tid; i < kOffParts / 16; i += kThreads)
            *reinterpret_cast<uint4 *>(smem + i * 16) = make_uint4(0, 0, 0, 0);
    if (warp == 3) {
        tmem_alloc(&bars->tmem_base, kTmemCols);
        tmem_relinquish();
    }
    fence_proxy_async();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    const float *lam = bars->lam;      // [0 .. 64]
    // Thread t of `of` splits its share of chunk c's W.
    auto split_chunk = [&](int c, int t, int of) {
        const int per = (vd + 7) / 8, total = kC * per;
        const bool whole = per == 16 || per == 8;
        const unsigned char *w = smem + kOffW + c % kStagesW * kTile;
        unsigned char *out = smem + kOffParts + (c & 1) * (3 * kTile);
        const float *leave = bars->leave[chunk_len(c) < kC];
        auto split = [&](uint32_t at, float d) {
            const uint4 raw = *reinterpret_cast<const uint4 *>(w + at);
            const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
            uint32_t r[4][3];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                split_parts<3>(__uint_as_float(in[q] << 16) * d, __uint_as_float(in[q] & 0xffff0000u) * d, r[q]);
#pragma unroll
            for (int i = 0; i < 3; ++i)
                *reinterpret_cast<uint4 *>(out + i * kTile + at) = make_uint4(r[0][i], r[1][i], r[2][i], r[3][i]);
        };
        if (whole) {
            // the rows of a thread's packets lie whole swizzle periods apart
            const int sh = per == 16 ? 4 : 3, apart = of >> sh;
            int r = t >> sh;
            uint32_t at = ((t & (per - 1)) >> 3) * kBlock + sw128_offset(r, t & 7);
#pragma unroll 1
            for (; r < kC; r += apart, at += apart * 128) split(at, leave[r]);
        } else {
#pragma unroll 1
            for (int i = t; i < total; i += of) {
                const int r = i / per, ch = i - r * per;
                split((ch >> 3) * kBlock + sw128_offset(r, ch & 7), leave[r]);
            }
        }
        fence_proxy_async();
        warp_arrive(&bars->parts_ready[c & 1]);
    };

    if (warp < 2) {
        // ------------------------------------------------ copies (without TMA:
        // warp 0 X and half of Y, warp 1 the other half and W)
        const __nv_bfloat16 *X = static_cast<const __nv_bfloat16 *>(a.X) + (long)(h / a.sx) * kd;
        const __nv_bfloat16 *Y = static_cast<const __nv_bfloat16 *>(a.Y) + (long)(h / a.sy) * kd;
        const __nv_bfloat16 *W = static_cast<const __nv_bfloat16 *>(a.W) + (long)(h / a.sw) * vd;
        const Maps &m = maps.pass[blockIdx.y];
        // W of chunk c + 1 is asked for with X and Y of chunk c.
        int issued = 0, issued_w = 0;
        auto copy_w = [&](int c) {
            const int st = c % kStagesW, n = chunk_len(c);
            if (c >= kStagesW && !warp_wait(&bars->empty_w[st], (c / kStagesW - 1) & 1, abort)) return false;
            unsigned char *tile = smem + kOffW + st * kTile;
            const long t0 = it.start + (long)chunk_at(c);
            if constexpr (kTma) {
                uint64_t *landed = n == kC ? &bars->full_w[st] : &bars->partial;
                const int blocks = (vd + 63) / 64;
                if (elect_one()) {
                    mbar_arrive_expect_tx(landed, kBlock * blocks);
                    for (int i = 0; i < blocks; ++i)
                        tma_load_3d(tile + i * kBlock, &m.w, landed, i * 64, h / a.sw, (int)t0);
                }
                __syncwarp();
            } else {
                copy_tile<V>(smem_u32(tile), W + t0 * a.ld_w, a.ld_w, vd, n, warp * (kC / 2), (warp + 1) * (kC / 2));
                if (V == 1) mbar_arrive(&bars->full_w[st]);
                else copies_arrive(&bars->full_w[st]);      // every lane, when its own copies have landed
            }
            ++issued_w;
            return true;
        };
        const int mine = kTma && warp ? 0 : chunks;
        bool fine = mine == 0 || copy_w(0);
        for (int c = 0; c < mine && fine; ++c) {
            const int st = c % kStages, n = chunk_len(c);
            if (c >= kStages && !(fine = warp_wait(&bars->empty[st], (c / kStages - 1) & 1, abort))) break;
            unsigned char *stage = smem + st * kStage;
            const long t0 = it.start + (long)chunk_at(c);
            if constexpr (kTma) {
                // (boxes of whole chunks: behind the last sequence's end they
                // are filled with zeros, behind another's the rows are replaced)
                uint64_t *landed = n == kC ? &bars->full[st] : &bars->partial;
                const int blocks = (kd + 63) / 64;
                if (elect_one()) {
                    mbar_arrive_expect_tx(landed, kBlock * (states_only ? 1 : 2) * blocks);
                    for (int i = 0; i < blocks; ++i) {
                        if (!states_only) tma_load_3d(stage + i * kBlock, &m.x, landed, i * 64, h / a.sx, (int)t0);
                        tma_load_3d(stage + kTile + i * kBlock, &m.y, landed, i * 64, h / a.sy, (int)t0);
                    }
                }
                __syncwarp();
                ++issued;
                if (n < kC) {
                    if (!(fine = warp_wait(&bars->partial, 0, abort))) break;      // a run has one such chunk
                    unsigned char *w = smem + kOffW + c % kStagesW * kTile;
                    for (int i = n * 8 + lane; i < kC * 8; i += 32) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            *reinterpret_cast<uint4 *>(stage + k * kBlock + i * 16) = make_uint4(0, 0, 0, 0);
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            *reinterpret_cast<uint4 *>(w + k * kBlock + i * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async();
                    warp_arrive(&bars->full[st]);
                    warp_arrive(&bars->full_w[c % kStagesW]);
                }
            } else {
                const uint32_t tile = smem_u32(stage);
                const int from = warp * (kC / 2), to = (warp + 1) * (kC / 2);
                copy_tile<V>(tile + kTile, Y + t0 * a.ld_y, a.ld_y, kd, n, from, to);
                if (!states_only) copy_tile<V>(tile, X + t0 * a.ld_x, a.ld_x, kd, n, from, to);
                if (V == 1) mbar_arrive(&bars->full[st]);
                else copies_arrive(&bars->full[st]);
            }
            if (c + 1 < chunks) fine = copy_w(c + 1);
        }
        if (kTma) {
            // every issued copy must land before the CTA may exit (a partial
            // chunk's has, or its wait ran out)
            int dummy = 0;
            if (lane < kStages && lane < issued) mbar_wait(&bars->full[lane], ((issued - 1 - lane) / kStages) & 1, &dummy);
            if (lane < kStagesW && lane < issued_w)
                mbar_wait(&bars->full_w[lane], ((issued_w - 1 - lane) / kStagesW) & 1, &dummy);
            __syncwarp();
        } else {
            commit_copies();
            wait_copies<0>();
        }
    } else if (warp < 4) {
        // ------------------------------------------------ MMA issuers (the
        // whole warp waits, one lane issues and commits).  The copies wrote
        // through the generic proxy: hence the proxy fence on this side.
        const uint32_t base = smem_u32(smem);
        // Lower words of the first stage's descriptors (the upper ones are alike);
        // another stage, K step or part is an addition to the address field (units
        // of 16 bytes).
        auto along_k = [](int k) { return (uint32_t)((k >> 2) * (kBlock / 16) + (k & 3) * 2); };
        const uint32_t hi = (uint32_t)(sdesc_sw128(base, 16, 1024) >> 32), x0 = (uint32_t)sdesc_sw128(base, 16, 1024);
        bool fine = true;
        auto wait = [&](uint64_t *bar, uint32_t parity) { return fine = fine && warp_wait(bar, parity, abort); };
        if (warp == 2) {
            const uint32_t idesc_a = idesc_bf16(64, 64, false, false), idesc_d = idesc_bf16(128, ksteps * 16, true, true);
            const uint32_t y0 = (uint32_t)sdesc_sw128(base + kTile, 16, 1024), yt0 = (uint32_t)sdesc_sw128(base + kTile, kBlock, 1024);
            const uint32_t part0 = (uint32_t)sdesc_sw128(base + kOffParts, kBlock, 1024);
            for (int c = 0; c < chunks; ++c) {
                const int st = c % kStages;
                const uint32_t stage = (uint32_t)st * (kStage / 16);
                if (!wait(&bars->full[st], (c / kStages) & 1)) break;
                if (!states_only) {
                    if (c >= 2 && !wait(&bars->o_free[c & 1], ((c >> 1) - 1) & 1)) break;
                    fence_proxy_async();
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t x = x0 + stage, y = y0 + stage;
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (k < ksteps) mma_lo(tmem + kColA + (c & 1) * 128, x + along_k(k), y + along_k(k), hi, idesc_a, k != 0);
                        mma_commit(&bars->a_ready[c & 1]);
                    }
                    __syncwarp();
                }
                // the state's increment
                if (!wait(&bars->parts_ready[c & 1], (c >> 1) & 1)) break;
                if (c >= 1 && !wait(&bars->d_free, (c - 1) & 1)) break;
                fence_proxy_async();
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t y = yt0 + stage, part = part0 + (uint32_t)((c & 1) * (3 * kTile / 16));
#pragma unroll
                    for (int k = 0; k < 12; ++k)      // the lowest part first: each MMA cuts the sum short
                        mma_lo(tmem + kColD, part + (uint32_t)((2 - (k >> 2)) * (kTile / 16) + (k & 3) * 128),
                               y + (uint32_t)((k & 3) * 128), hi, idesc_d, k != 0);
                    mma_commit(&bars->d_ready);
                    mma_commit(&bars->empty[st]);
                    if (states_only) {
                        mma_commit(&bars->parts_free[c & 1]);
                        mma_commit(&bars->empty_w[c % kStagesW]);
                    }
                }
                __syncwarp();
            }
        } else if (!states_only) {
            const uint32_t idesc_o1 = idesc_bf16(128, 64, false, false), idesc_o2 = idesc_bf16(128, 64, true, false);
            const uint32_t wt0 = (uint32_t)sdesc_sw128(base + kOffW, kBlock, 1024), p0 = (uint32_t)sdesc_sw128(base + kOffP, 16, 1024);
            for (int c = 0; c < chunks; ++c) {
                const int st = c % kStages;
                const uint32_t stage = (uint32_t)st * (kStage / 16), o = tmem + kColO + (c & 1) * 128;
                // what the state before the chunk gives
                if (!wait(&bars->full[st], (c / kStages) & 1)) break;
                if (c >= 2 && !wait(&bars->o_free[c & 1], ((c >> 1) - 1) & 1)) break;
                if (!wait(&bars->z_ready, c & 1)) break;
                fence_proxy_async();
                tc_fence_after();
                if (elect_one()) {
                    // (lower parts first, here and below)
                    const uint32_t x = x0 + stage;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (k < ksteps) mma_ta_lo(o, tmem + kColZ + 64 + k * 8, x + along_k(k), hi, idesc_o1, k != 0);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (k < ksteps) mma_ta_lo(o, tmem + kColZ + k * 8, x + along_k(k), hi, idesc_o1, 1);
                    mma_commit(&bars->o1_done);
                    mma_commit(&bars->empty[st]);
                }
                __syncwarp();
                if (!wait(&bars->full_w[c % kStagesW], (c / kStagesW) & 1)) break;
                if (!wait(&bars->p_ready, c & 1)) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t w = wt0 + (uint32_t)(c % kStagesW * (kTile / 16));
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mma_lo(o + 64, w + (uint32_t)((k & 3) * 128), p0 + (uint32_t)((1 - (k >> 2)) * (kBlock / 16) + (k & 3) * 2), hi,
                               idesc_o2, k != 0);
                    mma_commit(&bars->o_ready[c & 1]);
                    mma_commit(&bars->empty_w[c % kStagesW]);
                }
                __syncwarp();
            }
        }
        // all issued MMAs complete before TMEM is freed
        if (elect_one()) {
            mma_commit(&bars->drain[warp & 1]);
            int dummy = 0;
            mbar_wait(&bars->drain[warp & 1], 0, &dummy);
        }
        __syncwarp();
    } else if (states_only && warp < 12) {
        // ------------------------------------------------ D W for states alone
        for (int c = 0; c < chunks; ++c) {
            if (!warp_wait(&bars->full_w[c % kStagesW], (c / kStagesW) & 1, abort)) break;
            if (c >= 2 && !warp_wait(&bars->parts_free[c & 1], ((c >> 1) - 1) & 1, abort)) break;
            split_chunk(c, tid - 128, 256);
        }
    } else if (warp < 8) {
        // ------------------------------------------------ A -> P.  Row i of the
        // M = 64 product sits in lane 32 (i / 16) + i % 16; threads t and t + 16
        // of a warp take eight columns each of every 16.  A warp's rows see the
        // 16 columns of their own number with the mask, those on one side of it
        // whole and those on the other not at all.
        const int quad = warp & 3, i = quad * 16 + (lane & 15), j8 = (lane >> 4) * 8;
        if (!states_only) {
            const uint32_t from = tmem + kColA + ((uint32_t)(quad * 32) << 16);
            float power[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) power[q] = lam[rev ? q : 7 - q];
            for (int c = 0; c < chunks; ++c) {
                if (!warp_wait(&bars->a_ready[c & 1], (c >> 1) & 1, abort)) break;
                // (the products with the last P are done)
                if (c >= 1 && !warp_wait(&bars->o_ready[(c - 1) & 1], ((c - 1) >> 1) & 1, abort)) break;
                tc_fence_after();
                const uint32_t at = from + (c & 1) * 128;
                float s[8] = {};
                auto put = [&](int m) {
                    uint32_t r[4][2];
#pragma unroll
                    for (int q = 0; q < 4; ++q) split_parts<2>(s[2 * q], s[2 * q + 1], r[q]);
#pragma unroll
                    for (int i2 = 0; i2 < 2; ++i2)
                        *reinterpret_cast<uint4 *>(smem + kOffP + i2 * kBlock + sw128_offset(i, m * 2 + (lane >> 4))) =
                            make_uint4(r[0][i2], r[1][i2], r[2][i2], r[3][i2]);
                };
#pragma unroll 1
                for (int m = rev ? quad + 1 : 0; m < (rev ? 4 : quad); ++m) {
                    tmem_ld_16x2x8(at + m * 16, s);
                    const int j0 = m * 16 + j8;
                    const float f = bars->within[rev ? j0 - i : i - j0 - 7];
                    tmem_ld_wait();
#pragma unroll
                    for (int q = 0; q < 8; q += 2)
                        split_pair(mul2(make_pair(s[q], s[q + 1]), mul2(make_pair(power[q], power[q + 1]), make_pair(f, f))), s[q],
                                   s[q + 1]);
                    put(m);
                }
                tmem_ld_16x2x8(at + quad * 16, s);
                tmem_ld_wait();
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const int j = quad * 16 + j8 + q, e = rev ? j - i : i - j;
                    s[q] = e < 0 ? 0.f : s[q] * bars->within[max(e, 0)];
                }
                put(quad);
                fence_proxy_async();
                tc_fence_before();
                warp_arrive(&bars->p_ready);
            }
        }
    } else if (warp < 12) {
        // ------------------------------------------------ outputs
        const int quad = warp & 3, col = quad * 32 + lane;
        const uint32_t at = tmem + kColO + ((uint32_t)(quad * 32) << 16);
        const long step = (long)p.H * vd;
        const bool pairs = !(vd & 1) && !((uintptr_t)a.out & 3) && !a.out_f32;
        for (int c = 0; c < chunks && !states_only; ++c) {
            const int n = chunk_len(c);
            if (!warp_wait(&bars->o_ready[c & 1], (c >> 1) & 1, abort)) break;
            tc_fence_after();
            const uint32_t from = at + (c & 1) * 128;
            const long t0 = it.start + (long)chunk_at(c), row = (t0 * p.H + h) * vd + col;
            const float *enter = bars->enter[n < kC];
            if (pairs) {
                // neighbouring lanes trade halves: the even one writes two
                // columns of a token, the odd one of the next token
                uint32_t *out = reinterpret_cast<uint32_t *>(static_cast<unsigned short *>(a.out) + row + (lane & 1 ? step - 1 : 0));
                const uint32_t order = lane & 1 ? 0x3276 : 0x5410;
                int left = col < vd ? n - (lane & 1) : 0;             // of this lane's tokens 0, 2 ..
#pragma unroll 1
                for (int m = 0; m < 4; ++m, enter += 16, left -= 16) {
                    float o1[16], o2[16];
                    tmem_ld16(from + m * 16, o1);
                    tmem_ld16(from + 64 + m * 16, o2);
                    tmem_ld_wait();
                    if (m == 3) {
                        tc_fence_before();
                        warp_arrive(&bars->o_free[c & 1]);
                    }
#pragma unroll
                    for (int q = 0; q < 16; q += 2, out += step) {
                        const float2 f = *reinterpret_cast<const float2 *>(enter + q);
                        float v0, v1;
                        split_pair(fma2(make_pair(f.x, f.y), make_pair(o1[q], o1[q + 1]), make_pair(o2[q], o2[q + 1])), v0, v1);
                        const uint32_t mine = pack2(v0, v1), other = __shfl_xor_sync(0xffffffffu, mine, 1);
                        if (q < left) *out = __byte_perm(mine, other, order);
                    }
                }
                continue;
            }
#pragma unroll 1
            for (int m8 = 0; m8 < 8; ++m8) {
                float o1[8], o2[8];
                tmem_ld8(from + m8 * 8, o1);
                tmem_ld8(from + 64 + m8 * 8, o2);
                tmem_ld_wait();
                if (m8 == 7) {
                    tc_fence_before();
                    warp_arrive(&bars->o_free[c & 1]);
                }
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const int i = m8 * 8 + q;
                    if (col >= vd || i >= n) continue;
                    const float v = fmaf(enter[i], o1[q], o2[q]);
                    if (a.out_f32) static_cast<float *>(a.out)[row + i * step] = v;
                    else static_cast<__nv_bfloat16 *>(a.out)[row + i * step] = __float2bfloat16_rn(v);
                }
            }
        }
    } else {
        // ------------------------------------------------ the state: row `col`
        // of Z^T, columns k0 .. k0 + 31
        const int quad = warp & 3, col = quad * 32 + lane, k0 = ((warp - 12) >> 2) * 32;
        const bool mine = k0 < kd;
        const uint32_t at = tmem + ((uint32_t)(quad * 32) << 16);
        float z[32];
        attn_initial<32>(p, a, it, h, a.init_t ? (long)col * kd + k0 : (long)k0 * vd + col, a.init_t ? 1 : vd,
                         col < vd ? kd - k0 : 0, z);
        auto put = [&]() {
            if (mine) {
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    float v[2][8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        uint32_t r[2];
                        split_parts<2>(z[m * 16 + 2 * k], z[m * 16 + 2 * k + 1], r);
                        v[0][k] = __uint_as_float(r[0]);
                        v[1][k] = __uint_as_float(r[1]);
                    }
                    tmem_st8(at + kColZ + k0 / 2 + m * 8, v[0]);
                    tmem_st8(at + kColZ + 64 + k0 / 2 + m * 8, v[1]);
                }
                tmem_st_wait();
            }
            tc_fence_before();
            warp_arrive(&bars->z_ready);
        };
        bool fine = true;
        auto split_next = [&](int c) {
            if (!warp_wait(&bars->full_w[c % kStagesW], (c / kStagesW) & 1, abort)) return false;
            split_chunk(c, tid - 384, 512);
            return true;
        };
        if (!states_only && chunks) {
            fine = split_next(0);
            put();
        }
        for (int c = 0; c < chunks && fine; ++c) {
            // the next chunk's D W, in a buffer whose products were done with dZ
            // of the last chunk
            if (!states_only && c + 1 < chunks && !(fine = split_next(c + 1))) break;
            if (!(fine = warp_wait(&bars->d_ready, c & 1, abort))) break;
            tc_fence_after();
            const float f = lam[chunk_len(c)];
            if (mine)
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    float d[16];
                    tmem_ld16(at + kColD + k0 + m * 16, d);
                    tmem_ld_wait();
#pragma unroll
                    for (int q = 0; q < 16; q += 2) {
                        float &z0 = z[m * 16 + q], &z1 = z[m * 16 + q + 1];
                        split_pair(fma2(make_pair(f, f), make_pair(z0, z1), make_pair(d[q], d[q + 1])), z0, z1);
                    }
                }
            tc_fence_before();
            warp_arrive(&bars->d_free);
            if (states_only || c + 1 == chunks) continue;
            if (!(fine = warp_wait(&bars->o1_done, c & 1, abort))) break;
            tc_fence_after();
            put();
        }
        float *dst = nullptr;
        if (states_only) dst = a.seg_out + ((long)it.slot * p.H + h) * kd * vd;
        else if (a.fin && closes) dst = a.fin + ((long)it.seq * p.H + h) * kd * vd;
        if (dst && fine && col < vd)
#pragma unroll
            for (int k = 0; k < 32; ++k)
                if (k0 + k < kd) dst[(k0 + k) * vd + col] = z[k];
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && bars->abort) atomicExch(p.status, MDN_ERR_DEVICE_TIMEOUT);
    if (warp == 3) tmem_dealloc(tmem, kTmemCols);
}

template <int V>
cudaError_t launch(const AttnProblem &p, const AllMaps &maps, cudaStream_t st) {
    const cudaError_t err = allow_shared<attn_tc_kernel<V>>(kSmem);
    if (err != cudaSuccess) return err;
    return launch_after(attn_tc_kernel<V>, p, kThreads, kSmem, st, p, maps);
}

// [tokens, heads, width] rows as boxes of 64 tokens of 64 columns of a head.
bool map_rows(CUtensorMap *map, const void *base, long tokens, int heads, int width, long ld) {
    const uint64_t dims[3] = {(uint64_t)width, (uint64_t)heads, (uint64_t)tokens};
    const uint64_t strides[2] = {(uint64_t)width * 2, (uint64_t)ld * 2};
    const uint32_t box[3] = {64, 1, kC};
    return make_map_3d(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, dims, strides, box);
}

}  // namespace

cudaError_t launch_attn_tc(const AttnProblem &p, cudaStream_t st) {
    int V = packet_width(8, 2, [&](int V, int bytes) {
        for (int i = 0; i < p.n_pass; ++i) {
            const AttnPass &a = p.pass[i];
            if (a.kd % V || a.vd % V || !rows_aligned(a.X, a.ld_x, 2, bytes) || !rows_aligned(a.Y, a.ld_y, 2, bytes) ||
                !rows_aligned(a.W, a.ld_w, 2, bytes))
                return false;
        }
        return true;
    });
    AllMaps maps;
    for (int i = 0; i < p.n_pass && V == 8; ++i) {
        const AttnPass &a = p.pass[i];
        Maps &m = maps.pass[i];
        bool ok = map_rows(&m.y, a.Y, p.T_total, p.H / a.sy, a.kd, a.ld_y) &&
                  map_rows(&m.w, a.W, p.T_total, p.H / a.sw, a.vd, a.ld_w);
        if (a.out) ok = ok && map_rows(&m.x, a.X, p.T_total, p.H / a.sx, a.kd, a.ld_x);
        if (!ok) return cudaErrorInvalidValue;
    }
    return V == 8 ? launch<8>(p, maps, st) : V == 2 ? launch<2>(p, maps, st) : launch<1>(p, maps, st);
}

}  // namespace mdn
