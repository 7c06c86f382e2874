// What the tensor-core kernels of linear attention share (mdn_attn_tc.cu: bf16
// rows, mdn_attn_tc32.cu: fp32 rows).
#pragma once

#include "mdn_attn.cuh"
#include "mdn_sm100.cuh"

namespace mdn {
namespace attn_tc {

using namespace sm100;

constexpr int kC = 64;                            // tokens of a chunk
constexpr uint32_t kBlock = 8192;                 // 64 tokens x 64 columns, swizzled
constexpr uint32_t kTile = 2 * kBlock;            // 64 tokens x 128 columns

// mbar_wait for a whole warp.  Most of a CTA's warps wait at any time, and a try
// ends unsuccessful after some 270 cycles whatever its time limit, so what is
// done between tries counts: nothing but counting to 1024 here.  (With the look
// at the flag and the clock each time, the kernel issued 8600 instructions a
// chunk.)
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
    const uint32_t at = smem_u32(bar);
    uint64_t t0 = 0;
    for (;;) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .u32 n;\n\t"
            "mov.u32 n, 1024;\n"
            "again:\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "@p bra done;\n\t"
            "sub.u32 n, n, 1;\n\t"
            "setp.ne.u32 p, n, 0;\n\t"
            "@p bra again;\n"
            "done:\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(at), "r"(parity), "r"(1000000u)
            : "memory");
        if (__all_sync(0xffffffffu, ok)) return true;
        if (t0 == 0) t0 = globaltimer();
        bool over = *abort != 0;
        if (!over && globaltimer() - t0 > kWaitLimitNs) {
            *abort = 1;
            over = true;
        }
        if (__any_sync(0xffffffffu, over)) return false;
    }
}
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// D[tmem] (+)= A[tmem] * B[smem], bf16 x bf16 -> fp32; A: two neighbouring K of
// a row in each 32-bit column.
__device__ __forceinline__ void mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// The same two products with the descriptors' lower words (addresses and leading
// offsets) apart from the upper ones, which an MMA's neighbours share: one addition
// an operand.
__device__ __forceinline__ void mma_lo(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %3};\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_ta_lo(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
        : "memory");
}

// True in one lane of the warp.  Unlike a comparison of the lane's number it
// tells the compiler so, which then issues an MMA's operands as they are and not
// lane by lane: 43 to 106 cycles an MMA of the shapes here instead of 107.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one != 0;
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&v);
}

// a, b -> N bf16 parts, packed: each what the ones before it leave, rounded.
template <int N>
__device__ __forceinline__ void split_parts(float a, float b, uint32_t *part) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        part[i] = pack2(a, b);
        if (i == N - 1) break;
        split_pair(fma2(make_pair(__uint_as_float(part[i] << 16), __uint_as_float(part[i] & 0xffff0000u)), make_pair(-1.f, -1.f),
                        make_pair(a, b)), a, b);
    }
}

// Launches a pass's kernel: set up while the kernel before it ends, which it
// waits for (grid_dependency_wait) before it reads anything.
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), const AttnProblem &p, int threads, int smem, cudaStream_t st, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.slots * (long)p.H), p.n_pass);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace attn_tc
}  // namespace mdn
