// mx_gemv.cu -- products of a few tokens with 4-bit weights: y = alpha * x W^T
// with W in MXFP4 (E2M1 codes, an E8M0 scale per 32) or NVFP4 (E2M1 codes, an
// E4M3 scale per 16 and an fp32 encode scale per domain of rows), x in bf16 or
// fp32 as it is.  The weights' buffers are the block-scaled GEMM's operands.
//
// One warp per weight row: each lane takes words of eight codes, decodes them
// and adds their products with up to four tokens in fp32.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mx.h"
#include "mx_device.cuh"
#include "mx_internal.h"

namespace mxgemv {

using namespace mxk;

constexpr int TOKENS = 4;      // tokens per CTA row of the grid
constexpr int WARPS = 4;

struct GemvParams {
    const uint8_t *codes, *scales;
    const float *enc;          // NVFP4 encode scales, one per `lines` weight rows
    int64_t lines;
    int sl;
    const void *x;
    int64_t ldx;
    uint32_t tokens, n, k;
    uint32_t k_blocks, k_groups;
    float alpha;
    void *y;
    int y_f32;
    int64_t ldy;
};

__device__ __forceinline__ float e2m1_value(uint32_t code) {
    // times 2^126 (exact): the three magnitude bits are the low exponent bits and the top mantissa bit
    return __uint_as_float(((code & 8u) << 28) | ((code & 7u) << 22)) * 8.507059173023462e37f;
}

__device__ __forceinline__ uint8_t scale_byte(const GemvParams &p, uint32_t row, uint32_t kb) {
    if (p.sl == SL_PLAIN) return p.scales[static_cast<uint64_t>(row) * p.k_blocks + kb];
    return p.scales[p.sl == SL_MMA ? mma_scale_offset32(row, kb, p.k_groups) : x4_scale_offset32(row, kb, p.k_groups)];
}

__device__ __forceinline__ float e8m0_value(uint32_t s) {
    return s == 0xffu ? __uint_as_float(0x7fffffffu) : (s == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(s << 23));
}

__device__ __forceinline__ float e4m3_value(uint32_t s) {
    const uint32_t e = (s >> 3) & 15u, m = s & 7u;
    if ((s & 0x7fu) == 0x7fu) return __uint_as_float(0x7fffffffu);
    const float v = e == 0 ? static_cast<float>(m) * 0.001953125f : __uint_as_float(((e + 120u) << 23) | (m << 20));
    return s & 0x80u ? -v : v;
}

template <bool BF16, bool NV>
__global__ void __launch_bounds__(32 * WARPS) gemv_kernel(const __grid_constant__ GemvParams p) {
    const uint32_t row = blockIdx.x * WARPS + (threadIdx.x >> 5);
    const uint32_t lane = threadIdx.x & 31u;
    const uint32_t t0 = blockIdx.y * TOKENS;
    if (row >= p.n) return;
    float acc[TOKENS] = {};
    const uint8_t *codes = p.codes + static_cast<int64_t>(row) * (p.k / 2);
    for (uint32_t word = lane; word < p.k / 8; word += 32) {
        const uint32_t c = *reinterpret_cast<const uint32_t *>(codes + 4ull * word);
        const uint32_t s = scale_byte(p, row, NV ? word / 2 : word / 4);
        const float scale = NV ? e4m3_value(s) : e8m0_value(s);
#pragma unroll
        for (int t = 0; t < TOKENS; ++t) {
            if (t0 + t >= p.tokens) break;
            const int64_t off = static_cast<int64_t>(t0 + t) * p.ldx + 8ll * word;
            float part = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float xv = BF16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p.x)[off + j])
                                      : static_cast<const float *>(p.x)[off + j];
                part = __fmaf_rn(e2m1_value((c >> (4 * j)) & 15u), xv, part);
            }
            acc[t] = __fmaf_rn(scale, part, acc[t]);
        }
    }
    const float f = NV ? __fdiv_rn(p.alpha, p.enc[row / p.lines]) : p.alpha;
#pragma unroll
    for (int t = 0; t < TOKENS; ++t) {
        float s = acc[t];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0 && t0 + t < p.tokens) {
            const int64_t off = static_cast<int64_t>(t0 + t) * p.ldy + row;
            if (p.y_f32) static_cast<float *>(p.y)[off] = s * f;
            else static_cast<__nv_bfloat16 *>(p.y)[off] = __float2bfloat16_rn(s * f);
        }
    }
}

}  // namespace mxgemv

cudaError_t mx_launch_gemv(const MxGemvArgs &a, cudaStream_t st) {
    using namespace mxgemv;
    GemvParams p;
    p.codes = static_cast<const uint8_t *>(a.codes); p.scales = static_cast<const uint8_t *>(a.scales);
    p.enc = a.enc; p.lines = a.lines; p.sl = a.sl;
    p.x = a.x; p.ldx = a.ldx;
    p.tokens = static_cast<uint32_t>(a.M); p.n = static_cast<uint32_t>(a.N); p.k = static_cast<uint32_t>(a.K);
    p.k_blocks = p.k / (a.enc ? 16 : 32);
    p.k_groups = (p.k_blocks + 3) / 4;
    p.alpha = a.alpha; p.y = a.y; p.y_f32 = a.ydt == MX_F32; p.ldy = a.ldy;
    const dim3 grid((p.n + WARPS - 1) / WARPS, (p.tokens + TOKENS - 1) / TOKENS);
    if (a.xdt == MX_BF16) {
        if (a.enc) gemv_kernel<true, true><<<grid, 32 * WARPS, 0, st>>>(p);
        else gemv_kernel<true, false><<<grid, 32 * WARPS, 0, st>>>(p);
    } else {
        if (a.enc) gemv_kernel<false, true><<<grid, 32 * WARPS, 0, st>>>(p);
        else gemv_kernel<false, false><<<grid, 32 * WARPS, 0, st>>>(p);
    }
    return cudaGetLastError();
}
