// mx_norm.cu -- RMS norm with an optional residual addition in front of it and
// an optional MX cast of its result, and the norm's backward pass.
//
// Forward, per row of `cols` values:
//   h = x + residual (rounded to the tensors' type, which is what is kept), or x
//   rstd = 1 / sqrt(sum(h^2) / cols + eps)
//   y = (h * rstd) * weight                     each step one fp32 operation
//   codes, scales = Algorithm 1 of the MX summary page (section 3) on the fp32 y
// Backward, with n = h * rstd, a = dy * weight:
//   dx = rstd * (a - n * sum(a n) / cols) + dres
//   dweight = sum over rows of dy * n
#include <cstdint>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mx.h"
#include "mx_device.cuh"
#include "mx_internal.h"

namespace mxnorm {

using namespace mxk;

struct NormParams {
    const void *x, *res;
    int64_t rows, ldx, ldr, ldh, ldy;
    uint32_t cols, vecs;       // vecs = cols / 8
    const void *w;
    int w_f32;
    float eps;
    void *h, *y;
    float *rstd;
    uint8_t *codes, *scales;
    int fmt, sl;
    uint32_t key;              // stochastic-rounding seed key
    uint32_t k_blocks, k_groups;
    uint64_t codes_cap, scales_cap;
};

// Eight consecutive values, widened to fp32.
template <bool BF16>
__device__ __forceinline__ void load8(const void *base, int64_t off, float (&v)[8]) {
    if (BF16) {
        const uint4 a = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + off);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(base) + off);
        const float4 a = p[0], b = p[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {     // nearest even
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Stores eight values; for bf16, v becomes what was stored.
template <bool BF16>
__device__ __forceinline__ void store8(void *base, int64_t off, float (&v)[8]) {
    if (BF16) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + off) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(base) + off);
        p[0] = make_float4(v[0], v[1], v[2], v[3]);
        p[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
}

__device__ __forceinline__ void load_weight8(const void *w, int w_f32, uint32_t col, float (&v)[8]) {
    if (w_f32) load8<false>(w, col, v);
    else load8<true>(w, col, v);
}

// Sum over the CTA, in an order fixed by its shape; every thread gets it.
// `red` holds 32 floats that no other sum in flight uses.
__device__ __forceinline__ float cta_sum(float s, float *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const int nw = blockDim.x >> 5;
    if (nw == 1) return s;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    s = lane < nw ? red[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// Codes of eight values (a quarter of block `vec / 4`) from the block's exponent.
template <int FMT, bool SR>
__device__ __forceinline__ void encode8(const NormParams &p, int64_t row, uint32_t vec, const float (&y)[8], int e,
                                        uint32_t keep) {
    constexpr int BITS = Fmt<FMT>::bits;
    constexpr int SLOT = BITS == 4 ? 4 : 8;
    float u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = scale_down<FMT>(y[i], e);
    uint32_t pw[2];
    if (SR) {
        const uint32_t g = static_cast<uint32_t>((static_cast<uint64_t>(row) * p.cols + 8ull * vec) >> 2);
#pragma unroll
        for (int j = 0; j < 2; ++j)
            pw[j] = sr_quad<FMT>(u[4 * j], u[4 * j + 1], u[4 * j + 2], u[4 * j + 3], fmix32((g + j) ^ p.key));
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j)
            pw[j] = cvt_pair<FMT>(u[4 * j], u[4 * j + 1]) | (cvt_pair<FMT>(u[4 * j + 2], u[4 * j + 3]) << (2 * SLOT));
    }
    pw[0] &= keep;
    pw[1] &= keep;
    const int64_t off = row * (static_cast<int64_t>(p.cols) * BITS / 8) + static_cast<int64_t>(vec) * BITS;
    if (!in_bounds(static_cast<uint64_t>(off), BITS, p.codes_cap)) return;
    uint8_t *dst = p.codes + off;
    if (BITS == 8) {
        *reinterpret_cast<uint2 *>(dst) = make_uint2(pw[0], pw[1]);
    } else if (BITS == 4) {
        *reinterpret_cast<uint32_t *>(dst) = pw[0] | (pw[1] << 16);
    } else {
        // eight 6-bit codes, 48 bits at an even address
        uint64_t w = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            w |= static_cast<uint64_t>((pw[j >> 2] >> (8 * (j & 3))) & 0x3fu) << (6 * j);
        uint16_t *d = reinterpret_cast<uint16_t *>(dst);
        d[0] = static_cast<uint16_t>(w);
        d[1] = static_cast<uint16_t>(w >> 16);
        d[2] = static_cast<uint16_t>(w >> 32);
    }
}

// The cast of eight values: the four lanes that hold a 32-block share its
// largest magnitude (as bits: non-negative floats order as integers, and an
// Inf or NaN is at or above 0x7f800000).  All lanes of the warp call this.
template <int FMT, bool SR>
__device__ __forceinline__ void cast8(const NormParams &p, int64_t row, uint32_t vec, bool valid, const float (&y)[8]) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i += 2) m = max_abs3(m, y[i], y[i + 1]);
    uint32_t a = __float_as_uint(m);
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
    if (!valid) return;
    const bool nan_block = a >= 0x7f800000u;
    const int e = nan_block ? 0 : block_exponent<FMT>(a);
    encode8<FMT, SR>(p, row, vec, y, e, nan_block ? 0u : 0xffffffffu);
    if ((vec & 3u) == 0)
        put_scale(p.scales, p.sl, static_cast<uint32_t>(row), vec >> 2, p.k_blocks, p.k_groups,
                  nan_block ? 0xffu : static_cast<uint32_t>(e + 127), p.scales_cap);
}

// CAST: 0 no codes, 1 round to nearest even, 2 stochastic rounding.
template <int V, int CAST, typename F>
__device__ __forceinline__ void for_format(int fmt, F f) {
    constexpr bool SR = CAST == 2;
    switch (fmt) {
        case MX_E4M3: f(std::integral_constant<int, MX_E4M3>{}, std::bool_constant<SR>{}); break;
        case MX_E5M2: f(std::integral_constant<int, MX_E5M2>{}, std::bool_constant<SR>{}); break;
        case MX_E2M3: f(std::integral_constant<int, MX_E2M3>{}, std::bool_constant<SR>{}); break;
        case MX_E3M2: f(std::integral_constant<int, MX_E3M2>{}, std::bool_constant<SR>{}); break;
        case MX_E2M1: f(std::integral_constant<int, MX_E2M1>{}, std::bool_constant<SR>{}); break;
        case MX_INT8: f(std::integral_constant<int, MX_INT8>{}, std::bool_constant<SR>{}); break;
    }
}

// One CTA per row; a thread holds V vectors of eight values, vector i of
// thread t being i * blockDim + t (so four neighbouring lanes hold a block).
template <bool BF16, int V, int CAST>
__global__ void __launch_bounds__(1024) norm_kernel(const __grid_constant__ NormParams p) {
    __shared__ float red[32];
    const int64_t row = blockIdx.x;
    float v[V][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint32_t vec = i * blockDim.x + threadIdx.x;
        if (vec < p.vecs) {
            load8<BF16>(p.x, row * p.ldx + 8ll * vec, v[i]);
            if (p.res) {
                float r[8];
                load8<BF16>(p.res, row * p.ldr + 8ll * vec, r);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] += r[j];
                store8<BF16>(p.h, row * p.ldh + 8ll * vec, v[i]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = __fmaf_rn(v[i][j], v[i][j], ss);
    }
    ss = cta_sum(ss, red);
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(ss, static_cast<float>(p.cols)) + p.eps));
    if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint32_t vec = i * blockDim.x + threadIdx.x;
        const bool valid = vec < p.vecs;
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = 0.0f;
        if (valid) {
            float w[8];
            load_weight8(p.w, p.w_f32, 8 * vec, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = __fmul_rn(__fmul_rn(v[i][j], rstd), w[j]);
        }
        if (CAST != 0)
            for_format<V, CAST>(p.fmt, [&](auto f, auto sr) { cast8<f.value, sr.value>(p, row, vec, valid, y); });
        if (p.y && valid) store8<BF16>(p.y, row * p.ldy + 8ll * vec, y);
    }
}

struct BackParams {
    const void *dy, *h, *dres;
    int64_t rows, lddy, ldh, lddres, lddx;
    uint32_t cols, vecs;
    const void *w;
    int w_f32;
    const float *rstd;
    void *dx;
    float *dw, *part;
    uint32_t parts;
};

// Rows blockIdx.x, blockIdx.x + gridDim.x, ...; a thread keeps its columns'
// share of dweight in registers and writes it to part[blockIdx.x] at the end.
template <bool BF16, int V>
__global__ void __launch_bounds__(1024) norm_backward_kernel(const __grid_constant__ BackParams p) {
    __shared__ float red[2][32];
    float acc[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
        const float rstd = p.rstd[row];
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t vec = i * blockDim.x + threadIdx.x;
            if (vec >= p.vecs) continue;
            float g[8], n[8], w[8];
            load8<BF16>(p.dy, row * p.lddy + 8ll * vec, g);
            load8<BF16>(p.h, row * p.ldh + 8ll * vec, n);
            load_weight8(p.w, p.w_f32, 8 * vec, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float nn = n[j] * rstd;
                acc[i][j] = __fmaf_rn(g[j], nn, acc[i][j]);
                s = __fmaf_rn(g[j] * w[j], nn, s);
            }
        }
        const float c = cta_sum(s, red[turn]) / static_cast<float>(p.cols);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t vec = i * blockDim.x + threadIdx.x;
            if (vec >= p.vecs) continue;
            float g[8], n[8], w[8];
            load8<BF16>(p.dy, row * p.lddy + 8ll * vec, g);
            load8<BF16>(p.h, row * p.ldh + 8ll * vec, n);
            load_weight8(p.w, p.w_f32, 8 * vec, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) g[j] = rstd * __fmaf_rn(-(n[j] * rstd), c, g[j] * w[j]);
            if (p.dres) {
                float r[8];
                load8<BF16>(p.dres, row * p.lddres + 8ll * vec, r);
#pragma unroll
                for (int j = 0; j < 8; ++j) g[j] += r[j];
            }
            store8<BF16>(p.dx, row * p.lddx + 8ll * vec, g);
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint32_t vec = i * blockDim.x + threadIdx.x;
        if (vec < p.vecs) store8<false>(p.part, static_cast<int64_t>(blockIdx.x) * p.cols + 8ll * vec, acc[i]);
    }
}

// dweight[c] = the sum of the parts, in order of the part.
__global__ void norm_dweight_kernel(const float *part, uint32_t parts, uint32_t cols, float *dw) {
    const uint32_t c = blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= cols) return;
    float s = 0.0f;
    for (uint32_t i = 0; i < parts; ++i) s += part[static_cast<int64_t>(i) * cols + c];
    dw[c] = s;
}

template <bool BF16, int V>
void launch_norm(const NormParams &p, int threads, int cast, cudaStream_t st) {
    const unsigned grid = static_cast<unsigned>(p.rows);
    if (cast == 0) norm_kernel<BF16, V, 0><<<grid, threads, 0, st>>>(p);
    else if (cast == 1) norm_kernel<BF16, V, 1><<<grid, threads, 0, st>>>(p);
    else norm_kernel<BF16, V, 2><<<grid, threads, 0, st>>>(p);
}

template <bool BF16>
void launch_norm_v(const NormParams &p, int cast, cudaStream_t st) {
    const int v = p.vecs <= 1024 ? 1 : p.vecs <= 2048 ? 2 : 4;
    const int threads = static_cast<int>((p.vecs + v - 1) / v + 31) / 32 * 32;
    if (v == 1) launch_norm<BF16, 1>(p, threads, cast, st);
    else if (v == 2) launch_norm<BF16, 2>(p, threads, cast, st);
    else launch_norm<BF16, 4>(p, threads, cast, st);
}

template <bool BF16>
void launch_backward_v(const BackParams &p, cudaStream_t st) {
    const int v = p.vecs <= 1024 ? 1 : p.vecs <= 2048 ? 2 : 4;
    const int threads = static_cast<int>((p.vecs + v - 1) / v + 31) / 32 * 32;
    if (v == 1) norm_backward_kernel<BF16, 1><<<p.parts, threads, 0, st>>>(p);
    else if (v == 2) norm_backward_kernel<BF16, 2><<<p.parts, threads, 0, st>>>(p);
    else norm_backward_kernel<BF16, 4><<<p.parts, threads, 0, st>>>(p);
}

}  // namespace mxnorm

cudaError_t mx_launch_rmsnorm(const MxNormArgs &a, cudaStream_t st) {
    using namespace mxnorm;
    NormParams p;
    p.x = a.x; p.res = a.residual; p.rows = a.rows; p.ldx = a.ldx; p.ldr = a.ldr; p.ldh = a.ldh; p.ldy = a.ldy;
    p.cols = static_cast<uint32_t>(a.cols);
    p.vecs = p.cols / 8;
    p.w = a.weight; p.w_f32 = a.wdt == MX_F32; p.eps = a.eps;
    p.h = a.h; p.y = a.y; p.rstd = a.rstd;
    p.codes = static_cast<uint8_t *>(a.codes); p.scales = static_cast<uint8_t *>(a.scales);
    p.fmt = a.fmt; p.sl = a.sl;
    p.key = fmix32_host(static_cast<uint32_t>(a.seed)) ^ static_cast<uint32_t>(a.seed >> 32);
    p.k_blocks = p.cols / 32;
    p.k_groups = (p.k_blocks + 3) / 4;
    p.codes_cap = a.codes ? mx_codes_bytes(static_cast<mx_fmt>(a.fmt), a.rows, a.cols) : 0;
    p.scales_cap = a.codes ? mx_scales_bytes(static_cast<mx_scale_layout>(a.sl), a.rows, a.cols) : 0;
    const int cast = !a.codes ? 0 : (a.rnd == MX_SR ? 2 : 1);
    if (a.xdt == MX_BF16) launch_norm_v<true>(p, cast, st);
    else launch_norm_v<false>(p, cast, st);
    return cudaGetLastError();
}

cudaError_t mx_launch_rmsnorm_backward(const MxNormBackArgs &a, cudaStream_t st) {
    using namespace mxnorm;
    BackParams p;
    p.dy = a.dy; p.h = a.h; p.dres = a.dres; p.rows = a.rows;
    p.lddy = a.lddy; p.ldh = a.ldh; p.lddres = a.lddres; p.lddx = a.lddx;
    p.cols = static_cast<uint32_t>(a.cols);
    p.vecs = p.cols / 8;
    p.w = a.weight; p.w_f32 = a.wdt == MX_F32; p.rstd = a.rstd;
    p.dx = a.dx; p.dw = a.dweight; p.part = a.part; p.parts = static_cast<uint32_t>(a.parts);
    if (a.xdt == MX_BF16) launch_backward_v<true>(p, st);
    else launch_backward_v<false>(p, st);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    norm_dweight_kernel<<<(p.cols + 127) / 128, 128, 0, st>>>(p.part, p.parts, p.cols, p.dw);
    return cudaGetLastError();
}

int mx_read_norm_bounds_status() {
    int b = 0;
    if (cudaMemcpyFromSymbol(&b, mxk::g_bounds_status, sizeof(int)) != cudaSuccess) return MX_ERR_CUDA;
    const int zero = 0;
    if (cudaMemcpyToSymbol(mxk::g_bounds_status, &zero, sizeof(int)) != cudaSuccess) return MX_ERR_CUDA;
    return b;
}
