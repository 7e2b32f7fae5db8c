// mx_gemv.cu -- products of a few tokens with 4-bit weights: y = alpha * x W^T
// with W in MXFP4 (E2M1 codes, an E8M0 scale per 32) or NVFP4 (E2M1 codes, an
// E4M3 scale per 16 and an fp32 encode scale per domain of rows), x in bf16 or
// fp32 as it is.  The weights' buffers are the block-scaled GEMM's operands.
//
// The weight rows are cut into tiles of 16 and the tiles dealt out evenly over
// the clusters of CTAs, one CTA per SM; a warp takes a tile, or a part of K of
// a tile where there are fewer tiles than warps.  The parts of a tile are spread
// over its cluster's CTAs, so that each stages the activations of its parts
// alone, and their sums are added in order through (distributed) shared memory.
// A warp walks along its K in slices of 256 codes, 128 bytes of each row, copied
// asynchronously into its own ring, so that warps wait for one another only
// where activations are staged.  It multiplies its 16 rows with eight tokens at
// a time by m16n8k16 tensor-core products with fp32 sums, a 32-code chunk per
// pair of products; the chunk's sum times its scale is added to the running sum
// in fp32.  All operands of the products are exact:
//  - E2M1 codes become fp16 by the hardware conversion, two per instruction.
//    NVFP4's E4M3 scale multiplies them there: a code times a scale is a
//    multiple of 2^-10 up to 2688 with six significant bits.
//  - bf16 activations, times 2^6, are exact in fp16 from 2^-23 up to 2^10.  A
//    token with a value outside in a slice keeps that slice in bf16, and the
//    slice is then multiplied in bf16 (the weights, and the other tokens,
//    converted: exact too).
//  - fp32 activations are split into three bf16 terms (8 + 8 + 8 bits, by
//    truncation, exact down to bf16's smallest subnormal) whose products go
//    into the same sum.
// The number of parts depends on N, K, the device and the activations' type, and
// a token is a column of its own, so a token's result does not depend on the
// other tokens.
//
// What bounds it.  The weights are read once, at 5.9 TB/s while they stream (a
// copy makes 6.5): one token x 28672 x 4096 takes 15.2 us where their bytes take
// 9.6.  The rest is what a call has before and after the stream: 2.3 us of launch
// and first loads, 0.9 us of staging (2.6 for sixteen tokens, 2.2 for eight of
// K = 14336), 0.5 us of adding the parts (2.4 in a cluster, for its barriers and
// the slowest of its CTAs) and 1.3 us of products that do not hide behind copies
// (2.1 with eight tokens, 3.4 with two tiles of tokens).  So 1 x 4096 x 4096
// takes 5.5 us (bytes: 1.4), 8 x 4096 x 14336 13.5 and 16 x 14336 x 4096 16.2
// (4.8), NVFP4 18.3 (5.1).  fp32 activations have three times the products: 27.5
// us for 28672 x 4096.
//
// Measured against the choices here (us, one token x 28672 x 4096 where not said):
//  - rings of three or four slices 17.7, two 16.9; a slot refilled behind its
//    products, with two slices in flight, 15.9, before them, with one, 15.3: the
//    activations' loads queue behind the weights'
//  - rows copied in 64-byte pieces 16.9, whole slices by eight lanes 15.6
//  - at most 16, 20, 24, 26 and 28 warps to a CTA: 17.0, 17.2, 17.6, 15.4, 15.4 (13
//    have a tile, and 26 where two parts of K fit); 16 x 14336 x 4096 (2, 2, 3, 3 and
//    4 parts, a cluster's where they are even) 16.9, 16.6, 19.9, 21.2, 16.6, NVFP4
//    18.6, 18.2, 21.6, 23.6, 18.7; 16 x 4096 x 4096 9.7, 9.8, 10.1, 10.4, 10.5;
//    8 x 4096 x 14336 13.0, 13.5, 14.0, 14.0, 14.0.  28 is what 72 registers leave
//    room for; the kernels of two tiles of tokens spill 48 to 108 bytes a thread
//    there and 8 to 44 at 20 warps and 96 registers, the others up to 52
//  - fp32 activations as three fp16 terms 25.7 against 28.0, but 4 x 9000 x 4112
//    NVFP4 25.9 against 18.8 (K's tail mixes types), 3 x 1001 x 2080 8.2 against
//    6.8, and bf16's 16.1 against 15.3 by registers
//  - codes by matrix loads (ldmatrix) instead of words: the same, 15.0 and 15.1
#include <algorithm>
#include <cooperative_groups.h>
#include <cstdint>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mx.h"
#include "mx_device.cuh"
#include "mx_internal.h"

namespace mxgemv {

using namespace mxk;
namespace cg = cooperative_groups;

constexpr int ATOM = 128;            // weight rows of a scale atom: eight tiles
constexpr int SLICE = 256;           // codes of a row per slice: a 128-byte line
constexpr int DEPTH = 2;             // slices in a warp's ring
constexpr int PITCH = SLICE / 2 + 16;      // bytes of a row's slice in the ring: eight rows' words in different banks
constexpr int MAX_WARPS = 28;
constexpr int SMEM_MAX = 227 * 1024;

struct GemvParams {
    const uint8_t *codes, *scales;
    const float *enc;          // NVFP4 encode scales, one per `lines` weight rows
    int64_t lines;
    int sl;
    uint32_t full;             // slices that are whole, in 16-byte pieces of codes and scale words
    const void *x;
    int64_t ldx;
    uint32_t tokens, n, k;
    uint32_t tile;             // tokens of a CTA: min(tokens, 8 NT)
    uint32_t k_blocks, k_groups, slices;
    uint32_t tiles;            // of 16 rows
    uint32_t lanes, parts;     // tiles of a cluster at a time, parts of K of a tile
    uint32_t share;            // a CTA's parts: lanes x share of its warps have a tile, others only stage
    uint32_t lanes_inv, share_inv;      // 2^32 over them, rounded up: quotients of small numbers
    uint32_t size_log;         // CTAs of a cluster: 2^size_log
    uint32_t each, extra;      // tiles of a cluster, one more of the first `extra`
    uint32_t passes;           // times `lanes` tiles
    uint32_t steps;            // slices of a warp: ceil(slices / parts)
    uint32_t window;           // steps whose activations are staged together
    float alpha;
    void *y;
    int y_f32;
    int64_t ldy;
};

template <int B>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src) {
    if (B == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(B) : "memory");
}
// the first `bytes` from src, zeros behind them
template <int B>
__device__ __forceinline__ void copy_async_part(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(bytes), "n"(B) : "memory");
}

// Plain loads, in their place: the preceding kernel may still write when this one
// starts, which the read-only path does not allow for.
__device__ __forceinline__ uint4 load16(const void *src) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(src) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t load_byte(const uint8_t *src) {
    uint32_t v;
    asm volatile("ld.global.u8 %0, [%1];" : "=r"(v) : "l"(src) : "memory");
    return v;
}

// 16 x 8 x 16 products; FIRST: the sum starts from zero.
template <bool BF16, bool FIRST>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    const float z[4] = {FIRST ? 0.0f : c[0], FIRST ? 0.0f : c[1], FIRST ? 0.0f : c[2], FIRST ? 0.0f : c[3]};
    if (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %11, %12, %13};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(z[0]), "f"(z[1]), "f"(z[2]), "f"(z[3]));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %11, %12, %13};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(z[0]), "f"(z[1]), "f"(z[2]), "f"(z[3]));
}

// The eight codes of a word as fp16 pairs, code 2i in the low half of q[i].
__device__ __forceinline__ void decode8(uint32_t w, uint32_t (&q)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\tcvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(q[0]), "=r"(q[1]), "=r"(q[2]), "=r"(q[3]) : "r"(w));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ void unpack_f16(uint32_t h, float &lo, float &hi) {
    asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.f32.f16 %0, x;\n\tcvt.f32.f16 %1, y;\n\t}"
        : "=f"(lo), "=f"(hi) : "r"(h));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// fp16 pair times f as a bf16 pair (exact for the values here)
__device__ __forceinline__ uint32_t f16_to_bf16(uint32_t h, float f) {
    float lo, hi;
    unpack_f16(h, lo, hi);
    return __byte_perm(__float_as_uint(lo * f), __float_as_uint(hi * f), 0x7632u);
}

constexpr float ACT_UP = 64.0f, ACT_DOWN = 1.0f / 64.0f;

// Two E8M0 bytes (a half of the word) as fp32 2^(s - 127), 0xFF NaN; DOWN: times
// 2^-6 (2^-133 is bf16's smallest subnormal, so the packed product is exact).
template <bool DOWN>
__device__ __forceinline__ void e8m0_pair(uint32_t word, bool high, float &lo, float &hi) {
    uint32_t r;
    if (high) asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.bf16x2.ue8m0x2 %0, b;\n\t}" : "=r"(r) : "r"(word));
    else asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.bf16x2.ue8m0x2 %0, a;\n\t}" : "=r"(r) : "r"(word));
    if (DOWN) asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(r) : "r"(0x3c803c80u));
    lo = __uint_as_float(r << 16);
    hi = __uint_as_float(r & 0xffff0000u);
}

// Two E4M3 bytes (bits 0..15), each as an fp16 pair of equal halves.
__device__ __forceinline__ void e4m3_pair(uint32_t two, uint32_t &lo, uint32_t &hi) {
    uint32_t r;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(two));
    lo = __byte_perm(r, 0u, 0x1010u);
    hi = __byte_perm(r, 0u, 0x3232u);
}

// Eight bf16 activations as fp16 fragment words, times 2^6, if all 256 of the
// warp's are exact there, else as they are; returns whether they stayed bf16
// (the same in every lane).
__device__ __forceinline__ bool stage_bf16(uint8_t *dst, const uint4 &v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t h[4];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xffff0000u);
        float l2, h2;
        h[i] = pack_f16(lo * ACT_UP, hi * ACT_UP);
        unpack_f16(h[i], l2, h2);
        bad |= !(l2 * ACT_DOWN == lo) || !(h2 * ACT_DOWN == hi);
    }
    bad = __any_sync(0xffffffffu, bad);
    *reinterpret_cast<uint4 *>(dst) = bad ? v : make_uint4(h[0], h[1], h[2], h[3]);
    return bad;
}

// Eight fp32 activations as bf16 fragment words of their three terms, the
// smallest first, `plane` bytes apart.
__device__ __forceinline__ void stage_f32(uint8_t *dst, const uint4 &v0, const uint4 &v1, uint32_t plane) {
    const uint32_t b[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
    uint32_t t[3][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const bool special = (b[i] & 0x7f800000u) == 0x7f800000u;       // Inf or NaN: one term, NaN kept NaN
        t[2][i] = b[i] & 0xffff0000u;
        if ((b[i] & 0x7fffffffu) > 0x7f800000u) t[2][i] |= 0x00400000u;
        const float r = __uint_as_float(b[i]) - __uint_as_float(t[2][i]);
        t[1][i] = special ? 0u : __float_as_uint(r) & 0xffff0000u;
        t[0][i] = special ? 0u : __float_as_uint(r - __uint_as_float(t[1][i]));
    }
#pragma unroll
    for (int j = 0; j < 3; ++j)
        *reinterpret_cast<uint4 *>(dst + j * plane) =
            make_uint4(__byte_perm(t[j][0], t[j][1], 0x7632u), __byte_perm(t[j][2], t[j][3], 0x7632u),
                       __byte_perm(t[j][4], t[j][5], 0x7632u), __byte_perm(t[j][6], t[j][7], 0x7632u));
}

template <bool XF32, bool NV, int NT> struct Shape {
    static constexpr int PLANES = XF32 ? 3 : 1;
    static constexpr int GROUPS = NV ? 4 : 2;                  // scale words of a row per slice
    static constexpr int SLOT = 16 * PITCH + GROUPS * 64;      // a warp's slice
    static constexpr int RING = DEPTH * SLOT;                  // of a warp
    static_assert(NT * 8 * 16 * 4 <= RING, "the sums reuse the ring");
    // bytes of a token's activations of n slices; the odd 64 put neighbouring tokens in different banks
    __host__ __device__ static constexpr uint32_t token(uint32_t n) { return n * (SLICE * 2) + 64; }
    __host__ __device__ static constexpr uint32_t smem(uint32_t warps, uint32_t tile, uint32_t n) {
        return warps * RING + tile * PLANES * token(n) + n * 8 * NT;
    }
};

// The 16 rows x 8 tokens products of the eight chunks of a slice.
// codes: this lane's word of chunk 0 in its first row; scale: its rows' first
// scale words; act: its token's fragment of chunk 0, for each tile of tokens.
// EXACT16: every token's fragments are fp16, else `bf16` says it of this
// lane's token of each tile (always, for fp32 activations).
template <bool XF32, bool NV, int NT, bool EXACT16>
__device__ __forceinline__ void slice_products(const uint8_t *codes, uint32_t scale, const uint8_t *const (&act)[NT],
                                               uint32_t plane, uint32_t lane, const bool (&bf16)[NT], float (&acc)[NT][4]) {
    using S = Shape<XF32, NV, NT>;
    const uint32_t sel = (lane & 2u) ? 0x4431u : 0x4420u;     // NVFP4: this lane's block of chunks c and c + 1
    uint2 words = make_uint2(0u, 0u);
    float f_lo[2] = {1.0f, 1.0f}, f_hi[2] = {1.0f, 1.0f};
    uint32_t m_lo[2], m_hi[2];
    if (NV && EXACT16) f_lo[0] = f_lo[1] = f_hi[0] = f_hi[1] = ACT_DOWN;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        if (c % (NV ? 2 : 4) == 0)
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(words.x), "=r"(words.y) : "r"(scale + c / (NV ? 2 : 4) * 64));
        if (c % 2 == 0) {
            if (NV) {
                e4m3_pair(__byte_perm(words.x, 0u, sel), m_lo[0], m_lo[1]);
                e4m3_pair(__byte_perm(words.y, 0u, sel), m_hi[0], m_hi[1]);
            } else {
                e8m0_pair<EXACT16>(words.x, c % 4 != 0, f_lo[0], f_lo[1]);
                e8m0_pair<EXACT16>(words.y, c % 4 != 0, f_hi[0], f_hi[1]);
            }
        }
        uint32_t q[4], r[4];
        decode8(*reinterpret_cast<const uint32_t *>(codes + 16 * c), q);
        decode8(*reinterpret_cast<const uint32_t *>(codes + 16 * c + 8 * PITCH), r);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (NV) {
                q[i] = mul_f16x2(q[i], m_lo[c & 1]);
                r[i] = mul_f16x2(r[i], m_hi[c & 1]);
            }
            if (!EXACT16) {
                q[i] = f16_to_bf16(q[i], 1.0f);
                r[i] = f16_to_bf16(r[i], 1.0f);
            }
        }
        const uint32_t a0[4] = {q[0], r[0], q[1], r[1]}, a1[4] = {q[2], r[2], q[3], r[3]};
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            float part[4];
#pragma unroll
            for (int j = 0; j < S::PLANES; ++j) {
                uint4 b = *reinterpret_cast<const uint4 *>(act[i] + j * plane + 64 * c);
                if (!EXACT16 && !XF32 && !bf16[i]) {
                    b.x = f16_to_bf16(b.x, ACT_DOWN);
                    b.y = f16_to_bf16(b.y, ACT_DOWN);
                    b.z = f16_to_bf16(b.z, ACT_DOWN);
                    b.w = f16_to_bf16(b.w, ACT_DOWN);
                }
                if (j == 0) mma16816<!EXACT16, true>(part, a0, b.x, b.y);
                else mma16816<!EXACT16, false>(part, a0, b.x, b.y);
                mma16816<!EXACT16, false>(part, a1, b.z, b.w);
            }
            acc[i][0] = __fmaf_rn(f_lo[c & 1], part[0], acc[i][0]);
            acc[i][1] = __fmaf_rn(f_lo[c & 1], part[1], acc[i][1]);
            acc[i][2] = __fmaf_rn(f_hi[c & 1], part[2], acc[i][2]);
            acc[i][3] = __fmaf_rn(f_hi[c & 1], part[3], acc[i][3]);
        }
    }
}

// a / b for a, b < 2^16, inv = ceil(2^32 / b) (0 for b = 1): inv * b - 2^32 < b, so the product is off by less than a
__device__ __forceinline__ uint32_t small_quotient(uint32_t a, uint32_t inv) { return inv ? __umulhi(a, inv) : a; }

template <bool NV>
__device__ __forceinline__ void store_y(const GemvParams &p, uint32_t tok, uint32_t row, float v) {
    if (tok >= p.tokens || row >= p.n) return;
    v *= NV ? __fdiv_rn(p.alpha, p.enc[row / p.lines]) : p.alpha;
    const int64_t off = static_cast<int64_t>(tok) * p.ldy + row;
    if (p.y_f32) static_cast<float *>(p.y)[off] = v;
    else static_cast<__nv_bfloat16 *>(p.y)[off] = __float2bfloat16_rn(v);
}

// BYTES: plain scales whose rows are not whole aligned words.
template <bool XF32, bool NV, int NT, bool BYTES>
__global__ void __launch_bounds__(32 * MAX_WARPS, 1) gemv_kernel(const __grid_constant__ GemvParams p) {
    using S = Shape<XF32, NV, NT>;
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const uint32_t g = lane >> 2, t = lane & 3u;
    const uint32_t win = p.window * p.share;                   // slices in a window
    const uint32_t pitch = S::token(win), plane = p.tile * pitch;
    const uint32_t workers = p.lanes * p.share;                // warps with a tile
    uint8_t *ring = smem + warp * S::RING;                     // a worker's
    uint8_t *acts = smem + workers * S::RING;                // [planes][tile][pitch]
    uint8_t *flags = acts + S::PLANES * plane;                 // [win][8 NT]: the token is in bf16
    const uint32_t ring32 = static_cast<uint32_t>(__cvta_generic_to_shared(ring));

    // launched while the stream's last kernel may still run (see the launch): no
    // global memory is touched before it has ended and its writes are visible
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t t0 = blockIdx.y * (8 * NT), count = min(p.tokens - t0, 8u * NT);
    const uint32_t size = 1u << p.size_log, rank = blockIdx.x & (size - 1), cluster = blockIdx.x >> p.size_log;
    const uint32_t tile_lo = cluster * p.each + min(cluster, p.extra);
    const uint32_t tile_hi = tile_lo + p.each + (cluster < p.extra ? 1u : 0u);
    const uint32_t here = small_quotient(warp, p.lanes_inv), col = warp - here * p.lanes, part = rank * p.share + here;
    const uint32_t row_bytes = p.k / 2;

    // A tile is the rows 4 w + {0..3} + {0, 32, 64, 96} of a scale atom, a 64-byte
    // run of each of its 512-byte groups.  Place g of a slot holds row
    // g % 4 + 64 (g / 4), place g + 8 the row 32 behind it: the rows of lane
    // (g, t) in the products.  Lane 8 r + c copies the 16-byte piece c of rows r,
    // r + 64, r + 32 and r + 96 (places r, r + 4, r + 8, r + 12): a row's 128
    // bytes by eight lanes.  A row past the last reads the last one again; its
    // results are not stored.
    const uint32_t piece = lane & 7u, r0 = lane >> 3;
    const uint32_t cdst = ring32 + r0 * PITCH + piece * 16;
    // lane l copies scale word l % 16 (of rows r + 32 q: 4 r + q) of group l / 16
    const uint32_t word = lane & 15u, sgroup = lane >> 4;
    const uint32_t sstep = p.sl == SL_PLAIN ? 4u : (p.sl == SL_MMA ? 512u : 2048u);     // bytes between groups
    const uint32_t sdst = ring32 + 16 * PITCH + lane * 4;
    const uint8_t *src, *src_s;                                // this lane's pieces of the next slice: row r's,
    uint32_t off64, off32, off96;                              // and the others from there (K <= 2^24)
    auto set_tile = [&](uint32_t tile) {
        const uint32_t row0 = tile / 8 * ATOM, w = tile % 8, row = min(row0 + 4 * w + r0, p.n - 1);
        src = p.codes + static_cast<int64_t>(row) * row_bytes + static_cast<int64_t>(part) * (SLICE / 2) + piece * 16;
        off64 = (min(row0 + 4 * w + r0 + 64, p.n - 1) - row) * row_bytes;
        off32 = (min(row0 + 4 * w + r0 + 32, p.n - 1) - row) * row_bytes;
        off96 = (min(row0 + 4 * w + r0 + 96, p.n - 1) - row) * row_bytes;
        const uint32_t srow = min(row0 + 4 * w + (word >> 2) + 32 * (word & 3u), p.n - 1);
        src_s = p.scales + (part * S::GROUPS + sgroup) * static_cast<uint64_t>(sstep) +
                (p.sl == SL_PLAIN ? static_cast<uint64_t>(srow) * p.k_blocks
                                  : static_cast<uint64_t>(tile / 8) * p.k_groups * sstep + 64 * w + 4 * word);
    };
    const uint32_t code_step = p.parts * (SLICE / 2), scale_step = p.parts * S::GROUPS * sstep;
    auto advance = [&] {
        src += code_step;
        src_s += scale_step;
    };
    auto issue_whole = [&](uint32_t slot) {                    // a slice of whole 16-byte pieces and scale words
        copy_async<16>(cdst + slot, src);
        copy_async<16>(cdst + slot + 4 * PITCH, src + off64);
        copy_async<16>(cdst + slot + 8 * PITCH, src + off32);
        copy_async<16>(cdst + slot + 12 * PITCH, src + off96);
#pragma unroll
        for (int i = 0; i < S::GROUPS / 2; ++i) copy_async<4>(sdst + slot + i * 128, src_s + 2 * i * sstep);
        advance();
    };
    // Any slice.  BYTES: the scales are read byte by byte into registers, and
    // place_scales puts them into the slot after the products of the slice before,
    // when they have come.
    constexpr int WORDS = S::GROUPS / 2;
    uint32_t bytes[BYTES ? WORDS : 1][4];
    auto issue = [&](uint32_t s, uint32_t slot) {
        if (s < p.full) {
            issue_whole(slot);
            return;
        }
        const uint32_t b = s * (SLICE / 2) + piece * 16, left = b < row_bytes ? row_bytes - b : 0u;
        const bool whole = (s + 1) * (SLICE / 2) <= row_bytes;                 // (uniform)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t dst = cdst + slot + i * (4 * PITCH);
            const uint8_t *from = src + (i == 0 ? 0u : i == 1 ? off64 : i == 2 ? off32 : off96);
            if (whole && (!NV || row_bytes % 16 == 0)) {
                copy_async<16>(dst, from);
            } else if (whole) {                                // rows of an odd number of 8-byte blocks
                copy_async<8>(dst, from);
                copy_async<8>(dst + 8, from + 8);
            } else {
                copy_async_part<8>(dst, left ? from : p.codes, left ? 8u : 0u);
                copy_async_part<8>(dst + 8, left > 8 ? from + 8 : p.codes, left > 8 ? 8u : 0u);
            }
        }
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            const uint32_t kg = s * S::GROUPS + sgroup + 2 * i;
            const uint32_t n = kg * 4 < p.k_blocks ? min(p.k_blocks - kg * 4, 4u) : 0u;   // scales of this word
            const uint8_t *from = src_s + 2 * i * sstep;
            if (!BYTES) {
                copy_async_part<4>(sdst + slot + i * 128, n ? from : p.scales, n);
            } else {
#pragma unroll
                for (uint32_t j = 0; j < 4; ++j) bytes[BYTES ? i : 0][j] = j < n ? load_byte(from + j) : 0u;
            }
        }
        advance();
    };
    auto place_scales = [&](uint32_t slot) {
        if (!BYTES) return;
#pragma unroll
        for (int i = 0; i < WORDS; ++i)
            *reinterpret_cast<uint32_t *>(ring + slot + 16 * PITCH + lane * 4 + i * 128) =
                bytes[BYTES ? i : 0][0] | (bytes[BYTES ? i : 0][1] << 8) | (bytes[BYTES ? i : 0][2] << 16) |
                (bytes[BYTES ? i : 0][3] << 24);
    };
    auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };

    // Activations of the window's steps from w0, the slices of this CTA's parts:
    // a warp takes a (token, slice) at a time, lane l the eight values from 8 l.
    // Returns whether one of this warp's stayed bf16.
    auto stage = [&](uint32_t w0) {
        bool any = false;
        constexpr int BATCH = XF32 ? 2 : 4;                    // loads in flight
        const uint32_t n = min(p.window, p.steps - w0) * p.share;
        uint32_t tok = 0, j = warp;
        auto settle = [&] {
            while (j >= n && tok < count) {
                j -= n;
                ++tok;
            }
        };
        settle();
        while (tok < count) {
            uint4 v[BATCH][XF32 ? 2 : 1];
            uint32_t to[BATCH], flag[BATCH];
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                to[b] = ~0u;
                if (tok >= count) continue;
                const uint32_t step = small_quotient(j, p.share_inv);
                const uint32_t s = (w0 + step) * p.parts + rank * p.share + j - step * p.share, k = s * SLICE + lane * 8;
                const bool in = s < p.slices && k < p.k;
                const int64_t off = static_cast<int64_t>(t0 + tok) * p.ldx + k;
#pragma unroll
                for (int h = 0; h < (XF32 ? 2 : 1); ++h) {
                    v[b][h] = make_uint4(0, 0, 0, 0);
                    if (in)
                        v[b][h] = XF32 ? load16(static_cast<const float *>(p.x) + off + 4 * h)
                                       : load16(static_cast<const uint16_t *>(p.x) + off);
                }
                to[b] = tok * pitch + j * (SLICE * 2) + lane * 16;
                flag[b] = j * (8 * NT) + tok;
                j += warps;
                settle();
            }
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                if (to[b] == ~0u) break;
                if (XF32) {
                    stage_f32(acts + to[b], v[b][0], v[b][XF32], plane);
                } else {
                    const bool bad = stage_bf16(acts + to[b], v[b][0]);
                    if (lane == 0) flags[flag[b]] = bad;
                    any |= bad;
                }
            }
        }
        return any;
    };
    if (!XF32)
        for (uint32_t i = threadIdx.x; i < win * 8 * NT; i += blockDim.x)      // the tokens that are not there
            if (i % (8 * NT) >= count) flags[i] = 0;

    float acc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
    const uint8_t *act_mine[NT];            // columns past the last token repeat it; they are not stored
#pragma unroll
    for (int i = 0; i < NT; ++i) act_mine[i] = acts + min(8 * i + g, count - 1) * pitch + t * 16;

    // Step i of a pass is slice i * parts + part of tile pass * lanes + col; a
    // warp without a tile, or past the last slice, only waits with the others.
    uint32_t tile = tile_lo + col, slot = 0;
    const uint32_t mine = tile < tile_hi && warp < workers ? (p.slices - part + p.parts - 1) / p.parts : 0u;    // parts <= slices
    if (mine) {
        set_tile(tile);
        issue(part, 0);
        place_scales(0);
    }
    commit();
    const uint8_t *codes_mine = ring + g * PITCH + 4 * t;
    const uint32_t scale_mine = ring32 + 16 * PITCH + (g & 3u) * 16 + (g >> 2) * 8;
    const bool act16[NT] = {};              // no token in bf16
    bool mixed = false;                     // a token of the window is in bf16 somewhere
    for (uint32_t pass = 0; pass < p.passes; ++pass) {
        const uint32_t stop = tile < tile_hi ? mine : 0u;
        const bool more = tile + p.lanes < tile_hi;
        for (uint32_t w0 = 0; w0 < p.steps; w0 += p.window) {
            if (p.window < p.steps || pass == 0) {
                if (w0 + pass > 0) __syncthreads();            // the last window has been read
                mixed = __syncthreads_or(stage(w0));
            }
            const uint32_t w1 = min(w0 + p.window, stop);
            const uint8_t *act[NT], *fl = flags + here * (8 * NT);
#pragma unroll
            for (int j = 0; j < NT; ++j) act[j] = act_mine[j] + here * (SLICE * 2);
            uint32_t s = w0 * p.parts + part, i = w0;
            // steps whose next slice is whole, with every token in fp16: nothing to decide
            for (; !XF32 && !mixed && i < w1 && i + 1 < stop && s + p.parts < p.full && !BYTES; ++i) {
                asm volatile("cp.async.wait_group 0;" ::: "memory");
                __syncwarp();               // slice s is in, the other slot free
                issue_whole(S::SLOT - slot);
                commit();
                slice_products<XF32, NV, NT, !XF32>(codes_mine + slot, scale_mine + slot, act, plane, lane, act16, acc);
                slot = S::SLOT - slot;
                s += p.parts;
#pragma unroll
                for (int j = 0; j < NT; ++j) act[j] += p.share * (SLICE * 2);
            }
            for (; i < w1; ++i) {
                asm volatile("cp.async.wait_group 0;" ::: "memory");
                __syncwarp();
                s += p.parts;
                const bool ahead = i + 1 < stop || more;
                if (ahead) {
                    if (i + 1 == stop) set_tile(tile + p.lanes);
                    issue(i + 1 == stop ? part : s, S::SLOT - slot);
                }
                commit();
                bool bf16[NT], slow = XF32;
                if (mixed) {
                    uint64_t any = 0;
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        any |= reinterpret_cast<const uint64_t *>(fl + (i - w0) * p.share * (8 * NT))[j];
                        bf16[j] = fl[(i - w0) * p.share * (8 * NT) + min(8 * j + g, count - 1)];
                    }
                    slow = __any_sync(0xffffffffu, any != 0);
                }
                if (XF32 || slow) slice_products<XF32, NV, NT, false>(codes_mine + slot, scale_mine + slot, act, plane, lane, bf16, acc);
                else slice_products<XF32, NV, NT, !XF32>(codes_mine + slot, scale_mine + slot, act, plane, lane, act16, acc);
                slot = S::SLOT - slot;
                if (ahead) place_scales(slot);
#pragma unroll
                for (int j = 0; j < NT; ++j) act[j] += p.share * (SLICE * 2);
            }
        }
        if (p.parts == 1 && stop) {
            const uint32_t row = tile / 8 * ATOM + 4 * (tile % 8) + (g & 3u) + 64 * (g >> 2);    // this lane's: and + 32
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    store_y<NV>(p, t0 + 8 * i + 2 * t + (j & 1), row + 32 * (j >> 1), acc[i][j]);
                    acc[i][j] = 0.0f;
                }
        }
        tile += p.lanes;
    }
    if (p.parts == 1) return;

    // One pass: the parts' sums, [token][place in the tile] in each warp's ring (its copies have landed)
    __syncwarp();
    float *sums = reinterpret_cast<float *>(ring);
#pragma unroll
    for (int i = 0; i < NT && warp < workers; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sums[(8 * i + 2 * t + (j & 1)) * 16 + g + 8 * (j >> 1)] = acc[i][j];
    if (size > 1) cg::this_cluster().sync();
    else __syncthreads();
    const uint32_t rows = min(tile_hi - tile_lo, p.lanes) * 16;
    for (uint32_t e = rank * blockDim.x + threadIdx.x; e < count * rows; e += size * blockDim.x) {
        const uint32_t ti = e / rows, c = (e - ti * rows) / 16, q = e % 16, at = tile_lo + c;
        const float *theirs = reinterpret_cast<const float *>(smem + c * S::RING) + ti * 16 + q;
        float v = 0.0f;
        if (size == 1) {
            for (uint32_t k = 0; k < p.parts; ++k) v += theirs[k * p.lanes * (S::RING / 4)];
        } else {
            for (uint32_t k = 0; k < p.parts; k += 4) {        // in order, four loads in flight
                float f[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t one = min(k + j, p.parts - 1), r = small_quotient(one, p.share_inv);
                    f[j] = *cg::this_cluster().map_shared_rank(theirs + (one - r * p.share) * p.lanes * (S::RING / 4), r);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (k + j < p.parts) v += f[j];
            }
        }
        const uint32_t row = at / 8 * ATOM + 4 * (at % 8) + (q & 3u) + 64 * ((q >> 2) & 1u) + 32 * (q >> 3);
        store_y<NV>(p, t0 + ti, row, v);
    }
    if (size > 1) cg::this_cluster().sync();                   // the others still read this CTA's sums
}

uint32_t ceil_div(uint32_t a, uint32_t b) { return (a + b - 1) / b; }

template <bool XF32, bool NV, int NT, bool BYTES>
cudaError_t allow_smem() {
    static std::atomic<uint64_t> done{0};
    return ensure_smem_limit(gemv_kernel<XF32, NV, NT, BYTES>, SMEM_MAX, done);
}

// n = clusters of `size` CTAs with all the shared memory that the device runs at
// a time; asked once for each device and size.  The parts of K follow from it,
// so it is asked of one kernel for all (they have the same bounds): a token's
// bits depend neither on its kernel, that is on how many tokens there are, nor
// on which call came first.
cudaError_t max_clusters(uint32_t size, int sms, uint32_t &n) {
    static std::atomic<uint32_t> known[64][4];                     // the answer + 1
    n = static_cast<uint32_t>(sms);
    if (size == 1) return cudaSuccess;
    int dev = 0, count = 0;
    const int log = size == 2 ? 1 : size == 4 ? 2 : 3;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (const uint32_t k = known[dev][log].load(std::memory_order_relaxed)) {
        n = k - 1;
        return cudaSuccess;
    }
    e = allow_smem<false, false, 1, false>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(size);
    cfg.blockDim = dim3(32 * MAX_WARPS);
    cfg.dynamicSmemBytes = SMEM_MAX;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = size;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&count, gemv_kernel<false, false, 1, false>, &cfg);
    if (e != cudaSuccess) return e;
    n = count > 0 ? static_cast<uint32_t>(count) : 0u;
    known[dev][log].store(n + 1, std::memory_order_relaxed);
    return cudaSuccess;
}

template <bool XF32, bool NV, int NT, bool BYTES>
cudaError_t launch_kernel(GemvParams &p, int sms, cudaStream_t st) {
    using S = Shape<XF32, NV, NT>;
    auto kern = gemv_kernel<XF32, NV, NT, BYTES>;
    cudaError_t e = allow_smem<XF32, NV, NT, BYTES>();
    if (e != cudaSuccess) return e;
    p.tile = p.tokens < 8 * NT ? p.tokens : 8 * NT;

    // Parts of K, from N, K and the device alone: as many as there are warps for
    // with the tiles spread over all SMs, a multiple of four (or eight) so that
    // they can be shared out over a cluster.  That rounding leaves warps without a
    // tile at some widths, also where no cluster shares them: 1 x 5120 x 5120 has 4
    // parts of the 9 that fit, 12 warps, 7.4 us (bytes: 2.1); 8192 x 8192 4 of 7, 16
    // warps, 11.6 us (5.5); 11008 x 4096 4 of 5, 20 warps, 8.8 us (3.7).
    const uint32_t most = ceil_div(p.tiles, sms);                  // tiles per SM
    // SMs for each tile: a cluster's if there are so many, and slices enough to
    // make up for its barriers.  Measured (us, one SM to a tile and a cluster):
    // one token x 1024 x 4096 (16 slices) bf16 4.0 and 4.4, fp32 5.6 and 5.1;
    // 3 x 1001 x 2080 (9) 4.7 and 5.4, 6.5 and 6.6; 1 x 777 x 1056 (5) 3.4 and
    // 4.3, 4.5 and 5.4; 3 x 777 x 5120 (20) 6.9 and 5.5, 9.2 and 6.7;
    // 1 x 1024 x 14336 (56) 7.9 and 6.8, 12.5 and 10.1; 1 x 256 x 16384 (64)
    // 7.5 and 6.4, 14.1 and 7.1.
    uint32_t idle = 1;
    while (p.slices > (XF32 ? 8 : 16) && idle < 8) {
        uint32_t n;
        e = max_clusters(2 * idle, sms, n);
        if (e != cudaSuccess) return e;
        if (p.tiles > n) break;
        idle *= 2;
    }
    p.parts = 1;
    if (most <= MAX_WARPS / 2) {
        // with room for a step's activations of the most tokens that a CTA can have
        constexpr int MOST_NT = XF32 ? 1 : 2;
        uint32_t fit = MAX_WARPS / most;
        while (fit > 1 && Shape<XF32, NV, MOST_NT>::smem(most * fit, 8 * MOST_NT, fit) > SMEM_MAX) --fit;
        p.parts = fit * idle;
        p.parts = ceil_div(p.slices, ceil_div(p.slices, p.parts));
        const uint32_t unit = p.parts >= 8 && idle == 8 ? 8 : p.parts >= 4 ? 4 : 1;
        p.parts = p.parts / unit * unit;
    }
    p.steps = ceil_div(p.slices, p.parts);

    // CTAs of a cluster: as many as make the parts fit and leave no SM idle, and
    // more while a CTA stages the activations of more than 128 slices of tokens.
    // Staging one takes about 60 instructions of a warp, as much as 1.5 chunks'
    // products of a tile; a cluster's barriers take 1 to 2 us.  Measured (MXFP4,
    // bf16, us with clusters of 1, 2, 4): 8 tokens x 4096 x 4096 8.4, 8.5, 8.7
    // (128 slices); 8 x 4096 x 14336 22, 19, 16 (448); 1 x 4096 x 4096 6.0, 7.1,
    // 7.9 (16).
    uint32_t size = 0, clusters = 1;
    for (uint32_t c = 1; c <= 8 && p.parts % c == 0; c *= 2) {
        if (size >= idle && p.tile * p.slices <= 128 * size) break;
        uint32_t n;
        e = max_clusters(c, sms, n);
        if (e != cudaSuccess) return e;
        n = std::min(p.tiles, n);
        if (n == 0) continue;
        const uint32_t w = ceil_div(p.tiles, n) * (p.parts / c);
        if (p.parts > 1 && (w > MAX_WARPS || S::smem(w, p.tile, p.parts / c) > SMEM_MAX)) continue;
        size = c;
        clusters = n;
    }
    if (size == 0) return cudaErrorInvalidConfiguration;
    p.share = p.parts / size;
    p.size_log = size == 1 ? 0 : size == 2 ? 1 : size == 4 ? 2 : 3;
    p.each = p.tiles / clusters;
    p.extra = p.tiles % clusters;
    const uint32_t each = ceil_div(p.tiles, clusters);             // tiles of a cluster, at most
    p.passes = p.parts > 1 ? 1 : ceil_div(each, MAX_WARPS);
    p.lanes = ceil_div(each, p.passes);
    p.lanes_inv = p.lanes == 1 ? 0 : static_cast<uint32_t>(((1ull << 32) + p.lanes - 1) / p.lanes);
    p.share_inv = p.share == 1 ? 0 : static_cast<uint32_t>(((1ull << 32) + p.share - 1) / p.share);
    const uint32_t workers = p.lanes * p.share;
    // as many steps' activations at a time as fit, in windows of about the same size
    uint32_t windows = 1;
    for (p.window = p.steps; p.window > 1 && S::smem(workers, p.tile, p.window * p.share) > SMEM_MAX;
         p.window = ceil_div(p.steps, windows))
        ++windows;
    if (S::smem(workers, p.tile, p.window * p.share) > SMEM_MAX) return cudaErrorInvalidConfiguration;

    // Warps that stage a window in one batch of loads each: the CTA gets them if it
    // has much fewer with a tile.  Measured (us, without and with): 8 x 777 x 1056
    // (5 warps, 10 to stage) 6.7 and 4.5, 16 x 1024 x 4096 (8 and 32) 10.4 and 8.0,
    // 3 x 1001 x 2080 fp32 (9 and 14) 6.6 and 5.7, but 8 x 4096 x 14336 (24 and 30)
    // 13.5 and 13.8.
    const uint32_t staff = ceil_div(p.tile * p.window * p.share, XF32 ? 2 : 4);
    const uint32_t warps = 2 * staff >= 3 * workers ? std::max(workers, std::min(staff, uint32_t{MAX_WARPS})) : workers;

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(clusters * size, ceil_div(p.tokens, 8 * NT));
    cfg.blockDim = dim3(32 * warps);
    cfg.dynamicSmemBytes = S::smem(workers, p.tile, p.window * p.share);
    cfg.stream = st;
    // Programmatic serialization: this kernel's CTAs may start before the stream's
    // last kernel has drained.  Back to back, one token x 28672 x 4096 takes 15.9 us
    // a call instead of 18.4, eight x 4096 x 14336 15.1 instead of 16.6.
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = size;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = size > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <bool XF32, bool NV, int NT>
cudaError_t launch(GemvParams &p, bool bytes, int sms, cudaStream_t st) {
    return bytes ? launch_kernel<XF32, NV, NT, true>(p, sms, st) : launch_kernel<XF32, NV, NT, false>(p, sms, st);
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
    p.slices = (p.k + SLICE - 1) / SLICE;
    const bool bytes = a.sl == SL_PLAIN && (p.k_blocks % 4 != 0 || (reinterpret_cast<uintptr_t>(a.scales) & 3u) != 0);
    p.full = !bytes && p.k % 32 == 0 ? p.k / SLICE : 0;
    const uint32_t rest = p.n % ATOM;                              // rows of the last atom: a tile starts at each 4th of the first 32
    p.tiles = p.n / ATOM * 8 + (rest >= 32 ? 8 : (rest + 3) / 4);
    p.alpha = a.alpha; p.y = a.y; p.y_f32 = a.ydt == MX_F32; p.ldy = a.ldy;
    const bool nv = a.enc != nullptr;
    // Two tiles of tokens to a CTA from nine tokens on, as the registers allow with
    // bf16 alone: 16 x 14336 x 4096 takes 16.1 us, with a tile to each of two CTAs
    // (the weights read twice) 21.9.
    if (a.xdt == MX_F32) return nv ? launch<true, true, 1>(p, bytes, a.num_sms, st) : launch<true, false, 1>(p, bytes, a.num_sms, st);
    if (p.tokens <= 8) return nv ? launch<false, true, 1>(p, bytes, a.num_sms, st) : launch<false, false, 1>(p, bytes, a.num_sms, st);
    return nv ? launch<false, true, 2>(p, bytes, a.num_sms, st) : launch<false, false, 2>(p, bytes, a.num_sms, st);
}
