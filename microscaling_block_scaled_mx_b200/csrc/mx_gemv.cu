// mx_gemv.cu -- products of a few tokens with 4-bit weights: y = alpha * x W^T
// with W in MXFP4 (E2M1 codes, an E8M0 scale per 32) or NVFP4 (E2M1 codes, an
// E4M3 scale per 16 and an fp32 encode scale per domain of rows), x in bf16 or
// fp32 as it is.  The weights' buffers are the block-scaled GEMM's operands.
//
// A CTA of eight warps takes 128 weight rows (a scale atom's rows) and walks
// along K in slices of 256 codes: 128 bytes of each row, copied
// asynchronously into a ring of slices.  A warp multiplies 16 of the rows with
// eight tokens at a time by m16n8k16 tensor-core products with fp32 sums, a
// 32-code chunk per pair of products; the chunk's sum times its scale is added
// to the running sum in fp32.  All operands of the products are exact:
//  - E2M1 codes become fp16 by the hardware conversion, two per instruction.
//    NVFP4's E4M3 scale multiplies them there: a code times a scale is a
//    multiple of 2^-10 below 2688 with six significant bits.
//  - bf16 activations, times 2^6, are exact in fp16 from 2^-23 up to 2^10.  A
//    token with a value outside in a slice keeps that slice in bf16, and the
//    slice is then multiplied in bf16 (the weights, and the other tokens,
//    converted: exact too).
//  - fp32 activations are split into three bf16 terms (8 + 8 + 8 bits, by
//    truncation, exact down to bf16's smallest subnormal) whose products go
//    into the same sum.
// The CTAs of a cluster split K and add their sums through distributed shared
// memory in the order of their ranks.  The split depends on N and K alone, and
// a token is a column of its own, so a token's result does not depend on the
// other tokens.
#include <cooperative_groups.h>
#include <cstdint>
#include <cstdlib>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mx.h"
#include "mx_device.cuh"
#include "mx_internal.h"

namespace mxgemv {

using namespace mxk;
namespace cg = cooperative_groups;

constexpr int ROWS = 128;            // weight rows per CTA
constexpr int THREADS = 256;
constexpr int SLICE = 256;           // codes of a row per slice
constexpr int DEPTH = 3;             // slices in the ring
constexpr int PITCH = SLICE / 2 + 16;      // bytes of a row's slice in the ring: eight rows' words in different banks
constexpr int CODE_BYTES = ROWS * PITCH;

struct GemvParams {
    const uint8_t *codes, *scales;
    const float *enc;          // NVFP4 encode scales, one per `lines` weight rows
    int64_t lines;
    int sl;
    bool words;                // plain scales: rows of whole aligned words
    const void *x;
    int64_t ldx;
    uint32_t tokens, n, k;
    uint32_t k_blocks, k_groups, slices;
    float alpha;
    void *y;
    int y_f32;
    int64_t ldy;
};

__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, uint32_t bytes, std::integral_constant<int, 16>) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
template <int B>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, uint32_t bytes, std::integral_constant<int, B>) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(bytes), "n"(B) : "memory");
}

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// Two E8M0 bytes (bits 0..15) as fp32 2^(s - 127), 0xFF NaN; DOWN: times 2^-6
// (2^-133 is bf16's smallest subnormal, so the packed product is exact).
template <bool DOWN>
__device__ __forceinline__ void e8m0_pair(uint32_t two, float &lo, float &hi) {
    uint32_t r;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.bf16x2.ue8m0x2 %0, t;\n\t}" : "=r"(r) : "r"(two));
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

// Eight consecutive activations of one token, loaded and turned into the B
// fragments of a chunk (words of two neighbours).
template <bool XF32> struct Acts {
    uint4 v[XF32 ? 2 : 1];

    __device__ __forceinline__ void load(const void *x, int64_t off, bool valid) {
#pragma unroll
        for (int i = 0; i < (XF32 ? 2 : 1); ++i) {
            v[i] = make_uint4(0u, 0u, 0u, 0u);
            if (valid)
                v[i] = XF32 ? __ldg(reinterpret_cast<const uint4 *>(static_cast<const float *>(x) + off) + i)
                            : __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(x) + off));
        }
    }

    // bf16: fp16 fragments if every value of the warp's 256 is exact there, else
    // the bf16 words; returns whether they are bf16 (the same in every lane)
    __device__ __forceinline__ bool store_f16(uint4 *dst) const {
        const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
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
        *dst = bad ? v[0] : make_uint4(h[0], h[1], h[2], h[3]);
        return bad;
    }

    // fp32: bf16 fragments of the three terms, the smallest first
    __device__ __forceinline__ void store_terms(uint4 *dst, int plane_stride) const {
        const uint32_t b[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[XF32].x, v[XF32].y, v[XF32].z, v[XF32].w};
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
            dst[j * plane_stride] = make_uint4(__byte_perm(t[j][0], t[j][1], 0x7632u), __byte_perm(t[j][2], t[j][3], 0x7632u),
                                               __byte_perm(t[j][4], t[j][5], 0x7632u), __byte_perm(t[j][6], t[j][7], 0x7632u));
    }
};

template <bool XF32, bool NV, int NT> struct Shape {
    static constexpr int PLANES = XF32 ? 3 : 1;
    static constexpr int GROUPS = NV ? 4 : 2;                  // scale words of a row per slice
    static constexpr int SCALE_BYTES = GROUPS * 512;
    static constexpr int ACT_VECS = NT * PLANES * 256;         // 16-byte fragments of a slice's activations
    static constexpr int SMEM = DEPTH * (CODE_BYTES + SCALE_BYTES) + 2 * ACT_VECS * 16 + 2 * 8 * NT;
    static_assert(NT * 8 * ROWS * 4 <= CODE_BYTES, "the sums reuse the ring");
};

// The 16 rows x 8 tokens products of the eight chunks of a slice.
// codes: this lane's word of chunk 0 in its first row; scale: its rows' first
// scale words.  EXACT16: every token's fragments are fp16, else `bf16` says it
// of this lane's token of each tile (always, for fp32 activations).
template <bool XF32, bool NV, int NT, bool EXACT16>
__device__ __forceinline__ void slice_products(const uint8_t *codes, const uint2 *scale, const uint4 *act, uint32_t lane,
                                               const bool (&bf16)[NT], float (&acc)[NT][4]) {
    using S = Shape<XF32, NV, NT>;
    const uint32_t sel = (lane & 2u) ? 0x4431u : 0x4420u;     // NVFP4: this lane's block of chunks c and c + 1
    uint2 words = make_uint2(0u, 0u);
    float f_lo[2] = {1.0f, 1.0f}, f_hi[2] = {1.0f, 1.0f};
    uint32_t m_lo[2], m_hi[2];
    if (NV && EXACT16) f_lo[0] = f_lo[1] = f_hi[0] = f_hi[1] = ACT_DOWN;
#pragma unroll(EXACT16 ? 8 : 2)
    for (int c = 0; c < 8; ++c) {
        if (c % (NV ? 2 : 4) == 0) words = scale[c / (NV ? 2 : 4) * 64];
        if (c % 2 == 0) {
            if (NV) {
                e4m3_pair(__byte_perm(words.x, 0u, sel), m_lo[0], m_lo[1]);
                e4m3_pair(__byte_perm(words.y, 0u, sel), m_hi[0], m_hi[1]);
            } else {
                e8m0_pair<EXACT16>(c % 4 == 0 ? words.x & 0xffffu : words.x >> 16, f_lo[0], f_lo[1]);
                e8m0_pair<EXACT16>(c % 4 == 0 ? words.y & 0xffffu : words.y >> 16, f_hi[0], f_hi[1]);
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
            float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < S::PLANES; ++j) {
                uint4 b = act[(i * S::PLANES + j) * 256 + c * 32];
                if (!EXACT16 && !XF32 && !bf16[i]) {
                    b.x = f16_to_bf16(b.x, ACT_DOWN);
                    b.y = f16_to_bf16(b.y, ACT_DOWN);
                    b.z = f16_to_bf16(b.z, ACT_DOWN);
                    b.w = f16_to_bf16(b.w, ACT_DOWN);
                }
                mma16816<!EXACT16>(part, a0, b.x, b.y);
                mma16816<!EXACT16>(part, a1, b.z, b.w);
            }
            acc[i][0] = __fmaf_rn(f_lo[c & 1], part[0], acc[i][0]);
            acc[i][1] = __fmaf_rn(f_lo[c & 1], part[1], acc[i][1]);
            acc[i][2] = __fmaf_rn(f_hi[c & 1], part[2], acc[i][2]);
            acc[i][3] = __fmaf_rn(f_hi[c & 1], part[3], acc[i][3]);
        }
    }
}

template <bool XF32, bool NV, int NT>
__global__ void __launch_bounds__(THREADS) gemv_kernel(const __grid_constant__ GemvParams p) {
    using S = Shape<XF32, NV, NT>;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t *ring = smem;
    uint8_t *ring_s = smem + DEPTH * CODE_BYTES;
    uint4 *acts = reinterpret_cast<uint4 *>(ring_s + DEPTH * S::SCALE_BYTES);
    uint8_t *flags = reinterpret_cast<uint8_t *>(acts + 2 * S::ACT_VECS);      // [2][8 NT]: the token is in bf16

    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
    const uint32_t g = lane >> 2, t = lane & 3u;
    const uint32_t split = cg::this_cluster().num_blocks(), rank = cg::this_cluster().block_rank();
    const uint32_t row0 = blockIdx.x / split * ROWS;
    const uint32_t t0 = blockIdx.y * (8 * NT);
    const uint32_t s_begin = p.slices * rank / split, s_end = p.slices * (rank + 1) / split;
    const uint32_t row_bytes = p.k / 2;

    // Codes: thread (r, chunk) copies the 16 bytes of rows r, r + 32, r + 64,
    // r + 96 to the places 16 (r / 4) + r % 4 + {0, 8, 4, 12} of the ring, so
    // that lane (g, t) of warp w finds its rows at places 16 w + g and + 8.  A
    // row past the last reads the last one again; its results are not stored.
    const uint32_t chunk = tid & 7u, r0 = tid >> 3;
    const uint8_t *src[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        src[i] = p.codes + static_cast<int64_t>(min(row0 + r0 + 32 * i, p.n - 1)) * row_bytes + chunk * 16;
    const uint32_t ring32 = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
    const uint32_t dst0 = ring32 + ((r0 >> 2) * 16 + (r0 & 3u)) * PITCH + chunk * 16;

    auto issue = [&](uint32_t s, uint32_t slot) {
        const uint32_t b = s * (SLICE / 2) + chunk * 16;
        const uint32_t left = b < row_bytes ? row_bytes - b : 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t to = dst0 + slot * CODE_BYTES + (8 * (i & 1) + 4 * (i >> 1)) * PITCH;
            const uint8_t *from = left ? src[i] + s * (SLICE / 2) : p.codes;
            if (!NV || row_bytes % 16 == 0) {
                copy_async(to, from, left ? 16u : 0u, std::integral_constant<int, 16>{});
            } else {                                       // rows of an odd number of 8-byte blocks
                copy_async(to, from, left ? 8u : 0u, std::integral_constant<int, 8>{});
                copy_async(to + 8, left > 8 ? from + 8 : p.codes, left > 8 ? 8u : 0u, std::integral_constant<int, 8>{});
            }
        }
        uint8_t *sdst = ring_s + slot * S::SCALE_BYTES;
#pragma unroll
        for (int i = 0; i < S::GROUPS * 128 / THREADS; ++i) {
            const uint32_t idx = tid + THREADS * i, kg = s * S::GROUPS + (idx >> 7), word = idx & 127u;
            const uint32_t n = kg * 4 < p.k_blocks ? min(p.k_blocks - kg * 4, 4u) : 0u;   // scales of this word
            uint8_t *to = sdst + idx * 4;
            const uint32_t to_s = static_cast<uint32_t>(__cvta_generic_to_shared(to));
            if (p.sl != SL_PLAIN) {
                const uint64_t atom = static_cast<uint64_t>(row0 / 128) * p.k_groups + kg;
                copy_async(to_s, p.scales + (n ? atom * (p.sl == SL_MMA ? 512u : 2048u) + word * 4 : 0u), n,
                           std::integral_constant<int, 4>{});
            } else {
                const uint32_t row = min(row0 + (word >> 2) + 32 * (word & 3u), p.n - 1);
                const uint8_t *from = p.scales + (n ? static_cast<uint64_t>(row) * p.k_blocks + kg * 4 : 0u);
                if (p.words) {
                    copy_async(to_s, from, n, std::integral_constant<int, 4>{});
                } else {
                    uint32_t w = 0;
                    for (uint32_t j = 0; j < n; ++j) w |= static_cast<uint32_t>(__ldg(from + j)) << (8 * j);
                    *reinterpret_cast<uint32_t *>(to) = w;
                }
            }
        }
    };
    auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };

    // Activations: warp w takes token w of each tile, lane l the eight values
    // from 8 l of the slice.  The tokens that are not there stay zero.
    Acts<XF32> a_next[NT];
    uint4 *act_mine = acts + (lane >> 2) * 32 + warp * 4 + (lane & 3u);
    auto has = [&](int i) { return t0 + 8 * i + warp < p.tokens; };
    auto load_acts = [&](uint32_t s) {
        const uint32_t col = s * SLICE + lane * 8;
#pragma unroll
        for (int i = 0; i < NT; ++i)
            if (has(i) && s < s_end)
                a_next[i].load(p.x, static_cast<int64_t>(t0 + 8 * i + warp) * p.ldx + col, col < p.k);
    };
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        if (has(i)) continue;
        for (int b = 0; b < 2; ++b) {
            for (int j = 0; j < S::PLANES; ++j) act_mine[b * S::ACT_VECS + (i * S::PLANES + j) * 256] = make_uint4(0, 0, 0, 0);
            if (lane == 0) flags[(b * NT + i) * 8 + warp] = 0;
        }
    }

    float acc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;

#pragma unroll
    for (int i = 0; i < DEPTH - 1; ++i) {
        if (s_begin + i < s_end) issue(s_begin + i, i);
        commit();
    }
    load_acts(s_begin);

    uint32_t slot = 0;
    for (uint32_t s = s_begin; s < s_end; ++s) {
        const uint32_t buf = s & 1u;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            if (!has(i)) continue;
            uint4 *dst = act_mine + buf * S::ACT_VECS + i * S::PLANES * 256;
            if (XF32) {
                a_next[i].store_terms(dst, 256);
            } else {
                const bool bad = a_next[i].store_f16(dst);
                if (lane == 0) flags[(buf * NT + i) * 8 + warp] = bad;
            }
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 2) : "memory");
        __syncthreads();                                   // slice s is in; slice s - 1 and its activations are free
        if (s + DEPTH - 1 < s_end) issue(s + DEPTH - 1, slot == 0 ? DEPTH - 1 : slot - 1);
        commit();
        load_acts(s + 1);

        const uint8_t *codes = ring + slot * CODE_BYTES + (16 * warp + g) * PITCH + 4 * t;
        const uint2 *scale = reinterpret_cast<const uint2 *>(ring_s + slot * S::SCALE_BYTES) +
                             (4 * warp + (g & 3u)) * 2 + (g >> 2);
        const uint4 *act = acts + buf * S::ACT_VECS + lane;
        bool bf16[NT];
        if (XF32) {
            slice_products<XF32, NV, NT, false>(codes, scale, act, lane, bf16, acc);
        } else {
            uint64_t any = 0;
#pragma unroll
            for (int i = 0; i < NT; ++i) any |= *reinterpret_cast<const uint64_t *>(flags + (buf * NT + i) * 8);
            if (any == 0) {
                slice_products<XF32, NV, NT, !XF32>(codes, scale, act, lane, bf16, acc);
            } else {
#pragma unroll
                for (int i = 0; i < NT; ++i) bf16[i] = flags[(buf * NT + i) * 8 + g];
                slice_products<XF32, NV, NT, false>(codes, scale, act, lane, bf16, acc);
            }
        }
        slot = slot == DEPTH - 1 ? 0 : slot + 1;
    }

    // the sums of this CTA, [token][row], over the ring (all its copies have landed)
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    const uint32_t r_lo = 4 * warp + (g & 3u) + 64 * (g >> 2);    // this lane's rows: r_lo and r_lo + 32
    float *sums = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sums[(8 * i + 2 * t + (j & 1)) * ROWS + r_lo + 32 * (j >> 1)] = acc[i][j];
    if (split > 1) cg::this_cluster().sync();
    else __syncthreads();
    for (uint32_t e = rank * THREADS + tid; e < NT * 8 * ROWS; e += split * THREADS) {
        const uint32_t tok = t0 + e / ROWS, row = row0 + e % ROWS;
        if (tok >= p.tokens || row >= p.n) continue;
        float v = 0.0f;
        for (uint32_t c = 0; c < split; ++c) v += cg::this_cluster().map_shared_rank(sums, c)[e];
        v *= NV ? __fdiv_rn(p.alpha, p.enc[row / p.lines]) : p.alpha;
        const int64_t off = static_cast<int64_t>(tok) * p.ldy + row;
        if (p.y_f32) static_cast<float *>(p.y)[off] = v;
        else static_cast<__nv_bfloat16 *>(p.y)[off] = __float2bfloat16_rn(v);
    }
    if (split > 1) cg::this_cluster().sync();              // the others still read this CTA's sums
}

template <bool XF32, bool NV, int NT>
cudaError_t launch(const GemvParams &p, int split, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    auto kern = gemv_kernel<XF32, NV, NT>;
    constexpr int SMEM = Shape<XF32, NV, NT>::SMEM;
    const cudaError_t e = ensure_smem_limit(kern, SMEM, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((p.n + ROWS - 1) / ROWS * split, (p.tokens + 8 * NT - 1) / (8 * NT));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = split;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

// CTAs that share a row block.
int choose_split(uint32_t blocks, uint32_t slices) {
    if (const char *e = std::getenv("GV_SPLIT")) return std::atoi(e);
    int c = 1;
    while (c < 8 && blocks * c < 296 && static_cast<uint32_t>(2 * c) <= slices) c *= 2;
    return c;
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
    p.words = p.k_blocks % 4 == 0 && (reinterpret_cast<uintptr_t>(a.scales) & 3u) == 0;
    p.alpha = a.alpha; p.y = a.y; p.y_f32 = a.ydt == MX_F32; p.ldy = a.ldy;
    const int split = choose_split((p.n + ROWS - 1) / ROWS, p.slices);
    const bool nv = a.enc != nullptr;
    if (a.xdt == MX_F32) return nv ? launch<true, true, 1>(p, split, st) : launch<true, false, 1>(p, split, st);
    if (p.tokens <= 8) return nv ? launch<false, true, 1>(p, split, st) : launch<false, false, 1>(p, split, st);
    return nv ? launch<false, true, 2>(p, split, st) : launch<false, false, 2>(p, split, st);
}
